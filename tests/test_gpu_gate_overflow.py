"""Gradients that are infinite or NaN (an overflowed loss scale) do not reach ineligible experts, whose gradient is 0, nor
tokens whose own gradients are finite."""
import pytest
import torch

import mxfp8_quantized_moe_amd as fm
from gpu_helpers import DEV, note

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("E", [12, 16, 64, 255, 256, 1000])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [False, True])
def test_ineligible_experts_stay_zero(E, score, renorm):
    note(f"moe_gate_backward overflow {E} score {score} renorm {renorm}")
    g = torch.Generator(device=DEV).manual_seed(E)
    T, k = 50, 4
    z = torch.randn(T, E, generator=g, device=DEV)
    z[torch.rand(T, E, generator=g, device=DEV) < 0.3] = -INF
    z[torch.rand(T, E, generator=g, device=DEV) < 0.05] = NAN
    z[7] = -INF
    gone = ~(z > -INF)
    ids, _, _, _, dprob = fm.moe_gate_balance(z, k, 0.1, None, score, renormalize=renorm)
    dw = torch.randn(T, k, generator=g, device=DEV)
    plain = fm.moe_gate_backward(z, ids, dw, score, None, renorm, dprob=dprob)
    for bad in (INF, -INF, NAN):
        dl = torch.full((1,), bad, device=DEV)
        for dz in (fm.moe_gate_backward(z, ids, dw, score, None, renorm, dprob=dprob, dloss=dl),
                   fm.moe_balance_loss_backward(z, dprob, dl, None, score)):
            assert torch.count_nonzero(dz[gone]) == 0        # also counts NaN
        hit = torch.arange(T, device=DEV) % 3 == 0
        w2 = torch.where(hit[:, None] & (torch.arange(k, device=DEV) == 1), bad, dw)
        dz = fm.moe_gate_backward(z, ids, w2, score, None, renorm, dprob=dprob)
        assert torch.count_nonzero(dz[gone]) == 0
        assert torch.equal(dz[~hit], plain[~hit])            # the others' tokens are what they were


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [False, True])
def test_a_choice_of_an_ineligible_expert_passes_nothing(score, renorm):
    """ids made elsewhere that name experts the logits rule out, with infinite gradients at them."""
    note(f"moe_gate_backward ineligible choice score {score} renorm {renorm}")
    g = torch.Generator(device=DEV).manual_seed(2)
    z = torch.randn(30, 20, generator=g, device=DEV)
    z[:, 4], z[:, 9] = -INF, NAN
    ids = torch.tensor([[4, 1, 9, 2]], dtype=torch.int32, device=DEV).repeat(30, 1)
    dw = torch.randn(30, 4, generator=g, device=DEV)
    for bad in (1.0, INF, NAN):
        dw[:, 0], dw[:, 2] = bad, -bad
        dz = fm.moe_gate_backward(z, ids, dw, score, None, renorm)
        assert torch.count_nonzero(dz[:, [4, 9]]) == 0
        if score == 1 or renorm:                             # scores of their own: the two other choices alone
            alone = torch.tensor([[1, 2]], dtype=torch.int32, device=DEV).repeat(30, 1)
            want = fm.moe_gate_backward(z, alone, dw[:, [1, 3]].contiguous(), score, None, renorm)
            torch.testing.assert_close(dz, want, rtol=1e-5, atol=1e-6)
    dw[:, 0], dw[:, 1] = 1.0, INF                            # at an eligible choice beside them
    dz = fm.moe_gate_backward(z, ids, dw, score, None, renorm)
    assert torch.count_nonzero(dz[:, [4, 9]]) == 0
