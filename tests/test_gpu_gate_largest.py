"""The gate and the balance loss at the largest token count they take, 2^31 - 1025: chunks of 2048 tokens, whose sums with a
position pass 32 bits unless they are formed with care.  One expert, so every result is known: id 0, softmax weight 1, counts
and loss exact (sums of ones)."""
import numpy as np
import pytest
import torch

import mxfp8_quantized_moe_amd as fm
from gpu_helpers import DEV, note, host, i32_dev

pytestmark = pytest.mark.gpu

T = 2**31 - 1025


@pytest.fixture(scope="module")
def logits():
    return torch.zeros(T, 1, dtype=torch.bfloat16, device=DEV)


@pytest.mark.parametrize("offs", [None, [T], [3000, T - 5]])
def test_choice_and_loss(logits, offs):
    note(f"moe_gate_balance {T} tokens, ends {offs}")
    od = None if offs is None else i32_dev(offs)
    ids = torch.full((T, 1), 9, dtype=torch.int32, device=DEV)
    w = torch.full((T, 1), 9.0, device=DEV)
    _, _, loss, counts, dprob = fm.moe_gate_balance(logits, 1, 0.5, od, ids=ids, weights=w)
    assert int(ids.min()) == 0 and int(ids.max()) == 0
    assert float(w.min()) == 1.0 and float(w.max()) == 1.0
    n = np.diff([0] + (offs or [T]))
    np.testing.assert_array_equal(host(counts)[:, 0], n)
    np.testing.assert_allclose(host(dprob)[:, 0], 0.5 / len(n) / n, rtol=2.0 ** -22)
    assert float(loss) == 0.5                     # f = P = 1 in every sequence
    del w
    again = fm.moe_balance_loss(logits, ids, 0.5, od)
    assert all(torch.equal(a, b) for a, b in zip(again, (loss, counts, dprob)))


def test_gradient(logits):
    """A sigmoid score of 1/2: each token's gradient is a quarter of its weight's; the loss of one expert is constant."""
    note(f"moe_gate_backward {T} tokens")
    ids = torch.zeros(T, 1, dtype=torch.int32, device=DEV)
    dw = torch.ones(T, 1, device=DEV)
    out = torch.full((T, 1), 9.0, dtype=torch.bfloat16, device=DEV)
    dprob = torch.full((1, 1), 1.0 / T, device=DEV)
    fm.moe_gate_backward(logits, ids, dw, fm.GATE_SIGMOID, dprob=dprob, dlogits=out)
    assert float(out.min()) == 0.25 and float(out.max()) == 0.25
