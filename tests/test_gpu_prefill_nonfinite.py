"""pa_prefill_window with scores that are not finite, in tiles with and without a mask."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.helpers import bits, from_bits
from tests.test_gpu_prefill import run, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window,at", [(5000, 0), (5000, 13), (5000, 14), (5000, 15), (5000, 30),
                                       (5000, 31), (5000, 127), (5000, 128 + 62), (5000, 299),
                                       (64, 270)])
@pytest.mark.parametrize("kind", ["inf", "nan"])
def test_a_score_that_is_not_finite_makes_its_row_nan(window, at, kind):
    """One query head whose score at one position overflows to +inf, or is inf - inf: a NaN
    row, in tiles with and without a mask; every other row keeps its bits."""
    case, starts, q = setup([(9, 300), (20, 333)], 4, 2, 64, 16, "bf16", window, 0, 3, drop=False)
    k = from_bits(case["k"], "bf16").clone()
    row = k[int(case["tables"][0, at // 16]), :, at % 16]
    row[:] = 1e20
    if kind == "nan":
        row[:, 32:] = -1e20
    case["k"] = bits(k)
    plain, st = run(case, starts, q, window, 0)
    assert st == 0
    big = from_bits(q, "bf16").clone()
    big[8, 1] = 1e20                                 # the last new token, position 299
    out, st = run(case, starts, bits(big), window, 0)
    assert st == 0
    assert bool(out[8, 1].isnan().all())
    out[8, 1] = plain[8, 1]
    assert torch.equal(out.view(torch.int16), plain.view(torch.int16))


@pytest.mark.parametrize("window", [5000, 100])
def test_scores_of_minus_infinity_have_no_weight(window):
    """All scores of a row -inf: nothing to average, a zero row.  All but one: that one's V."""
    case, starts, q = setup([(1, 300), (20, 333)], 4, 2, 64, 16, "bf16", window, 0, 3, drop=False)
    k = from_bits(case["k"], "bf16").clone()
    t = case["tables"][0, :19].astype(np.int64)
    k[torch.from_numpy(t)] = 1e20
    big = from_bits(q, "bf16").clone()
    big[0] = -1e20
    out, st = run(dict(case, k=bits(k)), starts, bits(big), window, 0)
    assert st == 0 and bool((out[0] == 0).all())
    k[int(t[250 // 16]), :, 250 % 16] = 0
    out, st = run(dict(case, k=bits(k)), starts, bits(big), window, 0)
    v = from_bits(case["v"], "bf16")[int(t[250 // 16]), :, 250 % 16]
    # its weight is 1 and no other row's is more than 2^-126: exactly that row
    assert st == 0 and torch.equal(out[0].cpu(), v.repeat_interleave(2, 0))
