"""Attention over 4 bits of few rows: its weights to 15 bits, and the same bits whatever ran before.

The bounds of the other tests hold for weights rounded once to bf16; these would not."""
import numpy as np
import pytest

from tests import _verify_ref as ref
from tests._gpu import log
from tests.test_gpu_attention4 import Setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


# heads, dim, new, kv, window, sinks: at most 32 rows (new x heads to a key head), whole tiles and partial ones.
# Up to 16 rows and up to 32; row tiles that leave CUs idle (256 of them) and that do not.
FEW_ROWS = [
    ((8, 2), 128, [1, 1, 1], [9, 33, 70], 0, 0),
    ((32, 8), 64, [1], [40], 0, 0),
    ((16, 2), 256, [1, 2], [21, 64], 0, 0),
    ((8, 2), 128, [8, 2], [30, 64], 0, 0),
    ((8, 2), 64, [5, 8], [30, 96], 0, 0),
    ((4, 2), 256, [1, 13], [21, 50], 0, 0),
    ((8, 2), 128, [1, 2], [100, 64], 10, 3),
    ((32, 8), 128, [1] * 40, [9 + 7 * (i % 8) for i in range(40)], 0, 0),
    ((32, 8), 64, [2] * 40, [9 + 7 * (i % 8) for i in range(40)], 0, 0),
    ((16, 8), 256, [1] * 40, [9 + 7 * (i % 8) for i in range(40)], 0, 0),
    ((32, 8), 128, [8] * 20, [9 + 7 * (i % 8) for i in range(20)], 0, 0),
    ((32, 8), 64, [7] * 20, [9 + 7 * (i % 8) for i in range(20)], 0, 0),
    ((32, 8), 256, [5] * 20, [9 + 7 * (i % 8) for i in range(20)], 0, 0),
    # divided in earnest, few keys in each request but one
    ((8, 2), 128, [1, 1], [2100, 40], 2100, 0),
]


@pytest.mark.parametrize("case", FEW_ROWS, ids=lambda c: f"{c[0][0]}/{c[0][1]}-{c[1]}-{len(c[2])}x{max(c[2])}-{c[4]}")
def test_few_rows_keep_their_weights(case):
    """Up to 32 rows a weight is taken as two bf16 numbers.  The first is cut off after 8 bits (2^-7 of the weight is
    left), the second rounds that (2^-8 of it): off by at most 2^-15.  With the fp32 arithmetic that bounds the
    result before it is rounded, and rounding keeps order: the output lies between what the two ends round to."""
    import torch
    heads, dim, new, kv, window, sinks = case
    log(f"[gpu-test] weights over 4 bits {heads} {dim} {len(new)} x {max(new)} {window}")
    s = Setup(heads, dim, 16, new, kv, seed=31, extra_width=(5000 - max(kv)) // 16)
    s.q *= 0.25  # scores near each other: the bound is then mostly the weights' own
    widest = 0.0
    for kw in ({}, dict(max_kv=5000), dict(max_kv=max(kv))):  # bounds that cut requests into runs, and that do not
        out, _ = s.run(window=window, sinks=sinks, max_new=max(new), **kw)
        out = out.float().cpu().numpy().astype(np.float64)
        at = 0
        for b, n in enumerate(new):
            o, _, weight, reach = ref.attention(s.q[at:at + n].float().cpu().numpy(), s.keys[b], s.values[b], kv[b], window, sinks)
            tol, _ = ref.attention_bounds(o, weight, reach, kv[b], dim, False)
            tol = tol + 2.0 ** -15 * weight
            low, high = (torch.from_numpy(x).to(torch.bfloat16).double().numpy() for x in (o - tol, o + tol))
            bad = (out[at:at + n] < low) | (out[at:at + n] > high)
            assert not bad.any(), f"request {b}: {bad.sum()} of {bad.size} off"
            widest = max(widest, float(np.mean(high > low)))
            at += n
    log(f"[gpu-test]   ends that round apart: {widest:.2f}")


CALLS = [
    ((32, 8), 128, [1], [37]), ((8, 2), 128, [1, 1], [4000, 90]), ((8, 2), 64, [16] * 3, [3000, 16, 900]),
    ((32, 8), 128, [16] * 8, [2100, 700, 33, 16, 90, 1200, 400, 1700]), ((4, 1), 128, [2, 0, 1] * 27, [900, 0, 350] * 27),
    ((8, 2), 256, [16, 9], [1500, 30]), ((8, 2), 128, [300, 260], [2100, 400]), ((8, 2), 256, [90], [1900]),
]


@pytest.mark.parametrize("heads,dim,new,kv", CALLS)
def test_the_same_bits_after_other_calls(heads, dim, new, kv):
    """A call repeats itself to the bit, with other work of its handle before it: nothing that an earlier call left in
    the workspace counts, and no sum depends on which workgroup comes first."""
    import torch
    log(f"[gpu-test] the same bits over 4 bits {heads} {dim} {len(new)}")
    s = Setup(heads, dim, 16, new, kv, seed=3)
    bounds = dict(max_new=max(new), max_kv=max(kv))
    out, lse = s.run(**bounds)
    other = torch.full_like(s.q, float("nan"))
    for _ in range(3):
        s.run(q=other, **bounds)  # NaN through every part of the workspace
        s.run(window=7, sinks=1, **bounds)
        s.run(q=other)
        again, lse2 = s.run(**bounds)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
