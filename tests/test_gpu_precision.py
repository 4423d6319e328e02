"""How exact the operators of ``domino_verify.h`` are, with bounds near what their arithmetic gives.

The other tests bound every rounding by its worst case; these are for errors that hide below such bounds."""
import numpy as np
import pytest

from tests import _verify_ref as ref
from tests._gpu import log
from tests.test_gpu_attention import Setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


# heads, dim, new, kv, window, sinks: at most 32 rows (new x heads to a key head), whole tiles and partial ones
FEW_ROWS = [((8, 2), 128, [1, 1, 1], [9, 33, 70], 0, 0), ((32, 8), 64, [1], [40], 0, 0), ((8, 2), 128, [8, 2], [30, 64], 0, 0),
            ((4, 2), 256, [1, 3], [21, 50], 0, 0), ((8, 2), 128, [1, 2], [100, 64], 10, 3)]


@pytest.mark.parametrize("case", FEW_ROWS, ids=str)
def test_few_rows_keep_their_weights(case):
    """bf16, up to 32 rows: a weight is taken as two bf16 numbers.  The first is cut off after 8 bits (2^-7 of the
    weight is left), the second rounds that (2^-8 of it): off by at most 2^-15.  With the fp32 arithmetic that
    bounds the result before it is rounded, and rounding keeps order: the output lies between what the two ends
    round to.  Few keys, where weights are large."""
    import torch
    heads, dim, new, kv, window, sinks = case
    log(f"[gpu-test] attention weights {case}")
    s = Setup(heads, dim, 16, "bf16", new, kv, seed=31, k_scale=0.25)
    for kw in ({}, dict(max_kv=5000)):  # one workgroup a segment; room for pieces
        out, _ = s.run(window=window, sinks=sinks, max_new=max(new), **kw)
        out = out.float().cpu().numpy().astype(np.float64)
        at = 0
        for b, n in enumerate(new):
            o, _, weight, reach = ref.attention(*(x.float().cpu().numpy() for x in (s.q[at:at + n], s.keys[b], s.values[b])),
                                                kv[b], window, sinks)
            tol, _ = ref.attention_bounds(o, weight, reach, kv[b], dim, False)
            tol = tol + 2.0 ** -15 * weight
            low, high = (torch.from_numpy(x).to(torch.bfloat16).double().numpy() for x in (o - tol, o + tol))
            bad = (out[at:at + n] < low) | (out[at:at + n] > high)
            assert not bad.any(), f"request {b}: {bad.sum()} of {bad.size} off"
            at += n
