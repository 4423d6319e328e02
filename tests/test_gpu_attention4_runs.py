"""Attention over 4 bits with requests cut into runs, beyond 64 requests and up to that, in each size of head."""
import pytest

from tests._gpu import log
from tests.test_gpu_attention4 import Setup, _need_gpu  # noqa: F401

pytestmark = pytest.mark.gpu

# heads, dim, page, new, kv, window, sinks
CASES = [
    ((4, 1), 128, 16, [1, 2, 0] * 25, [700, 41, 0] * 25, 0, 0),
    ((16, 1), 128, 64, [1] * 100, [1 + 83 * (i % 11) for i in range(100)], 0, 0),
    ((4, 1), 128, 16, [3, 1] * 60, [900, 350] * 60, 500, 33),
    ((2, 1), 256, 32, [1, 8] * 34, [900, 33] * 34, 0, 0),
    ((2, 1), 256, 32, [2] * 128, [5 + 61 * (i % 13) for i in range(128)], 600, 5),
    ((8, 1), 64, 16, [2, 1] * 40, [1 + 97 * (i % 9) for i in range(80)], 0, 0),
    ((32, 8), 128, 16, [8] * 20, [8 + 50 * i for i in range(20)], 0, 0),
    ((32, 8), 128, 16, [8] * 32, [8 + 30 * i for i in range(32)], 0, 0),
    ((16, 2), 256, 16, [5] * 6, [5, 900, 31, 400, 0, 1200], 0, 0),
    ((16, 4), 64, 16, [4] * 16, [60 * i for i in range(16)], 700, 3),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace(" ", "")[:20] for x in c))
def test_against_64_bits(case):
    heads, dim, page, new, kv, window, sinks = case
    log(f"[gpu-test] attention over 4 bits in runs {heads} {dim} {len(new)} requests")
    bound = 8192  # on the keys of a request, far above those there are
    s = Setup(heads, dim, page, new, kv, seed=sum(kv), extra_width=bound // page - -(-max(kv) // page))
    # tokens before the first key see nothing
    s.check(*s.run(window=window, sinks=sinks, max_new=max(new), max_kv=bound), window, sinks)
    s.check(*s.run(window=window, sinks=sinks, max_new=max(new), max_kv=max(kv)), window, sinks)
