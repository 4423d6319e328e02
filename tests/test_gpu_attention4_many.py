"""Attention over a cache in 4 bits where the call's bounds promise much work: prompts and long caches, which
other kernels take than short ones; bounds looser than the lengths lead small requests there too."""
import numpy as np
import pytest

from tests import _verify_ref as ref
from tests._gpu import log
from tests.test_gpu_attention4 import Setup, _need_gpu  # noqa: F401

pytestmark = pytest.mark.gpu


def _setup(heads, dim, page, new, kv, bound, seed):
    width = max(-(-max(kv) // page), 1)
    return Setup(heads, dim, page, new, kv, seed=seed, extra_width=max(0, -(-bound // page) - width))


CASES = [
    # heads, dim, page, new, kv, window, sinks, bound on the keys of a request
    # 256 rows to a workgroup: pieces, shares and whole segments
    ((8, 2), 128, 128, [300, 40], [420, 900], 0, 0, 1 << 17),
    ((8, 2), 128, 64, [300, 1, 0], [520, 200, 30], 70, 5, 1 << 18),
    ((32, 8), 128, 16, [1040], [1100], 0, 0, 4096),
    ((32, 8), 128, 16, [700, 1024], [700, 1100], 0, 0, 4096),
    ((32, 8), 128, 32, [1024, 3], [1100, 900], 33, 2, 1 << 15),
    # 128 rows
    ((8, 2), 128, 128, [32, 7, 20], [420, 900, 20], 0, 0, 1 << 20),
    ((8, 2), 128, 64, [25, 1, 0], [520, 200, 30], 70, 5, 1 << 20),
    ((32, 8), 128, 16, [30] * 33, [50 + 29 * i for i in range(33)], 0, 0, 1 << 15),
    ((6, 2), 256, 32, [150], [161], 0, 0, 1 << 16),
    ((6, 2), 256, 32, [150, 9], [361, 700], 50, 2, 1 << 18),
    ((8, 4), 256, 16, [40] * 70, [60 + 9 * (i % 11) for i in range(70)], 0, 0, 4096),
    # windows over long caches
    ((32, 8), 128, 16, [30] * 33, [9300] + [50 + 29 * i for i in range(32)], 8900, 40, 1 << 14),
    ((16, 4), 256, 64, [30] * 8, [4700] + [50 + 29 * i for i in range(7)], 4500, 40, 1 << 13),
    # heads of 64
    ((16, 16), 64, 16, [700], [900], 0, 0, 0),
    ((16, 2), 64, 64, [300, 0, 5], [1300, 4, 700], 0, 0, 0),
    ((16, 2), 64, 64, [300, 1], [1300, 700], 100, 33, 0),
    ((4, 1), 64, 16, [40] * 70, [60 + 9 * (i % 11) for i in range(70)], 0, 0, 0),
    # requests cut into runs: up to 64 of them by their lengths, beyond that each into as many
    ((8, 2), 128, 16, [1, 1, 0, 1, 1], [5, 800, 3, 32, 900], 0, 0, 4096),
    ((8, 2), 128, 16, [1, 4, 2, 1], [500, 800, 31, 900], 300, 33, 4096),
    ((16, 4), 64, 16, [16, 7, 30], [500, 800, 1031], 0, 0, 4096),
    ((16, 4), 64, 16, [16, 7, 30], [500, 2800, 1031], 2200, 70, 4096),
    ((8, 2), 256, 16, [9, 1, 20], [500, 800, 31], 0, 0, 4096),
    ((16, 4), 128, 16, [9] * 20, [20 + 60 * i for i in range(20)], 0, 0, 4096),
    ((4, 1), 64, 16, [2, 0, 1] * 24, [900, 0, 350] * 24, 0, 0, 8192),
    ((4, 1), 128, 16, [5, 0, 1] * 24, [900, 4, 350] * 24, 0, 0, 8192),
    ((4, 1), 128, 16, [5, 0, 1] * 24, [900, 4, 2350] * 24, 2100, 40, 8192),
    ((8, 2), 256, 32, [1] * 66, [5 + 137 * (i % 9) for i in range(66)], 0, 0, 4096),
    ((8, 2), 256, 32, [1] * 66, [5 + 137 * (i % 9) for i in range(66)], 1100, 3, 4096),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace(" ", "")[:30] for x in c))
def test_against_64_bits(case):
    heads, dim, page, new, kv, window, sinks, bound = case
    log(f"[gpu-test] attention over 4 bits, much work promised {heads} {dim} {new[:4]} {kv[:4]}")
    s = _setup(heads, dim, page, new, kv, bound, seed=sum(kv))
    s.check(*s.run(window=window, sinks=sinks, max_new=max(new)), window, sinks)


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 2)])
@pytest.mark.parametrize("heads,dim,new,bound", [((8, 2), 128, 200, 1 << 18), ((8, 2), 128, 30, 1 << 20), ((8, 2), 256, 30, 1 << 19),
                                                 ((8, 2), 64, 200, 0)])
def test_spoilt_values_and_pages(heads, dim, new, bound, window, sinks):
    """A block of NaN among the values reaches the tokens that see it, in its 32 elements alone; a page out
    of range the tokens that see it; what no token sees may hold anything."""
    import torch
    log(f"[gpu-test] attention over 4 bits, spoilt values, much work promised {dim} {new}")
    kv = 300
    s = _setup(heads, dim, 32, [new, new], [kv, kv + 20], bound, seed=8)
    first = kv - new - window + 1 if window else 0
    spoil = new // 2
    pos = kv - new + spoil
    s.write(s.v_cache, 0, [pos], np.where(np.arange(dim) == 40, np.nan, s.values[0][pos])[None])
    if first > 32:
        unseen = np.arange(first // 32 * 32, first)
        for cache in (s.k_cache, s.v_cache):
            s.write(cache, 0, unseen, np.full((len(unseen), 2, dim), np.inf))
        s.table[0, 1:first // 32] = 2 ** 30
    out, lse = s.run(window=window, sinks=sinks, max_new=new)
    torch.cuda.synchronize()
    sees = np.zeros(new, bool)
    sees[spoil:spoil + window if window else new] = True
    o = out.float().cpu().numpy()
    assert np.isnan(o[:new][sees][:, :, 32:64]).all()
    q = s.q.float().cpu().numpy()
    for b in (0, 1):
        rows = slice(b * new, (b + 1) * new)
        a, l, c, reach = ref.attention(q[rows], s.keys[b], s.values[b], s.kv[b], window, sinks)
        tol, tol_l = ref.attention_bounds(a, c, reach, s.kv[b], dim, True)
        keep = np.ones_like(a, bool)
        if b == 0:
            keep[sees, :, 32:64] = False
        assert np.all((np.abs(o[rows] - a) <= tol)[keep])
        assert np.all(np.abs(lse[rows].cpu().numpy() - l) <= tol_l)
    s.table[1, (kv + 19) // 32] = s.num  # the last token's page
    s.kv_len[0] = -1
    out, lse = s.run(window=window, sinks=sinks, max_new=new)
    assert torch.isnan(out[:new]).all() and torch.isnan(lse[:new]).all()
    assert torch.isnan(out[-1]).all() and torch.isnan(lse[-1]).all()


def test_a_million_rows():
    """A prompt of so many rows that their tiles pass a grid's second dimension."""
    import torch
    log("[gpu-test] attention over 4 bits, 65540 tokens of 16 heads to a key head")
    tokens, heads, dim, window, sinks = 65540, 16, 64, 21, 3
    from gru_corrected_draft_amd import verify
    rng = np.random.default_rng(1)
    op = verify.PagedAttention4(heads, 1, dim, 128, max_requests=1)
    gen = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((tokens, 1, dim), generator=gen, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((tokens, heads, dim), generator=gen, device="cuda").bfloat16()
    pages = -(-tokens // 128)
    k_cache, v_cache = torch.zeros((2, pages, 1, op.page_bytes), dtype=torch.uint8, device="cuda")
    where = (k_cache, v_cache, torch.arange(pages, dtype=torch.int32, device="cuda")[None],
             torch.tensor([tokens], dtype=torch.int32, device="cuda"), torch.tensor([0, tokens], dtype=torch.int32, device="cuda"))
    op.append(k, v, *where)
    stored_k, stored_v = (x.float().cpu().numpy().astype(np.float64) for x in op.read(tokens, *where))
    out, lse = op.run(q, *where, window=window, sinks=sinks, return_lse=True)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all()
    for t in [0, 1, 2, 31, 2047, 2048, tokens - 5, tokens - 1, *rng.integers(0, tokens, 60)]:
        o, l, a, reach = ref.attention(q[t:t + 1].float().cpu().numpy(), stored_k[:t + 1], stored_v[:t + 1], t + 1, window, sinks)
        tol, tol_l = ref.attention_bounds(o, a, reach, t + 1, dim, True)
        assert np.all(np.abs(out[t:t + 1].float().cpu().numpy() - o) <= tol), t
        assert np.all(np.abs(lse[t:t + 1].cpu().numpy() - l) <= tol_l), t
