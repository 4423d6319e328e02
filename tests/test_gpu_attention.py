"""Paged attention and the append that fills the cache, against 64 bits.

Bounds follow from the arithmetic (``_verify_ref.attention_bounds``); sizes are the small ones at which
tiles, pages, windows and row tiles end in each other's middle."""
import numpy as np
import pytest

from tests import _verify_ref as ref
from tests._gpu import log

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def _types():
    import torch
    return {"bf16": torch.bfloat16, "fp32": torch.float32}


class Setup:
    """Random keys and values of some requests, laid into shuffled pages."""

    def __init__(self, heads, dim, page, dtype, new, kv, seed=0, order="phrd", extra_width=0, k_scale=1.0):
        import torch
        from gru_corrected_draft_amd import verify
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hq, self.hk = heads
        self.dim, self.page, self.new, self.kv = dim, page, list(new), list(kv)
        self.dtype = dt = _types()[dtype]
        self.bf16 = dtype == "bf16"

        def normal(*shape):
            return torch.randn(shape, generator=g, device="cuda").to(dt)

        self.tokens = sum(new)
        self.q = normal(self.tokens, self.hq, dim)
        self.keys = [(normal(n, self.hk, dim) * k_scale).to(dt) for n in kv]
        self.values = [normal(n, self.hk, dim) for n in kv]
        pages = [-(-n // page) for n in kv]
        self.num = sum(pages) + 2
        width = max(max(pages), 1) + extra_width
        perm = torch.randperm(self.num, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((len(kv), width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = perm[at:at + n]
            at += n
        dims = {"p": self.num, "h": self.hk, "r": page, "d": dim}
        both = torch.full((2,) + tuple(dims[c] for c in order), float("nan"), dtype=dt, device="cuda")
        back = [1 + order.index(c) for c in "phrd"]
        self.k_cache, self.v_cache = (both.permute(0, *back)[i] for i in (0, 1))
        for b, n in enumerate(kv):
            if n:
                pos = torch.arange(n, device="cuda")
                pg = self.table[b].long()[pos // page]
                self.k_cache[pg, :, pos % page] = self.keys[b]
                self.v_cache[pg, :, pos % page] = self.values[b]
        self.kv_len = torch.tensor(kv, dtype=torch.int32, device="cuda")
        self.q_start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
        self.op = verify.PagedAttention(self.hq, self.hk, dim, page, dt, max_requests=max(1, len(kv)))

    def run(self, **kw):
        return self.op.run(kw.pop("q", self.q), self.k_cache, self.v_cache, self.table, self.kv_len, self.q_start,
                           return_lse=True, **kw)

    def check(self, out, lse, window=0, sinks=0, scale=None, skip=()):
        import torch
        torch.cuda.synchronize()
        out, lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        start = 0
        for b, n in enumerate(self.new):
            rows = slice(start, start + n)
            start += n
            if b in skip or n == 0:
                continue
            kv = self.kv[b]
            o, l, a, reach = ref.attention(*(x.float().cpu().numpy() for x in
                                             (self.q[rows], self.keys[b], self.values[b])),
                                           kv, window, sinks, scale)
            tol, tol_l = ref.attention_bounds(o, a, reach, kv, self.dim, self.bf16)
            worst = np.max(np.abs(out[rows] - o) / tol)
            assert np.all(np.abs(out[rows] - o) <= tol), f"request {b}: {worst:.3g} of the bound"
            empty = np.isneginf(l)
            assert np.array_equal(np.isneginf(lse[rows]), empty), f"request {b}"
            assert np.all(np.abs(np.where(empty, 0, lse[rows]) - np.where(empty, 0, l)) <= tol_l), f"request {b}"


CASES = [
    # heads, dim, page, dtype, new, kv, window, sinks
    ((8, 2), 64, 16, "fp32", [1], [1], 0, 0),
    ((8, 2), 64, 16, "fp32", [7, 1, 3], [100, 17, 3], 0, 0),
    ((4, 4), 128, 32, "fp32", [5, 16], [33, 64], 0, 0),
    ((6, 2), 256, 16, "fp32", [2, 9], [50, 9], 0, 0),
    ((8, 2), 64, 16, "fp32", [16, 16], [300, 45], 20, 3),
    ((8, 1), 64, 64, "fp32", [40], [40], 0, 0),
    ((32, 8), 128, 16, "bf16", [1], [1], 0, 0),
    ((32, 8), 128, 16, "bf16", [1], [37], 0, 0),
    ((32, 8), 128, 16, "bf16", [1, 1, 1, 1], [31, 32, 33, 1000], 0, 0),
    ((32, 8), 128, 16, "bf16", [16, 16], [16, 700], 0, 0),
    ((32, 8), 128, 64, "bf16", [16, 5, 1, 0, 16], [129, 128, 127, 50, 400], 0, 0),
    ((40, 8), 128, 64, "bf16", [16], [515], 0, 0),
    ((40, 8), 128, 32, "bf16", [16, 16], [515, 90], 100, 4),
    ((7, 1), 128, 16, "bf16", [9], [200], 33, 0),
    ((8, 8), 64, 16, "bf16", [3, 16], [77, 260], 0, 0),
    ((8, 8), 64, 16, "bf16", [1, 16], [777, 260], 48, 70),
    ((16, 2), 256, 16, "bf16", [1, 16], [90, 300], 0, 0),
    ((16, 2), 256, 128, "bf16", [4], [1000], 64, 1),
    ((64, 1), 128, 16, "bf16", [1, 3], [500, 20], 0, 0),
    ((100, 1), 64, 32, "bf16", [2], [90], 0, 0),
    # prompts: many row tiles, ragged
    ((32, 8), 128, 16, "bf16", [200, 33], [200, 300], 0, 0),
    ((8, 2), 128, 64, "bf16", [513], [700], 0, 0),
    ((8, 2), 128, 64, "bf16", [300, 100], [500, 100], 64, 5),
    ((8, 2), 128, 64, "bf16", [300], [300], 1, 0),
    ((6, 2), 64, 16, "bf16", [350, 1], [350, 400], 0, 0),
    ((6, 2), 256, 32, "bf16", [150], [161], 0, 0),
    ((6, 2), 256, 32, "bf16", [150], [361], 50, 2),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c))
def test_against_64_bits(case):
    heads, dim, page, dtype, new, kv, window, sinks = case
    log(f"[gpu-test] attention {case}")
    s = Setup(heads, dim, page, dtype, new, kv, seed=sum(kv))
    s.check(*s.run(window=window, sinks=sinks), window, sinks)
    # tighter bounds choose other kernels for the same result
    s.check(*s.run(window=window, sinks=sinks, max_new=max(new), max_kv=max(kv)), window, sinks)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("order", ["prhd", "hprd", "rphd"])
def test_cache_orders_and_strided_rows(dtype, order):
    """A cache in any order of pages, heads and rows; q and out inside wider tensors."""
    import torch
    log(f"[gpu-test] attention cache order {order} {dtype}")
    s = Setup((8, 2), 128, 16, dtype, [5, 16], [90, 333], seed=5, order=order)
    wide = torch.zeros((s.tokens, 3, s.hq, s.dim), dtype=s.dtype, device="cuda")
    wide[:, 1] = s.q
    out = torch.full((s.hq, s.tokens, s.dim + 8), 7.0, dtype=s.dtype, device="cuda")
    got, lse = s.run(q=wide[:, 1], out=out[:, :, :s.dim].transpose(0, 1))
    s.check(got, lse)
    assert torch.all(out[:, :, s.dim:] == 7)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_few_keys_and_no_keys(dtype):
    """Cache lengths of zero and one, and fewer keys than new tokens: the first tokens see nothing."""
    log(f"[gpu-test] attention of few keys {dtype}")
    s = Setup((8, 2), 128, 16, dtype, [3, 4, 1, 2], [0, 2, 1, 40], seed=6)
    out, lse = s.run()
    s.check(out, lse)
    assert (out[:3] == 0).all() and (lse[:3] == float("-inf")).all()
    assert (out[3:5] == 0).all() and (lse[3:5] == float("-inf")).all()


@pytest.mark.parametrize("dtype,new,kv,max_new", [("bf16", 16, 300, 16), ("bf16", 16, 300, 200),
                                                  ("fp32", 16, 300, 16), ("bf16", 100, 300, 100)])
def test_unseen_values_do_not_matter(dtype, new, kv, max_new):
    """Values of positions that a token does not see may be anything: the unwritten rest of a page (NaN in
    every cache here), keys before the window in a page that is still read, later tokens of the block."""
    import torch
    log(f"[gpu-test] attention unseen values {dtype} {new} {kv}")
    window, sinks = 40, 2
    s = Setup((8, 2), 128, 32, dtype, [new], [kv], seed=8)
    spoil = new // 2  # a token of the block whose value is infinite in one element
    pos = kv - new + spoil
    s.values[0][pos, :, 5] = float("inf")
    s.values[0][pos, 1, 9] = float("nan")
    s.v_cache[s.table[0, pos // 32].long(), :, pos % 32] = s.values[0][pos]
    first = kv - new - window + 1  # the first key that any token sees past the sinks
    for p in range(first // 32 * 32, first):  # unseen, in a page that is seen
        s.v_cache[s.table[0, p // 32].long(), :, p % 32] = float("nan")
        s.k_cache[s.table[0, p // 32].long(), :, p % 32] = float("nan")
    for i in range(1, first // 32):
        s.table[0, i] = -1 if i % 2 else 2 ** 30  # pages of evicted keys
    out, lse = s.run(window=window, sinks=sinks, max_new=max_new)
    torch.cuda.synchronize()
    sees = torch.zeros(new, dtype=torch.bool)
    sees[spoil:min(new, spoil + window)] = True
    group = s.hq // s.hk
    o = out.float().cpu()
    assert torch.isinf(o[sees][:, :, 5]).all() and torch.isnan(o[sees][:, group:, 9]).all()
    assert torch.isfinite(o[~sees]).all()
    # all else as with a finite value there
    s.values[0][pos, :, 5] = 0
    s.values[0][pos, 1, 9] = 0
    out[sees.cuda(), :, 5] = 0
    out[sees.cuda(), group:, 9] = 0
    keep = torch.ones_like(o, dtype=torch.bool)
    keep[:, :, 5] = keep[:, :, 9] = False
    a, b, c, reach = ref.attention(*(x.float().cpu().numpy() for x in (s.q, s.keys[0], s.values[0])), kv, window, sinks)
    tol, _ = ref.attention_bounds(a, c, reach, kv, s.dim, s.bf16)
    err = np.abs(out.float().cpu().numpy() - a)
    assert np.all((err <= tol)[keep.numpy()])


@pytest.mark.parametrize("dtype,new", [("bf16", 4), ("fp32", 4), ("bf16", 200)])
def test_malformed_requests_get_nan(dtype, new):
    """Bad lengths and pages spoil their own request only; nothing is read through them."""
    import torch
    log(f"[gpu-test] attention malformed {dtype} {new}")
    s = Setup((8, 2), 128, 16, dtype, [new] * 5, [210 + 16 * i for i in range(5)], seed=9)
    s.kv_len[1] = -3
    s.kv_len[2] = s.table.shape[1] * 16 + 1
    s.table[3, 4] = s.num
    out, lse = s.run(max_new=new)
    s.check(out, lse, skip=(1, 2, 3))
    for b in (1, 2):
        assert torch.isnan(out[b * new:(b + 1) * new]).all() and torch.isnan(lse[b * new:(b + 1) * new]).all()
    assert torch.isnan(out[4 * new - 1]).all()
    # more new tokens than announced, and rows outside the token arrays
    s = Setup((8, 2), 128, 16, dtype, [new, new], [300, 250], seed=10)
    s.q_start[2] = 2 * new + 5
    out, lse = s.run(max_new=new)
    s.check(out, lse, skip=(1,))
    assert torch.isnan(out[new:]).all()


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes, its last pages in use."""
    import torch
    from gru_corrected_draft_amd import verify
    log("[gpu-test] attention over a 4.3 GB cache")
    hk, dim, page = 8, 128, 64
    num = (1 << 31) // (hk * page * dim) + 40
    k, v = (torch.empty((num, hk, page, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n, new = 2000, 16
    op = verify.PagedAttention(8, hk, dim, page, max_requests=1)
    s = Setup((8, 8), dim, page, "bf16", [new], [n], seed=11)
    table = torch.arange(num - 1, num - 1 - 32, -1, dtype=torch.int32, device="cuda")[None]
    kv_len = torch.tensor([n], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    op.append(s.keys[0], s.values[0], k, v, table, kv_len, start)
    s.k_cache, s.v_cache, s.table = k, v, table
    s.check(*s.run(max_new=new))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_append_then_attend(dtype):
    """The append writes exactly the new rows, from strided tensors, and skips what is out of range."""
    import torch
    log(f"[gpu-test] append {dtype}")
    s = Setup((8, 2), 64, 16, dtype, [5, 0, 16, 3, 2], [40, 7, 16, 2, 30], seed=12)
    want_k, want_v = s.k_cache.clone(), s.v_cache.clone()
    # a fresh cache without the new rows; k and v as slices of one projection
    fused = torch.zeros((s.tokens, 2 * s.hk, s.dim), dtype=s.dtype, device="cuda")
    s.k_cache.nan_to_num_(nan=3.0)
    s.v_cache.nan_to_num_(nan=3.0)
    want_k.nan_to_num_(nan=3.0)
    want_v.nan_to_num_(nan=3.0)
    at = 0
    for b, (n, kv) in enumerate(zip(s.new, s.kv)):
        for t in range(n):
            pos = kv - n + t
            if pos >= 0:
                fused[at + t, :s.hk], fused[at + t, s.hk:] = s.keys[b][pos], s.values[b][pos]
                s.k_cache[s.table[b, pos // 16].long(), :, pos % 16] = 9.0
                s.v_cache[s.table[b, pos // 16].long(), :, pos % 16] = 9.0
            else:
                fused[at + t] = 55.0  # position -1: must not be written
        at += n
    s.table[4, 1] = s.num + 3  # the last request's page is out of range: nothing written
    pg = 28 // 16
    keep = s.k_cache.clone()
    s.op.append(fused[:, :s.hk], fused[:, s.hk:], s.k_cache, s.v_cache, s.table, s.kv_len, s.q_start)
    torch.cuda.synchronize()
    assert pg == 1
    nine = keep == 9.0
    changed = s.k_cache != keep
    assert not (changed & ~nine).any()
    for b in range(4):
        n = s.kv[b]
        for p in range(n):
            row = s.table[b, p // 16].long(), slice(None), p % 16
            assert torch.equal(s.k_cache[row], want_k[row]) and torch.equal(s.v_cache[row], want_v[row]), (b, p)


def test_large_scores_and_scale():
    """Scores in the thousands (one weight is all but 1), a scale of its own."""
    log("[gpu-test] attention of large scores")
    for dtype in ("bf16", "fp32"):
        s = Setup((8, 2), 128, 16, dtype, [16, 1], [200, 333], seed=13, k_scale=60.0)
        s.check(*s.run())
        s.check(*s.run(scale=0.003), scale=0.003)


def test_same_bits_each_time_on_another_stream_and_in_a_graph():
    import torch
    log("[gpu-test] attention on streams and in a graph")
    for new, kv in (([16, 1, 7], [900, 2500, 60]), ([300, 20], [900, 400])):
        s = Setup((32, 8), 128, 16, "bf16", new, kv, seed=14)
        kw = dict(max_new=max(new), max_kv=max(kv))
        want, want_l = s.run(**kw)
        for _ in range(3):
            out, lse = s.run(**kw)
            assert torch.equal(out, want) and torch.equal(lse, want_l)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            out, lse = s.run(**kw)
        side.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_l)
        held = torch.empty_like(s.q)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            s.op.run(s.q, s.k_cache, s.v_cache, s.table, s.kv_len, s.q_start, out=held, **kw)
        for i in range(3):
            held.zero_()
            g.replay()
            assert torch.equal(held, want)
            # other lengths through the same graph
            full = s.kv_len.clone()
            s.kv_len -= 40 + i
            g.replay()
            got = held.clone()
            eager, _ = s.run(**kw)
            assert torch.equal(got, eager)
            s.kv_len.copy_(full)
            torch.cuda.synchronize()


def test_many_requests_of_one_token():
    """More (request, key head) pairs than workgroups, ragged from one key to a few hundred."""
    rng = np.random.default_rng(15)
    kv = [int(x) for x in rng.integers(1, 300, 150)]
    log("[gpu-test] attention of 150 requests")
    s = Setup((8, 8), 64, 16, "bf16", [1] * 150, kv, seed=15)
    s.check(*s.run(max_new=1, max_kv=300))


def test_refusals():
    import torch
    from gru_corrected_draft_amd import rollout as R
    from gru_corrected_draft_amd import verify
    log("[gpu-test] attention refusals")
    for kw, status in (((7, 2, 128, 16), R.DOMINO_ERR_INVALID_CONFIG), ((8, 2, 96, 16), R.DOMINO_ERR_UNSUPPORTED),
                       ((8, 2, 128, 24), R.DOMINO_ERR_UNSUPPORTED), ((8, 2, 128, 8), R.DOMINO_ERR_UNSUPPORTED)):
        with pytest.raises(R.DominoError) as e:
            verify.PagedAttention(*kw)
        assert e.value.status == status
    s = Setup((8, 2), 128, 16, "bf16", [2, 3], [20, 30], seed=16)
    bad = [dict(q=s.q.float()), dict(q=s.q[:, :4]), dict(window=-1), dict(sinks=-1), dict(scale=0.0),
           dict(scale=float("nan")), dict(max_new=-1), dict(out=torch.empty_like(s.q).cpu()),
           dict(out=torch.empty_like(s.q).transpose(1, 2).contiguous().transpose(1, 2))]
    for kw in bad:
        with pytest.raises((ValueError, R.DominoError)):
            s.run(**kw)
    with pytest.raises(ValueError):
        s.op.run(s.q, s.k_cache, s.v_cache, s.table, s.kv_len.long(), s.q_start)
    with pytest.raises(ValueError):
        s.op.run(s.q, s.k_cache, s.v_cache[:-1], s.table, s.kv_len, s.q_start)
    with pytest.raises(ValueError):
        s.op.run(s.q, s.k_cache, s.v_cache.clone(memory_format=torch.contiguous_format).permute(0, 2, 1, 3)
                 .contiguous().permute(0, 2, 1, 3), s.table, s.kv_len, s.q_start)
    # tensors of no token at all
    out = s.op.run(s.q[:0], s.k_cache, s.v_cache, s.table, s.kv_len, torch.zeros_like(s.q_start))
    assert out.shape == (0, 8, 128)


def _ragged(n, least, most, seed):
    rng = np.random.default_rng(seed)
    return np.exp(rng.uniform(np.log(least), np.log(most + 1), n)).astype(int).clip(least, most).tolist()


# heads, dim, page, dtype, new, kv, window, sinks: the ways to divide the work among workgroups
PLANS = {
    # more requests than lanes, equal shares that end inside segments
    "shares of 70 requests": ((8, 2), 128, 16, "bf16", [1] * 70, [0, 1] + _ragged(68, 3, 1500, 1), 0, 0),
    "shares of 70 requests, window": ((8, 2), 64, 16, "bf16", [1, 2] * 35, _ragged(70, 2, 1500, 2), 300, 5),
    "shares of 70 blocks": ((8, 2), 128, 16, "bf16", [16, 0, 9, 1, 12] * 14, _ragged(70, 16, 900, 3), 0, 0),
    "shares of 20 requests": ((32, 8), 128, 32, "bf16", [1] * 20, _ragged(20, 1, 2500, 4), 0, 0),
    "shares of 20 blocks": ((32, 8), 128, 16, "bf16", [16, 3] * 10, _ragged(20, 16, 900, 5), 0, 0),
    "shares of 20 wide blocks": ((64, 8), 128, 64, "bf16", [16, 9] * 10, _ragged(20, 16, 900, 6), 400, 4),
    "shares of 20 wide blocks, 64": ((64, 8), 64, 64, "bf16", [16, 9] * 10, _ragged(20, 16, 900, 6), 0, 0),
    "shares of 30 blocks, 256": ((24, 8), 256, 16, "bf16", [16, 2, 1] * 10, _ragged(30, 16, 500, 7), 0, 0),
    # each segment cut into pieces of its own
    "pieces of one request": ((8, 2), 128, 16, "bf16", [1], [6001], 0, 0),
    "pieces of ragged requests": ((8, 2), 64, 16, "bf16", [1, 1, 0, 1, 1], [3, 5000, 70, 0, 900], 0, 0),
    "pieces of blocks": ((32, 8), 128, 16, "bf16", [16, 1, 16], [2500, 2000, 31], 0, 0),
    "pieces of wide blocks, window": ((64, 8), 128, 16, "bf16", [16, 4], [5000, 2111], 1500, 40),
    "pieces, 256": ((16, 2), 256, 64, "bf16", [1, 3], [3000, 700], 0, 0),
    "pieces of blocks, 256": ((16, 2), 256, 64, "bf16", [16, 3], [3000, 700], 900, 3),
    # prompts: shares of row tiles, and a workgroup for each
    "shares of a prompt": ((8, 2), 128, 16, "bf16", [333], [1700], 0, 0),
    "shares of prompts, window": ((8, 2), 64, 16, "bf16", [333, 20, 0, 270], [1700, 900, 4, 290], 200, 7),
    "shares of 70 prompts": ((8, 2), 64, 16, "bf16", [40, 0, 90, 1, 33] * 14, _ragged(70, 90, 400, 8), 0, 0),
    "a workgroup a row tile": ((8, 2), 64, 16, "bf16", [400] * 40, _ragged(40, 400, 700, 9), 0, 0),
    "a workgroup a row tile, window": ((8, 2), 128, 16, "bf16", [400] * 40, _ragged(40, 400, 700, 10), 100, 35),
    # fp32, keys dealt to several workgroups
    "fp32 parts": ((8, 2), 64, 16, "fp32", [7, 1, 0, 16], [2100, 900, 4, 17], 0, 0),
    "fp32 parts, window": ((8, 2), 128, 16, "fp32", [3, 1, 2], [2100, 900, 1], 700, 3),
    "fp32 parts, 256": ((4, 2), 256, 16, "fp32", [3, 1], [1100, 0], 0, 0),
}


@pytest.mark.parametrize("plan", PLANS)
def test_division_of_work(plan):
    heads, dim, page, dtype, new, kv, window, sinks = PLANS[plan]
    log(f"[gpu-test] attention {plan}")
    s = Setup(heads, dim, page, dtype, new, kv, seed=len(plan))
    s.check(*s.run(window=window, sinks=sinks, max_new=max(new), max_kv=max(kv)), window, sinks)


@pytest.mark.parametrize("heads,new,kv", [((8, 2), 1, 3000), ((8, 2), 16, 3000), ((16, 2), 16, 3000),
                                          ((8, 2), 200, 1500)])
def test_odd_values_in_every_division(heads, new, kv):
    """Infinities and NaN among values that all tokens see reach the result; those past a token's position
    do not, wherever the keys are divided."""
    import torch
    log(f"[gpu-test] attention odd values {heads} {new} {kv}")
    s = Setup(heads, 128, 16, "bf16", [new], [kv], seed=15)
    for pos, i, x in ((5, 0, float("inf")), (kv // 2, 1, float("-inf")), (kv - new, 2, float("nan")),
                      (kv - 1, 3, float("inf")), (7, 4, float("inf")), (kv // 2 + 1, 4, float("-inf"))):
        s.v_cache[s.table[0, pos // 16].long(), :, pos % 16, i] = x
        s.values[0][pos, :, i] = 0
    out, lse = s.run(max_new=new, max_kv=kv)
    torch.cuda.synchronize()
    o = out.float()
    assert (o[:, :, 0] == float("inf")).all() and (o[:, :, 1] == float("-inf")).all()
    assert torch.isnan(o[:, :, 2]).all() and torch.isnan(o[:, :, 4]).all()
    assert (o[-1, :, 3] == float("inf")).all() and torch.isfinite(o[:-1, :, 3]).all()
    a, _, c, reach = ref.attention(*(x.float().cpu().numpy() for x in (s.q, s.keys[0], s.values[0])), kv, 0, 0)
    tol, _ = ref.attention_bounds(a, c, reach, kv, s.dim, True)
    err = np.abs(o.cpu().numpy() - a)
    assert np.all((err <= tol)[:, :, 5:]) and np.all((err <= tol)[:-1, :, 3])


def test_fp32_parts_give_the_same_bits_again():
    """Whichever workgroup comes last joins the parts in their order: the same bits each time, on replays of a
    graph with other lengths in between, and for a smaller call after a larger one."""
    import torch
    log("[gpu-test] attention fp32 parts again")
    s = Setup((8, 2), 64, 16, "fp32", [7, 1, 16], [2100, 900, 333], seed=16)
    kw = dict(max_new=16, max_kv=2100)
    want, want_l = s.run(**kw)
    s.check(want, want_l)
    held = torch.empty_like(s.q)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        s.op.run(s.q, s.k_cache, s.v_cache, s.table, s.kv_len, s.q_start, out=held, **kw)
    full = s.kv_len.clone()
    for i in range(4):
        held.zero_()
        g.replay()
        assert torch.equal(held, want)
        s.kv_len -= 100 + i
        g.replay()
        got = held.clone()
        eager, _ = s.run(**kw)
        assert torch.equal(got, eager)
        s.kv_len.copy_(full)
        out, lse = s.run(**kw)
        assert torch.equal(out, want) and torch.equal(lse, want_l)
        torch.cuda.synchronize()


# prompts that are divided: many row tiles to a request, many requests, a window longer than a few steps
PROMPTS = {
    "75 row tiles": ((64, 1), 64, 16, "bf16", [300], [2000], 0, 0),
    "75 row tiles of two requests": ((64, 1), 64, 16, "bf16", [300, 7], [3000, 100], 0, 0),
    "70 requests": ((8, 2), 64, 16, "bf16", [40, 33] * 35, _ragged(70, 40, 2500, 11), 0, 0),
    "window": ((8, 2), 64, 16, "bf16", [333, 270], [2600, 2900], 1500, 7),
    "window, 128": ((8, 2), 128, 32, "bf16", [100, 0, 333], [2600, 5, 400], 1500, 70),
    "heads of 256": ((6, 2), 256, 32, "bf16", [150, 40], [900, 700], 0, 0),
    "heads of 256, window": ((6, 2), 256, 32, "bf16", [150], [1300], 700, 2),
    "heads of 256, undivided": ((8, 8), 256, 16, "bf16", [140] * 5, _ragged(5, 140, 400, 12), 0, 0),
}


@pytest.mark.parametrize("prompt", PROMPTS)
def test_divided_prompts(prompt):
    heads, dim, page, dtype, new, kv, window, sinks = PROMPTS[prompt]
    log(f"[gpu-test] attention prompt {prompt}")
    s = Setup(heads, dim, page, dtype, new, kv, seed=100 + len(prompt))
    s.check(*s.run(window=window, sinks=sinks, max_new=max(new), max_kv=max(kv)), window, sinks)
