"""The cache in 4 bits: append, read and attention, against 64 bits over the numbers that it stands for.

bf16 holds those numbers exactly, so the attention's bounds are those of a bf16 cache
(``_verify_ref.attention_bounds``); what append stores and read gives back is compared bit by bit."""
import numpy as np
import pytest

from tests import _fp4_ref as fp4
from tests import _verify_ref as ref
from tests._gpu import log

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def _cuda(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


class Setup:
    """Random keys and values of some requests in shuffled pages; whatever no request owns is NaN."""

    def __init__(self, heads, dim, page, new, kv, seed=0, order="phb", extra_width=0, size=1.0):
        import torch
        from gru_corrected_draft_amd import verify
        rng = np.random.default_rng(seed)
        self.hq, self.hk = heads
        self.dim, self.page, self.new, self.kv, self.tokens = dim, page, list(new), list(kv), sum(new)
        self.q = _cuda(rng.standard_normal((self.tokens, self.hq, dim)).astype(np.float32)).bfloat16()
        self.op = verify.PagedAttention4(self.hq, self.hk, dim, page, max_requests=max(1, len(kv)))
        pages = [-(-n // page) for n in kv]
        self.num = sum(pages) + 2
        perm = rng.permutation(self.num).astype(np.int32)
        self.table = torch.full((len(kv), max(max(pages), 1) + extra_width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = _cuda(perm[at:at + n])
            at += n
        dims = {"p": self.num, "h": self.hk, "b": self.op.page_bytes}
        both = torch.full((2,) + tuple(dims[c] for c in order), 255, dtype=torch.uint8, device="cuda")
        back = [1 + order.index(c) for c in "phb"]
        self.k_cache, self.v_cache = (both.permute(0, *back)[i] for i in (0, 1))
        scale = rng.uniform(0.3, 2.0, (self.hk, dim)) * size
        self.keys, self.values = ([], [])
        for cache, rows in ((self.k_cache, self.keys), (self.v_cache, self.values)):
            for b, n in enumerate(kv):
                x = rng.standard_normal((n, self.hk, dim)) * scale
                rows.append(fp4.stored(x) if n else x)
                self.write(cache, b, np.arange(n), x)
        self.kv_len = torch.tensor(kv, dtype=torch.int32, device="cuda")
        self.q_start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")

    def places(self, b, pos):
        import torch
        pos = torch.as_tensor(pos, device="cuda").long()
        page, row = self.table[b].long()[pos // self.page], pos % self.page
        data = (row * (self.dim // 2))[:, None, None] + torch.arange(self.dim // 2, device="cuda")
        power = (self.page * (self.dim // 2) + row * (self.dim // 32))[:, None, None] + torch.arange(self.dim // 32, device="cuda")
        return page[:, None, None], torch.arange(self.hk, device="cuda")[None, :, None], data, power

    def write(self, cache, b, pos, x):
        if len(pos):
            page, head, data, power = self.places(b, pos)
            d, p = fp4.row_bytes(x)
            cache[page, head, data] = _cuda(d)
            cache[page, head, power] = _cuda(p)

    def bytes_at(self, cache, b, pos):
        page, head, data, power = self.places(b, pos)
        return cache[page, head, data].cpu().numpy(), cache[page, head, power].cpu().numpy()

    @property
    def where(self):
        return self.k_cache, self.v_cache, self.table, self.kv_len, self.q_start

    def run(self, **kw):
        return self.op.run(kw.pop("q", self.q), *self.where, return_lse=True, **kw)

    def check(self, out, lse, window=0, sinks=0, scale=None, skip=()):
        import torch
        torch.cuda.synchronize()
        out, lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        q = self.q.float().cpu().numpy()
        start = 0
        for b, n in enumerate(self.new):
            rows = slice(start, start + n)
            start += n
            if b in skip or n == 0:
                continue
            kv = self.kv[b]
            o, l, a, reach = ref.attention(q[rows], self.keys[b], self.values[b], kv, window, sinks, scale)
            tol, tol_l = ref.attention_bounds(o, a, reach, kv, self.dim, True)
            worst = np.max(np.abs(out[rows] - o) / tol)
            assert np.all(np.abs(out[rows] - o) <= tol), f"request {b}: {worst:.3g} of the bound"
            empty = np.isneginf(l)
            assert np.array_equal(np.isneginf(lse[rows]), empty), f"request {b}"
            assert np.all(np.abs(np.where(empty, 0, lse[rows]) - np.where(empty, 0, l)) <= tol_l), f"request {b}"


CASES = [
    # heads, dim, page, new, kv, window, sinks
    ((32, 8), 128, 16, [1], [1], 0, 0),
    ((32, 8), 128, 16, [1], [37], 0, 0),
    ((32, 8), 128, 16, [1, 1, 1, 1], [31, 32, 33, 1000], 0, 0),
    ((8, 8), 64, 16, [1, 1], [77, 260], 0, 0),
    ((16, 2), 256, 16, [1, 2], [90, 300], 0, 0),
    ((7, 1), 128, 32, [3], [200], 33, 0),
    ((64, 1), 128, 16, [1], [500], 0, 0),
    ((32, 8), 128, 16, [16, 16], [16, 700], 0, 0),
    ((32, 8), 128, 64, [16, 5, 1, 0, 16], [129, 128, 127, 50, 400], 0, 0),
    ((40, 8), 128, 64, [16], [515], 0, 0),
    ((40, 8), 128, 32, [16, 16], [515, 90], 100, 4),
    ((8, 8), 64, 16, [3, 16], [77, 260], 0, 0),
    ((8, 4), 64, 16, [1, 32], [777, 260], 48, 70),
    ((16, 2), 256, 16, [1, 16], [90, 300], 0, 0),
    ((16, 2), 256, 128, [4], [1000], 64, 1),
    ((100, 1), 64, 32, [2], [90], 0, 0),
    # prompts: many row tiles, ragged
    ((32, 8), 128, 16, [200, 33], [200, 300], 0, 0),
    ((8, 2), 128, 64, [513], [700], 0, 0),
    ((8, 2), 128, 64, [300, 100], [500, 100], 64, 5),
    ((8, 2), 128, 64, [300], [300], 1, 0),
    ((6, 2), 64, 16, [350, 1], [350, 400], 0, 0),
    ((6, 2), 256, 32, [150], [161], 0, 0),
    ((6, 2), 256, 32, [150], [361], 50, 2),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c))
def test_against_64_bits(case):
    heads, dim, page, new, kv, window, sinks = case
    log(f"[gpu-test] attention over 4 bits {case}")
    s = Setup(heads, dim, page, new, kv, seed=sum(kv))
    s.check(*s.run(window=window, sinks=sinks), window, sinks)
    # tighter bounds choose other kernels for the same result
    s.check(*s.run(window=window, sinks=sinks, max_new=max(new), max_kv=max(kv)), window, sinks)


# every way the keys are divided among workgroups: few and many requests, long and short, beyond 64
@pytest.mark.parametrize("heads,dim,new,kv", [
    ((8, 2), 128, [1] * 70, [5 + 37 * (i % 9) for i in range(70)]),
    ((8, 2), 128, [1] * 3, [4000, 1, 2500]),
    ((4, 1), 64, [1] * 70, [3 + 101 * (i % 9) for i in range(70)]),
    ((4, 1), 128, [2, 0, 1] * 27, [900, 0, 350] * 27),
    ((16, 8), 128, [1] * 40, [40 + 90 * (i % 7) for i in range(40)]),
    ((16, 8), 128, [4] * 40, [40 + 90 * (i % 7) for i in range(40)]),
    ((8, 1), 64, [16] * 3, [3000, 16, 900]),
    ((16, 4), 128, [16, 7], [2500, 700]),
    ((8, 2), 256, [16, 9], [1500, 30]),
    ((8, 2), 128, [300], [2100]),
])
def test_divided_keys(heads, dim, new, kv):
    log(f"[gpu-test] attention over 4 bits, divided {heads} {dim} {len(new)} requests")
    s = Setup(heads, dim, 16, new, kv, seed=3)
    s.check(*s.run(max_new=max(new), max_kv=max(kv)))


# numbers far from 1: powers at the ends of what append gives and between
@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** -20, 2.0 ** 30])
@pytest.mark.parametrize("new", [1, 16])
def test_powers(size, new):
    log(f"[gpu-test] attention over 4 bits, numbers of {size:.3g}")
    s = Setup((8, 2), 128, 16, [new], [100], seed=4, size=size)
    out, lse = s.run(scale=0.09 / size)
    s.check(out, lse, scale=0.09 / size)


@pytest.mark.parametrize("order", ["hpb"])
def test_cache_orders_and_strided_rows(order):
    """A cache in another order of pages and heads; q and out inside wider tensors."""
    import torch
    log(f"[gpu-test] attention over 4 bits, cache order {order}")
    s = Setup((8, 2), 128, 16, [5, 16], [90, 333], seed=5, order=order)
    wide = torch.zeros((s.tokens, 3, s.hq, s.dim), dtype=torch.bfloat16, device="cuda")
    wide[:, 1] = s.q
    out = torch.full((s.hq, s.tokens, s.dim + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    got, lse = s.run(q=wide[:, 1], out=out[:, :, :s.dim].transpose(0, 1))
    s.check(got, lse)
    assert torch.all(out[:, :, s.dim:] == 7)


def test_few_keys_and_no_keys():
    log("[gpu-test] attention over 4 bits of few keys")
    s = Setup((8, 2), 128, 16, [3, 4, 1, 2], [0, 2, 1, 40], seed=6)
    out, lse = s.run()
    s.check(out, lse)
    assert (out[:3] == 0).all() and (lse[:3] == float("-inf")).all()
    assert (out[3:5] == 0).all() and (lse[3:5] == float("-inf")).all()


@pytest.mark.parametrize("new,max_new", [(1, 1), (8, 8), (16, 16), (16, 200), (100, 100)])
def test_blocks_of_nan(new, max_new):
    """A block of NaN among the values reaches the tokens that see it, in its 32 elements alone; one among
    the keys all of theirs.  Unseen rows and pages may hold anything."""
    import torch
    log(f"[gpu-test] attention over 4 bits, blocks of NaN {new} {max_new}")
    kv, window, sinks = 300, 40, 2
    s = Setup((8, 2), 128, 32, [new], [kv], seed=8)
    first = kv - new - window + 1  # the first key that any token sees past the sinks
    spoil = new // 2
    pos = kv - new + spoil
    s.write(s.v_cache, 0, [pos], np.where(np.arange(128) == 40, np.nan, s.values[0][pos]) [None])
    unseen = np.arange(first // 32 * 32, first)
    for cache in (s.k_cache, s.v_cache):
        s.write(cache, 0, unseen, np.full((len(unseen), 2, 128), np.inf))
    for i in range(1, first // 32):
        s.table[0, i] = -1 if i % 2 else 2 ** 30  # pages of evicted keys
    out, lse = s.run(window=window, sinks=sinks, max_new=max_new)
    torch.cuda.synchronize()
    sees = np.zeros(new, bool)
    sees[spoil:min(new, spoil + window)] = True
    o = out.float().cpu().numpy()
    assert np.isnan(o[sees][:, :, 32:64]).all() and np.isfinite(o[~sees]).all()
    a, b, c, reach = ref.attention(s.q.float().cpu().numpy(), s.keys[0], s.values[0], kv, window, sinks)
    tol, tol_l = ref.attention_bounds(a, c, reach, kv, s.dim, True)
    keep = np.ones_like(o, bool)
    keep[sees, :, 32:64] = False
    assert np.all((np.abs(o - a) <= tol)[keep])
    assert np.all(np.abs(lse.cpu().numpy() - b) <= tol_l)
    # the same key in one head
    s.write(s.k_cache, 0, [pos], np.where(np.arange(2)[:, None] == 1, np.inf, s.keys[0][pos])[None])
    out, lse = s.run(window=window, sinks=sinks, max_new=max_new)
    assert torch.isnan(out[torch.as_tensor(sees).cuda()][:, 4:]).all()
    assert torch.isfinite(out[torch.as_tensor(~sees).cuda()]).all()


@pytest.mark.parametrize("new", [4, 16, 200])
def test_malformed_requests_get_nan(new):
    import torch
    log(f"[gpu-test] attention over 4 bits, malformed {new}")
    s = Setup((8, 2), 128, 16, [new] * 5, [210 + 16 * i for i in range(5)], seed=9)
    s.kv_len[1] = -3
    s.kv_len[2] = s.table.shape[1] * 16 + 1
    s.table[3, 4] = s.num
    out, lse = s.run(max_new=new)
    s.check(out, lse, skip=(1, 2, 3))
    for b in (1, 2):
        assert torch.isnan(out[b * new:(b + 1) * new]).all() and torch.isnan(lse[b * new:(b + 1) * new]).all()
    assert torch.isnan(out[4 * new - 1]).all()


def _numbers():
    """bf16 rows of 64 that meet every rounding: all significands over many powers, ties, zeros of both
    signs, the smallest and the largest numbers, numbers that are not finite."""
    rng = np.random.default_rng(11)
    rows = []
    for e in (-133, -126, -125, -60, -3, 0, 1, 5, 100, 124, 127):
        m = (1 + np.arange(128) / 128) * 2.0 ** e
        for top in (1.0, 1.5, 1.75, 1.7578125, 1.9921875):
            x = m.copy()
            x[::32] = top * 2.0 ** min(e + rng.integers(0, 4), 127)
            rows.append(np.where(rng.random(128) < 0.5, -x, x).reshape(2, 64))
    grid = np.array([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 6.9375])
    for e in (-100, -2, 0, 9):
        rows.append(np.concatenate([grid, -grid, grid[::-1], np.full(16, 6.5)] * 2).reshape(2, 64) * 2.0 ** e)
    rows.append(np.concatenate([np.zeros(32), np.full(32, -0.0), np.full(64, 2.0 ** -133)]).reshape(2, 64))
    for bad in (np.inf, -np.inf, np.nan):
        x = rng.standard_normal(128)
        x[rng.integers(0, 32)] = bad
        rows.append(x.reshape(2, 64))
    rows += list(rng.standard_normal((40, 2, 64)) * 2.0 ** rng.integers(-20, 20, (40, 1, 1)))
    return np.array(rows)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_append_and_read(dim):
    """The append writes exactly the new rows, from strided tensors, to the bit; read gives them back."""
    import torch
    log(f"[gpu-test] append of 4 bits {dim}")
    x = _numbers()
    n = len(x)
    wide = torch.from_numpy(np.concatenate([np.roll(x, i, 0) for i in range(dim // 64)], -1)).cuda().bfloat16()
    new = [n - 20, 0, 12, 8]
    s = Setup((4, 2), dim, 16, new, [n - 20 + 5, 7, 12, 90], seed=12, extra_width=2)
    before = s.k_cache.clone(), s.v_cache.clone()
    fused = torch.zeros((n, 6, dim), dtype=torch.bfloat16, device="cuda")
    fused[:, 2:4], fused[:, 4:] = wide, wide.flip(0)
    s.op.append(fused[:, 2:4], fused[:, 4:], *s.where, max_new=max(new))
    k, v = s.op.read(n, *s.where, max_new=max(new))
    want = wide.double().cpu().numpy()
    for cache, old, got, x in ((s.k_cache, before[0], k, want), (s.v_cache, before[1], v, want[::-1])):
        start = 0
        for b, m in enumerate(new):
            pos = np.arange(s.kv[b] - m, s.kv[b])
            rows = x[start:start + m]
            start += m
            if m == 0:
                continue
            data, power = s.bytes_at(cache, b, pos)
            want_data, want_power = fp4.row_bytes(rows)
            assert np.array_equal(power, want_power)
            assert np.array_equal(fp4.row_values(data, power), fp4.stored(rows), equal_nan=True)
            assert np.array_equal(data, want_data)
            s.write(old, b, pos, rows)
        assert torch.equal(cache, old)  # nothing besides
        assert np.array_equal(got.double().cpu().numpy(), fp4.stored(x), equal_nan=True)
    # a power of 255 is NaN whatever the elements
    assert np.isnan(fp4.stored(want)).any() and np.isinf(want).any()


def test_append_and_read_out_of_range():
    """Rows of malformed requests, at negative positions and in absent pages: not written, NaN when read."""
    import torch
    log("[gpu-test] append of 4 bits, out of range")
    s = Setup((4, 2), 64, 16, [3, 4, 2, 5], [40, 2, 30, 20], seed=13)
    s.kv_len[0] = 10_000
    s.table[2, 1] = s.num
    before = s.k_cache.clone(), s.v_cache.clone()
    x = torch.randn(14, 2, 64, device="cuda").bfloat16()
    s.op.append(x, x, *s.where)
    k, v = s.op.read(14, *s.where)
    there = torch.zeros(14, dtype=torch.bool)
    there[5:7] = there[9:] = True
    want = fp4.stored(x.double().cpu().numpy())
    for got in (k, v):
        got = got.double().cpu().numpy()
        assert np.isnan(got[~there.numpy()]).all() and np.array_equal(got[there.numpy()], want[there.numpy()])
    for cache, old in ((s.k_cache, before[0]), (s.v_cache, before[1])):
        s.write(old, 1, np.arange(2), x[5:7].double().cpu().numpy())
        s.write(old, 3, np.arange(15, 20), x[9:].double().cpu().numpy())
        assert torch.equal(cache, old)
    # rows past the last request are left as they were
    s = Setup((4, 2), 64, 16, [3], [40], seed=14)
    out = torch.full((6, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    s.run(q=torch.randn(6, 4, 64, device="cuda").bfloat16(), out=out)
    assert (out[3:] == 5).all() and not (out[:3] == 5).all()


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes, its last pages in use."""
    import torch
    log("[gpu-test] attention over a 4.3 GB cache of 4 bits")
    s = Setup((8, 8), 128, 64, [16], [2000], seed=11)
    num = (1 << 32) // (8 * s.op.page_bytes) + 40
    k, v = (torch.empty((num, 8, s.op.page_bytes), dtype=torch.uint8, device="cuda") for _ in range(2))
    table = torch.arange(num - 1, num - 1 - 32, -1, dtype=torch.int32, device="cuda")[None]
    x, y = (torch.from_numpy(r[0]).cuda().bfloat16() for r in (s.keys, s.values))
    start = torch.tensor([0, 2000], dtype=torch.int32, device="cuda")
    s.op.append(x, y, k, v, table, s.kv_len, start)
    s.k_cache, s.v_cache, s.table = k, v, table
    got = s.op.read(2000, k, v, table, s.kv_len, start)
    assert torch.equal(got[0], x) and torch.equal(got[1], y)
    s.check(*s.run(max_new=16))


@pytest.mark.parametrize("new,kv", [([1] * 8, [3000] * 8), ([16, 16], [900, 40]), ([200], [200])])
def test_graph_replays_match_eager_runs(new, kv):
    """Append and attention in a graph, replayed over changed inputs with eager work in between."""
    import torch
    log(f"[gpu-test] 4 bits in a graph {new[:2]} {kv[:2]}")
    s = Setup((8, 2), 128, 16, new, kv, seed=15)
    k, v = (torch.randn(s.tokens, 2, 128, device="cuda").bfloat16() for _ in range(2))
    bounds = dict(max_new=max(new), max_kv=max(kv))
    out = torch.empty_like(s.q)

    def step():
        s.op.append(k, v, *s.where, **bounds)
        s.op.run(s.q, *s.where, out=out, **bounds)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        for t in (k, v, s.q):
            t.copy_(torch.randn(t.shape, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        out.zero_()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out)
        (got.float() @ got.float().transpose(1, 2).contiguous()).sum().item()
