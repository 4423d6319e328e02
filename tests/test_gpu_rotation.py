"""Norm and rotation of query and key heads, against 64 bits.

Bounds: with u = 2^-24, the sum of D squares, the root and the division put at most (D + 12) u on the factor
of the norm, the two products 2 u.  The angle's fraction of a turn is rounded once (half of 2^-24 turns, 3.2 u
radians), sine and cosine add at most 8 u, the magnitude u, the two products and the sum of a rotation 2 u, all
of (|a| + |b|) times the magnitude: (D + 30) u in all.  A bf16 result is rounded once more, by 2^-8 of itself."""
import numpy as np
import pytest

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


def _frequencies(rotary, base=1e6):
    return base ** (-np.arange(0, rotary, 2) / rotary)


def reference(x, positions, freq, weight, eps, interleaved, magnitude, bf16):
    """One kind of heads, x [tokens, heads, d], a pair at a time: the result and its bound."""
    x = np.asarray(x, np.float64)
    d, r = x.shape[-1], 2 * len(freq)
    y = x.copy()
    if weight is not None:
        y = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    out, size = y.copy(), np.abs(y)
    for j, f in enumerate(freq):
        i, k = (2 * j, 2 * j + 1) if interleaved else (j, j + r // 2)
        turn = (np.asarray(positions, np.longdouble) * np.longdouble(f)) % (2 * np.pi * np.longdouble(1))
        c, s = (np.float64(magnitude) * g(turn.astype(np.float64))[:, None] for g in (np.cos, np.sin))
        out[..., i], out[..., k] = y[..., i] * c - y[..., k] * s, y[..., k] * c + y[..., i] * s
        size[..., i] = size[..., k] = abs(magnitude) * (np.abs(y[..., i]) + np.abs(y[..., k]))
    tol = 2.0 ** -24 * (d + 30) * size + 1e-37
    if bf16:
        tol = tol + 2.0 ** -8 * (np.abs(out) + tol)
    return out, tol


def _check(got, x, positions, freq, weight, eps=1e-6, interleaved=False, magnitude=1.0):
    import torch
    torch.cuda.synchronize()
    bf16 = got.dtype == torch.bfloat16
    want, tol = reference(x.double().cpu().numpy(), positions.cpu().numpy(), freq,
                          None if weight is None else weight.double().cpu().numpy(), eps, interleaved, magnitude, bf16)
    err = np.abs(got.double().cpu().numpy() - want)
    there = positions.cpu().numpy() >= 0
    assert np.all(err[there] <= tol[there]), f"{np.max((err / tol)[there]):.3g} of the bound"


CASES = [
    # tokens, heads, dim, rotary, dtype, norm, interleaved, magnitude, far
    (1, (32, 8), 128, 128, "bf16", True, False, 1.0, 40000),
    (1, (1, 1), 64, 16, "fp32", True, False, 1.0, 1),
    (3, (7, 1), 64, 64, "bf16", True, True, 1.0, 100),
    (5, (5, 5), 128, 48, "fp32", True, True, 1.25, 2 ** 31 - 1),
    (17, (16, 2), 256, 256, "bf16", True, False, 0.5, 2 ** 20),
    (17, (16, 2), 256, 112, "fp32", True, False, 1.0, 2 ** 20),
    (33, (40, 8), 128, 64, "bf16", False, False, 1.0, 5000),
    (130, (8, 2), 64, 32, "fp32", False, True, 1.0, 5000),
    (1025, (32, 8), 128, 128, "bf16", True, False, 1.0, 9000),
    (2049, (8, 2), 64, 64, "bf16", True, False, 1.0, 9000),
    (4099, (6, 2), 128, 96, "bf16", True, True, 1.0, 9000),
    (2050, (3, 1), 256, 256, "fp32", True, False, 1.0, 9000),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c))
def test_against_64_bits(case):
    import torch
    from gru_corrected_draft_amd import verify
    tokens, (hq, hk), dim, rotary, dtype, norm, interleaved, magnitude, far = case
    log(f"[gpu-test] rotation {case}")
    g = torch.Generator(device="cuda").manual_seed(tokens)
    dt = _types()[dtype]
    qkv = (torch.randn((tokens, hq + 2 * hk, dim), generator=g, device="cuda") * 3).to(dt)
    q, k, _ = qkv.split([hq, hk, hk], 1)
    weights = [(1 + 0.3 * torch.randn(dim, generator=g, device="cuda")).to(dt) if norm else None for _ in range(2)]
    positions = torch.randint(0, far, (tokens,), generator=g, device="cuda").to(torch.int32)
    positions[-1] = far - 1
    freq = _frequencies(rotary)
    op = verify.HeadRotation(hq, hk, dim, freq, dt, interleaved, magnitude)
    a, b = op.run(q, k, positions, *weights)
    _check(a, q, positions, freq, weights[0], 1e-6, interleaved, magnitude)
    _check(b, k, positions, freq, weights[1], 1e-6, interleaved, magnitude)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("tokens", [6, 2500])
def test_padding_is_left_as_it_was(dtype, tokens):
    """Tokens with a negative position; outputs inside wider tensors, heads before tokens; in place."""
    import torch
    from gru_corrected_draft_amd import verify
    log(f"[gpu-test] rotation of a padded batch {dtype} {tokens}")
    dt = _types()[dtype]
    q, k = torch.randn(tokens, 4, 64, device="cuda").to(dt), torch.randn(tokens, 2, 64, device="cuda").to(dt)
    w = torch.randn(64, device="cuda").to(dt)
    positions = torch.arange(tokens, device="cuda", dtype=torch.int32)
    positions[1::3] = -1
    positions[-1] = -2 ** 31
    freq = _frequencies(32)
    op = verify.HeadRotation(4, 2, 64, freq, dt)
    wide = [torch.full((n, tokens, 64 + 16), 7.0, dtype=dt, device="cuda") for n in (4, 2)]
    outs = [x[:, :, :64].transpose(0, 1) for x in wide]
    got = op.run(q, k, positions, w, w, out_q=outs[0], out_k=outs[1])
    for x, y, o in zip((q, k), got, wide):
        _check(y, x, positions, freq, w)
        assert torch.all(o[:, :, 64:] == 7) and torch.all(y[positions < 0] == 7)
    want = [x.clone() for x in got]
    same = op.run(q, k, positions, w, w, out_q=q, out_k=k)
    assert same[0] is q and same[1] is k
    there = positions >= 0
    assert torch.equal(q[there], want[0][there]) and torch.equal(k[there], want[1][there])


def test_zeros_large_numbers_and_nan():
    """A head of zeros stays zero (eps), one of small numbers is lifted, a NaN stays in its head."""
    import torch
    from gru_corrected_draft_amd import verify
    log("[gpu-test] rotation of special heads")
    q, k = torch.randn(4, 8, 128, device="cuda"), torch.randn(4, 2, 128, device="cuda")
    q[0, 1] = 0
    q[1, 2] *= 1e-6
    q[2, 3] *= 1e17
    q[3, 4, 77] = float("nan")
    w = torch.ones(128, device="cuda")
    positions = torch.tensor([0, 5, 1000, 77], dtype=torch.int32, device="cuda")
    freq = _frequencies(128, 1e4)
    a, b = verify.HeadRotation(8, 2, 128, freq, torch.float32).run(q, k, positions, w, w)
    assert torch.all(a[0, 1] == 0) and torch.isnan(a[3, 4]).all() and torch.isnan(a).sum() == 128
    q[3, 4] = a[3, 4] = 0
    _check(a, q, positions, freq, w)
    _check(b, k, positions, freq, w)


def test_rows_depend_on_themselves_alone():
    """The same token gives the same bits alone and among thousands, at either grid."""
    import torch
    from gru_corrected_draft_amd import verify
    log("[gpu-test] rotation, one token and many")
    q, k = torch.randn(3001, 32, 128, device="cuda").bfloat16(), torch.randn(3001, 8, 128, device="cuda").bfloat16()
    w = torch.randn(128, device="cuda").bfloat16()
    positions = torch.randint(0, 40000, (3001,), device="cuda", dtype=torch.int32)
    op = verify.HeadRotation(32, 8, 128, _frequencies(128))
    a, b = op.run(q, k, positions, w, w)
    for i in (0, 1, 1777, 3000):
        one = op.run(q[i:i + 1], k[i:i + 1], positions[i:i + 1], w, w)
        assert torch.equal(one[0][0], a[i]) and torch.equal(one[1][0], b[i])
    assert op.run(q[:0], k[:0], positions[:0], w, w)[0].shape == (0, 32, 128)


def test_graph_and_other_stream():
    import torch
    from gru_corrected_draft_amd import verify
    log("[gpu-test] rotation in a graph")
    q, k = torch.randn(64, 32, 128, device="cuda").bfloat16(), torch.randn(64, 8, 128, device="cuda").bfloat16()
    w = torch.randn(128, device="cuda").bfloat16()
    positions = torch.arange(64, device="cuda", dtype=torch.int32)
    op = verify.HeadRotation(32, 8, 128, _frequencies(128))
    outs = torch.empty_like(q), torch.empty_like(k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        op.run(q, k, positions, w, w, out_q=outs[0], out_k=outs[1])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.run(q, k, positions, w, w, out_q=outs[0], out_k=outs[1])
    for i in range(4):
        q.copy_(torch.randn(q.shape, device="cuda"))
        positions += 1000
        graph.replay()
        torch.cuda.synchronize()
        eager = op.run(q, k, positions, w, w)
        assert torch.equal(eager[0], outs[0]) and torch.equal(eager[1], outs[1])
