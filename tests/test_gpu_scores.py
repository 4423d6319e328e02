"""Log-probabilities of tokens, entropies and likeliest ids, against 64 bits.

Bounds, with u = 2^-24, y = (x - m) log2 e, p the probabilities and n the logits that one lane adds up at most:
an exponential is off by 2 u (|y| + 1) of itself, so the sum l by u (2 E|y| + 2) and u (n + 40) for the
additions; its logarithm by 2 u of itself, and x - m by u of itself.  The second sum, of e^y y, is off by u (2 E y^2 +
4 E|y|) for its terms and u (n + 40) E|y| for the additions, and takes the sum's error along in the quotient."""
import numpy as np
import pytest

from tests._gpu import log

pytestmark = pytest.mark.gpu
U, LOG2E = 2.0 ** -24, 1 / np.log(2)


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def _types():
    import torch
    return {"bf16": torch.bfloat16, "fp32": torch.float32}


def check(got, logits, tokens, top):
    import torch
    torch.cuda.synchronize()
    logprob, entropy, ids, values = (None if x is None else x.cpu().numpy().astype(np.float64) for x in got)
    x = logits.double().cpu().numpy()
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, float(np.finfo(np.float32).max)))
    rows, vocab = x.shape
    n = 8 * -(-vocab // 2048)
    for i in range(rows):
        row, m = x[i], x[i].max()
        order = np.argsort(-row, kind="stable")[:top]
        order = order[row[order] > -np.inf]
        if m == -np.inf:
            lp, h, tol, tol_h = np.full(vocab, -np.inf), 0.0, np.zeros(vocab), 0.0
        else:
            z = row - m
            e = np.exp(z)
            lp = z - np.log(e.sum())
            p = e / e.sum()
            y = np.where(p > 0, z * LOG2E, 0)
            s1, s2 = (p * np.abs(y)).sum(), (p * y * y).sum()
            h = -(p * np.where(p > 0, lp, 0)).sum()
            tol_l = U * (2 * s1 + n + 42)
            tol = tol_l + U * (2 * np.abs(np.where(np.isfinite(z), z, 0)) + 2 * np.log(e.sum()) + 2)
            tol_h = tol_l * (1 + s1) + U * (2 * s2 + (n + 44) * s1 + 2 * np.log(e.sum()) + 2 * h + 2)
        if tokens is not None:
            t = int(tokens[i])
            want = lp[t] if 0 <= t < vocab else -np.inf
            if np.isneginf(want):
                assert np.isneginf(logprob[i]), i
            else:
                assert abs(logprob[i] - want) <= tol[t], (i, logprob[i], want, tol[t])
        assert abs(entropy[i] - h) <= tol_h, (i, entropy[i], h, tol_h)
        if top:
            k = len(order)
            assert np.array_equal(ids[i, :k], order), (i, ids[i], order)
            assert np.all(np.abs(values[i, :k] - lp[order]) <= tol[order]), i
            assert np.all(ids[i, k:] == -1) and np.all(np.isneginf(values[i, k:])), i


def _logits(rows, vocab, dtype, seed, size=3.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((rows, vocab), generator=g, device="cuda") * size).to(_types()[dtype]), g


CASES = [
    # rows, vocab, dtype, top
    (1, 1, "bf16", 1), (2, 3, "fp32", 5), (5, 33, "bf16", 20), (3, 64, "fp32", 64), (3, 65, "fp32", 64),
    (1, 151936, "bf16", 20), (1, 151936, "fp32", 64), (3, 50257, "bf16", 5), (17, 50257, "fp32", 1),
    (7, 4096, "bf16", 64), (40, 5003, "bf16", 7), (130, 2049, "fp32", 3), (600, 5003, "bf16", 0),
    (2100, 300, "fp32", 2), (3, 500001, "bf16", 33),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(x) for x in c))
def test_against_64_bits(case):
    import torch
    from gru_corrected_draft_amd import verify
    rows, vocab, dtype, top = case
    log(f"[gpu-test] scores {case}")
    x, g = _logits(rows, vocab, dtype, rows + vocab)
    tokens = torch.randint(-1, vocab + 1, (rows,), generator=g, device="cuda").to(torch.int32)
    op = verify.TokenScores(vocab, _types()[dtype], max_rows=rows)
    check(op.run(x, tokens, top=top), x, tokens, top)
    # without tokens; rows apart, at an odd address
    wide = torch.full((rows, vocab + 3), 50.0, dtype=x.dtype, device="cuda")
    wide[:, 1:vocab + 1] = x
    got = op.run(wide[:, 1:vocab + 1], top=top)
    assert got[0] is None
    check(got, x, None, top)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("vocab", [97, 5003, 70000])
def test_masks_and_special_logits(dtype, vocab):
    """Rows with few ids or none, infinities, NaN (signaling too), the type's lowest value, equal logits."""
    import torch
    from gru_corrected_draft_amd import verify
    log(f"[gpu-test] scores of special rows {dtype} {vocab}")
    inf, low = float("inf"), torch.finfo(_types()[dtype]).min
    x, g = _logits(16, vocab, dtype, 3)
    x[0] = -inf
    x[1] = -inf
    x[1, 41] = -2.0                               # an only candidate
    x[2, :] = low
    x[2, [5, 90]] = torch.tensor([1.5, 1.5], dtype=x.dtype, device="cuda")
    x[3] = low                                    # all alike
    x[4] = 0.25
    x[5, 7] = inf
    x[5, 60] = inf
    x[6, 3::2] = float("nan")
    x[7] = float("nan")
    x[8] = -inf
    x[8, 20:31] = torch.arange(11, device="cuda").to(x.dtype)  # fewer ids than asked for, in one place
    x[9] = -inf
    x[9, 10:90] = -30000.0                        # many equal ones in few groups
    x[10] = torch.linspace(-20, 20, vocab, device="cuda").to(x.dtype)
    x[11] = torch.linspace(20, -20, vocab, device="cuda").to(x.dtype)
    x[12] = torch.arange(vocab, device="cuda").remainder(3).to(x.dtype)
    x[13] = torch.where(torch.arange(vocab, device="cuda") % 2 == 0, 0.0, -0.0).to(x.dtype)  # zeros of both signs
    kind = torch.int16 if dtype == "bf16" else torch.int32
    x[14].view(kind)[::5] = 0x7F81 if dtype == "bf16" else 0x7F800001  # signaling NaN
    x[15].view(kind)[1::7] = -0x7F if dtype == "bf16" else -0x7FFFFF
    tokens = torch.tensor([3, 41, 90, 1, vocab - 1, 60, 3, 8, 25, 11, vocab // 2, 0, 2, 96, 5, 8], dtype=torch.int32, device="cuda")
    op = verify.TokenScores(vocab, _types()[dtype], max_rows=16)
    for top in (1, 20, 64):
        got = op.run(x, tokens, top=top)
        check(got, x, tokens, top)
    # an only candidate is certain
    assert got[0][1] == 0 and got[1][1] == 0 and got[3][1, 0] == 0


def test_many_equal_logits_over_a_large_vocabulary():
    """Lists overflow: the bar is found bit by bit."""
    import torch
    from gru_corrected_draft_amd import verify
    log("[gpu-test] scores of equal logits, 151936 ids")
    x = torch.zeros((300, 151936), device="cuda").bfloat16()
    x[1::2] = torch.randint(0, 4, (150, 151936), device="cuda").bfloat16()
    x[2, 100000:] = 1.0
    tokens = torch.arange(300, device="cuda", dtype=torch.int32)
    op = verify.TokenScores(151936, max_rows=300)
    got = op.run(x, tokens, top=20)
    rows = [0, 1, 2, 3, 298, 299]
    check([t[rows] for t in got], x[rows], tokens[rows], 20)


def test_rows_depend_on_themselves_alone():
    import torch
    from gru_corrected_draft_amd import verify
    log("[gpu-test] scores, one row and many")
    x, _ = _logits(500, 50257, "bf16", 5)
    tokens = torch.arange(500, device="cuda", dtype=torch.int32)
    op = verify.TokenScores(50257, max_rows=500)
    many = op.run(x, tokens, top=10)
    again = op.run(x, tokens, top=10)
    for a, b in zip(many, again):
        assert torch.equal(a, b)
    few = op.run(x[77:80], tokens[77:80], top=10)
    check(few, x[77:80], tokens[77:80], 10)
    assert torch.equal(few[2], many[2][77:80])
    assert op.run(x[:0], tokens[:0], top=3)[2].shape == (0, 3)
    one = op.run(x[:1].expand(9, -1), tokens[:9], top=2)  # a row for all
    check(one, x[:1].expand(9, -1), tokens[:9], 2)


def test_offsets_past_32_bits():
    """Rows whose logits begin beyond 2^32 bytes."""
    import torch
    from gru_corrected_draft_amd import verify
    log("[gpu-test] scores of rows 4.4 GB apart")
    big = torch.empty((2, 1_100_000_000), dtype=torch.bfloat16, device="cuda")
    x, _ = _logits(2, 5003, "bf16", 6)
    big[:, :5003] = x
    tokens = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    wide = big.view(-1).as_strided((2, 5003), (2_199_990_000 - 5003, 1))
    wide[1] = x[1]
    check(verify.TokenScores(5003, max_rows=2).run(wide, tokens, top=9), x, tokens, 9)


def test_graph_replays_match_eager_runs():
    import torch
    from gru_corrected_draft_amd import verify
    log("[gpu-test] scores in a graph")
    x, _ = _logits(20, 50257, "bf16", 7)
    tokens = torch.arange(20, device="cuda", dtype=torch.int32)
    op = verify.TokenScores(50257, max_rows=20)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        op.run(x, tokens, top=8)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = op.run(x, tokens, top=8)
    for i in range(4):
        x.copy_(torch.randn(x.shape, device="cuda") * (i + 1))
        tokens += 3
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b in zip(got, op.run(x, tokens, top=8)):
            assert torch.equal(a, b)
        check(got, x, tokens, 8)


def test_many_rows_of_a_very_large_vocabulary():
    """Rows enough for a workgroup each, with more groups than its memory holds maxima of."""
    import torch
    from gru_corrected_draft_amd import verify
    rows, vocab, top = 521, 270001, 9
    log(f"[gpu-test] scores of {rows} rows of {vocab}")
    x, g = _logits(rows, vocab, "bf16", 12)
    x[3] = float("-inf")
    x[4, 100:] = float("-inf")
    x[520, :] = 1.0
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda").to(torch.int32)
    got = verify.TokenScores(vocab, torch.bfloat16, max_rows=rows).run(x, tokens, top=top)
    pick = torch.tensor([0, 1, 3, 4, 100, 255, 256, 300, 511, 512, 519, 520], device="cuda")
    check([y[pick] for y in got], x[pick], tokens[pick], top)


@pytest.mark.parametrize("rows,vocab,dtype", [(1, 151936, "fp32"), (24, 50257, "bf16"), (600, 5003, "fp32"), (3, 7, "bf16")])
def test_near_certain_tokens_keep_their_digits(rows, vocab, dtype):
    """With one id or two far ahead, ln(n + s) = ln n + ln(1 + s / n): the log-probability of such an id and
    the entropy are as exact, relative to themselves, as s, whose terms are off by 2 U (Y + 1) of themselves, Y
    the largest |y| that adds to it, and whose additions by U (n + 40) of it (the entropy's second sum by one U Y and
    three roundings more); logarithm, quotient and sum take 8 U."""
    import torch
    from gru_corrected_draft_amd import verify
    log(f"[gpu-test] scores of near certain tokens {rows} {vocab} {dtype}")
    x, g = _logits(rows, vocab, dtype, 21, 1.0)
    tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda").to(torch.int32)
    ahead = torch.linspace(13, 24, rows, device="cuda").to(x.dtype)
    x[torch.arange(rows, device="cuda"), tokens.long()] = ahead
    tied = torch.arange(rows, device="cuda") % 3 == 2
    x[tied, (tokens.long()[tied] + 1) % vocab] = ahead[tied]
    logprob, entropy, ids, values = verify.TokenScores(vocab, _types()[dtype], max_rows=rows).run(x, tokens, top=1)
    torch.cuda.synchronize()
    z = x.double().cpu().numpy()
    z -= z.max(1, keepdims=True)
    e = np.exp(z)
    n = (z == 0).sum(1)
    s = np.where(z == 0, 0, e).sum(1)
    want = -(np.log(n) + np.log1p(s / n))
    h = -want - (e * z).sum(1) / (n + s)
    tol = U * (2 * (-z.min(1) * LOG2E + 1) + 8 * -(-vocab // 2048) + 40 + 8)
    assert np.all(np.abs(logprob.double().cpu().numpy() - want) <= tol * -want)
    assert np.all(np.abs(values[:, 0].double().cpu().numpy() - want) <= tol * -want)
    assert np.all(np.abs(entropy.double().cpu().numpy() - h) <= (tol + U * (-z.min(1) * LOG2E + 3)) * h)
    assert -want.max() < 0.5
