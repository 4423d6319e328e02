"""Rules on logits and the acceptance of proposals, against 64 bits.

Processed logits are held to the rounding of the rules' own operations; tokens and counts have to be equal,
on inputs whose decisions the 64-bit reference makes by more than fp32 can blur."""
import numpy as np
import pytest

from tests import _verify_ref as ref
from tests._gpu import log

pytestmark = pytest.mark.gpu

# fp32 evaluates a score x - T ln E within a few ulp of numbers below 64, and a probability within 1e-5
MARGIN = 2e-5


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def make(batch, rows, vocab, dtype, seed, history=0, bias=0, mask=None, penalties=True, temperature=0.0,
         draft_len=None, agree=0.8):
    """Inputs as NumPy arrays; logits already rounded to the type."""
    import torch
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((batch, rows, vocab), np.float32) * 2
    rules = {}
    if rows > 1:
        d = rng.integers(0, vocab, (batch, rows - 1)).astype(np.int32)
        lift = np.where(rng.random((batch, rows - 1)) < agree, 12, 5).astype(np.float32)
        for b in range(batch):
            for t in range(rows - 1):
                x[b, t, d[b, t]] += lift[b, t]
        rules["draft"] = d
        if draft_len is not None:
            rules["draft_len"] = np.asarray(draft_len, np.int32)
    logits = torch.from_numpy(x).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    if history:
        rules["history"] = rng.integers(0, min(vocab, 3 * history), (batch, history)).astype(np.int32)
        rules["history_len"] = rng.integers(0, history + 1, batch).astype(np.int32)
        rules["prompt_len"] = (rules["history_len"] // 2).astype(np.int32)
    if history or penalties == "only":
        rules.update(repetition=rng.uniform(1, 1.4, batch).astype(np.float32),
                     frequency=rng.uniform(0, 0.3, batch).astype(np.float32),
                     presence=rng.uniform(0, 0.6, batch).astype(np.float32))
    if bias:
        rules["bias_ids"] = np.stack([rng.permutation(vocab)[:bias] for _ in range(batch)]).astype(np.int32)
        rules["bias_values"] = rng.uniform(-3, 3, (batch, bias)).astype(np.float32)
    if mask is not None:
        words = rng.integers(0, 2 ** 32, (batch, rows, (vocab + 31) // 32), dtype=np.uint64)
        if mask > 0.5:
            words |= rng.integers(0, 2 ** 32, words.shape, dtype=np.uint64)
        rules["mask"] = words.astype(np.uint32).view(np.int32)
    more = {}
    if temperature is not None and np.any(np.asarray(temperature) > 0):
        more["temperature"] = np.broadcast_to(np.asarray(temperature, np.float32), (batch,)).copy()
        more["noise"] = np.maximum(rng.standard_exponential((batch, vocab)), 1e-30).astype(np.float32)
        if rows > 1:
            more["accept_u"] = rng.random((batch, rows - 1)).astype(np.float32)
    return logits, rules, more


def dev(d):
    import torch
    return {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in d.items()}


_ops = {}


def op(vocab, dtype, batch=16, rows=16):
    import torch
    from gru_corrected_draft_amd import verify
    key = vocab, dtype, batch, rows
    if key not in _ops:
        _ops[key] = verify.DraftVerifier(vocab, torch.bfloat16 if dtype == "bf16" else torch.float32, batch, rows)
    return _ops[key]


def check_process(out, logits, rules, vocab, dtype):
    out = out.float().cpu().numpy().astype(np.float64)
    x = logits.float().numpy()
    for b in range(x.shape[0]):
        want, tol, _ = ref.processed(x, b, rules, vocab)
        if dtype == "bf16":
            tol = tol + 2.0 ** -8 * (np.abs(np.where(np.isfinite(want), want, 0)) + tol)
        gone = np.isneginf(want)
        assert np.array_equal(np.isneginf(out[b]), gone), f"request {b}"
        err = np.abs(np.where(gone, 0, out[b]) - np.where(gone, 0, want))
        assert np.all(err <= tol), f"request {b}: {np.max(err - tol)}"


def check_verify(got, logits, rules, more, vocab):
    tokens, accepted, logprob = (x.cpu().numpy() for x in got)
    x = logits.float().numpy()
    wt, wa, wl, margin = ref.verify(x, rules, vocab, more.get("temperature"), more.get("accept_u"), more.get("noise"))
    assert margin > MARGIN, f"the inputs decide by {margin:.2g} only"
    assert np.array_equal(accepted, wa), (accepted, wa)
    assert np.array_equal(tokens, wt)
    inf = np.isneginf(wl)
    assert np.array_equal(np.isneginf(logprob), inf)
    # x, m and ln s are each off by a few ulp of numbers below 64, over T at least 0.05
    low = 1.0 if "temperature" not in more else min(1.0, float(np.min(np.where(more["temperature"] > 0, more["temperature"], 1))))
    assert np.all(np.abs(np.where(inf, 0, logprob) - np.where(inf, 0, wl)) <= 2e-5 / low + 1e-6 * np.abs(np.where(inf, 0, wl)))
    return wa


PROCESS = [
    # batch, rows, vocab, history, bias, mask
    (1, 1, 1, 3, 0, None), (1, 1, 31, 5, 2, 0.3), (2, 3, 33, 0, 4, None), (3, 16, 1000, 50, 7, 0.5),
    (2, 5, 5003, 900, 0, 0.9), (1, 1, 5003, 3, 0, None), (4, 16, 4096, 64, 300, None), (2, 40, 777, 33, 3, 0.5),
    (1, 2, 50257, 4000, 300, 0.5), (3, 1, 20000, 0, 0, 0.5), (1, 64, 129, 1, 1, 0.9),
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("case", PROCESS, ids=str)
def test_process_against_64_bits(case, dtype):
    batch, rows, vocab, history, bias, mask = case
    log(f"[gpu-test] process {case} {dtype}")
    logits, rules, _ = make(batch, rows, vocab, dtype, 100 + vocab, history, bias, mask)
    v = op(vocab, dtype, rows=64)
    x = logits.cuda()
    out = v.process(x, **dev(rules))
    check_process(out, logits, rules, vocab, dtype)
    same = v.process(x, out=x, **dev(rules))
    assert same.data_ptr() == x.data_ptr() and np.array_equal(
        x.view(__import__("torch").uint8).cpu().numpy(), out.view(__import__("torch").uint8).cpu().numpy())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_process_only_proposals_and_bounds(dtype):
    """Penalties without a history count the proposals; ids and lengths out of range are passed over; the
    last entry of a repeated bias holds; draft_len cuts the proposals."""
    log(f"[gpu-test] process bounds {dtype}")
    vocab = 700
    logits, rules, _ = make(3, 6, vocab, dtype, 5, penalties="only", draft_len=[9, 2, -1])
    rules["draft"][0] = [5, 5, 5, -1, vocab]
    rules["bias_ids"] = np.array([[3, 3, 3, -1, vocab, 2 ** 31 - 1], [699, 0, 699, 1, 2, 3], [-2 ** 31, 4, 4, 4, 9, 9]], np.int32)
    rules["bias_values"] = np.array([[1, 2, -7, 1, 1, 1], [1, 2, 3, 4, 5, 6], [8, 1, 2, 3, 4, 5]], np.float32)
    rules["bias_len"] = np.array([6, 2, 99], np.int32)
    out = op(vocab, dtype).process(logits.cuda(), **dev(rules))
    check_process(out, logits, rules, vocab, dtype)
    logits, rules, _ = make(3, 6, vocab, dtype, 6, history=40)
    rules["history"][0, :5] = [-1, vocab, 2 ** 31 - 1, -2 ** 31, 7]
    rules["history_len"] = np.array([40, 1000, -5], np.int32)
    rules["prompt_len"] = np.array([-3, 1000, 7], np.int32)
    out = op(vocab, dtype).process(logits.cuda(), **dev(rules))
    check_process(out, logits, rules, vocab, dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_process_views(dtype):
    """Rows at an odd offset and stride, a mask and a history shared by all requests."""
    import torch
    log(f"[gpu-test] process views {dtype}")
    vocab = 1003
    logits, rules, _ = make(3, 4, vocab, dtype, 8, history=30, bias=5, mask=0.5)
    for k in ("history", "mask"):
        rules[k][:] = rules[k][:1]
    rules["mask"][:] = rules["mask"][:, :1]
    wide = torch.zeros((4, 3, vocab + 6), dtype=logits.dtype, device="cuda")
    wide[:, :, 3:3 + vocab] = logits.cuda().transpose(0, 1)
    x = wide[:, :, 3:3 + vocab].transpose(0, 1)
    d = dev(rules)
    d["mask"] = d["mask"][:1, :1].expand(3, 4, -1)
    d["history"] = d["history"][:1].expand(3, -1)
    out = torch.full((3, 4, vocab + 5), 9.0, dtype=logits.dtype, device="cuda")
    v = op(vocab, dtype)
    v.process(x, out=out[:, :, 1:1 + vocab], **d)
    check_process(out[:, :, 1:1 + vocab], logits, rules, vocab, dtype)
    assert (out[:, :, 0] == 9).all() and (out[:, :, 1 + vocab:] == 9).all()


def test_process_keeps_what_it_does_not_touch():
    """Infinities, NaN and the lowest value pass through untouched ids bit by bit."""
    import torch
    log("[gpu-test] process passes values through")
    vocab = 300
    for dtype in ("fp32", "bf16"):
        logits, rules, _ = make(1, 1, vocab, dtype, 9, history=4)
        logits[0, 0, :6] = torch.tensor([float("inf"), float("-inf"), float("nan"), -0.0, torch.finfo(logits.dtype).min, 1e-39])
        rules["history"][:] = 100
        out = op(vocab, dtype).process(logits.cuda(), **dev(rules)).cpu()
        keep = torch.arange(vocab) != 100
        assert torch.equal(out[0, 0, keep].view(torch.uint8), logits[0, 0, keep].view(torch.uint8))


VERIFY = [
    # batch, rows, vocab, history, bias, mask, temperature
    (1, 1, 1, 0, 0, None, 0.0), (1, 1, 1, 0, 0, None, 1.0), (2, 3, 33, 0, 0, None, 0.0),
    (5, 16, 1000, 0, 0, None, 0.0), (5, 16, 1000, 0, 0, None, 0.9), (3, 16, 5003, 300, 9, 0.5, 0.0),
    (3, 16, 5003, 300, 9, 0.5, 0.7), (1, 16, 50257, 1000, 0, None, 1.2), (16, 1, 4099, 20, 0, 0.9, 0.6),
    (2, 33, 259, 30, 2, 0.9, 0.8), (4, 9, 20001, 0, 300, None, 0.3), (1, 2, 50257, 0, 0, None, 0.0),
]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("case", VERIFY, ids=str)
def test_verify_against_64_bits(case, dtype):
    batch, rows, vocab, history, bias, mask, temp = case
    log(f"[gpu-test] verify {case} {dtype}")
    logits, rules, more = make(batch, rows, vocab, dtype, 200 + vocab + rows, history, bias, mask, temperature=temp)
    v = op(vocab, dtype, rows=33)
    got = v.run(logits.cuda(), return_logprob=True, **dev(rules), **dev(more))
    check_verify(got, logits, rules, more, vocab)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_verify_mixed_temperatures_and_lengths(dtype):
    """Greedy and sampling requests in one call, blocks of other lengths, proposals out of range."""
    log(f"[gpu-test] verify mixed {dtype}")
    vocab = 2003
    logits, rules, more = make(8, 8, vocab, dtype, 31, history=60, temperature=[0, 1, 0.5, -1, 2, 0.1, 0, 1],
                               draft_len=[7, 7, 0, 3, 100, 5, -4, 1], agree=0.95)
    rules["draft"][0, 2] = -1
    rules["draft"][1, 1] = vocab
    rules["draft"][4, 0] = 2 ** 31 - 1
    got = op(vocab, dtype).run(logits.cuda(), return_logprob=True, **dev(rules), **dev(more))
    took = check_verify(got, logits, rules, more, vocab)
    assert took[0] <= 2 and took[1] <= 1 and took[2] == 0 and took[4] == 0 and took[6] == 0


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_verify_ties_go_to_the_lowest_id(dtype):
    import torch
    log(f"[gpu-test] verify ties {dtype}")
    vocab = 9001
    logits = torch.zeros((6, 2, vocab))
    logits[:, 1] = -1
    logits[:, 1, 8000] = 4
    logits[0, 0] = -0.0                       # all equal: id 0
    logits[1, 0, [77, 4000, 8999]] = 3        # three at the top: 77
    logits[2, 0, [4000, 8999]] = 3
    logits[3, 0, [5, 6]] = 3
    logits[4, 0, [5, 6]] = 3
    logits[5, 0, 8992:] = 2.0
    logits = logits.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    rules = {"draft": np.array([[0], [4000], [4000], [6], [5], [8992]], np.int32)}
    t, a, l = op(vocab, dtype).run(logits.cuda(), return_logprob=True, **dev(rules))
    assert a.tolist() == [1, 0, 1, 0, 1, 1]
    assert t.tolist() == [[0, 8000], [77, -1], [4000, 8000], [5, -1], [5, 8000], [8992, 8000]]
    # touched ids tie with untouched ones: a bias of zero changes nothing
    rules.update(bias_ids=np.tile(np.array([[77, 0, 6, 8993]], np.int32), (6, 1)), bias_values=np.zeros((6, 4), np.float32))
    t2, a2, l2 = op(vocab, dtype).run(logits.cuda(), return_logprob=True, **dev(rules))
    assert torch.equal(t, t2) and torch.equal(a, a2) and torch.allclose(l, l2, rtol=0, atol=1e-5)


def test_verify_empty_rows_and_odd_values():
    """Rows without an allowed id, a single allowed id, NaN and infinities, the type's lowest value."""
    import torch
    log("[gpu-test] verify empty rows")
    vocab, inf = 700, float("inf")
    for dtype in ("fp32", "bf16"):
        logits, rules, more = make(7, 4, vocab, dtype, 41, mask=0.9, temperature=[0, 1, 0, 1, 0, 1, 1], agree=1.0)
        mask = np.full_like(rules["mask"], -1)
        mask[0, 0] = 0                           # nothing allowed at the first row
        mask[1, 2] = 0                           # nor at the third, sampling
        for b, t in ((2, 1), (3, 1)):            # the proposal alone is allowed: it stands whatever u is
            mask[b, t] = 0
            d = int(rules["draft"][b, t])
            mask[b, t, d // 32] = np.array([1 << (d % 32)], np.uint32).view(np.int32)[0]
        rules["mask"] = mask
        more["accept_u"][:] = 0.0
        more["accept_u"][3, 1] = 0.9999999
        logits[4, 0, 9] = float("nan")           # never chosen
        logits[4, 0, 10] = inf                   # the largest number
        logits[5, 0] = -inf                      # every logit is -inf
        logits[6, 0] = torch.finfo(logits.dtype).min   # all equal: a uniform row
        more["accept_u"][6, 0] = 0.5             # 1 / 700 < 0.5: refused
        got = op(vocab, dtype).run(logits.cuda(), return_logprob=True, **dev(rules), **dev(more))
        wt, wa, wl, _ = ref.verify(logits.float().numpy(), rules, vocab, more["temperature"], more["accept_u"], more["noise"])
        tokens, accepted, logprob = (x.cpu().numpy() for x in got)
        assert accepted[0] == 0 and tokens[0].tolist() == [-1] * 4 and logprob[0, 0] == -inf
        assert accepted[1] == 2 and tokens[1, 2] == -1 and logprob[1, 2] == -inf
        assert accepted[2] >= 2 and accepted[3] >= 2 and logprob[3, 1] == 0
        assert tokens[4, 0] == 10 and accepted[5] == 0 and tokens[5, 0] == -1 and accepted[6] == 0
        assert np.array_equal(tokens, wt) and np.array_equal(accepted, wa)
        assert abs(logprob[6, 0] + np.log(vocab)) < 1e-5


@pytest.mark.parametrize("temp", [0.0, 0.7])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_verify_passes_over_every_nan(dtype, temp):
    """NaN of both kinds and signs in every place of a row, next to the largest logit and away from it."""
    import torch
    log(f"[gpu-test] verify NaN {dtype} {temp}")
    vocab = 2050
    logits, rules, more = make(4, 3, vocab, dtype, 77, temperature=temp, agree=1.0)
    kinds = (0x7FC0, 0x7F81, 0xFFC0, 0xFF81) if dtype == "bf16" else (0x7FC00000, 0x7F800001, 0xFFC00000, 0xFF800001)
    raw = logits.view(torch.int16 if dtype == "bf16" else torch.int32).numpy()
    rng = np.random.default_rng(78)
    for b in range(4):
        for t in range(3):
            at = rng.permutation(vocab)[:600]
            top = int(np.nanargmax(logits[b, t].float().numpy()))
            at = np.concatenate([at, [top - 1, top + 1] if 0 < top < vocab - 1 else []]).astype(int)
            at = at[at != top]
            raw[b, t, at] = np.array(kinds, np.uint16 if dtype == "bf16" else np.uint32)[at % 4].view(raw.dtype)
    got = op(vocab, dtype).run(logits.cuda(), return_logprob=True, **dev(rules), **dev(more))
    check_verify(got, logits, rules, more, vocab)


def test_sampling_follows_the_distribution():
    """With one proposal and fresh noise, the first token's frequencies are the target's: 60000 draws over
    five ids, each within five standard deviations."""
    import torch
    log("[gpu-test] verify distribution")
    vocab, n = 5, 1000
    x = torch.tensor([0.3, 1.0, -0.5, 0.0, 0.8])
    p = torch.softmax(x / 0.7, 0).double()
    g = torch.Generator(device="cuda").manual_seed(3)
    v = op(vocab, "fp32", batch=n, rows=2)
    logits = x.expand(n, 2, vocab).contiguous().cuda()
    count = torch.zeros(vocab, dtype=torch.double)
    draft = torch.full((n, 1), 4, dtype=torch.int32, device="cuda")
    for _ in range(60):
        t, a = v.run(logits, draft, temperature=torch.full((n,), 0.7, device="cuda"),
                     accept_u=torch.rand((n, 1), generator=g, device="cuda"),
                     noise=torch.empty((n, vocab), device="cuda").exponential_(generator=g))
        count += torch.bincount(t[:, 0].long().cpu(), minlength=vocab).double()
    total = 60 * n
    assert torch.all((count - total * p).abs() <= 5 * (total * p * (1 - p)).sqrt()), count / total


def test_verify_equals_process_then_verify():
    """fp32: the fused rules and the rules alone give the same tokens and log-probabilities."""
    import torch
    log("[gpu-test] verify fused against process")
    vocab = 5003
    logits, rules, more = make(4, 16, vocab, "fp32", 51, history=500, bias=40, mask=0.9, temperature=0.8)
    v = op(vocab, "fp32")
    d, m = dev(rules), dev(more)
    a = v.run(logits.cuda(), return_logprob=True, **d, **m)
    b = v.run(v.process(logits.cuda(), **d), d["draft"], return_logprob=True, **m)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.allclose(a[2], b[2], rtol=0, atol=2e-5)


def test_same_bits_each_time_on_another_stream_and_in_a_graph():
    import torch
    log("[gpu-test] verify on streams and in a graph")
    vocab = 20001
    logits, rules, more = make(4, 16, vocab, "bf16", 61, history=2000, bias=40, mask=0.9, temperature=0.8)
    v = op(vocab, "bf16")
    x, d, m = logits.cuda(), dev(rules), dev(more)
    want, out = v.run(x, return_logprob=True, **d, **m), v.process(x, **d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, out2 = v.run(x, return_logprob=True, **d, **m), v.process(x, **d)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got)) and torch.equal(out, out2)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = v.run(x, return_logprob=True, **d, **m)
    for _ in range(3):
        for h in held:
            h.zero_()
        g.replay()
        assert all(torch.equal(p, q) for p, q in zip(want, held))
        again = v.run(x, return_logprob=True, **d, **m)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, again))


def test_refusals():
    import torch
    from gru_corrected_draft_amd import rollout as R
    from gru_corrected_draft_amd import verify
    log("[gpu-test] verify refusals")
    for kw in (dict(vocab=0), dict(vocab=10, max_rows=65), dict(vocab=10, max_requests=0)):
        with pytest.raises(R.DominoError) as e:
            verify.DraftVerifier(**kw)
        assert e.value.status == R.DOMINO_ERR_INVALID_CONFIG
    v = op(100, "fp32", batch=2, rows=4)
    x = torch.zeros((2, 4, 100), device="cuda")
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    f = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    for kw in (dict(draft=i(2, 4)), dict(draft=i(2, 3).long()), dict(draft=i(2, 3).cpu()),
               dict(temperature=f(2)), dict(draft=i(2, 3), temperature=f(2), noise=f(2, 100)),
               dict(temperature=f(2), noise=f(2, 99)), dict(bias_ids=i(2, 3)), dict(history=i(1, 3)),
               dict(mask=i(2, 4, 3)), dict(repetition=f(3)), dict(mask=i(2, 4, 8)[:, :, ::2])):
        with pytest.raises(ValueError):
            v.run(x, **kw)
    for bad in (x[:, :, :99], x.bfloat16(), x.cpu(), x[0]):
        with pytest.raises(ValueError):
            v.process(bad)
    with pytest.raises(R.DominoError) as e:
        v.run(torch.zeros((3, 4, 100), device="cuda"))
    assert e.value.status == R.DOMINO_ERR_INVALID_ARG
    with pytest.raises(R.DominoError):
        v.run(torch.zeros((2, 5, 100), device="cuda"))
    with pytest.raises(ValueError):
        v.process(x, out=x.transpose(0, 1))
