"""The operators of the target's pass together: heads normalised and rotated, their cache in 4 bits, attention
over it, scores of the logits; and generation with such a target."""
import numpy as np
import pytest

from tests import _fp4_ref as fp4
from tests import _verify_ref as ref
from tests._gpu import log
from tests.test_gpu_generate import LENGTHS, VOCAB, texts
from tests.test_gpu_rotation import _check as check_rotation
from tests.test_gpu_scores import check as check_scores

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def _generator(dtype, cache_bits=None, **more):
    import torch
    from gru_corrected_draft_amd.generate import Generator, Target
    target = Target(VOCAB, 96, 6, 2, 64, 2, 420, window=50, seed=3, rotary=1e4,
                    dtype=torch.float32 if dtype == "fp32" else torch.bfloat16)
    return Generator(target, texts(), 200, cache_bits=cache_bits, **more)


@pytest.mark.parametrize("new,kv,window", [([1, 1, 1], [40, 300, 1], 0), ([16, 5], [200, 33], 60), ([70, 3], [90, 250], 0)])
def test_a_layer_and_its_logits(new, kv, window):
    """Each operator on what the one before it made, against 64 bits; nothing synchronises in between."""
    import torch
    from gru_corrected_draft_amd import verify
    log(f"[gpu-test] operators together {new} {kv}")
    hq, hk, d, page, vocab, hidden = 8, 2, 64, 16, 1501, 128
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    freq = 1e5 ** (-np.arange(0, d, 2) / d)
    rotation = verify.HeadRotation(hq, hk, d, freq)
    attention = verify.PagedAttention4(hq, hk, d, page, max_requests=len(new))
    scores = verify.TokenScores(vocab, max_rows=512)
    weights = [(1 + 0.2 * torch.randn(d, generator=g, device="cuda")).bfloat16() for _ in range(2)]
    pages = [-(-n // page) for n in kv]
    table = torch.full((len(kv), max(pages)), -1, dtype=torch.int32, device="cuda")
    order = torch.randperm(sum(pages), generator=g, device="cuda").to(torch.int32)
    for b, n in enumerate(pages):
        table[b, :n] = order[sum(pages[:b]):sum(pages[:b]) + n]
    caches = [torch.full((sum(pages), hk, attention.page_bytes), 255, dtype=torch.uint8, device="cuda") for _ in range(2)]

    def step(lens, total):
        """New tokens of each request that end at `total`: what went in and came out."""
        n = sum(lens)
        where = (*caches, table, torch.tensor(total, dtype=torch.int32, device="cuda"),
                 torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda"))
        positions = torch.cat([torch.arange(t - m, t) for m, t in zip(lens, total)]).to("cuda", torch.int32)
        qkv = normal(n, hq + 2 * hk, d)
        q, k, v = qkv.split([hq, hk, hk], 1)
        q1, k1 = rotation.run(q, k, positions, *weights)
        attention.append(k1, v, *where)
        out = attention.run(q1, *where, window=window, sinks=2 if window else 0, max_new=max(lens), max_kv=max(total))
        logits = out.flatten(1)[:, :hidden].contiguous() @ normal(hidden, vocab)
        tokens = torch.randint(0, vocab, (n,), generator=g, device="cuda").to(torch.int32)
        return q, k, v, positions, q1, k1, out, logits, tokens, scores.run(logits, tokens, top=9)

    keys, values = [], []
    before = [t - n for n, t in zip(new, kv)]
    if max(before):
        first = step(before, before)  # what is cached already, in one ragged pass
        start = 0
        for n in before:
            keys.append(fp4.stored(first[5][start:start + n].double().cpu().numpy()) if n else np.zeros((0, hk, d)))
            values.append(fp4.stored(first[2][start:start + n].double().cpu().numpy()) if n else np.zeros((0, hk, d)))
            start += n
    else:
        keys, values = ([np.zeros((0, hk, d)) for _ in new] for _ in range(2))
    q, k, v, positions, q1, k1, out, logits, tokens, got = step(new, kv)
    check_rotation(q1, q, positions, freq, weights[0])
    check_rotation(k1, k, positions, freq, weights[1])
    start = 0
    for b, n in enumerate(new):
        rows = slice(start, start + n)
        start += n
        kk = np.concatenate([keys[b], fp4.stored(k1[rows].double().cpu().numpy())])
        vv = np.concatenate([values[b], fp4.stored(v[rows].double().cpu().numpy())])
        o, _, a, reach = ref.attention(q1[rows].double().cpu().numpy(), kk, vv, kv[b], window, 2 if window else 0)
        tol, _ = ref.attention_bounds(o, a, reach, kv[b], d, True)
        assert np.all(np.abs(out[rows].double().cpu().numpy() - o) <= tol), b
    check_scores(got, logits, tokens, 9)


def test_rotated_blocks_give_the_text_of_single_tokens():
    """fp32: proposals that are the target's own choices stand, others do not."""
    import torch
    log("[gpu-test] generate with rotated heads")
    one = _generator("fp32")
    for _ in range(40):
        one.block()
    want = [one.text[b, :n].tolist() for b, n in enumerate(one.length.tolist())]
    gen = _generator("fp32")
    rng = np.random.default_rng(7)
    for _ in range(12):
        if max(n - m for n, m in zip(gen.length.tolist(), LENGTHS)) > 24:
            break
        right = rng.integers(0, 9, len(LENGTHS))
        proposals = rng.integers(0, VOCAB, (len(LENGTHS), 8)).astype(np.int32)
        for b, n in enumerate(gen.length.tolist()):
            proposals[b, :right[b]] = want[b][n:n + right[b]]
        new, accepted = gen.block(torch.from_numpy(proposals).cuda())
        assert all(x >= y for x, y in zip(accepted.tolist(), right))
        for b, n in enumerate(gen.length.tolist()):
            have = gen.text[b, :n].tolist()
            assert have[:len(want[b])] == want[b][:len(have)]


@pytest.mark.parametrize("dtype,bits", [("fp32", None), ("bf16", None), ("bf16", 4)])
def test_score_of_continuations(dtype, bits):
    """Log-probabilities of given tokens are those of the logits after them; texts and caches stay."""
    import torch
    log(f"[gpu-test] scores of continuations {dtype} {bits}")
    gen = _generator(dtype, bits)
    b = len(LENGTHS)
    for _ in range(2):
        gen.block(torch.randint(0, VOCAB, (b, 15), dtype=torch.int32, device="cuda"))
    length, text = gen.length.clone(), gen.text.clone()
    tokens = torch.randint(0, VOCAB, (b, 7), dtype=torch.int32, device="cuda")
    got = gen.score(tokens, top=4)
    x = gen.logits(torch.cat([gen.last(), tokens[:, :-1]], 1))
    check_scores([t.flatten(0, 1) for t in got], x.flatten(0, 1), tokens.flatten(), 4)
    assert got[0].shape == (b, 7) and got[2].shape == (b, 7, 4)
    assert torch.equal(length, gen.length) and torch.equal(text, gen.text)
    again = gen.score(tokens)
    assert torch.equal(again[0], got[0]) and again[2] is None
    logprob, ids = gen.candidates(3)  # no rules: the same first choices
    assert torch.equal(ids[:, 0].int(), got[2][:, 0, 0])
    with pytest.raises(ValueError, match="at once"):
        gen.score(tokens.repeat(1, 3))
    gen.longest, gen._ahead = gen.max_kv, False
    with pytest.raises(ValueError, match="room"):
        gen.score(tokens)


def test_scores_of_padded_continuations():
    """Ids outside the vocabulary have no probability; those before them are what they would be."""
    import torch
    log("[gpu-test] scores of padded continuations")
    gen = _generator("bf16", 4)
    b = len(LENGTHS)
    tokens = torch.randint(0, VOCAB, (b, 5), device="cuda")
    want = gen.score(tokens)[0]
    padded = tokens.clone()
    padded[:, 3] = torch.tensor([-1, VOCAB, -2 ** 40, 2 ** 32], device="cuda")[torch.arange(b, device="cuda") % 4]
    got, entropy = gen.score(padded)[:2]
    assert torch.equal(got[:, :3], want[:, :3])
    assert torch.isneginf(got[:, 3]).all() and torch.isfinite(got[:, 4]).all() and torch.isfinite(entropy).all()


def test_the_cache_of_the_target():
    """Another cache, another answer; which targets can have one of 4 bits."""
    import torch
    log("[gpu-test] a cache of 4 bits and one of 16")
    a, b = _generator("bf16"), _generator("bf16", 4)
    x, y = (g.logits(g.last())[:, 0].float() for g in (a, b))
    assert torch.isfinite(x).all() and torch.isfinite(y).all() and not torch.equal(x, y)
    assert b.caches[0][0].dtype == torch.uint8 and 32 * b.caches[0][0].nbytes * 2 == 17 * a.caches[0][0].nbytes
    with pytest.raises(ValueError, match="bfloat16"):
        _generator("fp32", 4)
    with pytest.raises(ValueError, match="cache_bits"):
        _generator("bf16", 8)


def test_command():
    from gru_corrected_draft_amd import generate
    log("[gpu-test] generate command, rotated and in 4 bits")
    gen = generate.main(["--requests", "3", "--prompt", "40", "--blocks", "3", "--rotary", "--cache-bits", "4"])
    assert all(n >= m + 3 for n, m in zip(gen.length.tolist(), gen.prompt_len.tolist()))
