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


def plain_fp32(q, keys, values, scale):
    """Attention of one row over all keys, each operation rounded to fp32: scores by one fused sum after the
    other, weights against the maximum, sums in steps of 16 keys."""
    f = np.float32
    s = np.zeros(len(keys), f)
    for i in range(len(q)):
        s = (s.astype(np.float64) + np.float64(q[i]) * keys[:, i]).astype(f)
    s = (s * f(scale)).astype(f)
    m = s.max()
    p = np.exp(s - m).astype(f)
    den, num = f(0), np.zeros(values.shape[1], f)
    for a in range(0, len(p), 16):
        den = f(den + p[a:a + 16].sum(dtype=f))
        num = (num + (p[a:a + 16, None] * values[a:a + 16]).sum(0, dtype=f)).astype(f)
    return num / den, m + np.log(den)


@pytest.mark.parametrize("divided", [False, True])
@pytest.mark.parametrize("dim,kv,spread,early", [(64, 6001, 4.0, 0), (64, 6001, 1.0, 1), (128, 8192, 1.0, 0), (128, 8192, 4.0, 0)])
def test_fp32_errs_as_a_plain_evaluation_over_long_contexts(dim, kv, spread, early, divided):
    """fp32, thousands of keys: the kernel rounds as often as a plain fp32 evaluation does, in another order, so
    its error is that one's: within three times of it in the root mean square, for outputs and log-sum-exps.
    With other requests beside it a row's keys stay in one workgroup, alone they are dealt to many."""
    log(f"[gpu-test] attention fp32 long {dim} {kv} {spread} {early} {divided}")
    others = 0 if divided else 33  # x 8 key heads: more segments than CUs
    s = Setup((8, 8), dim, 64, "fp32", [1] * (1 + others), [kv] + [1] * others, seed=41)
    s.q *= spread
    if early:  # the largest score comes first
        s.keys[0][3] = s.q[0] / s.q[0].norm(dim=-1, keepdim=True) * (0.7 * dim ** 0.5)
        s.k_cache[s.table[0, 0].long(), :, 3] = s.keys[0][3]
    out, lse = s.run(max_new=1, max_kv=kv)
    out, lse = out[0].double().cpu().numpy(), lse[0].double().cpu().numpy()
    q, keys, values = (x.cpu().numpy() for x in (s.q[:1], s.keys[0], s.values[0]))
    want, want_l, _, _ = ref.attention(q, keys, values, kv)
    plain = [plain_fp32(q[0, h], keys[:, h], values[:, h], dim ** -0.5) for h in range(8)]

    def rms(x):
        return float(np.sqrt(np.mean(np.square(x))))

    for name, got, exact, base in (("out", out, want[0], np.stack([o for o, _ in plain])),
                                   ("lse", lse, want_l[0], np.array([n for _, n in plain]))):
        here, there = rms(got - exact), rms(base - exact)
        log(f"[gpu-test]   {name}: {here:.2e}, plain {there:.2e}")
        assert here <= 3 * there, f"{name}: {here:.3g}, a plain evaluation {there:.3g}"


def _rules(kind, batch, vocab):
    """No rule, or biases of 0 that put every third id on the list of touched ones."""
    import torch
    if kind == "plain":
        return {}
    ids = torch.arange(0, vocab, 3, dtype=torch.int32, device="cuda").repeat(batch, 1)
    return dict(bias_ids=ids, bias_values=torch.zeros(ids.shape, device="cuda"))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("kind", ["plain", "touched"])
@pytest.mark.parametrize("temp", [0.01, 0.05, 0.3, 1.0])
def test_log_probabilities_of_sampled_tokens(temp, kind, dtype):
    """Logits near 20, apart by about a temperature.  With u = 2^-24: z = (x - m) / T is off by 2 u |z|, a term of
    the sum by 3.5 u |z| (difference, product, two roundings of its factor) and 2 u of the exponential, the sum
    by u for each of at most 64 additions one after the other, the logarithm by 2 u of itself and the result by
    u.  m is at most 16 powers of two below the largest logit, so |z| <= 11.1 + ln V where it counts and
    |ln s| <= 11.1 + ln V: in all u (5 |lp| + 10 (11.1 + ln V) + 66)."""
    import torch
    from gru_corrected_draft_amd import verify
    vocab, batch, rows = 1501, 64, 2
    log(f"[gpu-test] log-probabilities {temp} {kind} {dtype}")
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(17)
    x = (20 + temp * torch.randn((batch, rows, vocab), generator=g, device="cuda")).to(dt)
    draft = torch.randint(0, vocab, (batch, rows - 1), generator=g, device="cuda", dtype=torch.int32)
    noise = torch.empty((batch, vocab), device="cuda").exponential_(generator=g).clamp_(min=1e-30)
    t = torch.full((batch,), temp, device="cuda")
    op = verify.DraftVerifier(vocab, dt, batch, rows)
    tokens, accepted, lp = op.run(x, draft, temperature=t, noise=noise, return_logprob=True,
                                  accept_u=torch.zeros((batch, rows - 1), device="cuda"), **_rules(kind, batch, vocab))
    assert (lp <= 0).all() and (accepted == rows - 1).all()
    want = torch.log_softmax(x.double() / t.double()[:, None, None], -1).gather(2, tokens.long()[..., None])[..., 0]
    err = (lp.double() - want).abs()
    tol = 2.0 ** -24 * (5 * want.abs() + 10 * (11.1 + np.log(vocab)) + 66)
    log(f"[gpu-test]   off by {err.max().item():.2e}, bound {tol.min().item():.2e}")
    assert (err <= tol).all(), f"{(err / tol).max().item():.3g} of the bound"


@pytest.mark.parametrize("kind", ["plain", "touched"])
def test_a_sampled_only_candidate_has_log_probability_zero(kind):
    import torch
    from gru_corrected_draft_amd import verify
    vocab, batch = 700, 200
    log(f"[gpu-test] only candidate {kind}")
    g = torch.Generator(device="cuda").manual_seed(19)
    x = 20 + 3 * torch.randn((batch, 1, vocab), generator=g, device="cuda")
    at = torch.randint(0, vocab, (batch,), generator=g, device="cuda")
    words = torch.zeros((batch, 1, (vocab + 31) // 32), dtype=torch.int64, device="cuda")
    words[torch.arange(batch, device="cuda"), 0, at // 32] = 1 << (at % 32)
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
    noise = torch.empty((batch, vocab), device="cuda").exponential_(generator=g).clamp_(min=1e-30)
    op = verify.DraftVerifier(vocab, torch.float32, batch, 1)
    for temp in (0.05, 0.3, 1.5):
        tokens, _, lp = op.run(x, temperature=torch.full((batch,), temp, device="cuda"), noise=noise, mask=words,
                               return_logprob=True, **_rules(kind, batch, vocab))
        assert torch.equal(tokens[:, 0].long(), at) and (lp == 0).all(), f"{(lp != 0).sum().item()} are not 0"
