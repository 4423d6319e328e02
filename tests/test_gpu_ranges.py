"""Rules and acceptance at the sizes that large calls have, where a workgroup's range of the vocabulary is
thousands of ids long (the other tests' calls are cut into the shortest ranges, 512 ids).

Four requests are made and checked against 64 bits; the batch repeats them, and each copy has to give the same
bits."""
import numpy as np
import pytest

from tests._gpu import log
from tests.test_gpu_verify import check_verify, dev, make

pytestmark = pytest.mark.gpu

KINDS = 4


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def repeated(batch, tensors):
    """Request b of each tensor is its request b % KINDS."""
    import torch
    at = torch.arange(batch, device="cuda") % KINDS
    return {k: t[at].contiguous() for k, t in tensors.items()}


def verifier(vocab, dtype, batch, rows):
    import torch
    from gru_corrected_draft_amd import verify
    return verify.DraftVerifier(vocab, torch.bfloat16 if dtype == "bf16" else torch.float32, batch, rows)


def all_alike(t):
    """Whether every copy of a request has the first one's bits."""
    import torch
    t = t.view(torch.int32 if t.element_size() == 4 else torch.int16)
    return all(torch.equal(t[k::KINDS], t[k].expand_as(t[k::KINDS])) for k in range(KINDS))


def run_verify(batch, logits, rules, more, vocab, dtype):
    import torch
    v = verifier(vocab, dtype, batch, logits.shape[1])
    x = repeated(batch, {"x": logits.cuda()})["x"]
    got = v.run(x, return_logprob=True, **repeated(batch, dev(rules)), **repeated(batch, dev(more)))
    torch.cuda.synchronize()
    v.close()
    assert all(all_alike(t) for t in got)
    return [t[:KINDS] for t in got]


# batch, vocab, history, bias: 73936, 67864, 71480 and 79616 bytes of LDS for a workgroup, all above 64 KB
LDS = [(24, 151936, 700, 0), (16, 151936, 0, 300), (48, 50257, 90, 20), (512, 50257, 700, 300)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("case", LDS, ids=str)
def test_ranges_that_fill_a_workgroups_share_of_lds(case, dtype):
    batch, vocab, history, bias = case
    log(f"[gpu-test] verify LDS {case} {dtype}")
    logits, rules, more = make(KINDS, 1, vocab, dtype, 300 + batch, history, bias, temperature=0.8)
    check_verify(run_verify(batch, logits, rules, more, vocab, dtype), logits, rules, more, vocab)


# 64 requests of 16 rows of 151937 ids: ranges of 4800 to 9536 ids, a wave to a row, so it takes several turns of
# 768 to 2048 ids without a check before the last one, whose vectors end anywhere; the last range ends inside one.
VOCAB, ROWS, BATCH = 151937, 16, 64


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rules", ["every rule", "history", "mask"])
def test_process_in_long_ranges(rules, dtype):
    import torch
    from tests.test_gpu_verify import check_process
    log(f"[gpu-test] process long ranges {rules} {dtype}")
    logits, r, _ = make(KINDS, ROWS, VOCAB, dtype, 401, 3000 if rules != "mask" else 0, 300 if rules == "every rule" else 0,
                        0.5 if rules != "history" else None)
    if "history" in r:  # many touched ids in every range, and runs of neighbours
        rng = np.random.default_rng(402)
        r["history"] = np.where(rng.random((KINDS, 3000)) < 0.5, rng.integers(0, VOCAB, (KINDS, 3000)),
                                60000 + rng.integers(0, 2500, (KINDS, 3000))).astype(np.int32)
        r["history_len"][:] = [3000, 2999, 1500, 1]
    v = verifier(VOCAB, dtype, BATCH, ROWS)
    out = v.process(repeated(BATCH, {"x": logits.cuda()})["x"], **repeated(BATCH, dev(r)))
    torch.cuda.synchronize()
    v.close()
    assert all_alike(out)
    check_process(out[:KINDS], logits, r, VOCAB, dtype)


def steepened(logits, draft):
    """Proposals that mostly stand among so many ids, and one request whose other logits grow along the row, so
    that the sums are rescaled again and again."""
    import torch
    x = logits.float()
    x[1] += torch.linspace(-40, 0, VOCAB)
    at = torch.from_numpy(draft).long()[..., None]
    x[:, :-1].scatter_add_(2, at, torch.full(at.shape, 6.0))
    x[1, :-1].scatter_(1, at[1], 20.0)
    return x.to(logits.dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("temp", [0.0, 0.7])
@pytest.mark.parametrize("rules", ["none", "history", "every rule"])
def test_verify_in_long_ranges(rules, temp, dtype):
    log(f"[gpu-test] verify long ranges {rules} {temp} {dtype}")
    logits, r, more = make(KINDS, ROWS, VOCAB, dtype, 411, 3000 if rules != "none" else 0, 300 if rules == "every rule" else 0,
                           0.9 if rules == "every rule" else None, temperature=temp, agree=0.97)
    logits = steepened(logits, r["draft"])
    check_verify(run_verify(BATCH, logits, r, more, VOCAB, dtype), logits, r, more, VOCAB)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("touched", [False, True])
def test_ties_and_odd_values_in_long_ranges(touched, dtype):
    """Greedy, in whole turns: ties go to the lowest id, NaN next to the largest and all over a row are passed
    over, +inf is the largest number, also beside ids that a bias of 0 puts on the list."""
    import torch
    log(f"[gpu-test] verify ties in long ranges {touched} {dtype}")
    logits = torch.from_numpy(np.random.default_rng(421).standard_normal((KINDS, ROWS, VOCAB), np.float32))
    ties = [300, 301, 2047, 2048, 4799, 4800, 9535, 9536, 77777, VOCAB - 1]
    for row in range(ROWS):
        logits[0, row, ties[row % 10:]] = 9.0          # the first of them
        at = ties[row % 10]
        logits[1, row, at] = 9.0
        logits[1, row, [at - 1, (at + 1) % VOCAB, 5, 100000]] = float("nan")
        logits[2, row, ::2] = float("nan")
        logits[2, row, 2 * (20000 + row) + 1] = 9.0
        logits[3, row, at] = float("inf")
    logits = logits.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    want = np.array([[ties[t % 10] for t in range(ROWS)]] * 2 + [[2 * (20000 + t) + 1 for t in range(ROWS)],
                                                              [ties[t % 10] for t in range(ROWS)]])
    draft = want[:, :-1].copy()
    draft[0, 12] += 1  # proposals that lose by a tie, and one that is refused early
    draft[3, 2] = 5
    r = {"draft": draft.astype(np.int32)}
    if touched:
        r.update(bias_ids=np.tile(np.array([[300, 2048, 9536, 40001, VOCAB - 1]], np.int32), (KINDS, 1)),
                 bias_values=np.zeros((KINDS, 5), np.float32))
    tokens, accepted, _ = (t.cpu().numpy() for t in run_verify(BATCH, logits, r, {}, VOCAB, dtype))
    for k, n in enumerate([12, ROWS - 1, ROWS - 1, 2]):
        assert accepted[k] == n and np.array_equal(tokens[k, :n + 1], want[k, :n + 1]) and (tokens[k, n + 1:] == -1).all(), k
