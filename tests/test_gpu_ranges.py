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
