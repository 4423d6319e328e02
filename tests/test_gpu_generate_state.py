"""What a generator's queries leave of its state."""
import pytest

from tests._gpu import log
from tests.test_gpu_generate import LENGTHS, VOCAB
from tests.test_gpu_generate_rotary import _generator

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


@pytest.mark.parametrize("dtype,bits", [("fp32", None), ("bf16", 4)])
def test_scores_between_blocks_change_nothing(dtype, bits):
    """Blocks with scores of several tokens between them and without: the same hidden states, texts and tokens."""
    import torch
    log(f"[gpu-test] scores between blocks {dtype} {bits}")
    a, b = _generator(dtype, bits), _generator(dtype, bits)
    g = torch.Generator(device="cuda").manual_seed(2)
    n = len(LENGTHS)
    a.score(torch.zeros((n, 9), dtype=torch.int32, device="cuda"))
    assert a.hidden.shape == (n, 1, 96)
    for _ in range(3):
        proposals = torch.randint(0, VOCAB, (n, 15), generator=g, dtype=torch.int32, device="cuda")
        first, second = a.block(proposals), b.block(proposals)
        assert torch.equal(first[0], second[0]) and torch.equal(first[1], second[1])
        before = a.hidden.clone()
        a.score(torch.randint(0, VOCAB, (n, 16), generator=g, dtype=torch.int32, device="cuda"), top=3)
        assert torch.equal(a.hidden, before) and torch.equal(a.hidden, b.hidden)
        assert torch.equal(a.text, b.text) and torch.equal(a.length, b.length)
