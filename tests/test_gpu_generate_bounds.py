"""How far a ``Generator`` goes: to ``max_new`` tokens, whatever its proposals were worth."""
import pytest

from tests._gpu import log
from tests.test_gpu_generate import LENGTHS, VOCAB, generator

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def test_refused_proposals_do_not_use_up_max_new():
    """Proposals outside the vocabulary are always refused, so each block of 16 positions adds one token; the
    text that comes of it is the target's own, and the limit holds where it is reached."""
    import torch
    log("[gpu-test] generate to max_new")
    gen, one = generator(None), generator(None)
    wrong = torch.full((len(LENGTHS), 15), VOCAB, dtype=torch.int32, device="cuda")
    for i in range(200):  # the generators' max_new
        new, accepted = gen.block(wrong)
        one.block()
        if i % 40 == 0:
            assert accepted.tolist() == [0] * len(LENGTHS) and (new[:, 0] >= 0).all()
    assert gen.length.tolist() == [n + 200 for n in LENGTHS]
    for b, n in enumerate(gen.length.tolist()):
        assert torch.equal(gen.text[b, :n], one.text[b, :n])
    # a block may start at max_new (there is room for its 16 positions), none past it
    gen.block(wrong)
    with pytest.raises(ValueError, match="outgrow"):
        gen.block(wrong)
    assert gen.length.tolist() == [n + 201 for n in LENGTHS]
