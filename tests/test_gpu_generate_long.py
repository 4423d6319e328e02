"""Texts of a rotary target that are longer than the number of positions it was made with."""
import pytest

from tests._gpu import log

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def test_text_longer_than_positions():
    """fp32: a text grown token by token past `positions`, and the same text as a prompt, go on alike."""
    import torch
    from gru_corrected_draft_amd.generate import Generator, Target
    log("[gpu-test] generate beyond the positions")
    target = Target(997, 96, 6, 2, 64, 2, 20, window=50, seed=3, rotary=1e4, dtype=torch.float32)
    gen = Generator(target, [[5, 9, 2], [7]], 90)
    for _ in range(80):
        gen.block()
    want = [gen.text[b, :n].tolist() for b, n in enumerate(gen.length.tolist())]
    assert [len(t) for t in want] == [83, 81]
    again = Generator(target, [t[:-8] for t in want], 40)
    for _ in range(8):
        again.block()
    assert [again.text[b, :n].tolist() for b, n in enumerate(again.length.tolist())] == want
