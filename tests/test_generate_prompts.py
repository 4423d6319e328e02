"""Prompts that ``Generator`` refuses before anything is on the GPU (CPU only)."""
import types

import pytest


@pytest.mark.parametrize("prompts,match", [
    ([[1, 2], [3, 97]], "ids"), ([[1, -1]], "ids"), ([[2 ** 40]], "ids"), ([[1], []], "needs a token"), ([], "needs a token"),
    ([[1] * 30], "positions"),
])
def test_refused(prompts, match):
    from gru_corrected_draft_amd.generate import Generator
    target = types.SimpleNamespace(heads=(8, 2, 64), device="cpu", vocab=97, position=[0] * 40)
    with pytest.raises(ValueError, match=match):
        Generator(target, prompts, 10)
