"""What scores of continuations leave behind, on a generator whose target is a stub (CPU only)."""
import types

import pytest


def _generator():
    """Texts of 3 and 5 tokens; the hidden state at a position is the token that stands there."""
    import torch
    from gru_corrected_draft_amd.generate import Generator
    gen = Generator.__new__(Generator)
    gen.requests, gen.longest, gen.max_kv, gen._ahead, gen.hidden = 2, 5, 40, False, None
    gen.text = torch.arange(80, dtype=torch.int32).view(2, 40)
    gen.length = torch.tensor([3, 5], dtype=torch.int32)
    gen.target = types.SimpleNamespace(vocab=97, dtype=torch.float32)

    def logits(tokens):
        gen.hidden = tokens.float()[..., None]
        return torch.zeros(*tokens.shape, 97)

    gen.logits = logits
    gen._scores = types.SimpleNamespace(run=lambda x, tokens, top: (tokens.float(), tokens.float(), None, None))
    return gen


@pytest.mark.parametrize("n", [1, 2, 16])
def test_score_leaves_the_hidden_states(n):
    """The next proposals are made from ``hidden``: it stays that of the text, not of what was scored."""
    import torch
    gen = _generator()
    tokens = torch.full((2, n), 90)
    gen.score(tokens)
    assert torch.equal(gen.hidden[:, -1, 0], gen.last()[:, 0].float()) and gen.hidden.shape == (2, 1, 1)
    gen.hidden = before = torch.rand(2, 16, 1)
    gen.score(tokens)
    assert gen.hidden is before
