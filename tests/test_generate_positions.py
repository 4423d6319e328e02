"""Which targets bound a text by their positions, without a GPU: the operators' handles are stubs."""
import pytest


@pytest.fixture
def generate(monkeypatch):
    from gru_corrected_draft_amd import generate
    for name in ("HeadRotation", "PagedAttention", "DraftVerifier"):
        monkeypatch.setattr(generate, name, lambda *args, **kw: None)
    return generate


def _target(generate, rotary):
    import torch
    return generate.Target(97, 32, 4, 2, 64, 2, 40, dtype=torch.float32, device="cpu", rotary=rotary)


def test_a_rotary_target_has_no_table_of_positions(generate):
    import torch
    learned, turned = _target(generate, None), _target(generate, 1e4)
    assert learned.position.shape == (40, 32) and turned.position is None
    # the weights of a seed are the same
    assert torch.equal(learned.embed, turned.embed) and torch.equal(learned.head, turned.head)
    for a, b in zip(learned.layers, turned.layers):
        assert all(torch.equal(a[name], b[name]) for name in a)


def test_a_rotary_target_bounds_no_text(generate):
    gen = generate.Generator(_target(generate, 1e4), [[3]], 100)
    assert gen.max_kv == 1 + 100 + generate.BLOCK and gen.text.shape == (1, gen.max_kv)
    with pytest.raises(ValueError, match="positions"):
        generate.Generator(_target(generate, None), [[3]], 100)
