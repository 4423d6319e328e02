"""Blocks that are checked in one pass against the same target taken token by token.

Whatever is proposed, greedy texts have to be the target's own: a proposal stands exactly if the target would
have chosen it, under the rules as they stand after the proposals before it.  fp32, so that the two ways to
batch the target's products decide alike."""
import pytest

from tests._gpu import log

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


VOCAB, POSITIONS, STEPS = 997, 420, 36
LENGTHS = [1, 17, 130, 64]


def texts():
    import numpy as np
    rng = np.random.default_rng(5)
    return [rng.integers(0, VOCAB, n).tolist() for n in LENGTHS]


def rules_of(kind):
    import numpy as np
    import torch
    if kind == "plain":
        return None
    rng = np.random.default_rng(6)
    b = len(LENGTHS)

    def to(a):
        return torch.from_numpy(a).cuda()

    words = rng.integers(0, 2 ** 32, (b, 1, (VOCAB + 31) // 32), dtype=np.uint64)
    return dict(repetition=to(np.full(b, 1.2, np.float32)), frequency=to(np.full(b, 0.3, np.float32)),
                presence=to(np.full(b, 0.5, np.float32)),
                bias_ids=to(np.stack([rng.permutation(VOCAB)[:9] for _ in range(b)]).astype(np.int32)),
                bias_values=to(rng.uniform(-2, 2, (b, 9)).astype(np.float32)),
                mask=to(words.astype(np.uint32).view(np.int32)))


def generator(rules, dtype="fp32", **more):
    import torch
    from gru_corrected_draft_amd.generate import Generator, Target
    target = Target(VOCAB, 96, 6, 2, 64, 2, POSITIONS, window=50,
                    dtype=torch.float32 if dtype == "fp32" else torch.bfloat16, seed=3)
    return Generator(target, texts(), 200, rules=rules, **more)


@pytest.mark.parametrize("kind", ["plain", "rules"])
def test_blocks_give_the_text_of_single_tokens(kind):
    import numpy as np
    import torch
    log(f"[gpu-test] generate {kind}")
    rules = rules_of(kind)
    one = generator(rules)
    for _ in range(STEPS + 16):
        one.block()
    want = [one.text[b, :n].tolist() for b, n in enumerate(one.length.tolist())]
    assert [len(t) for t in want] == [n + STEPS + 16 for n in LENGTHS]
    gen = generator(rules)
    rng = np.random.default_rng(7)
    took = set()
    while min(n - m for n, m in zip(gen.length.tolist(), LENGTHS)) < STEPS and gen.longest < 300:
        rows = rng.integers(2, 17)
        proposals = np.full((len(LENGTHS), rows - 1), -1, np.int32)
        right = rng.integers(0, rows, len(LENGTHS))
        for b, n in enumerate(gen.length.tolist()):
            good = want[b][n:n + right[b]]
            proposals[b] = rng.integers(0, VOCAB, rows - 1)
            proposals[b, :len(good)] = good
        new, accepted = gen.block(torch.from_numpy(proposals).cuda())
        new, accepted = new.tolist(), accepted.tolist()
        for b in range(len(LENGTHS)):
            took.add(accepted[b])
            assert all(t >= 0 for t in new[b][:accepted[b] + 1])
            assert all(t == -1 for t in new[b][accepted[b] + 1:])
            have = gen.text[b, :gen.length[b]].tolist()
            assert have[:len(want[b])] == want[b][:len(have)]
            assert accepted[b] >= min(right[b], len(want[b]) - (len(have) - accepted[b] - 1))
    assert len(took) > 6  # blocks that are refused early, late and not at all


def test_sampled_texts_obey_the_mask():
    import numpy as np
    import torch
    log("[gpu-test] generate sampled")
    rules = rules_of("rules")
    gen = generator(rules, "bf16", temperature=torch.full((len(LENGTHS),), 0.8, device="cuda"))
    logprob, ids = gen.candidates(5)
    for _ in range(4):
        gen.block(torch.randint(0, VOCAB, (len(LENGTHS), 15), dtype=torch.int32, device="cuda"))
    bits = np.unpackbits(rules["mask"][:, 0].cpu().numpy().view(np.uint8), axis=1, bitorder="little")
    for b, n in enumerate(gen.length.tolist()):
        assert n >= LENGTHS[b] + 4
        assert all(bits[b, v] for v in gen.text[b, LENGTHS[b]:n].tolist())
        assert all(bits[b, v] for v in ids[b].tolist())


def test_a_text_without_a_token_left():
    import torch
    log("[gpu-test] generate empty mask")
    mask = torch.full((len(LENGTHS), 1, (VOCAB + 31) // 32), -1, dtype=torch.int32, device="cuda")
    mask[2] = 0
    gen = generator(dict(mask=mask))
    new, accepted = gen.block()
    assert gen.length.tolist() == [n + (b != 2) for b, n in enumerate(LENGTHS)]
    assert new[2].tolist() == [-1]


def test_refusals():
    gen = generator(None)
    gen.longest = gen.max_kv
    with pytest.raises(ValueError, match="outgrow"):
        gen.block()
    from gru_corrected_draft_amd.generate import Generator
    with pytest.raises(ValueError, match="positions"):
        Generator(gen.target, [[1] * 300], 200)
    with pytest.raises(ValueError, match="prompt"):
        Generator(gen.target, [[1], []], 10)


def test_command():
    from gru_corrected_draft_amd import generate
    log("[gpu-test] generate command")
    gen = generate.main(["--requests", "3", "--prompt", "40", "--blocks", "3"])
    assert all(n >= m + 3 for n, m in zip(gen.length.tolist(), gen.prompt_len.tolist()))
    gen = generate.main(["--requests", "2", "--prompt", "9", "--blocks", "2", "--k", "0", "--temperature", "0.7"])
    assert all(n >= m + 2 for n, m in zip(gen.length.tolist(), gen.prompt_len.tolist()))
