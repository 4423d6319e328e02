"""Rotation at far positions by large frequencies: the angle's whole turns are taken off before it is rounded.

The reference's angles are fractions of whole numbers, reduced with 100 digits of pi.  Bounds, without norms and
with u = 2^-24: the fraction of a turn is rounded once (half of 2^-24 turns, 3.2 u radians), sine and cosine add
at most 8 u, the magnitude u, the two products and the sum 2 u, all of |a| + |b|: 16 u."""
from fractions import Fraction

import numpy as np
import pytest

from tests._gpu import log

pytestmark = pytest.mark.gpu

PI = Fraction("3.1415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170679")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield


def angle(position, frequency):
    """position x frequency less its whole turns, in radians."""
    turns = position * Fraction(frequency) / (2 * PI)
    return float((turns - round(turns)) * 2 * PI)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("largest", [1.0, 10.0, 1000.0])
def test_far_positions(largest, dtype):
    import torch
    from gru_corrected_draft_amd import verify
    log(f"[gpu-test] rotation far, frequencies to {largest} {dtype}")
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16
    freq = largest * 0.7 ** np.arange(32)
    freq[1] = -0.9997 * largest
    positions = [0, 1, 40000, 2 ** 20 + 1, 2 ** 24 + 1, 2 ** 30 - 7, 2 ** 31 - 12345678, 2 ** 31 - 2, 2 ** 31 - 1]
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k = (torch.randn(len(positions), n, 64, generator=g, device="cuda").to(dt) for n in (3, 2))
    op = verify.HeadRotation(3, 2, 64, freq, dt)
    got = op.run(q, k, torch.tensor(positions, dtype=torch.int32, device="cuda"))
    turn = np.array([[angle(p, f) for f in freq] for p in positions])[:, None]
    for x, y in zip((q, k), got):
        x, y = x.double().cpu().numpy(), y.double().cpu().numpy()
        a, b = x[..., :32], x[..., 32:]
        want = np.concatenate([a * np.cos(turn) - b * np.sin(turn), b * np.cos(turn) + a * np.sin(turn)], -1)
        tol = 16 * 2.0 ** -24 * np.tile(np.abs(a) + np.abs(b), 2)
        if dtype == "bf16":
            tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
        err = np.abs(y - want)
        assert np.all(err <= tol), f"{np.max(err / tol):.3g} of the bound"
