"""Padded batches of the target's pass: rows before the first sequence and behind the last are left as they were,
whatever they hold, and heads are rotated in place within the product that holds them."""
import numpy as np
import pytest

from tests import _fp4_ref as fp4
from tests._gpu import log
from tests.test_gpu_attention4 import Setup, _need_gpu  # noqa: F401
from tests.test_gpu_rotation import _check, _frequencies

pytestmark = pytest.mark.gpu

# heads, dim, new, kv, bound on the keys: undivided, cut into runs, tiles converted in LDS (whole, in parts)
CASES = [((8, 2), 128, [1, 1], [40, 90], 90), ((8, 2), 128, [1, 2], [700, 90], 8192), ((32, 8), 64, [16, 0, 3], [300, 4, 90], 300),
         ((8, 2), 256, [9, 16], [60, 700], 4096), ((8, 2), 128, [70, 300], [90, 420], 1 << 17), ((8, 2), 256, [150, 9], [361, 700], 1 << 18),
         ((32, 8), 128, [200, 1024], [700, 1100], 4096)]


@pytest.mark.parametrize("heads,dim,new,kv,bound", CASES)
def test_rows_of_no_request(heads, dim, new, kv, bound):
    import torch
    log(f"[gpu-test] padded attention over 4 bits {heads} {dim} {new} {bound}")
    s = Setup(heads, dim, 16, new, kv, seed=21, extra_width=max(0, bound // 16 - -(-max(kv) // 16)))
    before, behind = 3, 21
    tokens = before + s.tokens + behind
    inside = slice(before, before + s.tokens)
    s.q_start += before
    q = torch.full((tokens, s.hq, dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    q[inside] = s.q
    out = torch.full_like(q, 7.0)
    got, lse = s.op.run(q, *s.where, max_new=max(new), max_kv=bound, out=out, return_lse=True)
    assert got is out
    s.check(out[inside], lse[inside])
    outside = torch.ones(tokens, dtype=torch.bool, device="cuda")
    outside[inside] = False
    assert torch.all(out[outside] == 7)
    # appended rows outside the sequences do not reach the cache
    k, v = (torch.full((tokens, s.hk, dim), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[inside] = torch.randn(s.tokens, s.hk, dim, device="cuda").bfloat16()
    v[inside] = torch.randn(s.tokens, s.hk, dim, device="cuda").bfloat16()
    s.op.append(k, v, *s.where, max_new=max(new), max_kv=bound)
    k4, v4 = s.op.read(tokens, *s.where, max_new=max(new), max_kv=bound)
    start = before
    for n, m in zip(new, kv):
        rows = slice(start + max(0, n - m), start + n)
        assert torch.isfinite(k4[rows]).all() and torch.isfinite(v4[rows]).all()
        start += n
    for b, (n, m) in enumerate(zip(new, kv)):  # what stood before the new tokens is as it was
        for cache, rows in ((s.k_cache, s.keys[b]), (s.v_cache, s.values[b])):
            have = s.bytes_at(cache, b, np.arange(max(0, m - n)))
            want = fp4.row_bytes(rows[:max(0, m - n)])
            assert np.array_equal(fp4.row_values(*have), fp4.row_values(*want))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_heads_rotated_in_the_product(dtype, interleaved):
    """q and k as strided views of one product, rotated in place; v and the padded rows stay."""
    import torch
    from gru_corrected_draft_amd import verify
    log(f"[gpu-test] rotation within a product {dtype} {interleaved}")
    dt = torch.float32 if dtype == "fp32" else torch.bfloat16
    for tokens in (1, 37, 2600, 6001):
        qkv = torch.randn(tokens, 14, 64, device="cuda").to(dt)
        was = qkv.clone()
        q, k, v = qkv.split([8, 3, 3], 1)
        w = (1 + 0.1 * torch.randn(64, device="cuda")).to(dt)
        positions = torch.randint(0, 10 ** 6, (tokens,), device="cuda", dtype=torch.int32)
        positions[3::7] = -1
        op = verify.HeadRotation(8, 3, 64, _frequencies(48), dt, interleaved)
        op.run(q, k, positions, w, w, out_q=q, out_k=k)
        for x, y in ((was[:, :8], q), (was[:, 8:11], k)):
            _check(y, x, positions, _frequencies(48), w, interleaved=interleaved)
        there = positions >= 0
        assert torch.equal(v, was[:, 11:]) and torch.equal(qkv[~there], was[~there])
