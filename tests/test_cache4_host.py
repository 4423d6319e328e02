"""The host side of a cache in 4 bits: configurations, strides and tensors that are refused, and the launches
of its calls (CPU only)."""
import ctypes

import numpy as np
import pytest

from gru_corrected_draft_amd import rollout as R
from gru_corrected_draft_amd import verify
from tests import _fp4_ref as fp4
from tests.test_verify_host import runtime, walk  # noqa: F401

SETUP = """
torch.uint8 = "uint8"

def attention4(hq=8, hk=2, dim=128, page=16, requests=4, dtype=R.DTYPE_BF16):
    h = ctypes.c_void_p()
    return lib.domino_attention_create_fp4(ctypes.byref(verify.AttentionConfig(hq, hk, dim, page, requests, dtype)), ctypes.byref(h)), h

def cache4(dim=128, hk=2, page=16, requests=4, tokens=4, max_new=1, kv=4096, **kw):
    head = page * (dim // 2 + dim // 32)
    c = verify.CacheArgs(1 << 20, 1 << 20, hk * head, head, dim // 2, 4096, 1 << 20, 256, 256, 1 << 20, 1 << 20,
                         requests, tokens, max_new, kv)
    for name, x in kw.items():
        setattr(c, name, x)
    return ctypes.byref(c)

def run4(h, dim=128, out=None, **kw):
    return lib.domino_attention_run(h, cache4(dim, **kw), P, 1024, 128, 0, 0, 0.1, P, *(out or (8 * dim, dim)), None, None)

def rows4(h, call, dim=128, token=256, **kw):
    return getattr(lib, "domino_attention_" + call)(h, cache4(dim, **kw), P, token, dim, P, token, dim, None)

def tensors4(device=0, page_bytes=16 * 68, dtype="uint8"):
    i = "int32"
    c = [Tensor(dtype, 64, 2, page_bytes, device=device) for _ in range(2)]
    return c + [Tensor(i, 4, 8, device=device), Tensor(i, 4, device=device), Tensor(i, 5, device=device)]
"""


def walk4(runtime, body):
    import textwrap
    walk(runtime, SETUP + textwrap.dedent(body))


@pytest.mark.parametrize("cfg,status", [
    ((0, 1, 128, 16, 1, 0), R.DOMINO_ERR_INVALID_CONFIG), ((8, 2, 128, 16, 1, 1), R.DOMINO_ERR_UNSUPPORTED),
    ((8, 2, 96, 16, 1, 0), R.DOMINO_ERR_UNSUPPORTED), ((8, 2, 128, 8, 1, 0), R.DOMINO_ERR_UNSUPPORTED),
])
def test_create_refuses(cfg, status):
    lib, h = verify.load_library(), ctypes.c_void_p(1)
    assert lib.domino_attention_create_fp4(ctypes.byref(verify.AttentionConfig(*cfg)), ctypes.byref(h)) == status
    assert not h.value and lib.domino_attention_last_error(None).decode().startswith("create:")
    assert lib.domino_attention_create_fp4(None, None) == R.DOMINO_ERR_INVALID_ARG
    c, p = verify.CacheArgs(), ctypes.c_void_p(0x1000)
    assert lib.domino_attention_read(None, ctypes.byref(c), p, 0, 0, p, 0, 0, None) == R.DOMINO_ERR_INVALID_ARG


def test_caches_that_are_refused(runtime):  # noqa: F811
    walk4(runtime, """
        st, h = attention4()
        bad = R.DOMINO_ERR_INVALID_ARG
        assert st == 0 and run4(h) == 0 and rows4(h, "append") == 0 and rows4(h, "read") == 0
        n = rt.host_launches()
        for kw in (dict(row_stride=128), dict(row_stride=0), dict(page_stride=2 * 16 * 68 + 8), dict(head_stride=-16),
                   dict(requests=5), dict(requests=0), dict(num_pages=0), dict(k_cache=(1 << 20) + 8),
                   dict(kv_len=None), dict(max_kv=-1), dict(head_stride=1 << 31)):
            assert run4(h, **kw) == bad and rows4(h, "append", **kw) == bad and rows4(h, "read", **kw) == bad, kw
        # rows that several workgroups would write
        assert rows4(h, "read", token=0) == bad and rows4(h, "read", token=64) == bad
        assert b"overlap" in lib.domino_attention_last_error(h)
        assert rows4(h, "append", token=8) == 0 and rows4(h, "append", token=4) == bad
        assert rt.host_launches() == n + 1
        # nothing to do
        assert rows4(h, "read", tokens=0) == 0 and run4(h, max_new=0) == 0 and rt.host_launches() == n + 1
        st, plain = attention()
        c = verify.CacheArgs(1 << 20, 1 << 20, 4096, 2048, 128, 64, 1 << 20, 8, 8, 1 << 20, 1 << 20, 4, 4, 1, 128)
        assert lib.domino_attention_read(plain, ctypes.byref(c), P, 256, 128, P, 256, 128, None) == R.DOMINO_ERR_UNSUPPORTED
        """)


def test_launches_and_lds(runtime):  # noqa: F811
    walk4(runtime, """
        st, h = attention4()
        assert st == 0 and rt.host_attributes() > 0 and rt.host_launches() == 0
        rt.host_fail(0, -1)
        assert run4(h) == R.DOMINO_ERR_HIP and rt.host_launches() == 0
        for call in ("append", "read"):
            rt.host_fail(0, -1)
            assert rows4(h, call) == R.DOMINO_ERR_HIP and rt.host_launches() == 0
        live = rt.host_allocations()
        rt.host_fail(-1, 0)
        st, none = attention4()
        assert st == R.DOMINO_ERR_HIP and not none.value and rt.host_allocations() == live
        for dim in (64, 128, 256):
            for new in (1, 16, 32, 300):
                for kv in (64, 4096):
                    st, h = attention4(dim=dim)
                    assert st == 0 and run4(h, dim=dim, kv=kv, max_new=new, tokens=4 * new) == 0
        assert rt.host_lds_launched() > 65536 and rt.host_over() == 0
        """)


def test_tensors_that_are_refused(runtime):  # noqa: F811
    walk4(runtime, """
        a = verify.PagedAttention4(8, 2, 128, 16, max_requests=4)
        q, k, c = Tensor("bfloat16", 4, 8, 128), Tensor("bfloat16", 4, 2, 128), tensors4()
        a.run(q, *c); a.append(k, k, *c); a.read(4, *c)
        for other, match in ((tensors4(page_bytes=16 * 64), "k_cache must be"), (tensors4(dtype="bfloat16"), "k_cache must be")):
            for call in (lambda: a.run(q, *other), lambda: a.append(k, k, *other), lambda: a.read(4, *other)):
                refused(call, match)
        refused(lambda: a.append(Tensor("float32", 4, 2, 128), k, *c), "k must be")
        refused(lambda: a.read(2 ** 32 + 4, *c), "tokens")
        other = tensors4(device=1)
        refused(lambda: a.read(4, *other), "the handle is on cuda:0")
        refused(lambda: a.run(Tensor("bfloat16", 4, 8, 128, device=1), *other), "the handle is on cuda:0")
        try:
            a.read(-4, *c)
        except (R.DominoError, ValueError):
            pass
        else:
            raise AssertionError("not refused")
        """)


def test_reference_numbers():
    """Closed forms of the reference: rounding, ties, powers, bytes."""
    x = np.zeros(32)
    x[:9] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5.1]
    assert fp4.powers(x).tolist() == [0]
    assert fp4.stored(x)[:9].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -6]
    x[0] = 7
    assert fp4.powers(x).tolist() == [0] and fp4.stored(x)[0] == 6
    x[0] = 7.01
    assert fp4.powers(x).tolist() == [1] and fp4.stored(x)[0] == 8
    x[5] = np.inf
    assert fp4.powers(x).tolist() == [128] and np.isnan(fp4.stored(x)).all()
    assert fp4.powers(np.full(32, 2.0 ** 128 - 2.0 ** 120)).tolist() == [125]
    assert fp4.powers(np.zeros(32)).tolist() == [-125]
    y = np.random.default_rng(0).standard_normal((3, 64)) * 3
    data, power = fp4.row_bytes(y)
    assert data.shape == (3, 32) and power.shape == (3, 2)
    assert np.array_equal(fp4.row_values(data, power), fp4.stored(y))
    assert np.array_equal(fp4.stored(fp4.stored(y)), fp4.stored(y))
    e = 2.0 ** np.repeat(fp4.powers(y), 32, -1)
    assert np.all(np.abs(fp4.stored(y) - y) <= e)
