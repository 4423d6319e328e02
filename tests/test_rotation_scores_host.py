"""The host side of head rotation and token scores: configurations, arguments and tensors that are refused, and
the launches of their calls (CPU only)."""
import ctypes

import numpy as np
import pytest

from gru_corrected_draft_amd import rollout as R
from gru_corrected_draft_amd import verify
from tests.test_verify_host import runtime, walk  # noqa: F401

SETUP = """
import math

def rotation(q=8, kv=2, dim=128, rotary=128, dtype=R.DTYPE_BF16, interleaved=0, magnitude=1.0, freq=None):
    h = ctypes.c_void_p()
    f = (ctypes.c_double * 128)(*(freq or [0.5] * 64))
    cfg = verify.RotationConfig(q, kv, dim, rotary, dtype, interleaved, magnitude)
    return lib.domino_rotation_create(ctypes.byref(cfg), f, ctypes.byref(h)), h

def heads(n=8, dim=128, weight=1 << 20, **kw):
    a = verify.HeadsArgs(1 << 20, n * dim, dim, weight, 1 << 20, n * dim, dim)
    for name, x in kw.items():
        setattr(a, name, x)
    return a

def turn(h, q=None, k=None, positions=P, tokens=4, eps=1e-6):
    q, k = q or heads(), k or heads(2)
    return lib.domino_rotation_run(h, ctypes.byref(q), ctypes.byref(k), positions, tokens, eps, None)

def scores(vocab=151936, rows=64, top=64, dtype=R.DTYPE_BF16):
    h = ctypes.c_void_p()
    return lib.domino_scores_create(ctypes.byref(verify.ScoresConfig(vocab, rows, top, dtype)), ctypes.byref(h)), h

def rate(h, logits=P, stride=151936, rows=3, tokens=P, top=5, logprob=P, entropy=P, ids=P, values=P):
    return lib.domino_scores_run(h, logits, stride, rows, tokens, top, logprob, entropy, ids, values, None)
"""


def walk2(runtime, body):
    import textwrap
    walk(runtime, SETUP + textwrap.dedent(body))


@pytest.mark.parametrize("cfg,status", [
    ((0, 1, 128, 128, 0, 0, 1.0), R.DOMINO_ERR_INVALID_CONFIG), ((8, 1025, 128, 128, 0, 0, 1.0), R.DOMINO_ERR_INVALID_CONFIG),
    ((8, 2, 128, 128, 2, 0, 1.0), R.DOMINO_ERR_INVALID_CONFIG), ((8, 2, 128, 128, 0, 2, 1.0), R.DOMINO_ERR_INVALID_CONFIG),
    ((8, 2, 128, 128, 0, 0, float("nan")), R.DOMINO_ERR_INVALID_CONFIG), ((8, 2, 96, 96, 0, 0, 1.0), R.DOMINO_ERR_UNSUPPORTED),
    ((8, 2, 128, 0, 0, 0, 1.0), R.DOMINO_ERR_UNSUPPORTED), ((8, 2, 128, 40, 0, 0, 1.0), R.DOMINO_ERR_UNSUPPORTED),
    ((8, 2, 64, 128, 0, 0, 1.0), R.DOMINO_ERR_UNSUPPORTED),
])
def test_rotation_create_refuses(cfg, status):
    lib, h, f = verify.load_library(), ctypes.c_void_p(1), (ctypes.c_double * 128)()
    assert lib.domino_rotation_create(ctypes.byref(verify.RotationConfig(*cfg)), f, ctypes.byref(h)) == status
    assert not h.value and lib.domino_rotation_last_error(None).decode().startswith("create:")


@pytest.mark.parametrize("freq", [float("inf"), float("nan"), 1001.0, -2000.0])
def test_rotation_frequencies(freq):
    lib, h = verify.load_library(), ctypes.c_void_p(1)
    f = (ctypes.c_double * 64)(*([1.0] * 63 + [freq]))
    cfg = verify.RotationConfig(8, 2, 128, 128, 0, 0, 1.0)
    assert lib.domino_rotation_create(ctypes.byref(cfg), f, ctypes.byref(h)) == R.DOMINO_ERR_INVALID_CONFIG
    assert lib.domino_rotation_create(ctypes.byref(cfg), None, ctypes.byref(h)) == R.DOMINO_ERR_INVALID_ARG
    assert lib.domino_rotation_create(None, f, ctypes.byref(h)) == R.DOMINO_ERR_INVALID_ARG
    assert lib.domino_rotation_create(ctypes.byref(cfg), f, None) == R.DOMINO_ERR_INVALID_ARG
    a = verify.HeadsArgs()
    assert lib.domino_rotation_run(None, ctypes.byref(a), ctypes.byref(a), 4096, 1, 0.0, None) == R.DOMINO_ERR_INVALID_ARG
    lib.domino_rotation_destroy(None)


@pytest.mark.parametrize("cfg,status", [
    ((0, 1, 0, 0), R.DOMINO_ERR_INVALID_CONFIG), ((9, 0, 0, 0), R.DOMINO_ERR_INVALID_CONFIG),
    ((9, 1, 65, 0), R.DOMINO_ERR_INVALID_CONFIG), ((9, 1, -1, 0), R.DOMINO_ERR_INVALID_CONFIG),
    ((9, 1, 0, 3), R.DOMINO_ERR_INVALID_CONFIG), (((1 << 24) + 1, 1, 0, 0), R.DOMINO_ERR_UNSUPPORTED),
    ((9, 65536, 0, 0), R.DOMINO_ERR_UNSUPPORTED),
])
def test_scores_create_refuses(cfg, status):
    lib, h = verify.load_library(), ctypes.c_void_p(1)
    assert lib.domino_scores_create(ctypes.byref(verify.ScoresConfig(*cfg)), ctypes.byref(h)) == status
    assert not h.value and lib.domino_scores_last_error(None).decode().startswith("create:")
    assert lib.domino_scores_create(None, ctypes.byref(h)) == R.DOMINO_ERR_INVALID_ARG
    assert lib.domino_scores_create(ctypes.byref(verify.ScoresConfig(9, 1, 0, 0)), None) == R.DOMINO_ERR_INVALID_ARG
    assert lib.domino_scores_run(None, 4096, 9, 1, None, 0, None, None, None, None, None) == R.DOMINO_ERR_INVALID_ARG
    lib.domino_scores_destroy(None)


def test_rotation_arguments(runtime):  # noqa: F811
    walk2(runtime, """
        st, h = rotation()
        assert st == 0 and rt.host_launches() == 1 and rt.host_allocations() == 1
        assert turn(h) == 0 and turn(h, heads(weight=None), heads(2, weight=None)) == 0 and rt.host_launches() == 3
        bad = R.DOMINO_ERR_INVALID_ARG
        assert turn(h, tokens=0) == 0 and rt.host_launches() == 3
        for q in (heads(input=None), heads(out=None), heads(weight=None), heads(input=(1 << 20) + 8), heads(weight=(1 << 20) + 2),
                  heads(token_stride=1025), heads(head_stride=-128), heads(out_head_stride=64), heads(out_token_stride=0),
                  heads(out_token_stride=12)):
            assert turn(h, q) == bad
            assert turn(h, None, q) == bad
        for kw in (dict(tokens=-1), dict(positions=None), dict(positions=ctypes.c_void_p((1 << 20) + 2)), dict(eps=-1.0),
                   dict(eps=math.nan), dict(eps=math.inf)):
            assert turn(h, **kw) == bad, kw
        assert rt.host_launches() == 3
        rt.host_fail(0, -1)
        assert turn(h) == R.DOMINO_ERR_HIP and b"launch failed" in lib.domino_rotation_last_error(h) and turn(h) == 0
        live = rt.host_allocations()
        rt.host_fail(0, -1)
        st, none = rotation()
        assert st == R.DOMINO_ERR_HIP and not none.value and rt.host_allocations() == live
        # every shape has its kernel
        for dtype in (R.DTYPE_BF16, R.DTYPE_FP32):
            for dim in (64, 128, 256):
                for mode in (0, 1):
                    for tokens in (1, 5000):
                        st, h = rotation(dim=dim, rotary=48, dtype=dtype, interleaved=mode)
                        n = rt.host_launches()
                        assert st == 0 and turn(h, heads(dim=dim), heads(2, dim=dim), tokens=tokens) == 0
                        assert rt.host_launches() == n + 1
        """)


def test_scores_arguments(runtime):  # noqa: F811
    walk2(runtime, """
        st, h = scores()
        assert st == 0 and rt.host_launches() == 0 and rate(h) == 0 and rt.host_launches() == 1
        assert rate(h, tokens=None, logprob=None) == 0 and rate(h, top=0, ids=None, values=None) == 0
        assert rate(h, entropy=None) == 0 and rate(h, stride=0) == 0 and rt.host_launches() == 5
        bad, odd = R.DOMINO_ERR_INVALID_ARG, ctypes.c_void_p((1 << 20) + 2)
        for kw in (dict(rows=65), dict(rows=-1), dict(top=65), dict(top=-1), dict(stride=-1), dict(tokens=None), dict(logprob=None),
                   dict(ids=None), dict(values=None), dict(logits=None), dict(logits=ctypes.c_void_p((1 << 20) + 1)),
                   dict(tokens=odd), dict(entropy=odd), dict(ids=odd)):
            assert rate(h, **kw) == bad, kw
        # nothing to do
        assert rate(h, rows=0, logits=None) == 0
        assert rate(h, tokens=None, logprob=None, entropy=None, top=0) == 0 and rt.host_launches() == 5
        rt.host_fail(0, -1)
        assert rate(h) == R.DOMINO_ERR_HIP and b"launch failed" in lib.domino_scores_last_error(h) and rate(h) == 0
        # without alternatives there is no memory for them
        before = rt.host_bytes()
        scores(top=0)
        small = rt.host_bytes() - before
        scores(top=1)
        assert small < 64 * 1024 and rt.host_bytes() - before - small > 64 * 151936 // 32
        st, none = scores(top=0)
        assert rate(none, top=1) == bad
        """)


def test_tensors_that_are_refused(runtime):  # noqa: F811
    walk2(runtime, """
        i, bf = "int32", "bfloat16"
        a = verify.HeadRotation(8, 2, 128, [0.1] * 64)
        q, k, w, pos = Tensor(bf, 4, 8, 128), Tensor(bf, 4, 2, 128), Tensor(bf, 128), Tensor(i, 4)
        a.run(q, k, pos, w, w)
        a.run(q, k, pos, out_q=q, out_k=k)
        refused(lambda: a.run(q, k, pos, w), "together")
        refused(lambda: a.run(q, q, pos), "k must be")
        refused(lambda: a.run(q, k, Tensor("int64", 4)), "positions must be")
        refused(lambda: a.run(q, k, Tensor(i, 5)), "positions must be")
        refused(lambda: a.run(q, k, pos, w, Tensor("float32", 128)), "k_weight must be")
        refused(lambda: a.run(q, k, pos, out_q=k), "out_q must be")
        other = Tensor(bf, 4, 8, 128)
        other.strides = [2048, 128, 1]
        refused(lambda: a.run(q, k, pos, out_q=other), "strides")
        refused(lambda: a.run(Tensor(bf, 4, 8, 128, device=1), Tensor(bf, 4, 2, 128, device=1), Tensor(i, 4, device=1)), "the handle is on cuda:0")
        refused(lambda: verify.HeadRotation(2 ** 32 + 8, 2, 128, [0.1] * 64), "q_heads")
        s = verify.TokenScores(1000, max_rows=8, max_top=20)
        x, t = Tensor(bf, 4, 1000), Tensor(i, 4)
        s.run(x, t, top=20)
        s.run(x)
        refused(lambda: s.run(Tensor("float32", 4, 1000)), "logits must be")
        refused(lambda: s.run(Tensor(bf, 4, 999)), "logits must be")
        refused(lambda: s.run(x, Tensor(i, 3)), "tokens must be")
        refused(lambda: s.run(x, t, top=21), "top must be")
        refused(lambda: s.run(x, t, top=-1), "top must be")
        refused(lambda: s.run(Tensor(bf, 4, 1000, device=1)), "the handle is on cuda:0")
        refused(lambda: verify.TokenScores(2 ** 32 + 1000), "vocab")
        """)


def test_wrong_types_are_refused_by_the_binding():
    import torch
    with pytest.raises(TypeError):
        verify.HeadRotation(8, 2, 128, [0.1] * 64, torch.float16)
    with pytest.raises(TypeError):
        verify.TokenScores(100, torch.float16)


def test_reference_rotation():
    """The GPU test's reference: a quarter turn, both pairings, what stays."""
    from tests.test_gpu_rotation import reference
    x = np.zeros((1, 1, 64))
    x[0, 0, :4] = [1, 2, 3, 4]
    x[0, 0, 60] = 9
    out, _ = reference(x, [1], [np.pi / 2] + [0.0] * 15, None, 0, True, 1.0, False)
    assert np.allclose(out[0, 0, :4], [-2, 1, 3, 4]) and out[0, 0, 60] == 9
    out, _ = reference(x, [1], [np.pi / 2] + [0.0] * 15, None, 0, False, 2.0, False)
    assert np.allclose(out[0, 0, [0, 16]], [0, 2]) and np.allclose(out[0, 0, 1:4], [4, 6, 8]) and out[0, 0, 60] == 9
    w = np.full(64, 3.0)
    out, _ = reference(np.full((1, 1, 64), 5.0), [0], [1.0] * 8, w, 0, False, 1.0, False)
    assert np.allclose(out, 3.0)
