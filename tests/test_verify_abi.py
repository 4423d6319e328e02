"""The handles of ``domino_verify.h`` refuse bad configurations and NULL arguments on the host, before any
device call, and the 64-bit references agree with closed forms (CPU only)."""
import ctypes

import numpy as np
import pytest

from gru_corrected_draft_amd import rollout as R
from gru_corrected_draft_amd import verify
from tests import _verify_ref as ref


@pytest.fixture(scope="module")
def lib():
    return verify.load_library()


@pytest.mark.parametrize("cfg,status", [
    ((0, 1, 128, 16, 1, 0), R.DOMINO_ERR_INVALID_CONFIG), ((8, 3, 128, 16, 1, 0), R.DOMINO_ERR_INVALID_CONFIG),
    ((8, 0, 128, 16, 1, 0), R.DOMINO_ERR_INVALID_CONFIG), ((8, 2, 128, 16, 0, 0), R.DOMINO_ERR_INVALID_CONFIG),
    ((8, 2, 128, 16, 1025, 0), R.DOMINO_ERR_INVALID_CONFIG), ((8, 2, 128, 16, 1, 2), R.DOMINO_ERR_INVALID_CONFIG),
    ((8, 2, 80, 16, 1, 0), R.DOMINO_ERR_UNSUPPORTED), ((8, 2, 128, 48, 1, 0), R.DOMINO_ERR_UNSUPPORTED),
    ((8, 2, 128, 8192, 1, 1), R.DOMINO_ERR_UNSUPPORTED),
])
def test_attention_create_refuses(lib, cfg, status):
    h = ctypes.c_void_p(1)
    assert lib.domino_attention_create(ctypes.byref(verify.AttentionConfig(*cfg)), ctypes.byref(h)) == status
    assert not h.value and lib.domino_attention_last_error(None).decode().startswith("create:")


@pytest.mark.parametrize("cfg,status", [
    ((0, 1, 16, 0), R.DOMINO_ERR_INVALID_CONFIG), ((9, 0, 16, 0), R.DOMINO_ERR_INVALID_CONFIG),
    ((9, 1, 0, 0), R.DOMINO_ERR_INVALID_CONFIG), ((9, 1, 65, 0), R.DOMINO_ERR_INVALID_CONFIG),
    ((9, 1, 16, 5), R.DOMINO_ERR_INVALID_CONFIG), ((1 << 25, 1, 16, 0), R.DOMINO_ERR_UNSUPPORTED),
])
def test_verify_create_refuses(lib, cfg, status):
    h = ctypes.c_void_p(1)
    assert lib.domino_verify_create(ctypes.byref(verify.VerifyConfig(*cfg)), ctypes.byref(h)) == status
    assert not h.value and lib.domino_verify_last_error(None).decode().startswith("create:")


def test_null_arguments(lib):
    p, c, bad = ctypes.c_void_p(0x1000), verify.CacheArgs(), R.DOMINO_ERR_INVALID_ARG
    logits = verify.LogitsArgs()
    assert lib.domino_attention_create(None, None) == bad and lib.domino_verify_create(None, None) == bad
    h = ctypes.c_void_p(1)
    assert lib.domino_attention_create(None, ctypes.byref(h)) == bad and not h.value
    assert lib.domino_attention_append(None, ctypes.byref(c), p, 0, 0, p, 0, 0, None) == bad
    assert lib.domino_attention_run(None, ctypes.byref(c), p, 0, 0, 0, 0, 1.0, p, 0, 0, None, None) == bad
    assert lib.domino_verify_process(None, ctypes.byref(logits), p, 0, 0, None) == bad
    assert lib.domino_verify_run(None, ctypes.byref(logits), None, None, 0, None, 0, p, p, None, None) == bad
    lib.domino_attention_destroy(None)
    lib.domino_verify_destroy(None)


def test_wrong_dtype_is_refused_by_the_binding():
    import torch
    with pytest.raises(TypeError):
        verify.PagedAttention(8, 2, 128, 16, torch.float16)
    with pytest.raises(TypeError):
        verify.DraftVerifier(100, torch.float64)


def test_reference_attention_closed_forms():
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((9, 2, 4)), rng.standard_normal((9, 2, 4))
    out, lse, _, _ = ref.attention(np.zeros((3, 4, 4)), k, v, 9)
    # equal scores: the mean of what is visible, per key head
    for t in range(3):
        for h in range(4):
            assert np.allclose(out[t, h], v[:7 + t, h // 2].mean(0)) and np.isclose(lse[t, h], np.log(7 + t))
    out, lse, _, _ = ref.attention(np.zeros((3, 4, 4)), k, v, 9, window=2, sinks=1)
    assert np.allclose(out[2, 0], v[[0, 7, 8], 0].mean(0))
    out, lse, _, _ = ref.attention(np.zeros((3, 4, 4)), k[:1], v[:1], 1)
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.allclose(out[2, 0], v[0, 0])


def test_reference_rules_closed_forms():
    x = np.zeros((1, 3, 40))
    x[0, :, :4] = [2.0, -2.0, 2.0, 1.0]
    rules = {"draft": np.array([[3, 3]]), "history": np.array([[0, 1, 1, 99]]), "prompt_len": np.array([1]),
             "repetition": np.array([2.0]), "frequency": np.array([0.5]), "presence": np.array([0.25])}
    y, _, n = ref.processed(x, 0, rules, 40)
    assert n == 2
    # prompt only: the division; history twice: the product, 2 x frequency, presence; proposals add up
    assert np.allclose(y[0, :4], [1.0, -4.0 - 1.0 - 0.25, 2.0, 1.0])
    assert np.allclose(y[1, 3], 0.5 - 0.5 - 0.25) and np.allclose(y[2, 3], 0.5 - 1.0 - 0.25)
    mask = np.zeros((1, 3, 2), np.int32)
    mask[0, :, 1] = 1 << 7
    y, _, _ = ref.processed(x, 0, {"mask": mask}, 40)
    assert np.isneginf(y[0, :39]).all() and y[0, 39] == 0


def test_reference_verify_samples_without_the_refused_proposal():
    x = np.log(np.array([[[0.5, 0.3, 0.2], [0.1, 0.1, 0.8]]]))
    rules = {"draft": np.array([[0]])}
    kw = dict(temperature=np.array([1.0]), noise=np.array([[1e-9, 1.0, 1.0]]))
    t, a, l, _ = ref.verify(x, rules, 3, accept_u=np.array([[0.49]]), **kw)
    assert a[0] == 1 and t[0].tolist() == [0, 0] and np.allclose(l[0], np.log([0.5, 0.1]))
    t, a, l, _ = ref.verify(x, rules, 3, accept_u=np.array([[0.51]]), **kw)
    assert a[0] == 0 and t[0].tolist() == [1, -1] and np.isclose(l[0, 0], np.log(0.3))
