"""The host side of the handles of ``domino_verify.h``, walked without a GPU: what they ask of the runtime, and
what they do when it refuses (CPU only).

Each test runs in a process of its own whose HIP runtime is ``_host_runtime.cpp``: launches are counted, none
is carried out, so pointers need not point anywhere."""
import os
import shutil
import subprocess
import sys
import textwrap

import pytest

from tests.conftest import ROOT

PREAMBLE = """
import ctypes, sys, types
sys.path.insert(0, {root!r})
rt = ctypes.CDLL({runtime!r}, mode=ctypes.RTLD_GLOBAL)
for n in ("bytes", "lds_launched"):
    getattr(rt, "host_" + n).restype = ctypes.c_longlong
torch = types.ModuleType("torch")
torch.bfloat16, torch.float32, torch.int32 = "bfloat16", "float32", "int32"
torch._C = types.SimpleNamespace(_cuda_getCurrentRawStream=lambda i: None)
torch.cuda = types.SimpleNamespace(current_device=lambda: 0)
sys.modules["torch"] = torch
from gru_corrected_draft_amd import rollout as R, verify
lib = verify.load_library()
P = ctypes.c_void_p(1 << 20)

def attention(hq=8, hk=2, dim=128, page=16, requests=4, dtype=R.DTYPE_BF16):
    h = ctypes.c_void_p()
    st = lib.domino_attention_create(ctypes.byref(verify.AttentionConfig(hq, hk, dim, page, requests, dtype)), ctypes.byref(h))
    return st, h

def attend(h, kv=4096, width=256, tokens=4, max_new=1, hk=2, dim=128, page=16, requests=4, out=None):
    c = verify.CacheArgs(1 << 20, 1 << 20, hk * page * dim, page * dim, dim, 4096, 1 << 20, width, width, 1 << 20, 1 << 20,
                         requests, tokens, max_new, kv)
    return lib.domino_attention_run(h, ctypes.byref(c), P, 1024, 128, 0, 0, 0.1, P,
                                    *(out or (8 * dim, dim)), None, None)

def verifier(vocab=151936, requests=16, rows=16, dtype=R.DTYPE_BF16):
    h = ctypes.c_void_p()
    return lib.domino_verify_create(ctypes.byref(verify.VerifyConfig(vocab, requests, rows, dtype)), ctypes.byref(h)), h

def check(h, requests=16, rows=1, vocab=151936):
    a = verify.LogitsArgs(1 << 20, vocab * rows, vocab, requests, rows)
    return lib.domino_verify_run(h, ctypes.byref(a), None, None, 0, None, 0, P, P, None, None)

class Tensor:
    # what the binding looks at
    def __init__(self, dtype, *shape, device=0):
        self.dtype, self.shape, self.index = dtype, shape, device
        self.strides = [1]
        for n in reversed(shape[1:]):
            self.strides.insert(0, self.strides[0] * n)
    def dim(self): return len(self.shape)
    def stride(self, i=None): return tuple(self.strides) if i is None else self.strides[i]
    def get_device(self): return self.index
    def data_ptr(self): return 1 << 20
    @property
    def device(self): return f"cuda:{{self.index}}"

torch.empty = lambda shape, dtype=None, device=None: Tensor(dtype, *shape, device=int(str(device)[-1]))

def cache_tensors(requests=4, device=0):
    i = "int32"
    return (Tensor("bfloat16", 64, 2, 16, 128, device=device), Tensor("bfloat16", 64, 2, 16, 128, device=device),
            Tensor(i, requests, 8, device=device), Tensor(i, requests, device=device), Tensor(i, requests + 1, device=device))

def refused(call, match):
    n = rt.host_launches()
    try:
        call()
    except ValueError as e:
        assert match in str(e), e
    else:
        raise AssertionError("not refused")
    assert rt.host_launches() == n
"""


@pytest.fixture(scope="module")
def runtime(tmp_path_factory):
    include = "/opt/rocm/include"
    if not shutil.which("g++") or not os.path.isdir(include):
        pytest.skip("needs g++ and the HIP headers")
    so = str(tmp_path_factory.mktemp("runtime") / "libamdhip64.so.7")
    subprocess.run(["g++", "-shared", "-fPIC", "-O1", "-w", "-D__HIP_PLATFORM_AMD__", "-I", include, "-Wl,-soname,libamdhip64.so.7",
                    os.path.join(ROOT, "tests", "_host_runtime.cpp"), "-o", so], check=True)
    return so


def walk(runtime, body):
    """Runs `body`, whose assertions have to hold."""
    code = PREAMBLE.format(root=ROOT, runtime=runtime) + textwrap.dedent(body)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr[-2000:]


def test_a_failed_launch_ends_the_call(runtime):
    """The second launch of a call joins what the first one left: after a failed first there is none."""
    walk(runtime, """
        st, h = verifier()
        assert st == 0 and check(h) == 0 and rt.host_launches() == 2
        rt.host_fail(0, -1)
        assert check(h) == R.DOMINO_ERR_HIP and rt.host_launches() == 2
        assert b"launch failed" in lib.domino_verify_last_error(h)
        assert check(h) == 0 and rt.host_launches() == 4
        rt.host_fail(1, -1)
        assert check(h) == R.DOMINO_ERR_HIP and rt.host_launches() == 5

        st, h = attention()
        assert st == 0 and attend(h) == 0 and rt.host_launches() == 7
        rt.host_fail(0, -1)
        assert attend(h) == R.DOMINO_ERR_HIP and rt.host_launches() == 7
        assert b"launch failed" in lib.domino_attention_last_error(h)
        assert attend(h) == 0 and rt.host_launches() == 9
        """)


def test_lds_is_asked_for_at_create(runtime):
    """Before a handle's first launch its device has been asked for as much LDS as any launch takes, by each
    handle (another one may be on another device), and a refusal is the create's error."""
    walk(runtime, """
        for make, use in ((verifier, check), (attention, attend)):
            st, h = make()
            asked = rt.host_attributes()
            assert st == 0 and asked > 0 and rt.host_launches() == 0
            st, h = make()
            assert st == 0 and rt.host_attributes() == 2 * asked
            rt.host_fail(-1, asked - 1)
            live = rt.host_allocations()
            st, none = make()
            assert st == R.DOMINO_ERR_HIP and not none.value and rt.host_allocations() == live
            before = rt.host_attributes()
            assert use(h) == 0 and rt.host_attributes() == before
            rt.host_reset()

        for dim in (64, 128, 256):
            for new in (1, 16, 32, 300):
                for kv in (64, 4096):
                    st, h = attention(dim=dim)
                    assert st == 0 and attend(h, kv=kv, dim=dim, max_new=new, tokens=4 * new) == 0
        assert rt.host_lds_launched() > 65536 and rt.host_over() == 0
        rt.host_reset()
        for dtype in (R.DTYPE_BF16, R.DTYPE_FP32):
            st, h = verifier(dtype=dtype, requests=512)
            for requests in (1, 16, 24, 64, 512):
                for rules in (0, 1, 2, 3):
                    a = verify.LogitsArgs(1 << 20, 151936, 151936, requests, 1)
                    if rules & 1:
                        a.repetition = 1 << 20
                    if rules & 2:
                        a.bias_ids, a.bias_values, a.bias_width, a.bias_stride = 1 << 20, 1 << 20, 9, 9
                    assert lib.domino_verify_run(h, ctypes.byref(a), P, None, 0, P, 151936, P, P, None, None) == 0
        assert rt.host_lds_launched() > 65536 and rt.host_over() == 0
        """)


def test_tensors_of_another_gpu_are_refused(runtime):
    """A handle's workspace is on one GPU: tensors of another would be read from there on the wrong stream."""
    walk(runtime, """
        a = verify.PagedAttention(8, 2, 128, 16, max_requests=4)
        for device in (0, 1):
            q, k = (Tensor("bfloat16", 4, h, 128, device=device) for h in (8, 2))
            c = cache_tensors(device=device)
            calls = (lambda: a.run(q, *c), lambda: a.append(k, k, *c))
            for call in calls:
                if device == 0:
                    call()
                else:
                    refused(call, "the handle is on cuda:0")
        v = verify.DraftVerifier(1000, max_requests=4)
        for device in (0, 1):
            x = Tensor("bfloat16", 4, 3, 1000, device=device)
            for call in (lambda: v.run(x), lambda: v.process(x)):
                if device == 0:
                    call()
                else:
                    refused(call, "the handle is on cuda:0")
        """)


def test_numbers_beyond_32_bits_are_refused(runtime):
    """ctypes keeps the low 32 bits: a window of 2^32 + 64 would be one of 64."""
    walk(runtime, """
        a = verify.PagedAttention(8, 2, 128, 16, max_requests=4)
        q, k, c = Tensor("bfloat16", 4, 8, 128), Tensor("bfloat16", 4, 2, 128), cache_tensors()
        a.run(q, *c, window=2 ** 31 - 1, sinks=2 ** 31 - 1, max_new=2 ** 31 - 1, max_kv=2 ** 31 - 1)
        for name in ("window", "sinks", "max_new", "max_kv"):
            for x in (2 ** 32 + 64, 2 ** 31, -2 ** 31 - 1):
                refused(lambda: a.run(q, *c, **{name: x}), name)
                if name.startswith("max"):
                    refused(lambda: a.append(k, k, *c, **{name: x}), name)
        refused(lambda: verify.PagedAttention(2 ** 32 + 8, 2, 128, 16), "q_heads")
        refused(lambda: verify.PagedAttention(8, 2, 128, 2 ** 32 + 16), "page_size")
        refused(lambda: verify.DraftVerifier(2 ** 32 + 1000), "vocab")
        """)


def test_rows_of_out_that_overlap_are_refused(runtime):
    """An expanded tensor as the output of attention: several workgroups would write the same place."""
    walk(runtime, """
        st, h = attention()
        for token, head, status in ((1024, 128, 0), (128, 512, 0), (0, 128, R.DOMINO_ERR_INVALID_ARG),
                                    (1024, 0, R.DOMINO_ERR_INVALID_ARG), (1024, 64, R.DOMINO_ERR_INVALID_ARG)):
            assert attend(h, out=(token, head)) == status, (token, head)
        assert b"overlap" in lib.domino_attention_last_error(h)
        assert attend(h, tokens=1, requests=1, out=(0, 128)) == 0
        """)


def test_bounds_beyond_32_bit_sums_divide_nothing(runtime):
    """A divided call sums up steps in 32 bits from lengths that lie on the device.  Where the bounds allow more
    than that holds, each segment is taken whole, in one launch."""
    walk(runtime, """
        st, h = attention(hq=256, hk=256, dim=64, page=4096, requests=1)
        for kv, launches in ((1 << 20, 2), (1 << 29, 2), (1 << 30, 1)):
            n = rt.host_launches()
            assert st == 0 and attend(h, kv=kv, width=262144, tokens=1, hk=256, dim=64, page=4096, requests=1,
                                      out=(1 << 14, 64)) == 0
            assert rt.host_launches() == n + launches, kv
        """)
