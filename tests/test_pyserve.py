"""The C call path of the operators of include/hc_serve.h (``_hcpyserve``) hands the entry points
the same arguments as the ctypes path. Checked on the CPU against a stub library with the same
entry points that records what it receives."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import hyper_connection_residual_read_gb300._serve as w
from hyper_connection_residual_read_gb300 import _lib

from test_serve_abi import arguments

# every argument as 64 bits, in order; structs as their members
STUB = r"""
#include <stdint.h>
#include <string.h>
struct cache { void *codes, *scales; int blocks, kv_heads, block_size, head_dim; };
struct rotary { void *cos_sin, *axis_of, *q_norm, *k_norm; float eps; int length, dim, axes, interleaved; };
static int64_t got[64];
static int n;
static void start(int op) { n = 0; got[n++] = op; }
static void p(const void* x) { got[n++] = (int64_t)(uintptr_t)x; }
static void i(int64_t x) { got[n++] = x; }
static void f(float x) { int32_t bits; memcpy(&bits, &x, 4); i(bits); }
static void c(const struct cache* k) { p(k->codes); p(k->scales); i(k->blocks); i(k->kv_heads); i(k->block_size); i(k->head_dim); }
int hc_kv4_append_rotary(const struct cache* k, const struct rotary* r, int a, int b, int d, void* q, int64_t q1, int64_t q2,
                         void* x, int64_t x1, int64_t x2, void* v, int64_t v1, int64_t v2, void* e, void* s, void* o, void* st) {
    start(1); c(k); p(r->cos_sin); p(r->axis_of); p(r->q_norm); p(r->k_norm); f(r->eps); i(r->length); i(r->dim); i(r->axes);
    i(r->interleaved); i(a); i(b); i(d); p(q); i(q1); i(q2); p(x); i(x1); i(x2); p(v); i(v1); i(v2); p(e); p(s); p(o); p(st);
    return r->length == 77 ? -3 : 0;
}
int hc_kv4_attention_shared(const struct cache* k, int a, int b, int d, int e, int g, int h, int j, int l, float m, int t, void* q,
                            int64_t q1, int64_t q2, void* r1, void* r2, void* r3, void* r4, void* r5, void* r6, void* r7, void* r8,
                            void* r9, void* s1, void* s2) {
    start(2); c(k); i(a); i(b); i(d); i(e); i(g); i(h); i(j); i(l); f(m); i(t); p(q); i(q1); i(q2); p(r1); p(r2); p(r3); p(r4); p(r5);
    p(r6); p(r7); p(r8); p(r9); p(s1); p(s2);
    return 0;
}
int hc_sample_tokens(int a, int b, int d, void* x, int64_t r, void* u, void* t, void* k, void* q, void* m, void* o, void* l, void* s) {
    start(3); i(a); i(b); i(d); p(x); i(r); p(u); p(t); p(k); p(q); p(m); p(o); p(l); p(s);
    return 0;
}
int stub_n(void) { return n; }
int64_t stub_got(int k) { return got[k]; }
void stub_clear(void) { n = 0; }
"""


@pytest.fixture()
def stub(tmp_path, monkeypatch):
    try:
        from hyper_connection_residual_read_gb300 import _hcpyserve  # noqa: F401
    except ImportError:
        pytest.skip("the Python call module is not built")
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "stub.c"
    src.write_text(STUB)
    so = tmp_path / "libstub.so"
    subprocess.run([cc, "-O1", "-shared", "-fPIC", str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(os.fspath(so))
    lib.stub_got.restype = ctypes.c_int64
    real = w._bound
    monkeypatch.setattr(_lib, "load", lambda *a: lib)
    monkeypatch.setattr(_lib, "strerror", lambda code: str(code))
    monkeypatch.setattr(w, "_bound", None)
    monkeypatch.setattr(w, "_call", None)
    w._load()
    yield lib, w._call
    if real is not None:
        w._bind_call(real)


def both(stub, monkeypatch, f, **kw):
    """What the entry point receives by the C path and by ctypes; and the status codes."""
    lib, call = stub
    seen = []
    for path in (call, None):
        monkeypatch.setattr(w, "_call", path)
        lib.stub_clear()
        code = 0
        try:
            f(**kw, stream=77)
        except w._lib.HcReadError as e:
            code = e.code
        seen.append((code, [lib.stub_got(k) for k in range(lib.stub_n())]))
    assert seen[0] == seen[1]
    return seen[0]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_rotary(stub, monkeypatch, dtype):
    f, good = arguments("rotary")
    for name in ("q", "k", "v", "q_out", "q_norm", "k_norm"):
        good[name] = good[name].to(dtype)
    fused = torch.zeros(8, 8 * 64, dtype=dtype)
    variants = [{}, dict(q=None, q_out=None), dict(cos_sin=None, positions=None, axis_of=None), dict(q_norm=None), dict(k_norm=None),
                dict(axis_of=None, positions=torch.zeros(8, dtype=torch.int32)), dict(interleaved=True, eps=0.25),
                dict(q=fused[:, :256].view(8, 4, 64), k=fused[:, 256:384].view(8, 2, 64), v=fused[:, 384:].view(8, 2, 64)),
                dict(q=torch.zeros(4, 8, 64, dtype=dtype).transpose(0, 1)), dict(cos_sin=torch.zeros(77, 2, 16))]
    for other in variants:
        kw = dict(good, **other)
        code, got = both(stub, monkeypatch, f, **kw)
        assert got[0] == 1 and got[1] == kw["codes"].data_ptr() and got[-1] == 77
        assert code == (-3 if "cos_sin" in other and other["cos_sin"] is not None else 0)
        assert got[7] == (0 if kw["cos_sin"] is None else kw["cos_sin"].data_ptr())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_shared(stub, monkeypatch, dtype):
    f, good = arguments("shared")
    good["q"], good["out"] = good["q"].to(dtype), good["out"].to(dtype)
    for other in ({}, dict(lse=None), dict(mask=None), dict(lse=None, mask=None, scale=0.3), dict(workspace=torch.zeros(9999)),
                  dict(q=torch.zeros(5, 12, 64, dtype=dtype)[:, 3:7])):
        kw = dict(good, **other)
        code, got = both(stub, monkeypatch, f, **kw)
        assert code == 0 and got[0] == 2 and got[7:15] == [3, 2, 5, 4, 2, 4, 2, 3]
        assert got[-4:] == [kw["workspace"].data_ptr(), kw["out"].data_ptr(), kw["lse"].data_ptr() if kw["lse"] is not None else 0, 77]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_sample(stub, monkeypatch, dtype):
    f, good = arguments("sample")
    for other in ({}, dict(temperature=None), dict(top_k=None), dict(top_p=None), dict(min_p=None),
                  dict(temperature=None, top_k=None, top_p=None, min_p=None), dict(logits=torch.zeros(8, 20)[::2, 3:12])):
        kw = dict(good, **other)
        kw["logits"] = kw["logits"].to(dtype)
        code, got = both(stub, monkeypatch, f, **kw)
        assert code == 0 and got[0] == 3 and got[1:3] == [4, 9] and got[5] == kw["logits"].stride(0)


def test_other_objects_raise_as_python_does(stub):
    f, good = arguments("sample")
    for bad in (dict(uniform=3), dict(logits="x"), dict(top_k=[1])):
        with pytest.raises((AttributeError, TypeError)):
            f(**dict(good, **bad), stream=0)
