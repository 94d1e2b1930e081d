"""The window operators' C call path (``_hcpywindow``) hands the entry points the same
arguments as the ctypes path, and refuses the same tensors. Checked on the CPU against a
stub library with the same five entry points that records what it receives."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import hyper_connection_residual_read_gb300._window as w
from hyper_connection_residual_read_gb300 import _lib

# every argument as 64 bits, in order; a cache as its six members
STUB = r"""
#include <stdint.h>
#include <string.h>
struct cache { void *codes, *scales; int blocks, kv_heads, block_size, head_dim; };
static int64_t got[32];
static int n;
static void start(int op) { n = 0; got[n++] = op; }
static void p(void* x) { got[n++] = (int64_t)(uintptr_t)x; }
static void i(int64_t x) { got[n++] = x; }
static void c(const struct cache* k) { p(k->codes); p(k->scales); i(k->blocks); i(k->kv_heads); i(k->block_size); i(k->head_dim); }
int hc_window_plan(int a, int b, int d, int e, int f, void* g, void* h, void* j, void* k, void* l, void* m,
                   void* o, void* q, void* r, void* s, void* t, void* u) {
    start(1); i(a); i(b); i(d); i(e); i(f); p(g); p(h); p(j); p(k); p(l); p(m); p(o); p(q); p(r); p(s); p(t); p(u);
    return d == 99 ? -3 : 0;
}
int hc_kv4_append(const struct cache* k, int a, int b, void* d, int64_t e, int64_t f, void* g, int64_t h,
                  int64_t j, void* l, void* m) {
    start(2); c(k); i(a); i(b); p(d); i(e); i(f); p(g); i(h); i(j); p(l); p(m);
    return 0;
}
int hc_kv4_load(const struct cache* k, int a, void* b, int d, void* e, void* f, void* g) {
    start(3); c(k); i(a); p(b); i(d); p(e); p(f); p(g);
    return 0;
}
int hc_kv4_attention(const struct cache* k, int a, int b, int d, int e, int f, float g, int h, void* j, int64_t l,
                     int64_t m, void* o, void* q, void* r, void* s, void* t, void* u, void* v) {
    int32_t bits;
    memcpy(&bits, &g, 4);
    start(4); c(k); i(a); i(b); i(d); i(e); i(f); i(bits); i(h); p(j); i(l); i(m); p(o); p(q); p(r); p(s); p(t); p(u); p(v);
    return 0;
}
int hc_token_logprobs(int a, int b, int d, int e, void* f, int64_t g, void* h, void* j, void* k, void* l, void* m,
                      void* o, void* q, void* r) {
    start(5); i(a); i(b); i(d); i(e); p(f); i(g); p(h); p(j); p(k); p(l); p(m); p(o); p(q); p(r);
    return 0;
}
int stub_n(void) { return n; }
int64_t stub_got(int k) { return got[k]; }
void stub_clear(void) { n = 0; }
"""


@pytest.fixture()
def stub(tmp_path, monkeypatch):
    try:
        from hyper_connection_residual_read_gb300 import _hcpywindow  # noqa: F401
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


def both(stub, monkeypatch, fn, *args, **kw):
    """What the entry point receives by the C path and by ctypes; and the status codes."""
    lib, call = stub
    seen = []
    for path in (call, None):
        monkeypatch.setattr(w, "_call", path)
        lib.stub_clear()
        code = 0
        try:
            fn(*args, **kw, stream=77)
        except w.HcReadError as e:
            code = e.code
        seen.append((code, [lib.stub_got(k) for k in range(lib.stub_n())]))
    assert seen[0] == seen[1]
    return seen[0]


def i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


def test_plan(stub, monkeypatch):
    slots = torch.zeros(9, dtype=torch.int64)
    good = [i32(3), i32(3), i32(5), i32(1), 16, i32(3, 4), slots, i32(9), i32(9), i32(4), i32(3), i32(1)]
    code, got = both(stub, monkeypatch, w.hc_window_plan, *good)
    assert code == 0 and got[:6] == [1, 3, 4, 16, 9, 5] and got[-1] == 77
    assert got[6:17] == [t.data_ptr() for k, t in enumerate(good) if k != 4]
    assert both(stub, monkeypatch, w.hc_window_plan, *[99 if k == 4 else t for k, t in enumerate(good)])[0] == -3
    for at, bad in {0: i32(3, 1), 1: i32(4), 2: i32(5).long(), 3: i32(2), 5: i32(4, 3).t(), 6: i32(9), 8: i32(8),
                    9: i32(3), 10: i32(3).float(), 11: i32(0)}.items():
        code, got = both(stub, monkeypatch, w.hc_window_plan, *[bad if k == at else t for k, t in enumerate(good)])
        assert (code, got) == (w.HC_ERR_ARG, []), at


def cache():
    return (torch.zeros(3, 2, 2, 16, 32, dtype=torch.uint8), torch.zeros(3, 2, 2, 16, 2, dtype=torch.bfloat16))


def test_append_and_load(stub, monkeypatch):
    codes, scales = cache()
    slots = torch.zeros(7, dtype=torch.int64)
    for dtype, number in ((torch.bfloat16, 0), (torch.float16, 1), (torch.float32, 2)):
        fused = torch.zeros(7, 5, 64, dtype=dtype)
        k, v = fused[:, 1:3], torch.zeros(2, 7, 64, dtype=dtype).transpose(0, 1)
        code, got = both(stub, monkeypatch, w.hc_kv4_append, k, v, slots, codes, scales)
        assert code == 0 and got == [2, codes.data_ptr(), scales.data_ptr(), 3, 2, 16, 64, 7, number, k.data_ptr(),
                                     320, 64, v.data_ptr(), 64, 448, slots.data_ptr(), 77]
        out = [torch.zeros(7, 2, 64, dtype=dtype) for _ in range(2)]
        code, got = both(stub, monkeypatch, w.hc_kv4_load, slots, codes, scales, *out)
        assert code == 0 and got[7:] == [7, slots.data_ptr(), number, out[0].data_ptr(), out[1].data_ptr(), 77]
        assert both(stub, monkeypatch, w.hc_kv4_load, slots, codes, scales, out[0], fused[:, :2])[0] == w.HC_ERR_ARG
    k = torch.zeros(7, 2, 64)
    for args in [(k.double(), k.double(), slots, codes, scales), (k, k.half(), slots, codes, scales),
                 (k, k[:6], slots, codes, scales), (k[:, :1], k[:, :1], slots, codes, scales),
                 (k, k, slots.int(), codes, scales), (k, k, slots, codes.int(), scales),
                 (k, k, slots, codes[:, :, :, ::2], scales), (k, k, slots, codes, scales[:, :, :1]),
                 (k, k, slots, codes[0], scales), (k[0], k[0], slots, codes, scales),
                 (k, k.transpose(1, 2).contiguous().transpose(1, 2), slots, codes, scales)]:
        assert both(stub, monkeypatch, w.hc_kv4_append, *args) == (w.HC_ERR_ARG, [])


def test_attention(stub, monkeypatch):
    codes, scales = cache()
    q = torch.zeros(5, 6, 64, dtype=torch.float16)[:, 1:5]
    table, cu, kv, out = i32(2, 9), i32(3), i32(2), torch.zeros(5, 4, 64, dtype=torch.float16)
    lse, mask = torch.zeros(5, 4), torch.zeros(5, dtype=torch.int64)
    good = dict(q=q, codes=codes, scales=scales, block_table=table, cu_lens=cu, kv_lens=kv, max_new=3, out=out)
    bits = lambda x: int(torch.tensor(x, dtype=torch.float32).view(torch.int32))  # noqa: E731
    code, got = both(stub, monkeypatch, w.hc_kv4_attention, **good)
    assert code == 0 and got[7:] == [2, 5, 4, 3, 9, bits(0.125), 1, q.data_ptr(), 384, 64, cu.data_ptr(), kv.data_ptr(),
                                     table.data_ptr(), 0, out.data_ptr(), 0, 77]
    code, got = both(stub, monkeypatch, w.hc_kv4_attention, **good, lse=lse, mask=mask, scale=3)
    assert code == 0 and got[12] == bits(3.0) and got[20] == mask.data_ptr() and got[22] == lse.data_ptr()
    for bad in (dict(q=q[:, :3]), dict(q=q.transpose(1, 2)), dict(out=out.bfloat16()), dict(lse=lse.t()),
                dict(mask=mask[:4]), dict(mask=mask.int()), dict(kv_lens=i32(3)), dict(cu_lens=i32(2)),
                dict(block_table=i32(9)), dict(block_table=table.long()), dict(kv_lens=kv.view(1, 2))):
        assert both(stub, monkeypatch, w.hc_kv4_attention, **{**good, **bad}) == (w.HC_ERR_ARG, []), bad


def test_logprobs(stub, monkeypatch):
    x = torch.zeros(4, 50, dtype=torch.bfloat16)[:, 3:40]
    out = [torch.zeros(4), torch.zeros(4), torch.zeros(4), i32(4), i32(4, 6), torch.zeros(4, 6)]
    code, got = both(stub, monkeypatch, w.hc_token_logprobs, x, i32(4), *out)
    assert code == 0 and got[:7] == [5, 4, 37, 6, 0, x.data_ptr(), 50] and got[-1] == 77
    assert got[8:14] == [t.data_ptr() for t in out]
    for bad in [(x.t(), i32(4), *out), (x, i32(5), *out), (x.int(), i32(4), *out), (x, i32(4).long(), *out),
                (x, i32(4), *out[:4], i32(4, 5), out[5]), (x, i32(4), out[3], *out[1:]), (x[0], i32(4), *out),
                (x, i32(4), *out[:4], i32(24), out[5])]:
        assert both(stub, monkeypatch, w.hc_token_logprobs, *bad) == (w.HC_ERR_ARG, [])


def test_arguments_that_are_no_tensors_raise(stub):
    _, call = stub
    codes, scales = cache()
    with pytest.raises(AttributeError):
        call.append(1, 2, 3, codes, scales, 0)
    with pytest.raises(TypeError):
        call.append(codes)
    with pytest.raises(OverflowError):
        call.plan(*[i32(1)] * 4, 1 << 40, i32(1, 1), *[i32(1)] * 6, 0)
