"""Host-side checks of the operators of include/hc_serve.h (no GPU needed): the header and the
binding agree, every function is exported, calls without a device fail cleanly, and shapes that
disagree are refused before any call of the library."""
import os
import re

import pytest
import torch

import hyper_connection_residual_read_gb300 as hc
from hyper_connection_residual_read_gb300 import build as hcbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(hcbuild.LIB):
        hcbuild.build()
    return hc.load()


@pytest.fixture(scope="module")
def header():
    text = open(os.path.join(ROOT, "include", "hc_serve.h")).read()
    return re.sub(r"/\*.*?\*/", "", text, flags=re.S)


def test_header_declares_the_binding(header):
    assert sorted(set(re.findall(r"\bint (hc_\w+)\s*\(", header))) == sorted(hc.SERVE_EXPORTS)


def test_every_declared_symbol_is_exported(lib):
    for name in hc.SERVE_EXPORTS:
        assert hasattr(lib, name), name


def test_binding_constants_match_the_header(header):
    macros = dict((k, int(v)) for k, v in re.findall(r"#define\s+(HC_\w+)\s+(\d+)", header))
    assert len(macros) == 2
    for name, value in macros.items():
        assert getattr(hc, name) == value, name
    members = re.search(r"typedef struct hc_rotary \{(.*?)\}", header, flags=re.S).group(1)
    names = [m.group(1) for m in re.finditer(r"(\w+);", members)]
    assert names == [f for f, _ in hc.hc_rotary._fields_]


def arguments(op):
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    codes = torch.zeros(3, 2, 2, 16, 32, dtype=torch.uint8)
    scales = torch.zeros(3, 2, 2, 16, 2, dtype=torch.bfloat16)
    if op == "rotary":
        k, q = torch.zeros(8, 2, 64, dtype=torch.bfloat16), torch.zeros(8, 4, 64, dtype=torch.bfloat16)
        w = torch.zeros(64, dtype=torch.bfloat16)
        return hc.hc_kv4_append_rotary, dict(q=q, k=k, v=k.clone(), cos_sin=torch.zeros(9, 2, 16), positions=i(3, 8),
                                             slots=torch.zeros(8, dtype=torch.int64), codes=codes, scales=scales,
                                             q_out=q.clone(), q_norm=w, k_norm=w.clone(), axis_of=i(16))
    if op == "shared":
        q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
        return hc.hc_kv4_attention_shared, dict(q=q, codes=codes, scales=scales, prefix_table=i(2, 3), prefix_lens=i(2),
                                                cu_groups=i(3), max_shared=4, block_table=i(3, 2), cu_lens=i(4), kv_lens=i(3),
                                                max_new=2, workspace=torch.zeros(5 * 4 * 66), out=q.clone(),
                                                lse=torch.zeros(5, 4), mask=torch.zeros(5, dtype=torch.int64))
    f = torch.zeros(4)
    return hc.hc_sample_tokens, dict(logits=torch.zeros(4, 9), uniform=f, tokens=i(4), logprobs=f.clone(), temperature=f.clone(),
                                     top_k=i(4), top_p=f.clone(), min_p=f.clone())


BAD = {
    "rotary": [dict(q=None), dict(q_out=None), dict(cos_sin=None), dict(positions=None), dict(k=torch.zeros(8, 1, 64).bfloat16()),
               dict(v=torch.zeros(8, 2, 64)), dict(v=torch.zeros(7, 2, 64).bfloat16()), dict(q=torch.zeros(8, 4, 32).bfloat16()),
               dict(q_out=torch.zeros(8, 5, 64).bfloat16()), dict(slots=torch.zeros(8, dtype=torch.int32)),
               dict(positions=torch.zeros(3, 7, dtype=torch.int32)), dict(positions=torch.zeros(24, dtype=torch.int32)),
               dict(positions=torch.zeros(1, 3, 8, dtype=torch.int32)), dict(cos_sin=torch.zeros(9, 3, 16)),
               dict(cos_sin=torch.zeros(9, 2, 16).double()), dict(axis_of=torch.zeros(15, dtype=torch.int32)),
               dict(q_norm=torch.zeros(32).bfloat16()), dict(k_norm=torch.zeros(64)), dict(scales=torch.zeros(3, 2, 2, 16, 2)),
               dict(codes=torch.zeros(3, 2, 2, 16, 32)), dict(k=torch.zeros(8, 2, 128).bfloat16()[..., ::2])],
    "shared": [dict(workspace=torch.zeros(5 * 4 * 66 - 1)), dict(workspace=torch.zeros(5, 4 * 66)), dict(prefix_lens=torch.zeros(2)),
               dict(cu_groups=torch.zeros(2, dtype=torch.int32)), dict(prefix_table=torch.zeros(3, 3, dtype=torch.int32)),
               dict(prefix_table=torch.zeros(6, dtype=torch.int32)), dict(block_table=torch.zeros(2, 2, dtype=torch.int32)),
               dict(cu_lens=torch.zeros(3, dtype=torch.int32)), dict(out=torch.zeros(5, 4, 64)), dict(lse=torch.zeros(5, 3)),
               dict(mask=torch.zeros(4, dtype=torch.int64)), dict(q=torch.zeros(5, 4, 32).bfloat16())],
    "sample": [dict(uniform=torch.zeros(3)), dict(tokens=torch.zeros(4)), dict(logprobs=torch.zeros(4).double()),
               dict(temperature=torch.zeros(5)), dict(top_k=torch.zeros(4)), dict(top_p=torch.zeros(4, dtype=torch.int32)),
               dict(min_p=torch.zeros(4, 1)), dict(logits=torch.zeros(4, 9).double()), dict(logits=torch.zeros(36)),
               dict(logits=torch.zeros(9, 4).t())],
}


@pytest.mark.parametrize("c_path", [True, False])
@pytest.mark.parametrize("op", list(BAD))
def test_the_binding_refuses_shapes_that_disagree(lib, op, c_path, monkeypatch):
    import hyper_connection_residual_read_gb300._serve as w
    f, good = arguments(op)
    w._load()
    if not c_path:
        monkeypatch.setattr(w, "_call", None)
    elif w._call is None:
        pytest.skip("the Python call module is not built")
    for bad in BAD[op]:
        with pytest.raises(hc.HcReadError) as e:
            f(**dict(good, **bad), stream=0)
        assert e.value.code == hc.HC_ERR_ARG, {k: tuple(v.shape) if v is not None else None for k, v in bad.items()}


@pytest.mark.parametrize("op", list(BAD))
def test_calls_without_a_device_fail_cleanly(lib, op):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; covered by the GPU tests")
    f, good = arguments(op)
    with pytest.raises(hc.HcReadError) as e:
        f(**good, stream=0)
    assert e.value.code in (hc.HC_ERR_NOT_INIT, hc.HC_ERR_CUDA)
