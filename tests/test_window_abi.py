"""Host-side checks of the verify-window operators (no GPU needed): the header and the
binding agree, every function is exported, and calls without a device fail cleanly."""
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
    text = open(os.path.join(ROOT, "include", "hc_window.h")).read()
    return re.sub(r"/\*.*?\*/", "", text, flags=re.S)


def test_header_declares_the_binding(header):
    assert sorted(set(re.findall(r"\bint (hc_\w+)\s*\(", header))) == sorted(hc.WINDOW_EXPORTS)


def test_every_declared_symbol_is_exported(lib):
    for name in hc.WINDOW_EXPORTS:
        assert hasattr(lib, name), name


def test_binding_constants_match_the_header(header):
    enums = dict((k, int(v)) for k, v in re.findall(r"\b(HC_DTYPE_\w+)\s*=\s*(\d+)", header))
    macros = dict((k, int(v)) for k, v in re.findall(r"#define\s+(HC_\w+)\s+(\d+)", header))
    assert len(enums) == 3 and len(macros) == 5
    for name, value in {**enums, **macros}.items():
        assert getattr(hc, name) == value, name


def test_calls_without_a_device_fail_cleanly(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; covered by the GPU tests")
    i = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    with pytest.raises(hc.HcReadError) as e:
        hc.hc_window_plan(i(1), i(1), i(4), i(1), 16, i(4).view(1, 4), torch.zeros(8, dtype=torch.int64),
                          i(8), i(8), i(2), i(1), i(1), stream=0)
    assert e.value.code in (hc.HC_ERR_NOT_INIT, hc.HC_ERR_CUDA)
    with pytest.raises(hc.HcReadError):
        hc.hc_token_logprobs(torch.zeros(1, 8), i(1), torch.zeros(1), torch.zeros(1), torch.zeros(1),
                             i(1), i(2).view(1, 2), torch.zeros(1, 2), stream=0)


def test_the_binding_refuses_shapes_that_disagree(lib):
    """Before any call of the library: the same error as its own refusals."""
    i = lambda *n: torch.zeros(*n, dtype=torch.int32)  # noqa: E731
    slots = torch.zeros(8, dtype=torch.int64)
    good = [i(2), i(2), i(4), i(1), 16, i(2, 4), slots, i(8), i(8), i(3), i(2), i(1)]
    bad = {1: i(3), 5: i(3, 4), 6: slots.int(), 7: i(7), 9: i(2), 11: i(2), 3: i(1).long()}
    for at, x in bad.items():
        with pytest.raises(hc.HcReadError) as e:
            hc.hc_window_plan(*[x if k == at else y for k, y in enumerate(good)], stream=0)
        assert e.value.code == hc.HC_ERR_ARG
    codes = torch.zeros(3, 2, 2, 16, 32, dtype=torch.uint8)
    scales = torch.zeros(3, 2, 2, 16, 2, dtype=torch.bfloat16)
    k = torch.zeros(8, 2, 64, dtype=torch.bfloat16)
    for args in [(k[:, :1], k[:, :1], slots, codes, scales), (k, k.half(), slots, codes, scales),
                 (k, k, slots[:4], codes, scales), (k.double(), k.double(), slots, codes, scales),
                 (k, k, slots, codes[:, :1], scales), (k, k, slots, codes, scales[:2]),
                 (k[..., ::2], k[..., ::2], slots, codes, scales)]:
        with pytest.raises(hc.HcReadError) as e:
            hc.hc_kv4_append(*args, stream=0)
        assert e.value.code == hc.HC_ERR_ARG
