"""Small cases of the operators of include/hc_serve.h run in a fresh process against a given build of
the library (the bounds-checked one): each against its oracle, and the device status word clear
after each (a skipped out-of-range access would set HC_ERR_BOUNDS).

    python tests/_bounds_serve_cases.py PATH_TO_LIBRARY
"""
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, HERE)
sys.path.insert(0, os.path.dirname(HERE))

import torch  # noqa: E402

from hyper_connection_residual_read_gb300 import _lib  # noqa: E402


def main(path: str) -> None:
    _lib.load(path)
    import hyper_connection_residual_read_gb300 as hc
    import test_gpu_serve as T
    import test_gpu_serve_edges as E
    assert hc.hc_read_bounds_checked(), "not the bounds-checked build"
    hc.hc_read_init(0, 64, 1e-6)

    def done(label):
        code = hc.hc_read_status()
        assert code == hc.HC_OK, (label, code)
        print("ok", label, flush=True)

    for dtype in ("bf16", "fp32"):
        for args in ((1, 20, 4, 128, 128, 1, False, True), (17, 7, 1, 128, 96, 3, False, False), (33, 4, 2, 64, 32, 3, True, True),
                     (5, 0, 3, 128, 128, 1, True, True), (1025, 3, 1, 64, 64, 1, True, False)):
            T.test_rotary(dtype, *args)
            done(f"rotary {dtype} {args}")
    T.test_rotary_tokens_that_are_none()
    done("rotary of tokens that are none")
    for groups in T.GROUPS:
        T.test_shared(groups=groups, heads=(8, 2, 128), dtype="bf16")
        T.test_shared(groups=groups, heads=(8, 8, 64), dtype="fp16")
        done(f"shared: {groups}")
    T.test_shared_with_masks(heads=(20, 4, 128), mask=T.tree)
    T.test_shared_of_long_prefixes(prefix=4096, requests=40)
    T.test_shared_of_chunks(heads=(14, 2, 64), groups=[(500, [(64, 64), (100, 40), (40, 100)]), (77, [(0, 0), (300, 1)])])
    for columns in (0, 300):
        E.test_shared_of_many_short_requests(heads=(16, 4, 128), new=2, columns=columns)
    E.test_shared_prefixes_in_pieces_and_whole(prefix=4000, new=100)
    done("shared: masks, long prefixes, chunks, short requests, pieces")
    for dtype in ("bf16", "fp16", "fp32"):
        for args in ((1, 1), (5, 7), (64, 1000), (9, 50257), (2, 262144)):
            T.test_sample(dtype, *args)
    T.test_sample_of_difficult_rows("bf16", 1003)
    E.test_sample_of_lists_of_every_length("ties", torch.bfloat16)
    done("sample")
    print("all cases passed", flush=True)


if __name__ == "__main__":
    main(sys.argv[1])
