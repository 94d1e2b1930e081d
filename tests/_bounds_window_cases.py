"""Small cases of the window operators run in a fresh process against a given build of the
library (the bounds-checked one): each against its oracle, and the device status word clear
after each (a skipped out-of-range access would set HC_ERR_BOUNDS).

    python tests/_bounds_window_cases.py PATH_TO_LIBRARY
"""
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, HERE)
sys.path.insert(0, os.path.dirname(HERE))

import numpy as np  # noqa: E402
import torch  # noqa: E402

from hyper_connection_residual_read_gb300 import _lib  # noqa: E402


def main(path: str) -> None:
    _lib.load(path)
    import hyper_connection_residual_read_gb300 as hc
    import test_gpu_window as T
    assert hc.hc_read_bounds_checked(), "not the bounds-checked build"
    hc.hc_read_init(0, 64, 1e-6)

    def done(label):
        code = hc.hc_read_status()
        assert code == hc.HC_OK, (label, code)
        print("ok", label, flush=True)

    for args in ((1, 1, 0, 16, 1.0), (33, 4, 3000, 64, 1.0), (1500, 40, 200, 16, 0.7), (8192, 3, 20, 16, 0.3)):
        T.test_plan(*args)
        done(f"plan {args}")
    for dtype in ("bf16", "fp16", "fp32"):
        for args in ((1, 1, 64, 16), (17, 3, 128, 32), (200, 2, 128, 64)):
            T.test_append_and_load(dtype, *args)
            done(f"append and load {dtype} {args}")
    # windows of 8 and 16 rows; 17 to 128 rows; more; single tokens; split requests; strides
    for heads in ((8, 8, 64), (8, 2, 128), (7, 1, 64)):
        T.test_attention_of_single_tokens(heads, "bf16", 16)
        for mask in (None, T.tree, T.holes):
            T.test_attention_of_verify_windows(heads, "fp16", mask)
        done(f"attention of windows {heads}")
    for heads in ((8, 8, 64), (5, 1, 128)):
        for lens in ([(33, 33)], [(64, 64), (100, 40), (40, 100), (0, 0), (300, 1)], [(700, 300)]):
            T.test_attention_of_chunks(heads=heads, dtype="bf16", lens=lens)
        T.test_attention_with_masks_of_64_tokens(heads=(8, 2, 128))
        done(f"attention of chunks {heads}")
    for new in (1, 6, 40):
        T.test_attention_over_long_caches(length=4096, new=new)
    T.test_attention_of_many_short_requests()
    T.test_attention_of_many_chunks((8, 4, 128))
    T.test_attention_of_chunks_that_see_no_cache()
    T.test_attention_strides_streams_and_repeats()
    done("attention of many requests")
    for dtype in ("bf16", "fp16", "fp32"):
        for args in ((1, 1, 1), (1, 7, 7), (3, 33, 0), (5, 50257, 5), (300, 2048, 1), (1, 200003, 32)):
            T.test_logprobs(dtype, *args)
    for dtype in ("bf16", "fp32"):
        T.test_logprobs_of_difficult_rows(dtype, 1003)
    done("log probabilities")

    # what the checks compare with: lengths of arrays as the call's arguments give them, so that
    # an entry outside is still found, and nothing outside is touched
    codes, scales = T.blank_cache(2, 1, 16, 64)
    guard = codes.clone()
    k = torch.ones(3, 1, 64, device="cuda")
    hc.hc_kv4_append(k, k, torch.tensor([32, 1 << 40, -1]).cuda(), codes, scales)
    assert hc.hc_read_status() == hc.HC_ERR_BOUNDS and torch.equal(codes, guard)
    c = T.Case(12, [(100, 2), (50, 2)], 4, 2, 64, 16, "bf16")
    c.table[0, 3] = 1 << 20
    out, _ = c.run()
    assert hc.hc_read_status() == hc.HC_ERR_BOUNDS and bool(np.isfinite(T.f64(out)[2:]).all())
    done("entries outside")
    print("all cases passed", flush=True)


if __name__ == "__main__":
    main(sys.argv[1])
