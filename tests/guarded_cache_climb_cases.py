"""Decode over the 4-bit cache with climbing maxima, and the cases of test_gpu_cache_edges.py, through the guarded build (libmla_guard.so, path in argv[1]), as
guarded_cache_cases.py runs its own.  Prints "guarded ok" and exits 0 when every case passes."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch  # noqa: E402

from mla_attention_gb300 import _lib  # noqa: E402

_lib.LIB_PATH = sys.argv[1]

import mla_attention_gb300 as lib  # noqa: E402
import tests.test_gpu_cache_climb as climb  # noqa: E402
import tests.test_gpu_cache_edges as edges  # noqa: E402

if __name__ == "__main__":
    torch.cuda.set_device(torch.device("cuda", 0))
    climb.test_climb(5.7, 1, 1)
    climb.test_climb(6.5, 5, -1)
    climb.test_climb_rows(40, 2)
    edges.test_decode_a_nan_reaches_the_tokens_that_see_it_alone(3, 16, 0.07, 0x7F)
    edges.test_weights_of_an_infinite_key("fp4", 3, 100)
    edges.test_weights_rows_with_an_infinite_lse_add_nothing("bf16", 1, 16)
    edges.test_compact_weights_stay_with_rows_whose_page_is_none()
    torch.cuda.synchronize()
    lib.check_device_status()   # raises MLAError on a guarded-check code (0x3000 | site)
    print("guarded ok")
