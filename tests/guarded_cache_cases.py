"""Small cases of the smaller cache's calls run through the guarded build (libmla_guard.so, path in argv[1]),
each compared with the oracle, the status word read after each call: a guarded check that fires (an
access that would have left its buffer, which is skipped) fails the run.  Run as a child process by
tests/test_gpu_guarded_cache.py.  Prints "guarded ok" and exits 0 when every case passes."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch  # noqa: E402

from mla_attention_gb300 import _lib  # noqa: E402

_lib.LIB_PATH = sys.argv[1]

import mla_attention_gb300 as lib  # noqa: E402
import tests.test_gpu_cache as cases  # noqa: E402
import tests.test_gpu_cache_clusters as clusters  # noqa: E402


def decode_cases():
    for H in (1, 65, 128):
        cases.test_decode_lengths(H)
    cases.test_decode_page_sizes(7)
    cases.test_decode_several_tokens(5, 64)
    cases.test_decode_several_tokens(130, 1)
    cases.test_decode_splits(5)
    cases.test_decode_sinks()
    cases.test_decode_bad_pages_and_lengths_are_recorded()


def weights_cases():
    for fmt in cases.FORMATS:
        cases.test_weights_lengths(fmt, 16)
        cases.test_weights_page_sizes(fmt, 7)
        cases.test_weights_several_tokens(fmt, 4, 128)
        cases.test_weights_scales(fmt, 0.07, 0.25)
    cases.test_weights_bad_pages_and_lengths_are_recorded()


def select_cases():
    cases.test_select_kinds("few", 4, 32)
    cases.test_select_lengths([70000, 3, 129, 33000], 0.5)
    cases.test_select_refuses_bad_requests_alone()
    clusters.test_select_by_requests(77)
    clusters.test_select_keys_that_one_cta_cannot_hold()


def compact_cases():
    cases.test_compact(416, torch.uint8, 7)
    cases.test_compact(1152, torch.bfloat16, 64)
    cases.test_compact_skips_and_records_bad_entries()
    clusters.test_compact_by_requests(20, 1152)
    clusters.test_compact_by_requests(153, 416)
    clusters.test_compact_wide_rows(1921 * 16, 3)


def append_cases():
    cases.test_append(33, 5, False)
    cases.test_append(2, 128, True)
    cases.test_append_scales(0.75, True)
    cases.test_append_in_place_rows_and_strided_views()
    cases.test_append_bad_positions_and_slots_are_recorded()


if __name__ == "__main__":
    torch.cuda.set_device(torch.device("cuda", 0))
    for case in (decode_cases, weights_cases, select_cases, compact_cases, append_cases):
        case()
        torch.cuda.synchronize()
        lib.check_device_status()   # raises MLAError on a guarded-check code (0x3000 | site)
        print(case.__name__, "ok", flush=True)
    print("guarded ok")
