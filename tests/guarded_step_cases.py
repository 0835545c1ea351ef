"""Small cases of the serving step's calls run through the guarded build (libmla_guard.so, path in argv[1]),
each compared with the oracle, the status word read after each call: a guarded check that fires (an
access that would have left its buffer, which is skipped) fails the run.  Run as a child process by
tests/test_gpu_guarded_step.py.  Prints "guarded ok" and exits 0 when every case passes."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch  # noqa: E402

from mla_attention_gb300 import _lib  # noqa: E402

_lib.LIB_PATH = sys.argv[1]

import mla_attention_gb300 as lib  # noqa: E402
import tests.test_gpu_step as cases  # noqa: E402


def slot_map_cases():
    cases.test_slot_map_random_steps(65, 16, 7, 3)
    cases.test_slot_map_random_steps(1025, 32, 1, 6)
    cases.test_slot_map_one_long_prompt_among_single_tokens()
    cases.test_slot_map_refusals_keep_the_request(6)


def norm_cases():
    for T, D in ((3, 7), (5, 257), (130, 1024), (3, 1535), (9, 8200), (2, 32768)):
        cases._check_norm(T, D, pad=3, off=1)
    for D, group in ((576, 64), (8192, 128), (1535, 0)):
        cases._check_norm(5, D, pad=8, e4m3=True, group=group)


def append_cases():
    cases._check_append(33, 40, e4m3=True, rows_out=True)
    cases._check_append(7, 33, neox=True, norm=False)
    cases._check_append(40, 16, rows_out=True, bad=True)


def w4_cases():
    for args in ((1, 3, 512, 128, 32), (17, 2, 128, 512, 64), (65, 1, 100, 1024, 128), (5, 5, 33, 160, 32), (9, 1, 7, 4096, 128)):
        cases._check_w4(*args, f32=args[0] == 5, strided=args[0] == 9)
    cases.test_w4_large_and_small_values(9)
    for args in ((1, 128, 512, 128, 32), (17, 60, 700, 512, 64)):
        cases._check_w4(*args)


if __name__ == "__main__":
    torch.cuda.set_device(torch.device("cuda", 0))
    for case in (slot_map_cases, norm_cases, append_cases, w4_cases):
        case()
        torch.cuda.synchronize()
        lib.check_device_status()   # raises MLAError on a guarded-check code (0x3000 | site)
        print(case.__name__, "ok", flush=True)
    print("guarded ok")
