"""The serving step's binding on the host: sizes beyond the C ABI's 32-bit arguments, two threads' first calls (CPU
only: nothing is launched)."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import mla_attention_gb300 as m
from mla_attention_gb300 import _lib, _step


class Shaped:
    """Stands in for a tensor on GPU 0 of any size: what the binding asks of one, without its memory."""

    made = 0

    def __init__(self, dtype, *shape):
        self.dtype, self.shape, self.device = dtype, shape, torch.device("cuda", 0)
        Shaped.made += 1
        self.at = Shaped.made << 20

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def stride(self, dim=None):
        st = [1]
        for n in reversed(self.shape[1:]):
            st.insert(0, st[0] * n)
        return tuple(st) if dim is None else st[dim]

    def data_ptr(self):
        return self.at


def bf16(*shape):
    return Shaped(torch.bfloat16, *shape)


def i32(*shape):
    return Shaped(torch.int32, *shape)


@pytest.fixture
def word(monkeypatch):
    """A status word of GPU 0, so that no call makes one."""
    from mla_attention_gb300 import build as b
    b.build()
    monkeypatch.setitem(_lib._status_cache, 0, torch.zeros(256, dtype=torch.uint8))


BIG = 2 ** 32 + 128          # 128 in 32 bits


def norm(D):
    m.mla_rms_norm(bf16(1, D), bf16(D), out=bf16(1, D), stream=0)


def w4(H=1, N=64, K=128):
    m.mla_bmm_w4(bf16(1, H, K), Shaped(torch.uint8, H, N, K // 2), bf16(H, N, K // 128), out=bf16(1, H, N), stream=0)


def append(H=1, page=16, max_pos=64):
    m.mla_kv_append(bf16(1, 512), bf16(1, 64), i32(1), i32(1), Shaped(torch.float32, max_pos, 64), bf16(2, page, 576), q_pe=bf16(1, H, 64),
                    q_out=bf16(1, H, 576), stream=0)


def slot_map(page_size=16, max_pages=4):
    m.mla_slot_map(i32(2), i32(2), i32(2, max_pages), i32(8), i32(2), page_size, 4, positions=i32(4), slots=i32(4), cu_tokens=i32(3),
                   lens_out=i32(2), pool_state_out=i32(2), stream=0)


@pytest.mark.parametrize("call,kw,status,what", [
    (norm, dict(D=BIG), 2, "D"), (w4, dict(H=BIG), 1, "H"), (w4, dict(N=BIG), 1, "N"), (w4, dict(K=BIG), 1, "K"),
    (append, dict(H=BIG), 1, "H"),
    (append, dict(page=BIG), 1, "page"), (append, dict(max_pos=BIG), 1, "max_pos"), (slot_map, dict(page_size=BIG), 1, "page_size"),
    (slot_map, dict(page_size=16 - 2 ** 32), 1, "page_size"), (slot_map, dict(max_pages=BIG), 1, "max_pages")])
def test_sizes_beyond_32_bits_are_refused(word, call, kw, status, what):
    with pytest.raises(m.MLAError) as e:
        call(**kw)
    assert e.value.status == status and what in str(e.value), e.value


def test_two_threads_first_calls_share_one_status_word(monkeypatch):
    """Both threads find no buffer and wait for their own; the address that each goes on with must be the one that is kept."""
    meet = threading.Barrier(2)

    class Stream:
        def synchronize(self):   # lets the other thread run up to here
            try:
                meet.wait(timeout=2)
            except threading.BrokenBarrierError:
                pass             # the other one waits for a lock, or has found the buffer

    zeros = torch.zeros
    monkeypatch.setattr(_lib, "_status_cache", {})
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **k: zeros(*a, **k))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: Stream())
    got = []
    threads = [threading.Thread(target=lambda: got.append(_step._workspace(None, 0))) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    kept = _lib._status_cache[0]
    assert got == [(kept.data_ptr(), 256)] * 2


def test_a_thread_that_finds_the_function_knows_the_number_of_devices(monkeypatch):
    """A second thread's call on GPU 1, made as soon as the first thread's call has looked the function up, runs on GPU 1."""
    on, current = [], [0]

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.was, current[0] = current[0], self.dev

        def __exit__(self, *_):
            current[0] = self.was

    def second(*_):
        on.append(current[0])
        return 0

    class Functions(dict):
        def __setitem__(self, name, fn):        # the first thread stops here, just behind the store
            super().__setitem__(name, second)
            _step._call(name, 1, 0)

    monkeypatch.setattr(_step, "_functions", Functions())
    monkeypatch.setattr(_step, "_several_devices", None)
    monkeypatch.setattr(_lib, "lib", lambda: type("L", (), {"mla_rms_norm": second}))
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    _step._call("mla_rms_norm", 0, 0)
    assert on == [1, 0]


def test_the_package_imports_with_a_torch_without_cuda():
    """Such a build has no _cuda_* functions; the oracle's and the inputs' users need none."""
    code = ("import torch\nfor n in dir(torch._C):\n    if n.startswith('_cuda_'): delattr(torch._C, n)\n"
            "import mla_attention_gb300 as m\nprint(len(m.__all__))")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and int(r.stdout) == len(m.__all__), r.stderr[-2000:]
