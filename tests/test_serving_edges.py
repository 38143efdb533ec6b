"""Edges of the serving calls' host side, without a GPU: CPU tensors without elements and plain objects stand in for CUDA
tensors, and nothing is launched."""
import ctypes
import os
import struct
import subprocess
import sys
import sysconfig
import threading
import time

import pytest
import torch

import ring_attention_slope_gb300 as slope
from _lib import ROOT, built_lib
from ring_attention_slope_gb300 import _build
from test_serving_abi import F32, S_OK, cache, ref, t
from test_serving_marshal import Fake

BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    return built_lib()


@pytest.fixture
def on_cpu(lib, monkeypatch):
    """The public calls with the host's memory in the place of the device's."""
    slope.serving._bound()
    monkeypatch.setattr(slope.serving, "_device", lambda: 0)
    monkeypatch.setattr(slope.serving, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(slope.serving, "_alloc", lambda size, stride, dtype: torch.empty_strided(size, stride, dtype=dtype))


# ---------------------------------------------------------------- no tokens

@pytest.mark.parametrize("stride", [[0, 1], [1, 1], [7, 1]])
def test_lse_strides_without_rows(lib, stride):
    """A dense [H, S] has strides (S, 1): without rows the first is 0, and no address is made with it."""
    lse = t([8, 0], F32, data=0, stride=stride)
    q, k = t([0, 8, 64], data=0), t([0, 2, 64], data=0)
    cu = (ctypes.c_int64 * 2)(0, 0)
    assert lib.slope_attn_varlen(ref(q), ref(k), ref(k), cu, 1, 1, 0, 0.0, ref(q), ref(lse), None) == S_OK
    assert lib.slope_kv4_attn(ref(q), ref(cache()), 0x6000, 5, 5, 0x7000, 1, 0, 0.0, ref(q), ref(lse), None, 0, None) == S_OK


def test_lse_strides_with_rows_are_still_checked(lib):
    q, k = t([3, 8, 64]), t([3, 2, 64])
    cu = (ctypes.c_int64 * 2)(0, 0)
    for stride in ([0, 1], [3, 0], [-3, 1]):
        lse = t([8, 3], F32, stride=stride)
        assert lib.slope_attn_varlen(ref(q), ref(k), ref(k), cu, 1, 1, 0, 0.0, ref(q), ref(lse), None) == -4


@pytest.mark.parametrize("stride", [[64, 0, 1], [0, 0, 0], [1, 7, 3]])
def test_strides_without_rows(lib, stride):
    """PyTorch gives a [0, 1, d] that an operation made strides of (d, 0, 1): they say nothing."""
    q, lse = t([0, 1, 64], data=0, stride=stride), t([1, 0], F32, data=0, stride=[0, 1])
    cu = (ctypes.c_int64 * 1)(0)
    assert lib.slope_attn_varlen(ref(q), ref(q), ref(q), cu, 0, 1, 0, 0.0, ref(q), ref(lse), None) == S_OK
    assert lib.slope_kv4_attn(ref(q), ref(cache(H=1)), 0x6000, 5, 5, 0x7000, 1, 0, 0.0, ref(q), ref(lse), None, 0, None) == S_OK
    assert lib.slope_attn_partial(ref(q), ref(q), ref(q), 0, 0, 1, 0, 0.0, ref(q), ref(lse), None) == S_OK
    assert lib.slope_kv4_write(ref(cache(H=1)), ref(q), ref(q), None, None) == S_OK
    assert lib.slope_qk_norm_rope(ref(q), None, None, None, 1, 1e-6, None, None, 0, ref(q), None, None) == S_OK


def test_calls_without_tokens_make_their_outputs(on_cpu):
    """Every output left to the call: a batch without sequences is a no-op, not an error."""
    q, k = torch.empty(0, 8, 64, dtype=BF), torch.empty(0, 2, 64, dtype=BF)
    for cu in ([0], [0, 0], [0, 0, 0]):
        out, lse = slope.attn_varlen(q, k, k, cu)
        assert out.shape == (0, 8, 64) and lse.shape == (8, 0)
    held = slope.KV4Cache(0, 16, 2, 64, 64, device="cpu")
    none = torch.empty(0, dtype=torch.int32)
    for pages in (0, 5):
        out, lse = slope.kv4_attn(q, held, torch.empty(0, pages, dtype=torch.int32), none, q_len=3,
                                  workspace=workspace())
        assert out.shape == (0, 8, 64) and lse.shape == (8, 0)
    slope.kv4_write(held, k, k, none)
    assert [x.shape for x in slope.kv4_read(held, none)] == [(0, 2, 64)] * 2
    assert [x.shape for x in slope.qk_norm_rope(q, k)] == [(0, 8, 64), (0, 2, 64)]


def workspace():
    ws = Fake([1 << 24], torch.uint8, ptr=0x100000)
    ws.nbytes, ws.is_contiguous = 1 << 24, lambda: True
    return ws


# ---------------------------------------------------------------- a cache whose memory moves

class FakeData(Fake):
    """Bytes at an address."""

    def __init__(self, n, ptr, dtype=torch.uint8, cuda=True, dense=True):
        super().__init__([n], dtype, ptr=ptr, device=0 if cuda else -1)
        self.is_cuda, self.device, self.dense, self.held = cuda, "cuda:0" if cuda else "cpu", dense, n

    def is_contiguous(self):
        return self.dense

    def untyped_storage(self):
        return self

    def nbytes(self):
        return self.held

    def storage_offset(self):
        return 0


class Recorder:
    """Stands in for the C module: keeps the cache structure that a call was given."""

    def __init__(self, real):
        self.real, self.got = real, None

    def __getattr__(self, name):
        if name in ("cache_bytes", "attn_workspace_size"):
            return getattr(self.real, name)

        def call(*args):
            packed = next(a for a in args if isinstance(a, bytes))
            self.got = struct.unpack("@Pqiiii", packed)
            return 0
        return call


def test_cache_follows_its_data(on_cpu, monkeypatch):
    """Another tensor in the place of `data`, or the same one with other memory: the next call goes there."""
    recorder = Recorder(slope.serving._bound())
    monkeypatch.setattr(slope.serving, "_marshal", recorder)
    n = 4 * 4 * 2 * 1280
    held = slope.KV4Cache(4, 64, 2, 64, 64, data=FakeData(n, 0x10000))
    k, slots, q = Fake([3, 2, 64]), Fake([3], torch.int32), Fake([3, 8, 64])
    calls = (lambda: slope.kv4_write(held, k, k, slots), lambda: slope.kv4_read(held, slots, k_out=k, v_out=k),
             lambda: slope.kv4_attn(q, held, Fake([3, 4], torch.int32), slots, out=q, lse=Fake([8, 3], torch.float32),
                                    workspace=workspace()))
    for i, call in enumerate(calls):
        call()
        assert recorder.got == (held.data.ptr, 4, 64, 2, 64, 64)
        held.data = FakeData(n + i, 0x20000 + 0x10000 * i)
        call()
        assert recorder.got == (0x20000 + 0x10000 * i, 4, 64, 2, 64, 64)
        held.data.ptr = 0x70000 + 0x10000 * i
        call()
        assert recorder.got == (0x70000 + 0x10000 * i, 4, 64, 2, 64, 64)
    now = held.data
    for other, error in ((FakeData(n - 1, 0x50000), ValueError), (FakeData(n, 0x50000, torch.int8), TypeError),
                         (FakeData(n, 0x50000, cuda=False), TypeError), (FakeData(n, 0x50000, dense=False), TypeError)):
        with pytest.raises(error):
            held.data = other
        calls[0]()
        assert held.data is now and recorder.got[0] == now.ptr
    now.ptr, now.held = 0x90000, n - 1  # its storage has shrunk
    for call in calls:
        with pytest.raises(ValueError):
            call()
    for name in ("n_pages", "page_size", "Hkv", "dqk", "dv"):
        with pytest.raises(AttributeError):
            setattr(held, name, 1)
    assert (held.n_pages, held.page_size, held.Hkv, held.dqk, held.dv) == (4, 64, 2, 64, 64)


def test_strided_workspace_is_refused(on_cpu, monkeypatch):
    """The workspace's bytes are used as one run: of a view with gaps that would be the gaps' memory too."""
    monkeypatch.setattr(slope.serving, "_marshal", Recorder(slope.serving._bound()))
    held = slope.KV4Cache(4, 64, 2, 64, 64, data=FakeData(4 * 4 * 2 * 1280, 0x10000))
    q, lens = Fake([3, 8, 64]), Fake([3], torch.int32)
    call = lambda ws: slope.kv4_attn(q, held, Fake([3, 4], torch.int32), lens, out=q, want_lse=False, workspace=ws)  # noqa: E731
    ws = workspace()
    call(ws)
    ws.is_contiguous = lambda: False
    with pytest.raises(ValueError):
        call(ws)


# ---------------------------------------------------------------- other threads during a call

WAITER = """
#include <time.h>
volatile int entered, released;
/* Stands in for a library call whose launch waits: 0 once another thread has set `released`, -99 after five seconds. */
int wait_for_release(void) {
  const struct timespec ms = {0, 1000000};
  entered = 1;
  for (int i = 0; i < 5000 && !released; ++i) nanosleep(&ms, 0);
  return released ? 0 : -99;
}
"""


def test_other_threads_run_during_a_call(lib, tmp_path):
    """A call that waits, as a launch into a full queue does, leaves the interpreter to the other threads."""
    (tmp_path / "waiter.c").write_text(WAITER)
    subprocess.check_call(["gcc", "-O1", "-shared", "-fPIC", str(tmp_path / "waiter.c"), "-o", str(tmp_path / "waiter.so")])
    waiter = ctypes.CDLL(str(tmp_path / "waiter.so"))
    address = ctypes.cast(waiter.wait_for_release, ctypes.c_void_p).value
    entered, released = (ctypes.c_int.in_dll(waiter, n) for n in ("entered", "released"))
    m = slope.serving._bound()
    packed = slope.serving._pack_cache(0x40000, 4, 64, 2, 64, 64)
    q, k, ints, lse = Fake([3, 8, 64]), Fake([3, 2, 64]), Fake([3], torch.int32), Fake([8, 3], torch.float32)
    calls = {
        "qk_norm_rope": lambda: m.qk_norm_rope(q, k, None, None, True, 1e-6, None, None, 0, q, k, 0, 0),
        "attn_varlen": lambda: m.attn_varlen(q, k, k, [0, 3], True, 0, 0.0, q, lse, 0, 0),
        "kv4_write": lambda: m.kv4_write(packed, k, k, ints, 0, 0),
        "kv4_read": lambda: m.kv4_read(packed, ints, k, k, 0, 0),
        "kv4_attn": lambda: m.kv4_attn(q, packed, Fake([3, 4], torch.int32), ints, 1, 0, 0.0, q, lse, 0, 0, 0, 0),
    }
    m.bind(torch.bfloat16, torch.float32, torch.int32, *[address] * 7)
    try:
        for name, call in calls.items():
            entered.value = released.value = 0

            def release():
                while not entered.value:
                    time.sleep(0.001)
                released.value = 1

            thread = threading.Thread(target=release)
            thread.start()
            status = call()
            entered.value = 1
            thread.join()
            assert status == 0, name
    finally:
        slope.serving._bound()


CHANGING_LIST = """
import sys; sys.path[:0] = [{root!r}, {tests!r}]
import torch, ring_attention_slope_gb300 as slope
from test_serving_marshal import Fake
class Entry:
    def __index__(self):
        del cu[1:]
        junk.append([object() for _ in range(2000)])
        return 10 ** 6
cu, junk = [], []
q, k, lse = Fake([4 * 10 ** 6, 8, 64]), Fake([4 * 10 ** 6, 2, 64]), Fake([8, 4 * 10 ** 6], torch.float32)
m = slope.serving._bound()
for n in (3, 300, 5000):
    cu[:] = [10 ** 6] * 2 + [Entry()] + [10 ** 6 for _ in range(n)]
    assert m.attn_varlen(q, k, k, cu, True, 0, 0.0, q, lse, 0, 0) == 0 and len(cu) == 1
    cu[:] = [int(str(10 ** 6)), Entry()] + [int(str(10 ** 6 + i)) for i in range(n)] + [0]
    assert m.attn_varlen(q, k, k, cu, True, 0, 0.0, q, lse, 0, 0) == -5  # the 0 that stood at its end
print("done")
"""


def test_list_that_changes_while_it_is_read(lib):
    """Row indices whose own conversion shortens the list: what the list held when the call began counts."""
    code = CHANGING_LIST.format(root=ROOT, tests=os.path.join(ROOT, "tests"))
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=100)
    assert run.returncode == 0 and run.stdout == "done\n", (run.returncode, run.stderr[-2000:])


# ---------------------------------------------------------------- building

def test_library_builds_without_python_headers(lib, tmp_path, monkeypatch):
    """libslope needs no Python: where marshal.c cannot be compiled it is built all the same, and says so."""
    monkeypatch.setattr(_build, "MARSHAL_PATH", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(_build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    for older in (False, True):  # a module of older sources is not left to be loaded
        if older:
            (tmp_path / "_marshal.so").write_bytes(b"")
            os.utime(tmp_path / "_marshal.so", (0, 0))
        with pytest.warns(UserWarning, match="marshal"):
            assert _build.build() == _build.LIB_PATH
        assert os.listdir(tmp_path) == []


def test_marshalling_belongs_to_its_interpreter(lib, tmp_path, monkeypatch):
    """The C module carries the interpreter's tag, and no other file is loaded in its place."""
    m = slope.serving._bound()
    assert m.__file__ == _build.MARSHAL_PATH
    assert os.path.basename(m.__file__) == "_marshal" + sysconfig.get_config_var("EXT_SUFFIX") != "_marshal.so"
    (tmp_path / "_marshal.so").write_bytes(open(m.__file__, "rb").read())
    monkeypatch.setattr(_build, "MARSHAL_PATH", str(tmp_path / "_marshal.other-interpreter.so"))
    monkeypatch.delitem(sys.modules, m.__name__)
    with pytest.raises(RuntimeError, match="not built"):
        slope.serving._bound()


WITHOUT_TORCH = """
import sys; sys.path.insert(0, {root!r}); sys.modules["torch"] = None  # as where it is not installed
from ring_attention_slope_gb300 import *
import ring_attention_slope_gb300 as slope
assert slope.load().slope_kv4_block_bytes(64, 64) == 1280 and len(slope.rope_inv_freq(64)[0]) == 32
assert Rope([1.0] * 8)._c and version()
try:
    qk_norm_rope(None)
except ModuleNotFoundError as e:
    assert e.name == "torch"
    print("done")
"""


def test_package_without_torch(lib):
    """Importing the package, its library and its host-only calls need no PyTorch; calls on tensors say that they do."""
    run = subprocess.run([sys.executable, "-c", WITHOUT_TORCH.format(root=ROOT)], capture_output=True, text=True, timeout=100)
    assert run.returncode == 0 and run.stdout == "done\n", (run.returncode, run.stderr[-2000:])
    lazy = f"import sys; sys.path.insert(0, {ROOT!r}); import ring_attention_slope_gb300 as s; s.load(); print('torch' in sys.modules)"
    assert subprocess.check_output([sys.executable, "-c", lazy], text=True, timeout=100) == "False\n"
