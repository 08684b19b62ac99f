"""Which workspace a call of the attention gets: by stream and by recording (no GPU: the library is stood in for)."""
import ctypes
import gc
import struct
import weakref

import pytest

import compressed_linear_amd as cla
from compressed_linear_amd import serving

torch = pytest.importorskip("torch")


class Library:
    """Takes the calls of `tree_attention` and notes the workspace they were given."""

    def __init__(self):
        self.need, self.recording, self.calls = 1 << 20, {}, []

    def cl_call(self, entry, args):
        work, size, stream = struct.unpack("16qd4q", args)[18:21]
        if size < self.need:
            return -3
        self.calls.append((stream, work, size))
        return 0

    def cl_recording(self, stream, ref):
        ref._obj.value = self.recording.get(stream, 0)
        return 0

    def cl_tree_attention_work_bytes(self, *sizes):
        return self.need


class OnDevice(torch.Tensor):
    is_cuda = True


class Stand:
    """A cache on the CPU and calls of the attention on streams that are numbers."""

    def __init__(self, monkeypatch):
        serving._setup()
        self.lib, self.stream = Library(), 1
        monkeypatch.setattr(serving, "_lib", self.lib)
        monkeypatch.setattr(serving, "_stream", lambda dev: self.stream)
        monkeypatch.setattr(serving, "_capturing", lambda: bool(self.lib.recording.get(self.stream)), raising=False)
        k, v = (torch.zeros(1, 2, 16, 64, dtype=torch.uint8).as_subclass(OnDevice) for _ in range(2))
        ks, vs = (torch.zeros(1, 2, 16, dtype=torch.float16).as_subclass(OnDevice) for _ in range(2))
        self.cache = cla.KVCache(k=k, v=v, k_scale=ks, v_scale=vs)

    def call(self, stream, recording=0):
        self.stream, self.lib.recording[stream] = stream, recording
        i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
        serving.tree_attention(torch.zeros(1, 4, 64, dtype=torch.float16), self.cache, i32(0)[None], i32(0), i32(0, 1),
                               max_q=1, max_ctx=100)
        return self.lib.calls[-1][1]


@pytest.fixture
def stand(monkeypatch):
    return Stand(monkeypatch)


def test_a_recorded_call_shares_no_workspace(stand):
    # a replay runs on any stream, next to eager calls on the one it was recorded on, and to other graphs
    eager = stand.call(1)
    first, again = stand.call(1, recording=7), stand.call(1, recording=7)
    second = stand.call(1, recording=8)
    other = stand.call(2, recording=8)  # a branch of the same recording
    assert first == again and len({eager, first, second, other}) == 4
    # the recordings end: here their memory may be given out again, on the GPU it is the graphs'
    assert stand.call(1) == eager and stand.call(2) != eager


def test_counters_are_cleared_where_a_workspace_is_made(stand):
    for stream, recording in ((1, 0), (1, 5), (2, 0)):
        stand.call(stream, recording)
    assert len({work for _, work, _ in stand.lib.calls}) == 3
    assert all(not any(ctypes.string_at(work, serving.COUNTER_BYTES)) for _, work, _ in stand.lib.calls)


def test_workspace_stays_bounded():
    # the longest contexts on many sequences with many rows, as a wide block table asks for
    need = cla.lib().cl_tree_attention_work_bytes
    for B in (1, 3, 64, 1000, 65535):
        for hq, hkv in ((1, 1), (64, 8), (64, 64), (8, 1)):
            for dim in (64, 128):
                for T in (1, 16, 64, 256):
                    for ctx in (0, 5000, 131072, 2 ** 31 - 1):
                        assert 0 <= need(B, hq, hkv, dim, T, ctx) <= serving.COUNTER_BYTES + 2 ** 29, (B, hq, hkv, dim, T, ctx)
    # ordinary sizes still cut their keys
    assert need(1, 64, 8, 128, 1, 131001) > 0 and need(64, 64, 8, 128, 16, 8000) > 0


class Alive:
    """Counts the workspaces that are still held."""

    def __init__(self, monkeypatch):
        self.refs, empty = [], serving._empty

        def noted(*a, **kw):
            t = empty(*a, **kw)
            if t.dtype == torch.uint8:
                self.refs.append(weakref.ref(t))
            return t
        monkeypatch.setattr(serving, "_empty", noted)

    def sizes(self):
        gc.collect()
        return [r().numel() for r in self.refs if r() is not None]


def test_outgrown_workspaces_are_returned(stand, monkeypatch):
    alive = Alive(monkeypatch)
    for need in (1 << 20, 5 << 20, 30 << 20, 100 << 20):
        stand.lib.need = need
        stand.call(1)
        (size,) = alive.sizes()
        assert need <= size <= need + (32 << 20)  # room to grow, but not another hundred megabytes
    stand.lib.need = 1 << 20
    stand.call(1)
    assert len(alive.refs) == 4


def test_recordings_that_ended_hold_no_workspace(stand, monkeypatch):
    # a graph's memory is its own: once it is recorded, the cache lets its workspace go
    alive = Alive(monkeypatch)
    stand.call(1)
    for i in range(1, 4):
        stand.call(2, recording=i)
        stand.call(2, recording=i)
    stand.call(3, recording=9)  # still under way below
    stand.lib.recording[2] = 0
    mine = stand.call(3, recording=9)
    stand.call(1)
    assert len(alive.sizes()) == 2 and stand.call(3, recording=9) == mine
    stand.lib.recording[3] = 0
    stand.call(1)
    assert len(alive.sizes()) == 1
    for i in range(20, 60):  # recorded again and again, with no other call between
        stand.call(2, recording=i)
    assert len(alive.sizes()) <= 6
