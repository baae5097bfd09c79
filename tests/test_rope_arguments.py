"""What the binding of the rotation and prefill calls hands to the library, seen through a library that only records it."""
import types

import pytest
import torch

import paged_kv_cache_282_gb300 as pkv
from paged_kv_cache_282_gb300 import PagedKVCache, Rope

BF = torch.bfloat16
H, HK, D = 4, 2, 64


class Recorder:
    """Stands for the library in the calls that need a device; the rest goes to the library itself."""

    def __init__(self, lib, *names):
        self.lib, self.names, self.calls = lib, names, []

    def __getattr__(self, name):
        if name not in self.names:
            return getattr(self.lib, name)

        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


def _cache(*names):
    c = PagedKVCache(8, H, HK, D, 2, 4, host_only=True)
    c.device = torch.device("cpu")
    c.k_pool = torch.empty(8, HK, 16, D, dtype=BF)  # the binding asks it for the device
    c.lib = Recorder(c.lib, *names)
    return c


STREAM = types.SimpleNamespace(cuda_stream=0)


@pytest.mark.parametrize("rot,positions", [(0, torch.arange(3)), (0, torch.zeros(1, dtype=torch.int32)), (0, None),
                                           (32, torch.arange(3, dtype=torch.int32))])
def test_positions_are_handed_over_only_where_something_rotates(rot, positions):
    """Without a rotation they are not read, so anything may be given: it must not reach the device."""
    c = _cache("pkv_qk_norm_rope")
    rope = Rope(16, rot, device="cpu")
    q, k = torch.zeros(3, H, D, dtype=BF), torch.zeros(3, HK, D, dtype=BF)
    c.qk_norm_rope(q, k, positions, rope, q_out=q, k_out=k, stream=STREAM)
    assert c.lib.calls[0][1][4] == (positions.data_ptr() if rot else None)
    c = _cache("pkv_append_rope")
    if rot or positions is None:
        c.append_rope([0], k, k, rope, counts=[3], positions=positions, stream=STREAM)
        assert c.lib.calls[0][1][6] == (positions.data_ptr() if rot else None)


def test_prefill_scratch_belongs_to_the_stream(monkeypatch):
    """Calls on two streams, and decode, never get the same scratch; nothing that a call allocates is of another stream."""
    c = _cache("pkv_prefill_attn", "pkv_append_rope", "pkv_qk_norm_rope")
    inside = []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            inside.append(self.stream)

        def __exit__(self, *a):
            inside.append(None)

    monkeypatch.setattr(pkv, "_on", On, raising=False)
    empty, made = torch.empty, []

    def note(*a, **kw):
        made.append(inside[-1] if inside else None)
        return empty(*a, **kw)
    monkeypatch.setattr(torch, "empty", note)
    streams = [types.SimpleNamespace(cuda_stream=i) for i in (1, 2, 1, 2)]
    q = torch.zeros(2, H, D, dtype=BF)
    decode = c.workspace(1)
    made.clear()
    used = []
    for s in streams:
        out, lse = c.prefill([0], [2], q, stream=s)
        used.append(c.lib.calls[-1][1][12])
        assert c.lib.calls[-1][1][1] == s.cuda_stream
    assert used[0] == used[2] != used[1] == used[3] and decode.data_ptr() not in used
    assert c.workspace(1) is decode
    k = torch.zeros(2, HK, D, dtype=BF)
    rope = Rope(16, 0, device="cpu")
    c.append_rope([0], k, k, rope, counts=[2], q=q, stream=streams[0])
    c.qk_norm_rope(q, k, None, rope, stream=streams[1])
    assert [s.cuda_stream for s in made] == [1, 1, 1, 2, 2, 2, 1, 1, 2, 2, 1, 2, 2]


def test_prefill_refuses_a_workspace_that_the_kernel_cannot_use():
    c = _cache("pkv_prefill_attn")
    q = torch.zeros(2, H, D, dtype=BF)
    kw = dict(out=torch.zeros_like(q), lse=False, stream=STREAM)
    for bad in (torch.empty(1 << 20, dtype=torch.uint8, device="meta"), torch.empty(1 << 20, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError):
            c.prefill([0], [2], q, workspace=bad, **kw)
    assert not c.lib.calls
    good = torch.empty(1 << 20, dtype=torch.float32)
    c.prefill([0], [2], q, workspace=good, **kw)
    assert c.lib.calls[0][1][12:] == (good.data_ptr(), 4 << 20)
