"""Prefill and qk_norm_rope on streams other than the current one, ordered by events as their caller has to."""
import pytest
import torch

from paged_kv_cache_282_gb300 import PagedKVCache, Rope
from test_gpu_prefill import _check, _pool, _q
from test_gpu_rope import BF

pytestmark = pytest.mark.gpu


def _busy(us=2000):
    """About that much work on the current stream."""
    x = torch.zeros(1 << 26, device="cuda")
    for _ in range(us // 100):
        x += 1.0
    return x


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_prefill_on_two_streams(kv):
    """Cut items (whose partial records lie in the scratch) on two streams and decodes between them, each call behind the one
    before: the results of one stream, and a scratch for each stream that decode leaves alone."""
    cache, ids = _pool(kv, 8, 2, 128, [3000, 4000], seed=2)
    qs = [_q(cache, 40 + i, seed=i) for i in range(6)]
    want = [cache.prefill(ids, [20, 20 + i], q) for i, q in enumerate(qs)]
    _check(cache, ids, [20, 20], qs[0], *want[0])
    step = cache.decode(ids, qs[0][:2].contiguous())
    torch.cuda.synchronize()
    main, side = torch.cuda.current_stream(), torch.cuda.Stream()
    got = []
    _busy()
    for i, q in enumerate(qs):
        s, other = (side, main) if i % 2 else (main, side)
        s.wait_stream(other)
        got.append(cache.prefill(ids, [20, 20 + i], q, stream=s))
        if i == 3:
            main.wait_stream(side)
            d = cache.decode(ids, qs[0][:2].contiguous())  # on the current stream
    main.wait_stream(side)
    cache.sync_status()
    for (o, l), (x, y) in zip(got, want):
        assert torch.equal(o, x) and torch.equal(l, y)
    assert torch.equal(d[0], step[0]) and torch.equal(d[1], step[1])
    a, b = (cache._prefill_scratch[int(s.cuda_stream)].data_ptr() for s in (main, side))
    assert a != b and cache._workspace.data_ptr() not in (a, b)


def test_what_a_call_allocates_is_not_handed_on_early():
    """A result of a call on a side stream is dropped while the call waits there; memory taken on the current stream
    meanwhile must not be it."""
    cache, ids = _pool("bf16", 8, 2, 128, [2000], seed=4)
    rope = Rope(64, 128)
    q = _q(cache, 50)
    k = torch.zeros((50, 2, 128), dtype=BF, device="cuda")
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        _busy(20000)
    out, lse = cache.prefill(ids, [50], q, stream=side)
    qo, ko = cache.qk_norm_rope(q, k, pos, rope, stream=side)
    was = [x.data_ptr() for x in (out, lse, qo, ko)]
    shapes = [(x.shape, x.dtype) for x in (out, lse, qo, ko)]
    del out, lse, qo, ko
    new = [torch.full(s, 7, dtype=t, device="cuda") for s, t in shapes]
    assert not set(was) & {x.data_ptr() for x in new}
    torch.cuda.synchronize()
    assert all(bool((x == 7).all()) for x in new)
