"""pkv_append_rope and pkv_qk_norm_rope on the GPU against the formulas in 64
bits.

Tolerances.  A result is an fp32 evaluation of a c - b s (and b c + a s) with
a, b the (normed) pair, rounded once.  Counting roundings relative to
|a| + |b|: the sum of squares (at most D / 2 + 6 additions, halved by the root), the
reciprocal root (2 ulp), two products of the norm, the table entry, a product
and a sum: below 64 x 2^-24 = 2^-18 for D <= 128 (the sum of squares has non-negative
terms, 16 lanes or fewer added pairwise, 8 values or fewer each in sequence: under 16
roundings).  The output's own rounding adds half a step, eps / 2 relative
(bf16 2^-8, fp32 2^-24).  Codes: half a step of the code, times the scale."""
import numpy as np
import pytest
import torch

import paged_kv_cache_282_gb300 as pkv
from paged_kv_cache_282_gb300 import PagedKVCache, PKVError, Rope

pytestmark = pytest.mark.gpu

EVAL = 2.0 ** -18
BF, F32 = torch.bfloat16, torch.float32


def _dtype(kv):
    return F32 if kv == "fp32" else BF


def _rand(shape, dtype, seed, spread=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if spread:
        x = x * 10.0 ** (spread * (2 * torch.rand((*shape[:-1], 1), generator=g) - 1))
    return x.to(dtype)


def _rotated(x, w, pos, rot, inter, eps=1e-6, base=10000.0):
    """(y, |a| + |b|) in 64 bits: x [tok][heads][D], w [D] or None."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    y, mag = x.clone(), x.abs()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        t = pos.double() * base ** (-2.0 * i / rot)
        c, s = t.cos()[:, None], t.sin()[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        mag[..., a] = mag[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, mag


def _close(got, y, mag, dtype):
    tol = torch.finfo(dtype).eps / 2 * (y.abs() + EVAL * mag) + EVAL * mag
    d = (got.cpu().double() - y).abs()
    assert bool((d <= tol).all()), float((d - tol).max())


def _weights(D, dtype, seed):
    return [(1 + 0.3 * _rand((D,), F32, seed + i)).to(dtype).cuda() for i in range(2)]


SHAPES = [(32, 8, 128), (8, 8, 64), (3, 3, 64), (16, 2, 128), (8, 1, 64)]


@pytest.mark.parametrize("kv", ["bf16", "fp32"])
@pytest.mark.parametrize("H,Hk,D", SHAPES)
@pytest.mark.parametrize("rot_of,inter,norm", [(1, False, True), (1, True, False), (2, False, False), (4, True, True),
                                               (0, False, True), ("16", False, True), ("48", False, False)])
def test_qk_norm_rope(kv, H, Hk, D, rot_of, inter, norm):
    rot = int(rot_of) if isinstance(rot_of, str) else 0 if rot_of == 0 else D // rot_of
    dt = _dtype(kv)
    cache = PagedKVCache(1, H, Hk, D, 1, 1, kv_dtype=kv)
    qw, kw = _weights(D, dt, 5) if norm else (None, None)
    rope = Rope(131072, rot, interleaved=inter, q_weight=qw, k_weight=kw)
    for n in (1, 2, 7, 33, 700):
        x = _rand((n, H + 2 * Hk, D), dt, n + D, spread=2.0 if n == 33 else 0.0)
        pos = torch.randint(0, 131072, (n,), generator=torch.Generator().manual_seed(n), dtype=torch.int32)
        xd = x.cuda()
        q, k = cache.qk_norm_rope(xd[:, :H], xd[:, H:H + Hk], pos.cuda(), rope)
        cache.sync_status()
        assert torch.equal(xd.cpu(), x)
        for got, part, w in ((q, x[:, :H], qw), (k, x[:, H:H + Hk], kw)):
            _close(got, *_rotated(part, None if w is None else w.cpu(), pos, rot, inter), dt)
        # in place inside the packed tensor, with the values left alone
        cache.qk_norm_rope(xd[:, :H], xd[:, H:H + Hk], pos.cuda(), rope, q_out=xd[:, :H], k_out=xd[:, H:H + Hk])
        assert torch.equal(xd[:, :H], q) and torch.equal(xd[:, H:H + Hk], k)
        assert torch.equal(xd[:, H + Hk:].cpu(), x[:, H + Hk:])
        # either side alone
        xd = x.cuda()
        assert torch.equal(cache.qk_norm_rope(xd[:, :H], None, pos.cuda(), rope)[0], q)
        assert torch.equal(cache.qk_norm_rope(None, xd[:, H:H + Hk], pos.cuda(), rope)[1], k)


def test_qk_norm_rope_marks_positions_outside_the_table():
    cache = PagedKVCache(1, 4, 2, 64, 1, 1)
    rope = Rope(100, 64)
    x = _rand((5, 6, 64), BF, 1).cuda()
    pos = torch.tensor([99, 100, 3, -1, 0], dtype=torch.int32).cuda()
    q = torch.full((5, 4, 64), 7.0, dtype=BF, device="cuda")
    cache.qk_norm_rope(x[:, :4], None, pos, rope, q_out=q)
    with pytest.raises(PKVError) as e:
        cache.sync_status()
    assert e.value.status == 7
    assert bool((q[[1, 3]] == 7).all())
    y, mag = _rotated(x[:, :4].cpu(), None, pos.cpu().clamp(0, 99), 64, False)
    good = [0, 2, 4]
    _close(q[good], y[good], mag[good], BF)
    cache.sync_status()  # the status was cleared


def test_qk_norm_rope_captured_and_replayed():
    cache = PagedKVCache(1, 8, 2, 128, 1, 1)
    rope = Rope(4096, 128, q_weight=_weights(128, BF, 3)[0])
    x = _rand((9, 12, 128), BF, 2).cuda()
    pos = torch.arange(9, dtype=torch.int32).cuda()
    q, k = torch.empty(9, 8, 128, dtype=BF, device="cuda"), torch.empty(9, 2, 128, dtype=BF, device="cuda")
    g = torch.cuda.CUDAGraph()
    cache.qk_norm_rope(x[:, :8], x[:, 8:10], pos, rope, q_out=q, k_out=k)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        cache.qk_norm_rope(x[:, :8], x[:, 8:10], pos, rope, q_out=q, k_out=k)
    for seed in (4, 5):
        x.copy_(_rand((9, 12, 128), BF, seed))
        pos.copy_(torch.randint(0, 4096, (9,), dtype=torch.int32))
        g.replay()
        want = cache.qk_norm_rope(x[:, :8], x[:, 8:10], pos, rope)
        assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    # what a graph cannot hold is refused without disturbing the capture
    s = cache.seq_add()
    out = torch.empty_like(q)
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        for call in (lambda: cache.append_rope([s], x[:1, 8:10], x[:1, 10:], rope),
                     lambda: cache.prefill([], [], x[:0, :8], lse=False, out=out[:0])):
            with pytest.raises(PKVError) as e:
                call()
            assert e.value.status == 2
        cache.timing_enable(["qk_rope"])
        with pytest.raises(PKVError):
            cache.qk_norm_rope(x[:, :8], None, pos, rope, q_out=out)
        cache.timing_enable(False)
        cache.qk_norm_rope(x[:, :8], None, pos, rope, q_out=out)
    assert cache.seq_len(s) == 0


def _sentinel(cache):
    for x in (cache.k_pool, cache.v_pool, cache.k_scale, cache.v_scale):
        if x is not None:
            x.view(torch.uint8).fill_(0x5A)


def _pools(cache):
    return [x for x in (cache.k_pool, cache.v_pool, cache.k_scale, cache.v_scale) if x is not None]


def _rows(cache, seq, lo, hi):
    """(K, V) rows of positions [lo, hi) in 64 bits, dequantised, and the K and V scales."""
    t = torch.from_numpy(cache.block_table(seq).astype(np.int64)).cuda()
    p = torch.arange(lo, hi, device="cuda")
    at, off = t[p // 16], p % 16
    out = []
    for x, sc in ((cache.k_pool, cache.k_scale), (cache.v_pool, cache.v_scale)):
        x = x.view(torch.float8_e4m3fn) if cache.kv_dtype == "fp8" else x
        x = x.to(F32) if x.element_size() == 1 else x
        r = x[at, :, off].double()
        out.append((r.cpu(), None if sc is None else sc[at, :, off].double().cpu()))
    return out


def _check_rows(cache, got, y, mag, channel=None):
    rows, sc = got
    if sc is None:
        return _close(rows, y, mag, _dtype(cache.kv_dtype))
    if channel is not None:
        y, mag = y / channel.cpu().double(), mag / channel.cpu().double()
    top = y.abs().amax(-1)
    most = 448.0 if cache.kv_dtype == "fp8" else 127.0
    want = torch.where(top == 0, torch.ones_like(top), top / most)
    assert bool(((sc - want).abs() <= (EVAL * mag.amax(-1) + 2.0 ** -23 * top) / most).all())
    y, mag = y / sc[..., None], mag / sc[..., None]
    if cache.kv_dtype == "fp8":  # half a step: 2^-4 relative, 2^-10 for subnormal codes
        half = torch.maximum(y.abs() * 2.0 ** -4, torch.full_like(y, 2.0 ** -10))
    else:
        half = torch.full_like(y, 0.5)
    d = (rows - y).abs()
    tol = half * (1 + EVAL) + EVAL * mag + 2.0 ** -22 * y.abs()
    assert bool((d <= tol).all()), float((d - tol).max())


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8", "fp32"])
@pytest.mark.parametrize("H,Hk,D", SHAPES)
def test_append_rope(kv, H, Hk, D):
    dt = _dtype(kv)
    lens = [0, 1, 15, 16, 17, 40]
    cache = PagedKVCache(200, H, Hk, D, 8, 60, kv_dtype=kv, alloc_seed=3)
    channel = [None, None]
    if kv in ("fp8", "int8") and D == 64:
        channel = [(2.0 ** torch.randint(-3, 4, (Hk, D), generator=torch.Generator().manual_seed(i))).cuda() for i in (1, 2)]
        cache.set_channel_scales(*channel)
    ids = [cache.seq_add() for _ in lens]
    for s, n in zip(ids, lens):
        cache.reserve_slots([s], n)
    qw, kw = _weights(D, dt, 9)
    for step, (counts, rot, inter, norm, far) in enumerate([
            ((1, 1, 1, 1, 1, 1), D, False, False, False), ((1, 0, 1, 1, 0, 1), D // 2, True, True, True),
            ((300, 0, 17, 1, 16, 5), D, False, True, False), ((0, 31, 0, 0, 0, 0), 16, False, False, True),
            ((0, 0, 0, 0, 0, 0), D, False, False, False), ((2, 700, 3, 33, 100, 15), 48, True, True, True)]):
        if sum((n + 15) // 16 for n in counts) > 30:
            for s in ids:
                cache.seq_truncate(s, min(cache.seq_len(s), 20))
        n = sum(counts)
        rope = Rope(131072 if far else 1200, rot, interleaved=inter, q_weight=qw if norm else None,
                    k_weight=kw if norm else None)
        x = _rand((n, H + 2 * Hk, D), dt, step, spread=1.5 if step == 2 else 0.0)
        old = [cache.seq_len(s) for s in ids]
        pos = torch.tensor([o + t for o, c in zip(old, counts) for t in range(c)], dtype=torch.int32)
        if far:
            pos += 130000
        xd = x.cuda()
        _sentinel(cache)
        before = [p.clone() for p in _pools(cache)]
        q = cache.append_rope(ids, xd[:, H:H + Hk], xd[:, H + Hk:], rope, counts=counts, q=xd[:, :H],
                              positions=pos.cuda() if far else None)
        cache.sync_status()
        assert [cache.seq_len(s) for s in ids] == [o + c for o, c in zip(old, counts)]
        w = (qw.cpu(), kw.cpu()) if norm else (None, None)
        if n:
            _close(q, *_rotated(x[:, :H], w[0], pos, rot, inter), dt)
            y, mag = _rotated(x[:, H:H + Hk], w[1], pos, rot, inter)
            v = x[:, H + Hk:].double()
            at = 0
            for s, o, c in zip(ids, old, counts):
                (kr, vr), e = _rows(cache, s, o, o + c), at + c
                _check_rows(cache, kr, y[at:e], mag[at:e], channel[0])
                _check_rows(cache, vr, v[at:e], torch.zeros_like(v[at:e]), channel[1])
                at = e
        # nothing else of the pool changed
        slots = [int(cache.block_table(s)[p // 16]) * 16 + p % 16 for s, o, c in zip(ids, old, counts) for p in range(o, o + c)]
        for b, p in zip(before, _pools(cache)):
            b, p = (z.view(torch.uint8).view(z.shape[0], Hk, 16, -1).transpose(1, 2).reshape(-1, Hk * z.element_size() * (
                D if z.dim() == 4 else 1)) for z in (b, p))
            keep = torch.ones(b.shape[0], dtype=torch.bool, device="cuda")
            keep[slots] = False
            assert torch.equal(b[keep], p[keep])
    # the device's block table agrees with the host's
    for s in ids:
        t = cache.block_table(s)
        assert np.array_equal(cache.block_tables[s, :len(t)].cpu().numpy(), t)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8", "fp32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 3, 90])
def test_append_without_rotation_is_append(kv, D, T):
    """rot_dim 0 and no norm store the same bytes as the plain append, copies of shared blocks included."""
    dt = _dtype(kv)
    k, v = _rand((3, T, 2, D), dt, 1, spread=2.0).cuda(), _rand((3, T, 2, D), dt, 2).cuda()
    caches = [PagedKVCache(64, 4, 2, D, 6, 16, kv_dtype=kv, alloc_seed=7) for _ in range(2)]
    for c in caches:
        _sentinel(c)
        a = c.seq_add()
        c.append([a], *(_rand((1, 21, 2, D), dt, 5 + i).cuda() for i in range(2)))
        ids = [a, c.seq_fork(a), c.seq_add()]
    caches[0].append(ids, k, v)
    caches[1].append_rope(ids, k, v, Rope(1, 0))
    for c in caches:
        c.sync_status()
        assert c.stats()["cow_copies"] == 1
    for x, y in zip(_pools(caches[0]), _pools(caches[1])):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert torch.equal(caches[0].block_tables, caches[1].block_tables)


def test_append_rope_of_a_fork_leaves_the_parent():
    cache = PagedKVCache(32, 4, 2, 64, 4, 8)
    a = cache.seq_add()
    rope = Rope(128, 64)
    cache.append_rope([a], *(_rand((1, 20, 2, 64), BF, i).cuda() for i in range(2)), rope)
    parent = _rows(cache, a, 0, 20)
    b = cache.seq_fork(a)
    k = _rand((5, 2, 64), BF, 8)
    cache.append_rope([b, a], k.cuda(), k.cuda(), rope, counts=[3, 2])
    cache.sync_status()
    for s, n, part in ((b, 3, k[:3]), (a, 2, k[3:])):
        for (x, _), (y, _) in zip(parent, _rows(cache, s, 0, 20)):
            assert torch.equal(x, y)
        y, mag = _rotated(part, None, torch.arange(20, 20 + n), 64, False)
        _close(_rows(cache, s, 20, 20 + n)[0][0], y, mag, BF)


def test_append_rope_skips_tokens_at_positions_outside_the_table():
    cache = PagedKVCache(8, 4, 2, 64, 2, 4, kv_dtype="fp8")
    s = cache.seq_add()
    _sentinel(cache)
    x = _rand((3, 8, 64), BF, 3).cuda()
    pos = torch.tensor([0, 64, 2], dtype=torch.int32).cuda()
    q = torch.full((3, 4, 64), 7.0, dtype=BF, device="cuda")
    cache.append_rope([s], x[:, 4:6], x[:, 6:], Rope(64, 64), counts=[3], q=x[:, :4], q_out=q, positions=pos)
    with pytest.raises(PKVError) as e:
        cache.sync_status()
    assert e.value.status == 7
    b = int(cache.block_table(s)[0])
    assert bool((q[1] == 7).all()) and bool((q[0] != 7).any())
    assert bool((cache.k_pool[b, :, 1] == 0x5A).all()) and bool((cache.v_pool[b, :, 1] == 0x5A).all())
    assert bool((cache.v_pool[b, :, 2] != 0x5A).any()) and cache.seq_len(s) == 3


def test_append_rope_on_another_stream_and_own_frequencies():
    cache = PagedKVCache(64, 8, 4, 128, 4, 16)
    s = cache.seq_add()
    f = [1.0 / (1 + i) for i in range(32)]
    rope = Rope(500, 64, frequencies=f)
    x = _rand((400, 16, 128), BF, 3)
    side = torch.cuda.Stream()
    xd = x.cuda()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for lo in range(0, 100, 10):
            cache.append_rope([s], xd[lo:lo + 10, 8:12], xd[lo:lo + 10, 12:], rope, counts=[10])
        q = cache.append_rope([s], xd[100:, 8:12], xd[100:, 12:], rope, counts=[300], q=xd[100:, :8]) \
            if cache.max_blocks_per_seq * 16 >= 400 else None
    assert q is None
    cache.sync_status(side)
    y = x[:100, 8:12].double()
    for i, fi in enumerate(f):
        t = torch.arange(100).double() * fi
        a, b = x[:100, 8:12, i].double(), x[:100, 8:12, i + 32].double()
        y[..., i], y[..., i + 32] = a * t.cos()[:, None] - b * t.sin()[:, None], b * t.cos()[:, None] + a * t.sin()[:, None]
    mag = 2 * x[:100, 8:12].double().abs().amax(-1, keepdim=True).expand(y.shape)
    _close(_rows(cache, s, 0, 100)[0][0], y, mag, BF)


def test_binding_refusals():
    cache = PagedKVCache(8, 4, 2, 64, 2, 4)
    s = cache.seq_add()
    rope = Rope(64, 64)
    x = _rand((3, 8, 64), BF, 3).cuda()
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    pos = torch.arange(3, dtype=torch.int32).cuda()
    bad_w = Rope(64, 64, q_weight=torch.ones(64, device="cuda"))
    for call in (lambda: cache.append_rope([s], k, v[:2], rope, counts=[3]),
                 lambda: cache.append_rope([s], k, v, rope, counts=[2]),
                 lambda: cache.append_rope([s], k.float(), v, rope, counts=[3]),
                 lambda: cache.append_rope([s], k.cpu(), v, rope, counts=[3]),
                 lambda: cache.append_rope([s], k, v, rope, counts=[3], q=q[:2]),
                 lambda: cache.append_rope([s], k, v, rope, counts=[3], q=q, q_out=q),  # not contiguous
                 lambda: cache.append_rope([s], k, v, rope, counts=[3], positions=pos.long()),
                 lambda: cache.append_rope([s], k, v, bad_w, counts=[3]),
                 lambda: cache.append_rope([s], k, v, Rope(64, 64, device="cpu"), counts=[3]),
                 lambda: cache.qk_norm_rope(q, k[:2], pos, rope),
                 lambda: cache.qk_norm_rope(q, k, pos[:2], rope),
                 lambda: cache.qk_norm_rope(q, k, None, rope),
                 lambda: cache.prefill([s], [2], q.contiguous()),
                 lambda: cache.prefill([s], [3], q),
                 lambda: Rope(64, 64, frequencies=[1.0]),
                 lambda: Rope(64, 64, q_weight=torch.ones(2, 64, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    assert cache.seq_len(s) == 0
    with pytest.raises(PKVError):
        cache.append_rope([s], k, v, Rope(2, 64), counts=[3])  # past the table
    with pytest.raises(PKVError):
        cache.append_rope([s], x[:, 4:6, :].as_strided((3, 2, 64), (0, 64, 1)), v, rope, counts=[3])
    assert cache.seq_len(s) == 0
    cache.append_rope([s], k, v, rope, counts=[3])
    cache.append_rope([], k[:0], v[:0], rope, counts=[])
    cache.sync_status()
    assert cache.seq_len(s) == 3 and pkv.version()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_positions_are_not_read_without_a_rotation(kv):
    """The library is given an address that no int32 can be read from."""
    cache = PagedKVCache(4, 4, 2, 64, 1, 4, kv_dtype=kv)
    w = _weights(64, BF, 7)
    rope = Rope(1, 0, q_weight=w[0], k_weight=w[1])
    x = _rand((5, 8, 64), BF, 4).cuda()
    y, mag = _rotated(x[:, :4].cpu(), w[0].cpu(), torch.zeros(5), 0, False)
    q = torch.empty((5, 4, 64), dtype=BF, device="cuda")
    k = torch.empty((5, 2, 64), dtype=BF, device="cuda")
    odd = torch.zeros(64, dtype=torch.uint8, device="cuda").data_ptr() + 1
    pkv._abi.check(cache.lib.pkv_qk_norm_rope(cache.handle, pkv._stream_ptr(None), 5, rope._ref, odd, x.data_ptr(), 8 * 64,
                                              q.data_ptr(), 4 * 64, x.data_ptr() + 4 * 64 * 2, 8 * 64, k.data_ptr(), 2 * 64))
    cache.sync_status()
    _close(q, y, mag, BF)
    s, one = np.array([cache.seq_add()], np.int32), np.array([5], np.int32)
    q2 = torch.empty_like(q)
    pkv._abi.check(cache.lib.pkv_append_rope(cache.handle, pkv._stream_ptr(None), 1, s.ctypes.data, one.ctypes.data, rope._ref, odd,
                                             x.data_ptr(), 8 * 64, q2.data_ptr(), x.data_ptr() + 4 * 64 * 2, 8 * 64,
                                             x.data_ptr() + 6 * 64 * 2, 8 * 64))
    cache.sync_status()
    assert torch.equal(q2, q)
    # the binding: positions on the host, and too few of them
    for positions in (torch.arange(5), torch.zeros(1, dtype=torch.int32, device="cuda"), None):
        assert torch.equal(cache.qk_norm_rope(x[:, :4], None, positions, rope)[0], q)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_long_append_on_another_stream_with_own_frequencies(kv):
    """More tokens than travel in the kernel's parameters (they are staged and uploaded) behind earlier work of the stream,
    queries among them."""
    cache = PagedKVCache(64, 8, 4, 128, 2, 26, kv_dtype=kv)
    s = cache.seq_add()
    f = [1.0 / (1 + i) for i in range(32)]
    rope = Rope(500, 64, frequencies=f)
    x = _rand((400, 16, 128), BF, 3)
    side = torch.cuda.Stream()
    xd = torch.zeros((400, 16, 128), dtype=BF, device="cuda")
    host = x.pin_memory()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        y = torch.zeros(1 << 26, device="cuda")
        for _ in range(20):
            y += 1.0
        xd.copy_(host, non_blocking=True)  # the rows arrive there only now
    cache.append_rope([s], xd[:100, 8:12], xd[:100, 12:], rope, counts=[100], stream=side)
    q = cache.append_rope([s], xd[100:, 8:12], xd[100:, 12:], rope, counts=[300], q=xd[100:, :8], stream=side)
    cache.sync_status(side)
    side.synchronize()
    turned = x.double()
    for i, fi in enumerate(f):
        t = torch.arange(400).double() * fi
        a, b = x[..., i].double(), x[..., i + 32].double()
        turned[..., i] = a * t.cos()[:, None] - b * t.sin()[:, None]
        turned[..., i + 32] = b * t.cos()[:, None] + a * t.sin()[:, None]
    mag = 2 * x.double().abs().amax(-1, keepdim=True).expand(turned.shape)
    _close(q, turned[100:, :8], mag[100:, :8], BF)
    for got, y, m in zip(_rows(cache, s, 0, 400), (turned[:, 8:12], x[:, 12:].double()), (mag[:, 8:12], x[:, 12:].double().abs())):
        _check_rows(cache, got, y, m)
