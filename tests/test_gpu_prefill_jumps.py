"""Prefill of rows whose logits rise steeply from one key tile to a later one, against the formula in 64 bits.

Tolerances: those of test_gpu_prefill (an fp32 evaluation, weights rounded to bf16 on the tensor cores), and one term for
weights that vanish.  A weight below 2^-126, relative to the row's largest, may be flushed to zero, which takes at most
2^-126 |V_jd| from the sum over j; the sum of the weights is at least 1, so that the result is off by at most
2^-126 sum_j |V_jd|.  It is all that is left of a result where the key that holds the weight has V_jd = 0 exactly (INT8
codes): a key 89 below weighs e^-89 = 2^-128.4.

The tensor-core kernel takes a tile's weights relative to a reference it knows before the tile.  A rise of j over n keys
gives a tile sum of n e^j: the steps below lie around 2^126 and 2^128 (j = 87.3 and 88.7 for one key, 82.5 and 83.9 for
128), where fp32 ends, while V stays small enough for every O to be finite."""
import math

import pytest
import torch

from paged_kv_cache_282_gb300 import PagedKVCache, _abi
from test_gpu_prefill import BF, _kept, _pool, _q, _run, _stored

pytestmark = pytest.mark.gpu

JUMPS = [60.0, 82.0, 82.4, 82.8, 83.2, 83.6, 84.0, 85.0, 86.0, 87.0, 87.2, 87.4, 87.6, 87.8, 88.0, 88.2, 88.5, 88.7, 88.8,
         89.0, 200.0, 2000.0]
FACTORS = (1.0, 1.0, 0.5, 1.0, 0.25, -1.0, 1.0, 1.0)  # of the jump, per query head


def _cache(kv, D, L, at, size=0.1):
    """One sequence of L keys of about 0 and values of about `size`; the keys at positions `at` (a list of (first, count,
    value)) hold `value` in every dimension."""
    cache = PagedKVCache((L + 15) // 16 + 4, 8, 2, D, 1, (L + 15) // 16 + 2, kv_dtype=kv, alloc_seed=3)
    g = torch.Generator(device="cuda").manual_seed(L + D)
    k, v = (x * torch.randn((1, L, 2, D), generator=g, device="cuda") for x in (1e-3, size))
    for first, count, value in at:
        k[:, first:first + count] = value
    s = cache.seq_add()
    cache.append([s], k.to(BF), v.to(BF))
    return cache, s


def _check(cache, s, q, out, lse, scale, mask="full", S=0, W=0):
    G, D, T = cache.group, cache.head_dim, q.shape[0]
    k, v = (x.repeat_interleave(G, 1) for x in _stored(cache, s))
    L = k.shape[0]
    keep = _kept(mask, S, W, torch.arange(L - T, L, device="cuda")[:, None], torch.arange(L, device="cuda")[None])
    lg = (torch.einsum("thd,jhd->htj", q.double(), k) * scale).masked_fill(~keep, -math.inf)
    mag = (torch.einsum("thd,jhd->htj", q.double().abs(), k.abs()) * abs(scale)).masked_fill(~keep, 0.0)
    p = torch.softmax(lg, -1)
    ref, ref_lse = torch.einsum("htj,jhd->thd", p, v), torch.logsumexp(lg, -1).T
    e = (D + 8) * 2.0 ** -24 * (1 + mag.amax(-1)).T  # [t][H]
    w = 2 * e + L * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -8
    tol = torch.einsum("htj,jhd->thd", p, v.abs()) * w[..., None] * 1.01 + 2.0 ** -126 * v.abs().sum(0)
    tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    d = (out.double() - ref).abs()
    assert bool((d <= tol).all()), (scale * D, float((d - tol).max()), float(d.max()))
    dl = (lse.double() - ref_lse).abs()
    assert bool((dl <= e + 2.0 ** -20 * (1 + ref_lse.abs())).all()), (scale * D, float(dl.max()))


def _jump(cache, s, T, jump):
    """The jump's logits are jump times the head's factor."""
    D = cache.head_dim
    q = torch.ones((T, 8, D), device="cuda") * torch.tensor(FACTORS, device="cuda")[None, :, None]
    q = q.to(BF)
    out, lse = _run(cache, [s], [T], q, scale=jump / D)
    _check(cache, s, q, out, lse, jump / D)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("n", [1, 2, 16, 128])
@pytest.mark.parametrize("at", [512, 256, 300])
def test_logits_that_rise_in_a_later_tile(kv, D, n, at):
    """In the last key tile, in one with others behind it, and across two; 140 queries of 8 heads."""
    cache, s = _cache(kv, D, 640, [(at, n, 1.0)])
    for jump in JUMPS:
        _jump(cache, s, 140, jump)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("D", [128, 64])
def test_logits_that_rise_twice(kv, D):
    cache, s = _cache(kv, D, 900, [(200, 3, 1.0), (700, 40, 2.0), (890, 2, 2.5)])
    for jump in JUMPS:
        _jump(cache, s, 300, jump)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("n", [1, 128])
def test_logits_that_rise_in_cut_items(kv, D, n):
    """Two query tokens whose 20000 keys are split over CTAs: the rise lies in one piece, in several, at a piece's end."""
    for at in ([(9000, n, 1.0)], [(5000 + 1300 * i + 128 * i, n, 1.0) for i in range(8)], [(19800, n, 1.0)]):
        cache, s = _cache(kv, D, 20000, at)
        for jump in JUMPS:
            _jump(cache, s, 2, jump)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
def test_values_of_zero_behind_a_rise(kv):
    """All values zero: O is zero whatever the weights are, lse is not."""
    cache, s = _cache(kv, 128, 640, [(300, 5, 1.0)], size=0.0)
    for jump in JUMPS:
        _jump(cache, s, 140, jump)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
def test_such_rows_may_outlast_the_wait_limit(kv):
    """64 tokens of 8 heads behind 30000 keys, the rise in the last tile, so that every row is computed twice, which takes
    longer than the waits' limit of 1 ms (as more keys would than the default of 4 s)."""
    cache, s = _cache(kv, 128, 30000, [(29900, 1, 1.0)])
    _abi.check(cache.lib.pkv_set_wait_limit(cache.handle, 1_000_000))
    _jump(cache, s, 64, 50.0)  # ordinary rows take less
    _jump(cache, s, 64, 100.0)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("G,D", [(1, 128), (2, 64), (8, 128), (8, 64)])
@pytest.mark.parametrize("mask,S,W", [("full", 0, 0), ("sliding", 0, 200), ("sink_window", 20, 333)])
@pytest.mark.parametrize("L,T", [(700, 200), (9000, 5)])
def test_random_logits_of_a_wide_range(kv, G, D, mask, S, W, L, T):
    """Logits with a deviation of 100, so that rows rise in some tiles and not in others; per-channel scales."""
    cache, ids = _pool(kv, 2 * G, 2, D, [L], seed=G, channel=kv != "bf16")
    q = _q(cache, T, seed=D)
    scale = 100.0 / float(torch.einsum("thd,jhd->htj", q[:50].double(), _stored(cache, ids[0])[0][:50].repeat_interleave(G, 1)).std())
    out, lse = _run(cache, ids, [T], q, scale=scale, mask=mask, num_sinks=S, window=W)
    _check(cache, ids[0], q, out, lse, scale, mask, S, W)
