"""Attention over an 8-bit cache whose values differ in size by powers of two that weights of 11 or 22 bits could not
span: heavy weights on small values beside light weights on large ones."""
import numpy as np
import pytest
import torch

import serving_reference as R
from test_gpu_serving import cache8, cuda, randn, zha

pytestmark = pytest.mark.gpu


def two_kinds(n, d, C, gap, drop, heavy):
    """A tree of keys of two kinds, by chunk: large values (2^gap) whose scores are `drop` below those of small values
    (1), for queries near `axis`. heavy: of every this many chunks the first is of small values."""
    Z = zha()
    small = (torch.arange(n, device="cuda") // C) % heavy == 0
    axis = torch.zeros(d, device="cuda")
    axis[:16] = 1.0
    k = 0.25 * randn(1, 1, 1, n, d)
    k[..., :16] = 0.0
    k = k + torch.where(small, drop / 16, 0.0)[:, None] * axis
    v = randn(2, 1, 1, n, d) * torch.where(small, 0, gap).float().exp2()[:, None]
    K, V, ks, vs = cache8(1, 1, n, d)
    Z.kv_write(k, v, K, V, ks, vs, 0)
    t = Z.Tree(K, V, randn(3, 1, 1, d), n, C, 1, 1.0, k_scale=ks, v_scale=vs)
    return t, axis, *R.cache_values(K, V, ks, vs)


def assert_close(out, lse, ref, keys):
    """As serving_reference.assert_attention, but the weights' own error against sum p |v| / sum p, not the largest of
    all values, however light: what a walk's 22 (11) bits of weights leave, and at most 2^-22 (2^-18) of its largest
    result a key where they leave less (2^-25 * 448 of a weight and a code, against results of 2^6 (2^2) and more)."""
    o, l, to, tl, spread = ref
    got = R.host(out).reshape(o.shape)
    one = out.dtype == torch.bfloat16
    weights = 2 * (tl + 2.0 ** -21) + (2.0 ** -11 if one else 0.0)
    floor = keys * 2.0 ** (-18 if one else -22) * np.abs(o).max(1)
    allow = weights[:, None] * spread + floor[:, None] + R.half_step(out.dtype) * np.maximum(np.abs(o), np.abs(got))
    bad = ~(np.abs(got - o) <= allow)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.abs(got - o)[bad].max():.3g} of {np.abs(o).max():.3g}"
    some = ~np.isneginf(l)
    assert np.isneginf(R.host(lse)[~some]).all() and (np.abs(R.host(lse)[some] - l[some]) <= tl[some]).all()


@pytest.mark.parametrize("q_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gap,drop", [(6, 10), (9, 20), (13, 30), (20, 30), (30, 40), (33, 40), (40, 60), (60, 80)])
@pytest.mark.parametrize("d,n,heavy", [(64, 40, 2), (128, 67, 3), (128, 2403, 100), (256, 403, 7)])
def test_heavy_weights_on_small_values(d, n, heavy, gap, drop, q_dtype):
    C, W = 8, 11
    t, axis, K64, V64 = two_kinds(n, d, C, gap, drop, heavy)
    n1 = n // C
    Q = (0.25 * randn(4, 1, 1, W, d) + axis).to(torch.bfloat16 if q_dtype == "bf16" else torch.float32)
    sel = np.tile(np.arange(n1, dtype=np.int32), (W, 1))
    cnt = np.full(W, n1, dtype=np.int32)
    cnt[3] = 1  # small values and the tail's
    cnt[5] = 0
    ref = R.attention(K64, V64, n, C, 1.0, R.host(Q), sel, cnt)
    args = Q, cuda(sel), cuda(cnt)
    for dt in (torch.float32, torch.bfloat16):
        out, lse = t.attend(*args, out_dtype=dt)
        assert_close(out, lse, ref, n)
        o2, l2 = torch.empty_like(out), torch.empty_like(lse)
        t.attend_noalloc(*args, o2, l2)
        assert_close(o2, l2, ref, n)
    kd = 0.25 * randn(5, 1, 1, W, d)
    vd = randn(6, 1, 1, W, d)
    mask = R.draft_mask(np.random.default_rng(7), 1, W, "chain")
    mask[0, 4] = 0
    ref = R.attention(K64, V64, n, C, 1.0, R.host(Q), sel, cnt, R.host(kd), R.host(vd), mask)
    for dt in (torch.float32, torch.bfloat16):
        out, lse = t.attend_draft(*args, kd, vd, cuda(mask), out_dtype=dt)
        assert_close(out, lse, ref, n + W)
    t.sync_status()


@pytest.mark.parametrize("q_dtype", ["f32", "bf16"])
def test_the_least_values_beside_others(q_dtype):
    """Rows at the format's least exponent, which zeros have too, beside a neighbour's rows of ordinary values."""
    Z, C, d, n = zha(), 8, 128, 64
    size = torch.full((n,), 0.0)
    size[8:16], size[16:24], size[24:32] = -121.0, -113.0, -300.0
    v = randn(1, 1, 1, n, d).double() * torch.exp2(size.double()).cuda()[:, None]
    K, V, ks, vs = cache8(1, 1, n, d)
    Z.kv_write(randn(2, 1, 1, n, d), v.float(), K, V, ks, vs, 0)
    t = Z.Tree(K, V, randn(3, 1, 1, d), n, C, 1, d ** -0.5, k_scale=ks, v_scale=vs)
    sel = np.array([[0, 4], [1, 3], [2, 3], [3, 3], [1, 2]], dtype=np.int32)
    cnt = np.array([2, 2, 2, 1, 2], dtype=np.int32)
    Q = randn(4, 1, 1, 5, d, dtype=torch.bfloat16 if q_dtype == "bf16" else torch.float32)
    K64, V64 = R.cache_values(K, V, ks, vs)
    ref = R.attention(K64, V64, n, C, d ** -0.5, R.host(Q), sel, cnt)
    assert (np.abs(ref[0]).max(1) > 0).tolist() == [True, True, True, False, True]
    for dt in (torch.float32, torch.bfloat16):
        out, lse = t.attend(Q, cuda(sel), cuda(cnt), out_dtype=dt)
        # results of the codes' least steps, 2^-126: below it fp32 is taken as zero by the exponential's and other units
        got, least = R.host(out).reshape(5, d), 2.0 ** -126
        o, _, to, tl, spread = ref
        allow = 2 * (tl + 2.0 ** -21)[:, None] * spread + (2.0 ** -11) * spread + R.half_step(dt) * np.abs(o) + 2 * least
        assert (np.abs(got - o) <= allow).all()
