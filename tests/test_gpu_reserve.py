"""zha_reserve before a capture: the attention of many walks, which takes both of a tree's scratch blocks."""
import numpy as np
import pytest
import torch

import serving_reference as R
from test_gpu_serving import cuda, make_tree, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,walks", [("bf16", 1024), ("e4m3", 4096)])
def test_a_capture_after_reserve_alone(kind, walks):
    """Reserved while the cache is short, captured when it is full; no call in between but extend."""
    n, cap, d, C = 130, 1300, 128, 8
    t, _, _ = make_tree(kind, 1, 2, n, d, C, depth=2, cap=cap)
    t.reserve(2 * walks, 20)
    dt = torch.float32 if kind == "e4m3" else torch.bfloat16
    t.extend(randn(1, 1, 2, cap - n, d, dtype=dt), randn(2, 1, 2, cap - n, d, dtype=dt))
    K64, V64 = R.cache_values(t.K, t.V, t.k_scale, t.v_scale)
    sel, cnt = R.selection(np.random.default_rng(3), 2, walks, cap // C, 20)
    Q = randn(4, 1, 2, walks, d, dtype=torch.bfloat16)
    s, c = cuda(sel), cuda(cnt)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = t.attend(Q, s, c)
    Q.copy_(randn(5, *Q.shape, dtype=torch.bfloat16))
    g.replay()
    torch.cuda.synchronize()
    t.sync_status()
    some = np.arange(0, 2 * walks, 37)  # each walk's reference is a loop on the host
    o, l, to, tl, spread = R.attention(K64, V64, cap, C, d ** -0.5, R.host(Q), sel, np.where(np.isin(np.arange(2 * walks), some), cnt, 0))
    # the kernels of many walks: queries and keys exact in bf16, weights in two bf16 terms, 2^-17 of each
    pick = lambda x: x.reshape(2 * walks, -1)[some]
    ref = pick(o), l[some], to[some] + 2.0 ** -16 * spread[some].max(1), tl[some], spread[some]
    R.assert_attention(out.view(2 * walks, d)[torch.from_numpy(some).cuda()], lse[torch.from_numpy(some).cuda()], ref, kind, False)


def test_reserve_takes_any_number_of_walks():
    """More walks a tree than the tensor-core attention takes: what it can take is reserved."""
    t, _, _ = make_tree("bf16", 1, 1, 200, 128, 8)
    t.reserve(70000, 4)
    sel, cnt = R.selection(np.random.default_rng(6), 1, 65535, 25, 4)
    Q = randn(7, 1, 1, 65535, 128, dtype=torch.bfloat16)
    s, c = cuda(sel), cuda(cnt)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, _ = t.attend(Q, s, c)
    g.replay()
    torch.cuda.synchronize()
    t.sync_status()
    assert torch.isfinite(out).all()
