"""A tree's two scratch blocks when calls are captured into CUDA graphs: what a captured
call leaves behind for the eager calls after it, and what keeps its graph replayable."""
import numpy as np
import pytest
import torch

import serving_reference as R
from test_gpu_serving import cuda, make_tree, randn, zha

pytestmark = pytest.mark.gpu


def inputs(t, n_q, seed=1, most=4):
    """Queries [B][2 H][n_q][d] in bf16 and chunk lists of their walks."""
    B, H, _, d = t.K.shape
    Q = randn(seed, B, 2 * H, n_q, d, dtype=torch.bfloat16)
    sel, cnt = R.selection(np.random.default_rng(seed), B * H, 2 * n_q, t.n_keys // t.cfg.chunk, most)
    return Q, cuda(sel), cuda(cnt)


def captured(call):
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    return g, out


def walk(t, Q):
    """The context-parallel walk of a shard that holds every key."""
    W = Q.shape[0] * Q.shape[1] * Q.shape[2]
    counts = [t.n_keys]
    for _ in range(t.depth):
        counts.append(counts[-1] // t.cfg.chunk)
    i32 = lambda *shape: torch.empty(*shape, dtype=torch.int32, device="cuda")
    ids, n, sel, cnt = i32(W, counts[1]), i32(W), i32(W, counts[1]), i32(W)
    scores = torch.empty(W, counts[1], device="cuda")
    level = t.cp_begin(Q, 0, counts)
    while level > 0:
        t.cp_export(ids, scores, n)
        level = t.cp_select(ids[None], scores[None], n[None], zha().TOP_P, 0.9, 1, sel, cnt)
    return sel, cnt


EAGER = {
    "dense_scan": lambda t, Q: t.dense_scan(Q, zha().TOP_K, k=5, max_sel=5),
    "chunk_mass": lambda t, Q: t.chunk_mass(Q, 8, 0.8)[:2],
    "ref_grad": lambda t, Q: t.ref_grad(Q),
    "walk": walk,
}


def lists(sel, cnt):
    return [row[:c].tolist() for row, c in zip(sel.cpu(), cnt.tolist())]


def assert_same(name, got, want):
    if name == "ref_grad":  # its sums are atomic: the terms of at most 60 walks and 600 keys in any order
        for a, b in zip(got, want):
            assert float((a - b).abs().max()) <= 60 * 600 * R.U * float(b.abs().max())
    else:
        assert lists(*got) == lists(*want)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", list(EAGER))
def test_an_eager_call_after_a_captured_one(name, kind):
    """An eager call that needs more scratch than the tree holds, once a call has been captured."""
    t, _, _ = make_tree(kind, 1, 2, 600, 64, 8, depth=2)
    Q, sel, cnt = inputs(t, 2)
    t.search(Q, zha().TOP_P, 0.9)
    t.attend(Q, sel, cnt)
    _, (out, _) = captured(lambda: t.attend(Q, sel, cnt))
    more, _, _ = inputs(t, 15, seed=2)  # 30 walks a tree, where the search had 4
    got = EAGER[name](t, more)
    t.sync_status()
    fresh, _, _ = make_tree(kind, 1, 2, 600, 64, 8, depth=2)
    assert_same(name, got, EAGER[name](fresh, more))


@pytest.mark.parametrize("name", ["dense_scan", "chunk_mass", "ref_grad"])
def test_a_captured_call_outlives_a_larger_one(name):
    """The block that a captured call of the second kind of scratch uses is kept when a larger call outgrows it."""
    t, _, _ = make_tree("bf16", 1, 2, 600, 64, 8, depth=2)
    Q, _, _ = inputs(t, 1)
    EAGER[name](t, Q)
    g, got = captured(lambda: EAGER[name](t, Q))
    more, _, _ = inputs(t, 15, seed=2)
    EAGER["chunk_mass"](t, more)
    EAGER["dense_scan"](t, more)
    Q.copy_(randn(9, *Q.shape, dtype=torch.bfloat16))
    for x in got:
        x.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert_same(name, got, EAGER[name](t, Q))
    t.sync_status()


@pytest.mark.parametrize("name", ["dense_scan", "chunk_mass", "ref_grad"])
def test_a_captured_call_of_the_second_block_does_not_allocate(name):
    t, _, _ = make_tree("bf16", 1, 1, 600, 64, 8, depth=2)
    Q, _, _ = inputs(t, 1)

    def both():
        with pytest.raises(zha().ZhaError, match="captured"):
            EAGER[name](t, Q)
        Q.mul_(1)  # the capture goes on

    captured(both)
    EAGER[name](t, Q)
    t.sync_status()


def test_only_blocks_that_a_graph_uses_are_kept():
    """After a capture, scratch that eager calls alone used is given back when it is outgrown."""
    big, _, _ = make_tree("bf16", 1, 1, 2 ** 19, 64, 8, depth=2, refs=1)
    Q1 = randn(3, 1, 1, 1, 64, dtype=torch.bfloat16)
    EAGER["dense_scan"](big, Q1)
    captured(lambda: EAGER["dense_scan"](big, Q1))
    torch.cuda.synchronize()
    free0 = torch.cuda.mem_get_info()[0]
    for n_q in range(2, 33):  # 8 bytes a walk and key: 2 blocks of 4 MB kept, and not 31 of 4 to 128 MB
        sel = torch.empty(n_q, 1, dtype=torch.int32, device="cuda")
        big.dense_scan(randn(4, 1, 1, n_q, 64, dtype=torch.bfloat16), zha().TOP_K, k=1, max_sel=1,
                       out=(sel, sel.new_empty(n_q)))
    torch.cuda.synchronize()
    # the last block, 132 MB, and what torch holds for 32 small tensors
    assert free0 - torch.cuda.mem_get_info()[0] <= 200 * 2 ** 20
