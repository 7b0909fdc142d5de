"""A tree's calls run on its own GPU and stream, whatever GPU is current, and refuse tensors of another: checked on the
binding, with a library and tensors that only record."""
import contextlib
import ctypes

import pytest
import torch

import tree_indexed_sparse_append_b200 as Z


class Gpu:
    """As much of a tensor on GPU `index` as the binding asks for."""

    def __init__(self, shape, dtype=torch.float32, index=1):
        self.shape, self.dtype, self.index, self.is_cuda = torch.Size(shape), dtype, index, index >= 0
        self.device = torch.device("cuda", index) if index >= 0 else torch.device("cpu")

    def get_device(self):
        return self.index

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def unsqueeze(self, i):
        return Gpu(self.shape[:i] + (1,) + self.shape[i:], self.dtype, self.index)

    def new_empty(self, *shape, dtype=None):
        return Gpu(shape, dtype or self.dtype, self.index)


class Lib:
    def __init__(self, log, current):
        self.log, self.current = log, current

    def __getattr__(self, name):
        def call(*args):
            self.log.append((name, self.current[-1], args))
            return {"zha_num_keys": 64, "zha_depth": 1}.get(name, Z.OK)

        return call


@pytest.fixture
def world(monkeypatch):
    """GPU 0 current; stream handles 100 + GPU. Returns the log of (call, GPU current at it, arguments)."""
    log, current = [], [0]

    @contextlib.contextmanager
    def device(d):
        current.append(d)
        yield
        current.pop()

    fake = Lib(log, current)
    monkeypatch.setattr(Z, "lib", lambda: fake)
    monkeypatch.setattr(Z, "_get_device", lambda: current[-1])
    monkeypatch.setattr(Z, "_raw_stream", lambda d: 100 + d)
    monkeypatch.setattr(torch.cuda, "device", device)
    for name in ("empty", "zeros"):
        def make(*shape, dtype=torch.float32, device=None, real=getattr(torch, name), **kw):
            if isinstance(device, torch.device) and device.type == "cuda":
                return Gpu(shape, dtype, device.index)
            return real(*shape, dtype=dtype, device=device, **kw)
        monkeypatch.setattr(torch, name, make)
    monkeypatch.setattr(torch, "empty_like", lambda x, dtype=None, **kw: Gpu(x.shape, dtype or x.dtype, x.index))
    return log


I32 = torch.int32
HOST = ("zha_num_keys", "zha_depth", "zha_level")  # calls that touch no GPU
B, H, n, d, W = 1, 2, 64, 64, 6


def tree(kind):
    dt = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[kind]
    K, V, refs = Gpu((B, H, n, d), dt), Gpu((B, H, n, d), dt), Gpu((H, 2, d))
    e = Gpu((B, H, n), torch.uint8)
    return Z.Tree(K, V, refs, n, 8, 1, 0.1, **(dict(k_scale=e, v_scale=e) if kind == "e4m3" else {}))


def calls(t, i=1):
    """Every call with a stream, its first tensor on GPU i."""
    Q, row = Gpu((B, H, 3, d), torch.bfloat16, i), Gpu((B, H, d), torch.bfloat16, i)
    rows = Gpu((B, H, 3, d), torch.bfloat16, i)
    sel, cnt, lse = Gpu((W, 4), I32), Gpu((W,), I32), Gpu((W,))
    ids, scores, counts = Gpu((2, W, 4), I32, i), Gpu((2, W, 4)), Gpu((2, W), I32)
    return {
        "append": lambda: t.append(row, row),
        "extend": lambda: t.extend(rows, rows),
        "search": lambda: t.search(Q, Z.TOP_P, 0.9),
        "attend": lambda: t.attend(Q, sel, cnt),
        "attend_noalloc": lambda: t.attend_noalloc(Q, sel, cnt, Gpu((B, H, 3, d), torch.bfloat16), lse),
        "attend_draft": lambda: t.attend_draft(Q, sel, cnt, Gpu((B, H, 3, d)), Gpu((B, H, 3, d)), Gpu((B, 3, 3), torch.uint8)),
        "dense_scan": lambda: t.dense_scan(Q),
        "chunk_mass": lambda: t.chunk_mass(Q),
        "ref_grad": lambda: t.ref_grad(Q),
        "cp_begin": lambda: t.cp_begin(Q, 0, [64, 8]),
        "cp_export": lambda: t.cp_export(Gpu((W, 4), I32, i), Gpu((W, 4)), cnt),
        "cp_select": lambda: t.cp_select(ids, scores, counts, Z.TOP_P, 0.9, 1, sel, cnt),
    }


STREAMS_ONLY = {
    "rebuild": lambda t: t.rebuild(),
    "profile_read": lambda t: t.profile_read(),
    "last_search_info": lambda t: t.last_search_info(),
    "sync_status": lambda t: t.sync_status(),
}


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_calls_run_on_the_trees_gpu(world, kind):
    t = tree(kind)
    for call in [*calls(t).values(), *(lambda f=f: f(t) for f in STREAMS_ONLY.values()), lambda: t.reserve(4, 4)]:
        call()
    names = [name for name, _, _ in world]
    assert len(set(names)) >= 15
    for name, current, args in world:
        if name in HOST:
            continue
        assert current == 1, name
        if name == "zha_reserve":
            continue
        handles = [a for a in args if isinstance(a, int) and a in (100, 101)]
        assert handles == [101], (name, args)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("index", [0, -1])
def test_tensors_of_another_device_are_refused(world, kind, index):
    t = tree(kind)
    for name, call in calls(t, index).items():
        del world[:]
        with pytest.raises((ValueError, TypeError), match="cuda:1"):
            call()
        assert not [x for x in world if x[0] not in HOST], name


def test_a_given_stream_is_taken(world):
    t = tree("bf16")
    stream = type("S", (), {"cuda_stream": 7})()
    t.attend(Gpu((B, H, 3, d)), Gpu((W, 4), I32), Gpu((W,), I32), stream=stream)
    assert world[-1][0] == "zha_attend" and world[-1][1] == 1 and world[-1][2][-1] == 7


def test_partial_results_are_combined_on_their_gpu(world):
    Z.lse_combine(Gpu((2, 5, d)), Gpu((2, 5)))
    assert world[-1][0] == "zha_lse_combine" and world[-1][1] == 1 and world[-1][2][-1] == 101
