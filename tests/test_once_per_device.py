"""A kernel's shared-memory limit is set once on each device (csrc/zha_once.cuh), not once in a process."""
import os
import re
import subprocess

import numpy as np
import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tree_indexed_sparse_append_b200", "csrc")

PROGRAM = r"""
#include "zha_once.cuh"
#include <cstdio>
int main() {
    zha::OncePerDevice once;
    int calls = 0, fail = 0;
    auto set = [&] { ++calls; return fail; };
    fail = 7;
    const int first = once(0, set);            // fails: tried again
    fail = 0;
    for (int i = 0; i < 2; ++i)
        for (int d = 0; d < 8; ++d) once(d, set);
    const int eight = calls;
    once(63, set), once(63, set);
    const int nine = calls;
    once(64, set), once(64, set);              // behind the bits: each time
    std::printf("%d %d %d %d\n", first, eight, nine, calls);
}
"""


def test_every_device_and_every_failure(tmp_path):
    src = tmp_path / "once.cpp"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, "-o", tmp_path / "once", src], check=True)
    out = subprocess.run([tmp_path / "once"], check=True, capture_output=True, text=True).stdout
    assert out.split() == ["7", "9", "10", "12"]


def test_no_limit_is_set_once_in_a_process():
    """Every limit is set at each launch or through OncePerDevice: no flag of its own stands before one."""
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as f:
            assert not re.search(r"static\s+(thread_local\s+)?(bool|int)[^;]*;[^;]*\)?\s*\{[^}]*cudaFuncSetAttribute", f.read()), name


@pytest.mark.gpu
@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_the_second_gpu_takes_many_walks_too():
    import serving_reference as R
    import tree_indexed_sparse_append_b200 as Z

    got = []
    for dev in (0, 1):
        with torch.cuda.device(dev):
            g = torch.Generator().manual_seed(1)
            x = lambda *shape: torch.randn(*shape, generator=g).bfloat16().cuda()
            t = Z.Tree(x(1, 1, 1003, 128), x(1, 1, 1003, 128), x(1, 4, 128).float(), 1003, 8, 2, 128 ** -0.5)
            Q = x(1, 1, 1024, 128)
            sel, cnt = R.selection(np.random.default_rng(2), 1, 1024, 125, 9)
            sel, cnt = torch.from_numpy(sel).cuda(), torch.from_numpy(cnt).cuda()
            out, _ = t.attend(Q, sel, cnt, out_dtype=torch.float32)
            found, n, _ = t.search(Q, Z.TOP_P, 0.9)
            t.sync_status()
            got.append((out.cpu(), n.cpu()))
    # the sums' order is the atomics': weights of 2^-17 and 72 keys' terms
    assert float((got[0][0] - got[1][0]).abs().max()) <= (2.0 ** -17 + 80 * R.U) * 2 * 6
    assert torch.equal(got[0][1], got[1][1])
