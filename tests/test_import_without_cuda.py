"""The package imports where torch was built without CUDA (its private CUDA names are missing there), and takes the
current stream without them."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import types, torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
del torch.float8_e8m0fnu  # younger than the rest of what the package uses
import tree_indexed_sparse_append_b200 as Z

# as a torch with a GPU and without those names would answer
asked = []
stream = lambda dev=None: asked.append(dev) or types.SimpleNamespace(cuda_stream=77 if dev in (None, 3) else 78)
torch.cuda.current_stream, torch.cuda.current_device = stream, lambda: 3
seen = []
Z._launch(lambda *a: seen.append(a) or Z.OK, 3, None, 5)
Z._launch(lambda *a: seen.append(a) or Z.OK, 3, types.SimpleNamespace(cuda_stream=9), 5)
assert seen == [(5, 77), (5, 9)], seen
try:
    Z.kv_read(*[torch.zeros(1, 1, 4, 64).to(torch.float8_e4m3fn)] * 2, *[torch.zeros(1, 1, 4, dtype=torch.uint8)] * 2, 0, 1)
except ValueError as e:
    assert "CUDA" in str(e)
else:
    raise AssertionError("a CPU cache was taken")
print("imported")
"""


def test_the_package_imports_without_torchs_cuda_names():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and "imported" in r.stdout, r.stderr
