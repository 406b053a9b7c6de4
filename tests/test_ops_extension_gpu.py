"""The compiled form of the operators' calls (_flce_ops): what it does with errors that come
after its checks. A small library whose symbols
come first stands in for calls that fail."""
import os
import shutil
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FAILING = r"""
static int count;
int flce_clip_grads(const void *g) { (void)g; ++count; return 6; }   /* FLCE_ERR_CUDA */
int flce_layer_norm(const void *x) { (void)x; ++count; return 6; }
int failing_calls(void) { return count; }
"""

PROGRAM = r"""
import ctypes, sys, torch
failing = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
import linear_cross_entropy_flce_gb300 as flce
g = torch.full((100,), 3.0, device="cuda:0")
for k, call in enumerate((lambda: flce.clip_grads([g], 1.0), lambda: flce.layer_norm(g))):
    try:
        call()
    except flce.FLCEError as e:
        assert e.code == flce.FLCE_ERR_CUDA and "flce_" in str(e), e
    else:
        raise SystemExit("tried again")
    assert failing.failing_calls() == k + 1
assert bool((g == 3).all())
print("ok")
"""


def _run(program, *args):
    r = subprocess.run([sys.executable, "-c", program, *args], capture_output=True, text=True, timeout=300,
                       cwd=ROOT, env={**os.environ, "PYTHONPATH": ROOT})
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), (r.stdout, r.stderr[-2000:])


def test_a_cuda_error_is_raised_and_the_call_not_made_again(tmp_path):
    gcc = shutil.which("gcc") or shutil.which("cc")
    if gcc is None:
        pytest.skip("no C compiler")
    src, lib = tmp_path / "failing.c", tmp_path / "failing.so"
    src.write_text(FAILING)
    r = subprocess.run([gcc, "-shared", "-fPIC", "-o", str(lib), str(src)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    _run(PROGRAM, str(lib))


OUT_OF_MEMORY = r"""
import torch
import linear_cross_entropy_flce_gb300 as flce
x = torch.ones(40000, 1024, device="cuda:0")     # 164 MB, of 280 MB that the process may take
torch.cuda.set_per_process_memory_fraction(280e6 / torch.cuda.get_device_properties(0).total_memory)
try:
    flce.layer_norm(x)
except torch.OutOfMemoryError:
    print("ok")
"""


def test_out_of_memory_is_pytorchs_own_error():
    _run(OUT_OF_MEMORY)
