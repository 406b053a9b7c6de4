"""The compiled form of the operators' calls (_flce_ops) is for speed only: without it, or with
one for another PyTorch, the package and the loss work all the same."""
import concurrent.futures as cf
import os
import subprocess
import sys

import pytest

import linear_cross_entropy_flce_gb300 as flce
from linear_cross_entropy_flce_gb300 import _ops_binding, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
import sys, types, warnings
name = "linear_cross_entropy_flce_gb300._flce_ops"
sys.modules[name] = eval(sys.argv[1])
with warnings.catch_warnings(record=True) as said:
    warnings.simplefilter("always")
    import linear_cross_entropy_flce_gb300 as flce
assert any("_flce_ops" in str(w.message) and sys.argv[2] in str(w.message) for w in said), said
import torch
assert flce.workspace_size(64, 128, 1000) > 0
for call in (lambda t: flce.layer_norm(t), lambda t: flce.token_logprobs(t, None), lambda t: flce.clip_grads([t], 1.0),
             lambda t: flce.linear_token_logprobs(t, t, None)):
    try:
        call(torch.zeros(2, 8))
    except (ValueError, RuntimeError, AssertionError):   # a host tensor, or no GPU
        pass
    else:
        raise SystemExit("a host tensor was taken")
print("ok")
"""


@pytest.mark.parametrize("module,why", [("None", ""), ("types.SimpleNamespace(torch_version='1.0.0')", "1.0.0")])
def test_the_package_works_without_its_extension(module, why):
    r = subprocess.run([sys.executable, "-c", PROGRAM, module, why], capture_output=True, text=True, timeout=300,
                       cwd=ROOT, env={**os.environ, "PYTHONPATH": ROOT})
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.stdout, r.stderr[-2000:])


def test_this_tree_has_it():
    assert not isinstance(_ops_binding._fast, _ops_binding._NoExtension)
    assert flce.lib is not None


def test_a_build_that_cannot_compile_it_goes_on_without(tmp_path, monkeypatch):
    old = tmp_path / "_flce_ops.so"
    old.write_bytes(b"of another build")
    monkeypatch.setattr(build, "EXT", str(old))
    failed = cf.Future()
    failed.set_exception(RuntimeError("no torch headers"))
    with pytest.warns(RuntimeWarning, match="no torch headers"):
        build._finish_ext(failed)
    assert not old.exists()
