"""include/flce_ops.h: the library exports what it declares, a C program can use it, and bad
arguments are refused on the host before any device work (no compute call is made here)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import linear_cross_entropy_flce_gb300 as flce
from linear_cross_entropy_flce_gb300 import _binding, _ops_binding

torch = pytest.importorskip("torch")

HEADER = os.path.join(os.path.dirname(_binding.HEADER_PATH), "flce_ops.h")
lib = flce.lib
NULL, SHAPE, ALIGN, WS, OPTION = (flce.FLCE_ERR_NULL, flce.FLCE_ERR_SHAPE, flce.FLCE_ERR_ALIGN,
                                  flce.FLCE_ERR_WORKSPACE, flce.FLCE_ERR_OPTION)


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(flce_\w+)\s*\(", text)))
    assert len(names) == 11
    for name in names:
        assert hasattr(lib, name), name


def test_default_options():
    o = flce.LogprobOptions()
    lib.flce_default_logprob_options(ctypes.byref(o))
    assert (o.ignore_index, o.top_k, o.temperature, o.dw_dtype, o.timeout_ns) == (-100, 0, 1.0, 0, 0)
    assert ctypes.sizeof(o) == 24


def _opt(**kw):
    o = flce.LogprobOptions(-100, 0, 1.0, 0, 0)
    for k, v in kw.items():
        setattr(o, k, v)
    return o


BAD_OPTIONS = [dict(top_k=-1), dict(top_k=33), dict(temperature=0.0), dict(temperature=-1.0),
               dict(temperature=float("inf")), dict(temperature=float("nan")), dict(temperature=1e-45),
               dict(dw_dtype=2), dict(timeout_ns=-1)]


def test_token_logprobs_refusals():
    ok = dict(z=0x1000, dtype=0, ld=100, y=0x2000, N=8, V=100, o=None, lp=0x3000, ent=0x4000,
              lse=0x5000, tl=None, ti=None, st=None)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.flce_token_logprobs(a["z"], a["dtype"], a["ld"], a["y"], a["N"], a["V"], a["o"],
                                       a["lp"], a["ent"], a["lse"], a["tl"], a["ti"], a["st"], None)

    assert call(z=None) == NULL
    assert call(o=_opt(top_k=4)) == NULL
    assert call(o=_opt(top_k=4), tl=0x6000) == NULL
    assert call(N=-1) == SHAPE and call(V=0) == SHAPE and call(V=(1 << 30) + 1, ld=1 << 31) == SHAPE
    assert call(ld=99) == SHAPE
    assert call(dtype=2) == OPTION
    for bad in BAD_OPTIONS:
        assert call(o=_opt(**bad)) == OPTION, bad
    assert call(o=_opt(top_k=5), V=4, ld=4, tl=0x6000, ti=0x7000) == OPTION
    assert call(z=0x1002) == ALIGN and call(z=0x1001, dtype=1) == ALIGN
    for k in ("y", "lp", "ent", "lse", "st"):
        assert call(**{k: 0x2002}) == ALIGN, k
    assert call(N=0) == flce.FLCE_OK      # nothing to do, nothing enqueued


def test_token_logprobs_backward_refusals():
    ok = dict(z=0x1000, dtype=0, ld=100, y=0x2000, N=8, V=100, o=None, lp=0x3000, ent=0x4000,
              lse=0x5000, a=0x6000, b=0x7000, c=None, dz=0x8000, dld=100)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.flce_token_logprobs_backward(
            a["z"], a["dtype"], a["ld"], a["y"], a["N"], a["V"], a["o"], a["lp"], a["ent"], a["lse"],
            a["a"], a["b"], a["c"], a["dz"], a["dld"], None)

    assert call(z=None) == NULL and call(dz=None) == NULL and call(lse=None) == NULL
    assert call(a=None, b=None) == NULL              # no upstream gradient
    assert call(ent=None) == NULL and call(lp=None) == NULL
    assert call(dld=99) == SHAPE and call(ld=99) == SHAPE and call(N=-1) == SHAPE
    assert call(dz=0x1000, dld=104) == OPTION and call(dtype=7) == OPTION
    assert call(dz=0x8002) == ALIGN and call(c=0x9001) == ALIGN
    for bad in BAD_OPTIONS[2:7]:
        assert call(o=_opt(**bad)) == OPTION
    assert call(N=0) == flce.FLCE_OK


def _linear_ws(N=64, D=128, V=1000, backward=0, **kw):
    size = ctypes.c_size_t()
    rc = lib.flce_linear_logprobs_workspace_size(N, D, V, _opt(**kw), backward, ctypes.byref(size))
    return rc, size.value


def test_linear_workspace_size():
    assert _linear_ws(D=12)[0] == ALIGN
    assert _linear_ws(V=0)[0] == SHAPE and _linear_ws(N=-1)[0] == SHAPE
    for bad in BAD_OPTIONS:
        assert _linear_ws(**bad)[0] == OPTION, bad
    assert lib.flce_linear_logprobs_workspace_size(1, 8, 8, None, 0, None) == NULL
    assert _linear_ws(N=0) == (flce.FLCE_OK, 0)
    # far below the logits, with and without rankings and gradients
    for N, D, V in ((1, 4096, 128256), (8192, 4096, 128256), (4096, 2048, 32000)):
        small, ranked = _linear_ws(N, D, V)[1], _linear_ws(N, D, V, top_k=20)[1]
        assert 0 < small <= ranked   # equal for a few tokens, whose logits are held either way
        if N > 1:
            assert ranked < N * V * 4 // 10
            assert _linear_ws(N, D, V, backward=1)[1] < N * V * 4 // 2
    assert flce.linear_logprobs_workspace_size(8, 64, 500, top_k=3) == _linear_ws(8, 64, 500, top_k=3)[1]


def test_linear_refusals():
    ok = dict(H=0x1000, W=0x2000, y=0x3000, N=64, D=128, V=1000, o=None, lp=0x4000, ent=0x5000,
              lse=0x6000, tl=None, ti=None, ws=0x7000, wb=1 << 30, st=None)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.flce_linear_token_logprobs(
            a["H"], a["W"], a["y"], a["N"], a["D"], a["V"], a["o"], a["lp"], a["ent"], a["lse"],
            a["tl"], a["ti"], a["ws"], a["wb"], a["st"], None)

    for k in ("H", "W", "ws"):
        assert call(**{k: None}) == NULL and call(**{k: 0x1008}) == ALIGN
    assert call(o=_opt(top_k=3)) == NULL
    assert call(wb=8) == WS
    assert call(D=100) == ALIGN and call(V=0) == SHAPE
    assert call(lp=0x4002) == ALIGN and call(st=0x4001) == ALIGN
    assert call(N=0) == flce.FLCE_OK

    def back(dH=0x8000, dW=0x9000, a=0xA000, lse=0x6000, wb=1 << 30, N=64, lp=0x4000, **o):
        return lib.flce_linear_token_logprobs_backward(
            0x1000, 0x2000, 0x3000, N, 128, 1000, _opt(**o), lp, 0x5000, lse, a, None, None, dH, dW,
            0x7000, wb, None, None)

    assert back(dH=None, dW=None) == NULL and back(a=None) == NULL and back(lse=None) == NULL
    assert back(lp=None) == NULL
    assert back(dH=0x8008) == ALIGN and back(dW=0x9004) == ALIGN
    assert back(wb=16) == WS
    assert back(temperature=0.0) == OPTION and back(dw_dtype=5) == OPTION
    assert back(N=0, dW=None) == flce.FLCE_OK


def test_layer_norm_refusals():
    def call(x=0x1000, dtype=0, ldx=64, w=0x2000, b=0x3000, wd=0, N=4, D=64, eps=1e-5, y=0x4000,
             ldy=64, mean=None, rstd=None):
        return lib.flce_layer_norm(x, dtype, ldx, w, b, wd, N, D, eps, y, ldy, mean, rstd, None)

    assert call(x=None) == NULL and call(y=None) == NULL
    assert call(N=-1) == SHAPE and call(D=0) == SHAPE and call(ldx=63) == SHAPE and call(ldy=63) == SHAPE
    assert call(dtype=3) == OPTION and call(wd=-1) == OPTION
    for eps in (-1.0, float("nan"), float("inf")):
        assert call(eps=eps) == OPTION
    assert call(y=0x1000, ldy=65) == OPTION        # in place with another stride
    assert call(x=0x1002) == ALIGN and call(w=0x2001) == ALIGN and call(mean=0x5002) == ALIGN
    assert call(N=0) == flce.FLCE_OK
    size = ctypes.c_size_t()
    assert lib.flce_layer_norm_workspace_size(8192, 4096, ctypes.byref(size)) == flce.FLCE_OK
    assert 0 < size.value <= 304 * 2 * 4096 * 4
    assert lib.flce_layer_norm_workspace_size(4, 0, ctypes.byref(size)) == SHAPE
    assert lib.flce_layer_norm_workspace_size(4, 8, None) == NULL

    def back(dy=0x1000, x=0x2000, mean=0x3000, rstd=0x4000, dx=0x5000, dw=0x6000, db=0x7000,
             ws=0x8000, wb=1 << 20, lddx=64, lddy=64, N=4):
        return lib.flce_layer_norm_backward(dy, lddy, x, 0, 64, None, 0, mean, rstd, N, 64, dx, lddx,
                                            dw, db, ws, wb, None)

    for k in ("dy", "x", "mean", "rstd", "ws"):
        assert back(**{k: None}) == NULL, k
    assert back(wb=100) == WS
    assert back(lddx=1) == SHAPE and back(lddy=1) == SHAPE
    assert back(dx=0x1000, lddx=70) == OPTION and back(dx=0x2000) == OPTION
    assert back(dx=0x5002) == ALIGN and back(dw=0x6001) == ALIGN and back(ws=0x8008) == ALIGN
    assert back(N=0, dw=None, db=None) == flce.FLCE_OK


def test_clip_refusals():
    def call(ptr=0x1000, out=0x2000, n=8, dtype=0, count=1, max_norm=1.0, norm=0x3000, ws=0x4000,
             wb=1 << 20, grads=True):
        g, o = (ctypes.c_void_p * 1)(ptr), (ctypes.c_void_p * 1)(out)
        return lib.flce_clip_grads(g if grads else None, o, (ctypes.c_int64 * 1)(n),
                                   (ctypes.c_int32 * 1)(dtype), count, max_norm, norm, ws, wb, None)

    assert call(ptr=None) == NULL and call(out=None) == NULL and call(norm=None) == NULL
    assert call(ws=None) == NULL and call(grads=False) == NULL
    assert call(n=-1) == SHAPE and call(count=-1) == SHAPE
    assert call(dtype=4) == OPTION and call(max_norm=-0.5) == OPTION and call(max_norm=float("nan")) == OPTION
    assert call(ptr=0x1002) == ALIGN and call(out=0x2001, dtype=1) == ALIGN and call(norm=0x3001) == ALIGN
    assert call(wb=64) == WS


def test_binding_refuses_host_tensors_and_bad_arguments():
    z = torch.zeros(2, 10)
    y = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        flce.token_logprobs(z, y)
    with pytest.raises(ValueError):
        flce.linear_token_logprobs(z.bfloat16(), z.bfloat16(), y)
    with pytest.raises(ValueError):
        flce.layer_norm(z)
    with pytest.raises(KeyError):
        flce.linear_logprobs_workspace_size(4, 64, 100, dw_dtype="float16")
    with pytest.raises(flce.FLCEError):
        flce.linear_logprobs_workspace_size(4, 63, 100)


def test_dense_layouts():
    a = torch.zeros(4, 5, 6)
    assert _ops_binding._dense(a.permute(2, 0, 1)) and _ops_binding._dense(a[:1].transpose(1, 2))
    assert not _ops_binding._dense(a[:, :3]) and not _ops_binding._dense(a[:, :1].expand(4, 5, 6))
    assert not _ops_binding._dense(torch.zeros(3, 4)[:, ::2])


C_PROGRAM = r"""
#include <stdio.h>
#include "flce_ops.h"
int main(void) {
  flce_logprob_options o;
  size_t bytes = 0;
  flce_default_logprob_options(&o);
  if (sizeof(o) != 24 || o.temperature != 1.0f || o.ignore_index != -100) return 1;
  o.top_k = FLCE_MAX_TOP_K;
  if (flce_linear_logprobs_workspace_size(16, 64, 1000, &o, 0, &bytes) != FLCE_OK || bytes == 0) return 2;
  if (flce_layer_norm_workspace_size(16, 64, &bytes) != FLCE_OK) return 3;
  if (flce_clip_grads_workspace_size(3, &bytes) != FLCE_OK || bytes < 8) return 4;
  if (flce_token_logprobs(NULL, FLCE_DTYPE_F32, 4, NULL, 1, 4, &o, NULL, NULL, NULL, NULL, NULL,
                          NULL, NULL) != FLCE_ERR_OPTION) return 5;   /* top_k above V */
  printf("ok\n");
  return 0;
}
"""


def test_header_compiles_as_c_and_links(tmp_path):
    gcc = shutil.which("gcc") or shutil.which("cc")
    if gcc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "ops.c"
    src.write_text(C_PROGRAM)
    libdir = os.path.dirname(_binding.LIB_PATH)
    exe = str(tmp_path / "ops")
    r = subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.dirname(HEADER), str(src),
                        "-L", libdir, "-lflce", "-Wl,-rpath," + libdir, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.returncode, r.stdout, r.stderr)
