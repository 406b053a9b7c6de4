"""include/flce_embed.h: the library exports what it declares, and bad arguments are refused on
the host before any device work."""
import ctypes
import os
import re

import linear_cross_entropy_flce_gb300 as flce
from linear_cross_entropy_flce_gb300 import _binding

HEADER = os.path.join(os.path.dirname(_binding.HEADER_PATH), "flce_embed.h")
lib = flce.lib
NULL, SHAPE, ALIGN, WS, OPTION, OK = (flce.FLCE_ERR_NULL, flce.FLCE_ERR_SHAPE, flce.FLCE_ERR_ALIGN,
                                      flce.FLCE_ERR_WORKSPACE, flce.FLCE_ERR_OPTION, flce.FLCE_OK)


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(flce_\w+)\s*\(", text)))
    assert len(names) == 3
    for name in names:
        assert hasattr(lib, name), name


def test_lookup_refusals():
    ok = dict(w=0x1000, wt=1, ldw=64, t=0x2000, N=8, V=100, D=64, s=1.0, y=0x3000, dt=1, ldy=64, st=None)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.flce_embedding(a["w"], a["wt"], a["ldw"], a["t"], a["N"], a["V"], a["D"], a["s"], -100,
                                  a["y"], a["dt"], a["ldy"], a["st"], None)

    for k in ("w", "t", "y"):
        assert call(**{k: None}) == NULL and call(**{k: 0x1001}) == ALIGN
    assert call(w=0x1002, wt=0) == ALIGN and call(st=0x4002) == ALIGN
    assert call(N=-1) == SHAPE and call(V=0) == SHAPE and call(D=0) == SHAPE and call(D=1 << 25) == SHAPE
    assert call(ldw=63) == SHAPE and call(ldy=63) == SHAPE and call(V=(1 << 30) + 1) == SHAPE
    assert call(wt=2) == OPTION and call(dt=-1) == OPTION and call(y=0x1000) == OPTION
    for s in (float("nan"), float("inf")):
        assert call(s=s) == OPTION
    assert call(N=0) == OK


def _ws(N, V=100, D=64):
    size = ctypes.c_size_t()
    return lib.flce_embedding_backward_workspace_size(N, V, D, ctypes.byref(size)), size.value


def test_gradient_refusals():
    ok = dict(dy=0x1000, dt=1, lddy=64, t=0x2000, N=8, V=100, D=64, s=1.0, dW=0x3000, wt=0, ldw=64, acc=0,
              ws=0x4000, wb=1 << 30)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.flce_embedding_backward(a["dy"], a["dt"], a["lddy"], a["t"], a["N"], a["V"], a["D"], a["s"],
                                           -100, a["dW"], a["wt"], a["ldw"], a["acc"], a["ws"], a["wb"], None)

    for k in ("dy", "t", "dW", "ws"):
        assert call(**{k: None}) == NULL and call(**{k: 0x1001}) == ALIGN
    assert call(ws=0x4008) == ALIGN and call(dW=0x3002) == ALIGN
    assert call(N=-1) == SHAPE and call(V=0) == SHAPE and call(D=0) == SHAPE
    assert call(lddy=63) == SHAPE and call(ldw=63) == SHAPE
    assert call(dt=2) == OPTION and call(wt=2) == OPTION and call(dW=0x1000) == OPTION and call(s=float("inf")) == OPTION
    assert call(wb=_ws(8)[1] - 1) == WS
    assert call(N=0, acc=1, dy=None, t=None, dW=None) == OK      # nothing to add


def test_workspace_size():
    assert lib.flce_embedding_backward_workspace_size(1, 1, 1, None) == NULL
    assert _ws(-1)[0] == SHAPE and _ws(1, V=0)[0] == SHAPE and _ws(1, D=0)[0] == SHAPE
    assert _ws(0) == (OK, 0)
    # the sorted order, and two fp32 rows for each of at most 2048 ranges; past one cluster's tokens the
    # order twice, and 512 counters for each tile of 4096
    assert _ws(8192, 128256, 4096)[1] <= 8192 * 8 + 256 * 2 * 4096 * 4 + 1024
    assert _ws(1 << 24, 128256, 4096)[1] <= (1 << 24) * 16 + 2049 * 2 * 4096 * 4 + 4096 * 512 * 4 + 4096
    assert flce.embedding_backward_workspace_size(100, 50, 33) == _ws(100, 50, 33)[1]
