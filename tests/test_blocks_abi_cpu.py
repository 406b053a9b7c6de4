"""include/flce_blocks.h: the library exports what it declares, and bad arguments are refused on
the host before any device work."""
import ctypes
import os
import re

import linear_cross_entropy_flce_gb300 as flce
from linear_cross_entropy_flce_gb300 import _binding

HEADER = os.path.join(os.path.dirname(_binding.HEADER_PATH), "flce_blocks.h")
lib = flce.lib
NULL, SHAPE, ALIGN, WS, OPTION, OK = (flce.FLCE_ERR_NULL, flce.FLCE_ERR_SHAPE, flce.FLCE_ERR_ALIGN,
                                      flce.FLCE_ERR_WORKSPACE, flce.FLCE_ERR_OPTION, flce.FLCE_OK)


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(flce_\w+)\s*\(", text)))
    assert len(names) == 9
    for name in names:
        assert hasattr(lib, name), name


def test_records():
    size = ctypes.c_int64()
    assert lib.flce_packed_row_bytes(1, None) == NULL
    for D in (0, -1, (1 << 24) + 1):
        assert lib.flce_packed_row_bytes(D, ctypes.byref(size)) == SHAPE
    for D, want in ((1, 48), (32, 48), (33, 80), (512, 528), (513, 544 + 32), (4096, 4224)):
        assert flce.packed_row_bytes(D) == want


def test_pack_refusals():
    for f, order in ((lib.flce_pack_e4m3, ("x", "t", "ld", "N", "D", "p")), (lib.flce_unpack_e4m3, ("p", "N", "D", "x", "t", "ld"))):
        def call(**kw):
            a = dict(dict(x=0x1000, t=1, ld=64, N=8, D=64, p=0x2000), **kw)
            return f(*[a[k] for k in order], None)

        assert call(x=None) == NULL and call(p=None) == NULL
        assert call(x=0x1001) == ALIGN and call(x=0x1002, t=0) == ALIGN and call(p=0x2008) == ALIGN
        assert call(N=-1) == SHAPE and call(D=0) == SHAPE and call(ld=63) == SHAPE and call(N=(1 << 30) + 1) == SHAPE
        assert call(t=2) == OPTION and call(p=0x1000) == OPTION
        assert call(N=0) == OK


def test_layer_norm_refusals():
    def forward(x=0x1000, t=1, ldx=64, w=0x2000, b=0x3000, wt=0, N=8, D=64, eps=1e-5, y=0x4000, ldy=64, m=0x5000,
                r=0x6000, p=0x7000):
        return lib.flce_layer_norm_packed(x, t, ldx, w, b, wt, N, D, eps, y, ldy, m, r, p, None)

    assert forward(x=None) == NULL and forward(y=None) == NULL and forward(p=None) == NULL
    assert forward(ldx=63) == SHAPE and forward(ldy=63) == SHAPE and forward(N=-1) == SHAPE and forward(D=0) == SHAPE
    assert forward(t=3) == OPTION and forward(wt=2) == OPTION and forward(eps=-1.0) == OPTION
    assert forward(eps=float("nan")) == OPTION and forward(p=0x1000) == OPTION and forward(y=0x1000, ldy=72) == OPTION
    for k in ("x", "w", "b", "y", "m", "r", "p"):
        assert forward(**{k: 0x1001}) == ALIGN, k
    assert forward(N=0) == OK

    def back(dy=0x1000, t=1, lddy=64, p=0x2000, w=0x3000, wt=0, m=0x4000, r=0x5000, N=8, D=64, dx=0x6000, lddx=64,
             dw=0x7000, db=0x8000, ws=0x9000, wb=1 << 30):
        return lib.flce_layer_norm_packed_backward(dy, t, lddy, p, w, wt, m, r, N, D, dx, lddx, dw, db, ws, wb, None)

    for k in ("dy", "p", "m", "r", "ws"):
        assert back(**{k: None}) == NULL, k
    for k in ("dy", "p", "w", "m", "r", "dx", "dw", "db", "ws"):
        assert back(**{k: 0xA001}) == ALIGN, k
    assert back(lddy=63) == SHAPE and back(lddx=63) == SHAPE and back(D=0) == SHAPE
    assert back(t=2) == OPTION and back(wt=2) == OPTION and back(dx=0x2000) == OPTION and back(dx=0x1000, lddx=72) == OPTION
    assert back(wb=8 * 2 * 64 * 4 - 1) == WS
    assert back(N=0, dw=None, db=None) == OK


def _sizes(N, D, fmt):
    row, scales = ctypes.c_int64(), ctypes.c_size_t()
    rc = lib.flce_fp4_sizes(N, D, fmt, ctypes.byref(row), ctypes.byref(scales))
    return rc, row.value, scales.value


def test_fp4_sizes():
    assert lib.flce_fp4_sizes(1, 1, 0, None, None) == NULL
    assert _sizes(-1, 1, 0)[0] == SHAPE and _sizes(1, 0, 0)[0] == SHAPE and _sizes(1, 1, 2)[0] == OPTION
    assert _sizes(0, 64, 1) == (OK, 32, 0)
    assert _sizes(1, 1, 1) == (OK, 32, 2048) and _sizes(1, 1, 0) == (OK, 32, 1024)
    assert _sizes(129, 257, 1) == (OK, 160, 2 * 2 * 2048)
    assert _sizes(128256, 4096, 1) == (OK, 2048, 128256 * 4096 // 16)


def test_fp4_refusals():
    def quant(x=0x1000, t=1, ld=64, N=8, D=64, fmt=1, c=0x2000, s=0x3000, r=0x4000):
        return lib.flce_quantize_fp4(x, t, ld, N, D, fmt, c, s, r, None)

    def values(c=0x2000, s=0x3000, r=0x4000, N=8, D=64, fmt=1, x=0x1000, t=1, ld=64):
        return lib.flce_dequantize_fp4(c, s, r, N, D, fmt, x, t, ld, None)

    for call in (quant, values):
        for k in ("x", "c", "s", "r"):
            assert call(**{k: None}) == NULL and call(**{k: 0x1001}) == ALIGN, k
        assert call(c=0x2008) == ALIGN and call(s=0x3008) == ALIGN and call(x=0x1002, t=0) == ALIGN
        assert call(N=-1) == SHAPE and call(D=0) == SHAPE and call(ld=63) == SHAPE
        assert call(fmt=2) == OPTION and call(t=2) == OPTION and call(c=0x1000) == OPTION and call(s=0x1000) == OPTION
        assert call(N=0) == OK

    def linear(N=8, D=64, V=100, fmt=1, y=0xA000, t=1, ldy=100, tmo=0, st=None, **kw):
        a = dict(dict(hc=0x1000, hs=0x2000, hr=0x3000, wc=0x4000, wsc=0x5000, wr=0x6000), **kw)
        return lib.flce_linear_fp4(a["hc"], a["hs"], a["hr"], a["wc"], a["wsc"], a["wr"], N, D, V, fmt, y, t, ldy,
                                   tmo, st, None)

    for k in ("hc", "hs", "hr", "wc", "wsc", "wr", "y"):
        assert linear(**{k: None}) == NULL and linear(**{k: 0x1001}) == ALIGN, k
    assert linear(y=0xA002, t=0) == ALIGN and linear(st=0xB002) == ALIGN and linear(wc=0x4008) == ALIGN
    assert linear(N=-1) == SHAPE and linear(D=0) == SHAPE and linear(V=0) == SHAPE and linear(ldy=99) == SHAPE
    assert linear(fmt=-1) == OPTION and linear(t=2) == OPTION and linear(tmo=-1) == OPTION
    assert linear(N=0) == OK
