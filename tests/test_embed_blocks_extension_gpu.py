"""The compiled calls of the embedding and of the block-scaled formats give what the general forms
give, and leave to those what they do not take."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import linear_cross_entropy_flce_gb300 as flce
    from linear_cross_entropy_flce_gb300 import _ops_binding

DEV = "cuda:0"


def _same(a, b):
    if isinstance(a, (tuple, list)):
        return len(a) == len(b) and all(_same(x, y) for x, y in zip(a, b))
    if isinstance(a, torch.Tensor):
        return a.dtype == b.dtype and a.shape == b.shape and torch.equal(a, b)
    if hasattr(a, "__dataclass_fields__"):
        return _same([getattr(a, f) for f in a.__dataclass_fields__], [getattr(b, f) for f in b.__dataclass_fields__])
    return a == b


def _calls():
    g = torch.Generator(device=DEV).manual_seed(1)
    W = torch.randn(50, 72, generator=g, device=DEV)
    x = torch.randn(3, 7, 72, generator=g, device=DEV).bfloat16()
    t = torch.randint(-1, 50, (3, 7), generator=g, device=DEV).int()
    w = torch.randn(72, generator=g, device=DEV)
    r, p = flce.layer_norm_packed(x, w)
    h, v = flce.quantize_fp4(x), flce.quantize_fp4(W)
    m, n = flce.quantize_fp4(x, format="mxfp4"), flce.quantize_fp4(W, format="mxfp4")
    return {
        "embedding": lambda **k: flce.embedding(W, t, scale=2.0, ignore_index=-1, dtype=torch.bfloat16, **k),
        "embedding_backward": lambda **k: flce.embedding_backward(x, t, 50, ignore_index=-1, dtype=torch.float32, **k),
        "pack_e4m3": lambda **k: flce.pack_e4m3(x, **k),
        "unpack_e4m3": lambda **k: flce.unpack_e4m3(p, **k),
        "layer_norm_packed": lambda **k: flce.layer_norm_packed(x, w, w, **k),
        "layer_norm_packed_backward": lambda **k: flce.layer_norm_packed_backward(x, p, w, r, need_dbias=False, **k),
        "quantize_fp4": lambda **k: (flce.quantize_fp4(x, **k), flce.quantize_fp4(W, format="mxfp4", **k)),
        "dequantize_fp4": lambda **k: (flce.dequantize_fp4(h, **k), flce.dequantize_fp4(m, dtype=torch.bfloat16, **k)),
        "linear_fp4": lambda **k: (flce.linear_fp4(h, v, **k), flce.linear_fp4(m, n, dtype=torch.float32, **k)),
    }


def test_compiled_and_general_forms_agree(monkeypatch):
    if isinstance(_ops_binding._fast, _ops_binding._NoExtension):
        pytest.skip("built without the extension")
    taken = []
    for name, call in _calls().items():
        real = getattr(_ops_binding._fast, name)
        fast = call()
        here = torch.cuda.current_stream()
        general = call(stream=here)
        assert _same(fast, general), name
        taken.append(real)
    assert len(taken) == 9


def test_what_the_compiled_forms_do_not_take():
    x = torch.randn(4, 6, 40, device=DEV)
    view = x.transpose(0, 1)   # rows in another order than they lie
    t = torch.zeros(6, 4, dtype=torch.int32, device=DEV)
    assert _ops_binding._fast.pack_e4m3(view) is None and _ops_binding._fast.quantize_fp4(view, 1) is None
    assert torch.equal(flce.unpack_e4m3(flce.pack_e4m3(view)), flce.unpack_e4m3(flce.pack_e4m3(view.contiguous())))
    want = flce.embedding_backward(view.contiguous(), t, 3)
    assert torch.equal(flce.embedding_backward(view, t, 3), want)
    with torch.cuda.stream(torch.cuda.Stream()):
        pass


def test_errors_are_named():
    W = torch.zeros(4, 8, device=DEV)
    with pytest.raises(flce.FLCEError, match="flce_embedding"):
        flce.embedding(W, torch.zeros(1, dtype=torch.int32, device=DEV), scale=float("nan"))
