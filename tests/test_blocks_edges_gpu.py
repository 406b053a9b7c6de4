"""Calls of the embedding and of the block-scaled formats at the ends of their ranges: few rows of W under many
tokens, long and short rows, two calls at once on two streams, outputs among other data, one result for one
input however it is reached."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import linear_cross_entropy_flce_gb300 as flce
    from test_fp4_gpu import _check, _pair

DEV = "cuda:0"


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("N,D,V", [
    (70, 64, 1), (200, 300, 31), (128, 16, 129), (256, 80, 255), (100, 520, 257), (300, 40, 1), (1000, 272, 129),
    (257, 1, 385), (1, 20000, 65), (65, 20000, 33), (16, 1, 1), (33, 257, 128 * 152 + 1), (520, 255, 256 * 76 + 32)])
def test_products_of_few_rows_and_of_many_tiles(fmt, N, D, V):
    h, w = _pair(N, D, V, fmt, N + D)
    for dtype in (torch.float32, torch.bfloat16):
        _check(flce.linear_fp4(h, w, dtype=dtype), h, w)


def test_products_into_columns_of_a_wider_matrix():
    h, w = _pair(300, 128, 256, "nvfp4", 5)
    wide = torch.full((300, 1024), 3.0, dtype=torch.bfloat16, device=DEV)
    flce.linear_fp4(h, w, out=wide[:, 512:768])   # rows in whole 16 bytes, 2048 apart
    assert torch.equal(wide[:, 512:768], flce.linear_fp4(h, w))
    assert bool((wide[:, :512] == 3).all()) and bool((wide[:, 768:] == 3).all())
    some = torch.full((4, 300, 256), 3.0, device=DEV)
    flce.linear_fp4(h, w, out=some[2])
    assert bool((some[1] == 3).all()) and bool((some[3] == 3).all())


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("N,V", [(33, 40), (64, 96), (65, 40), (129, 264), (257, 1000), (300, 520)])
def test_products_whose_last_rows_are_not_whole(fmt, N, V):
    h, w = _pair(N, 144, V, fmt, N + V)
    dense = flce.linear_fp4(h, w, dtype=torch.bfloat16)
    _check(dense, h, w)
    wide = torch.full((N + 2, V + 40), 3.0, dtype=torch.bfloat16, device=DEV)
    for first in (0, 8, 1, 39):   # rows of whole 16 bytes, and not
        for to in (wide[1:-1, first:first + V], wide.view(-1)[:(N + 2) * (V + 39)].view(N + 2, V + 39)[1:-1, :V]):
            wide.fill_(3.0)
            flce.linear_fp4(h, w, out=to)
            assert torch.equal(to, dense)
            to.fill_(3.0)
            assert bool((wide == 3).all())


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("N,D,V", [(700, 144, 19456), (1150, 64, 19432), (634, 300, 19456), (534, 1111, 19424)])
def test_products_of_many_tokens_and_rows(fmt, N, D, V):
    h, w = _pair(N, D, V, fmt, N + D)
    y = flce.linear_fp4(h, w, dtype=torch.bfloat16)
    _check(y, h, w)
    wide = torch.full((N + 1, V + 8), 3.0, dtype=torch.bfloat16, device=DEV)
    flce.linear_fp4(h, w, out=wide[:N, :V])
    assert torch.equal(wide[:N, :V], y) and bool((wide[N] == 3).all()) and bool((wide[:, V:] == 3).all())


def test_two_calls_at_once():
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(700, 2048, generator=g, device=DEV).bfloat16()
    W = torch.randn(9000, 2048, generator=g, device=DEV).bfloat16()
    t = torch.randint(0, 9000, (700,), generator=g, device=DEV).int()
    w = torch.randn(2048, generator=g, device=DEV)
    W4 = flce.quantize_fp4(W)

    def work():
        r, p = flce.layer_norm_packed(x, w)
        return (flce.linear_fp4(flce.quantize_fp4(r.y), W4), flce.embedding_backward(x, t, 9000), p.data,
                *flce.layer_norm_packed_backward(x, p, w, r), flce.linear_fp4(flce.quantize_fp4(x[:3]), W4))

    want = work()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(3):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(work())
    torch.cuda.synchronize()
    for results in got:
        for r in results:
            assert all(torch.equal(a, b) for a, b in zip(r, want))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [1024, 1001])
def test_a_row_alone_and_among_others(dtype, D):
    """A row's codes, values and packed record are its own; the layer norm's statistics too, by one kernel."""
    g = torch.Generator(device=DEV).manual_seed(D)
    x = torch.randn(3000, D, generator=g, device=DEV).to(dtype)
    p = flce.pack_e4m3(x)
    for fmt in flce.FP4_FORMATS:
        m = flce.quantize_fp4(x, format=fmt)
        one = flce.quantize_fp4(x[1234:1235], format=fmt)
        assert torch.equal(one.codes[0], m.codes[1234]) and torch.equal(one.block_scales()[0], m.block_scales()[1234])
        assert torch.equal(flce.dequantize_fp4(one)[0], flce.dequantize_fp4(m)[1234])
    assert torch.equal(flce.pack_e4m3(x[77:78]).data[0], p.data[77])
    r, q = flce.layer_norm_packed(x)
    assert torch.equal(q.data, p.data)
    few, qf = flce.layer_norm_packed(x[5:9])
    assert torch.equal(qf.data, p.data[5:9])
    # by another kernel: other orders of the sums, whose rounding is below 2^-18 of these values
    assert float((few.mean - r.mean[5:9]).abs().max()) <= 2.0 ** -18
    assert float((few.rstd / r.rstd[5:9] - 1).abs().max()) <= 2.0 ** -18


@pytest.mark.parametrize("N", [1, 2, 1023, 1024, 1025, 2049, 4097, 8192, 16383, 16384, 16385, 20481])
@pytest.mark.parametrize("V", [1, 2, 511, 512, 513, 262143, 262144, 300000])
def test_the_sorts_sizes(N, V):
    """Sums of whole numbers are exact: any token lost, counted twice or put in the wrong row shows."""
    g = torch.Generator(device=DEV).manual_seed(N + V)
    t = torch.randint(0, V, (N,), generator=g, device=DEV).int()
    t[torch.rand(N, generator=g, device=DEV) < 0.05] = -100
    dy = torch.randint(-8, 9, (N, 4), generator=g, device=DEV).float()
    live = t >= 0
    want = torch.zeros(V, 4, device=DEV).index_add_(0, t[live].long(), dy[live])
    assert torch.equal(flce.embedding_backward(dy, t, V), want)
    got = flce.embedding_backward(dy, t, V, out=want.clone(), accumulate=True)
    assert torch.equal(got, 2 * want)


def test_padding_that_is_an_id_of_the_table():
    W = torch.randn(10, 8, device=DEV)
    t = torch.tensor([3, 0, 5, 0, 3], dtype=torch.int32, device=DEV)
    y = flce.embedding(W, t, ignore_index=0)
    assert bool((y[1] == 0).all()) and torch.equal(y[0], W[3])
    dW = flce.embedding_backward(torch.ones(5, 8, device=DEV), t, 10, ignore_index=0)
    assert bool((dW[0] == 0).all()) and bool((dW[3] == 2).all()) and bool((dW[5] == 1).all())


def test_gradients_that_are_not_finite_stay_in_their_rows():
    dy = torch.ones(6, 40, device=DEV)
    dy[1, 3], dy[4, 7] = float("inf"), float("nan")
    t = torch.tensor([0, 1, 2, 3, 4, 1], dtype=torch.int32, device=DEV)
    dW = flce.embedding_backward(dy, t, 7)
    assert bool(torch.isinf(dW[1, 3])) and bool(torch.isnan(dW[4, 7]))
    dW[1, 3], dW[4, 7] = 2, 1
    assert torch.equal(dW.sum(1), torch.tensor([40., 80, 40, 40, 40, 0, 0], device=DEV))
