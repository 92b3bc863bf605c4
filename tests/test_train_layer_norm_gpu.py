"""Layer norm forward and backward on the GPU against the formulas in 64 bits.

Tolerances, with u = 2^-24 (one float32 rounding, relative) and half = 2^-8
(one rounding to bfloat16, which has 8 significant bits):
  - a sum over a row is a tree: at most 16 sequential terms per thread, 6
    lane levels, 16 waves; with the product and the factor 1/cols fewer than
    48 roundings touch a term, so its error is below 48 u sum|terms|; rows
    past 16384 columns add up to cols / 1024 sequential terms;
  - a column sum of the backward has at most `rows` sequential terms in a
    part (4 waves' sums and 512 / 16 + 16 parts join after it);
  - an output adds a few roundings of its own terms.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def tb():
    from tropical_semiring_tensor_amd import binding
    binding.tropical_train_init(0)
    yield binding
    # give the memory back: torch keeps its matrix products' workspace inside
    # whatever cached block it came from
    torch.cuda.synchronize()
    torch._C._cuda_clearCublasWorkspaces()
    torch.cuda.empty_cache()


def half(dtype):
    return 2.0 ** -8 if dtype == BF16 else 2 * U


def matrix(rows, cols, pad, dtype, gen, offset=0.0):
    """rows x cols view of a wider buffer whose other elements are NaN."""
    buf = torch.full((rows, cols + pad), float("nan"))
    buf[:, :cols] = torch.randn(rows, cols, generator=gen) + offset
    return buf.to(dtype).to(DEV)[:, :cols]


def forward_reference(x, gamma, beta, eps):
    x = x.double()
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = 1 / ((xc * xc).mean(1) + eps).sqrt()
    xh = xc * rstd[:, None]
    g = gamma.double() if gamma is not None else torch.ones_like(x[0])
    b = beta.double() if beta is not None else torch.zeros_like(x[0])
    return xh * g + b, mean, rstd, xh, g, b


def assert_within(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, worst {float((err - tol).max()):.3g} over"


def check_forward(tb, x, gamma, beta, eps=1e-5):
    y, mean, rstd = tb.tropical_layer_norm_forward(x, gamma, beta, eps=eps)
    ry, rm, rr, xh, g, b = forward_reference(x, gamma, beta, eps)
    n = 48 + x.shape[1] / 1024
    mabs = x.double().abs().mean(1)
    # the mean's error enters the variance as its square: below the other terms
    rel = n * U + 2 * (n * U * mabs * rr) ** 2
    assert_within(mean, rm, n * U * mabs, "mean")
    assert_within(rstd, rr, rel * rr, "rstd")
    tol = ((n * U * mabs * rr)[:, None] + (rel + 4 * U)[:, None] * xh.abs()) * g.abs()
    assert_within(y, ry, tol + half(x.dtype) * (ry.abs() + (xh * g).abs() * 2 * U + tol), "y")
    return mean, rstd


def check_backward(tb, dy, x, mean, rstd, gamma, **kw):
    dx, dgamma, dbeta = tb.tropical_layer_norm_backward(dy, x, mean, rstd, gamma, **kw)
    rows, cols = x.shape
    d, r = dy.double(), rstd.double()[:, None]
    h = (x.double() - mean.double()[:, None]) * r
    w = d * (gamma.double() if gamma is not None else 1.0)
    c1, c2 = w.mean(1, keepdim=True), (w * h).mean(1, keepdim=True)
    n = 48 + cols / 1024
    if dx is not None:
        want = r * (w - c1 - h * c2)
        tol = r * (n * U * (w.abs().mean(1, keepdim=True) + h.abs() * (w * h).abs().mean(1, keepdim=True))
                   + 8 * U * (w.abs() + c1.abs() + (h * c2).abs()))
        assert_within(dx, want, tol + half(x.dtype) * (want.abs() + tol), "dx")
    n = rows + 64
    ptype = gamma.dtype if gamma is not None else F32
    if dgamma is not None:
        want, tol = (d * h).sum(0), n * U * (d * h).abs().sum(0)
        assert_within(dgamma, want, tol + half(ptype) * (want.abs() + tol), "dgamma")
    if dbeta is not None:
        want, tol = d.sum(0), n * U * d.abs().sum(0)
        assert_within(dbeta, want, tol + half(ptype) * (want.abs() + tol), "dbeta")
    return dx, dgamma, dbeta


SHAPES = [(1, 1), (1, 64), (3, 7), (5, 8), (4, 1000), (7, 1023), (9, 1024), (2, 1025), (6, 2047), (3, 4096),
          (3, 4097), (2, 8191), (2, 16384), (2, 16385), (1, 40001), (2049, 24), (700, 520)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype,ptype", [(F32, F32), (BF16, BF16), (BF16, F32)])
def test_forward_and_backward(tb, rows, cols, dtype, ptype):
    gen = torch.Generator().manual_seed(rows * 100003 + cols)
    pad = (rows + cols) % 4  # row strides of every alignment
    x = matrix(rows, cols, pad, dtype, gen, offset=1.5)
    dy = matrix(rows, cols, (pad + 1) % 3, dtype, gen)
    gamma = (1 + 0.2 * torch.randn(cols, generator=gen)).to(ptype).to(DEV)
    beta = torch.randn(cols, generator=gen).to(ptype).to(DEV)
    mean, rstd = check_forward(tb, x, gamma, beta)
    if rows <= 600:
        check_backward(tb, dy, x, mean, rstd, gamma)
    else:  # two calls give the same bits
        a = check_backward(tb, dy, x, mean, rstd, gamma)
        b = tb.tropical_layer_norm_backward(dy, x, mean, rstd, gamma)
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_without_weights_and_partial_gradients(tb):
    gen = torch.Generator().manual_seed(5)
    x, dy = matrix(33, 130, 1, F32, gen), matrix(33, 130, 0, F32, gen)
    gamma = torch.randn(130, generator=gen).to(DEV)
    mean, rstd = check_forward(tb, x, None, None)
    check_forward(tb, x, gamma, None)
    check_forward(tb, x, None, gamma)
    check_backward(tb, dy, x, mean, rstd, None)
    check_backward(tb, dy, x, mean, rstd, gamma, dx=None)
    check_backward(tb, dy, x, mean, rstd, gamma, dgamma=None)
    check_backward(tb, dy, x, mean, rstd, gamma, dbeta=None)
    check_backward(tb, dy, x, mean, rstd, gamma, dgamma=None, dbeta=None)


@pytest.mark.parametrize("cols", [50, 3000, 9000, 20000])
def test_in_place(tb, cols):
    gen = torch.Generator().manual_seed(cols)
    x, dy = matrix(6, cols, 2, F32, gen), matrix(6, cols, 2, F32, gen)
    gamma = torch.randn(cols, generator=gen).to(DEV)
    y, mean, rstd = tb.tropical_layer_norm_forward(x, gamma)
    want = tb.tropical_layer_norm_backward(dy, x, mean, rstd, gamma)
    got = tb.tropical_layer_norm_backward(dy, x, mean, rstd, gamma, dx=dy)
    assert got[0] is dy and all(torch.equal(a, b) for a, b in zip(got, want))
    tb.tropical_layer_norm_forward(x, gamma, y=x)
    assert torch.equal(x, y)


def test_rows_keep_to_themselves(tb):
    """A NaN or an infinity in one row reaches that row only (and the column
    sums, which hold every row)."""
    gen = torch.Generator().manual_seed(9)
    for cols in (100, 2000, 5000, 17000):
        x, dy = matrix(6, cols, 0, F32, gen), matrix(6, cols, 0, F32, gen)
        clean = tb.tropical_layer_norm_forward(x)
        cdx = tb.tropical_layer_norm_backward(dy, x, clean[1], clean[2])[0]
        x2 = x.clone()
        x2[2, 5] = float("nan")
        x2[4, cols - 1] = float("inf")
        out = tb.tropical_layer_norm_forward(x2)
        dx = tb.tropical_layer_norm_backward(dy, x2, out[1], out[2])[0]
        keep = [0, 1, 3, 5]
        for a, b in zip((*clean, cdx), (*out, dx)):
            assert torch.equal(a[keep], b[keep])
            assert not torch.isfinite(b[[2, 4]]).all(dim=-1).any()


def test_constant_rows_and_large_offsets(tb):
    # a constant row has no spread: rstd = 1 / sqrt(eps), y = beta
    x = torch.full((3, 700), 3.0, device=DEV)
    y, mean, rstd = tb.tropical_layer_norm_forward(x, None, None, eps=1e-4)
    assert torch.equal(mean, torch.full_like(mean, 3.0)) and torch.equal(y, torch.zeros_like(y))
    assert torch.allclose(rstd, torch.full_like(rstd, 100.0), rtol=4 * U, atol=0)
    # an offset a thousand times the spread: the variance about the mean keeps its digits
    gen = torch.Generator().manual_seed(3)
    check_forward(tb, matrix(4, 3000, 0, F32, gen, offset=1000.0), None, None)


def test_gradient_against_differences(tb):
    """The gradients along random directions against central differences of
    the forward's formula in 64 bits (step 1e-4: error near 1e-8 of the scale)."""
    gen = torch.Generator().manual_seed(17)
    x, dy = matrix(5, 300, 0, F32, gen), matrix(5, 300, 0, F32, gen)
    gamma, beta = torch.randn(300, generator=gen).to(DEV), torch.randn(300, generator=gen).to(DEV)
    _, mean, rstd = tb.tropical_layer_norm_forward(x, gamma, beta)
    grads = tb.tropical_layer_norm_backward(dy, x, mean, rstd, gamma)
    base = [x.double(), gamma.double(), beta.double()]

    def loss(args):
        return (forward_reference(*args, 1e-5)[0] * dy.double()).sum()

    for i, g in enumerate(grads):
        for _ in range(3):
            d = torch.randn(base[i].shape, generator=gen).double().to(DEV)
            plus, minus = list(base), list(base)
            plus[i], minus[i] = base[i] + 1e-4 * d, base[i] - 1e-4 * d
            want = (loss(plus) - loss(minus)) / 2e-4
            got = (g.double() * d).sum()
            scale = (g.double() * d).abs().sum()
            assert abs(got - want) <= 1e-6 * scale + 1e-6 * dy.numel() ** 0.5, (i, float(got), float(want))


def test_other_stream_and_no_rows(tb):
    gen = torch.Generator().manual_seed(2)
    x, dy = matrix(40, 600, 0, BF16, gen), matrix(40, 600, 0, BF16, gen)
    want = tb.tropical_layer_norm_forward(x)
    wantb = tb.tropical_layer_norm_backward(dy, x, want[1], want[2])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = tb.tropical_layer_norm_forward(x, stream=s)
    gotb = tb.tropical_layer_norm_backward(dy, x, got[1], got[2], stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*want, *wantb), (*got, *gotb)))
    # no rows: the column sums are zero
    e = torch.empty(0, 600, device=DEV)
    st = torch.empty(0, device=DEV)
    dx, dg, db = tb.tropical_layer_norm_backward(e, e, st, st)
    assert dx.shape == (0, 600) and not dg.any() and not db.any()
    assert tb.tropical_layer_norm_forward(e)[0].shape == (0, 600)


def test_offsets_past_32_bits(tb):
    """Rows more than 2^32 bytes apart."""
    ld = 1_300_000_001
    buf = torch.empty(2 * ld + 70, dtype=BF16, device=DEV)
    x = torch.as_strided(buf, (3, 70), (ld, 1))
    gen = torch.Generator().manual_seed(1)
    x.copy_(torch.randn(3, 70, generator=gen))
    mean, rstd = check_forward(tb, x, None, None)
    dy = torch.randn(3, 70, generator=gen).to(BF16).to(DEV)
    want = tb.tropical_layer_norm_backward(dy, x.contiguous(), mean, rstd)
    got = tb.tropical_layer_norm_backward(dy, x, mean, rstd)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_graph_replays(tb):
    gen = torch.Generator().manual_seed(4)
    x, dy = matrix(300, 900, 0, F32, gen), matrix(300, 900, 0, F32, gen)
    gamma = torch.randn(900, generator=gen).to(DEV)
    y, mean, rstd = tb.tropical_layer_norm_forward(x, gamma)
    outs = [torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(gamma)]
    ws = torch.empty(tb.tropical_layer_norm_backward_workspace_size(300, 900), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tb.tropical_layer_norm_forward(x, gamma, y=y, mean=mean, rstd=rstd)
        tb.tropical_layer_norm_backward(dy, x, mean, rstd, gamma, *outs, workspace=ws)
    for i in range(3):
        x.copy_(matrix(300, 900, 0, F32, gen))
        g.replay()
        torch.cuda.synchronize()
        ref = tb.tropical_layer_norm_forward(x, gamma)
        refb = tb.tropical_layer_norm_backward(dy, x, ref[1], ref[2], gamma)
        assert all(torch.equal(a, b) for a, b in zip((*ref, *refb), (y, mean, rstd, *outs))), i


def test_refusals(tb):
    x = torch.randn(4, 8, device=DEV)
    v = torch.randn(4, device=DEV)
    with pytest.raises(tb.TropicalError) as e:
        tb.tropical_layer_norm_forward(torch.randn(4, 8), y=x)
    assert e.value.status == tb.NOT_DEVICE_MEMORY
    with pytest.raises(tb.TropicalError) as e:
        tb.tropical_layer_norm_backward(x, x, v, v, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
    assert e.value.status == tb.WORKSPACE_TOO_SMALL
    with pytest.raises(tb.TropicalError) as e:
        tb.tropical_layer_norm_forward(x, eps=-1.0)
    assert e.value.status == tb.INVALID_ARGUMENT
    with pytest.raises(TypeError):
        tb.tropical_layer_norm_forward(x.half())
    with pytest.raises(ValueError):
        tb.tropical_layer_norm_forward(x.t())
    with pytest.raises(ValueError):
        tb.tropical_layer_norm_forward(x, torch.ones(7, device=DEV))
    with pytest.raises(ValueError):
        tb.tropical_layer_norm_backward(x, x, v[:3], v)
    with pytest.raises(tb.TropicalError) as e:  # float32 rows take float32 weights
        tb.tropical_layer_norm_forward(x, torch.ones(8, device=DEV, dtype=BF16))
    assert e.value.status == tb.INVALID_ARGUMENT
    torch.cuda.empty_cache()
    raw = torch.empty(16 << 20, device=DEV)
    st = tb.lib().tropical_layer_norm_forward(0, 0, raw.data_ptr(), 1 << 20, None, None, 1e-5, x.data_ptr(), 1 << 20,
                                              None, None, 4096, 8, None)
    assert st == tb.INVALID_ARGUMENT and "allocation" in tb.tropical_last_error()


def test_more_rows_than_a_launch_holds(tb):
    """2^32 threads are four waves to 2^26 rows, 256 threads to 2^24, 1024 to 2^22."""
    gen = torch.Generator(device=DEV).manual_seed(6)
    x = torch.randn((1 << 26) + 5, 2, generator=gen, device=DEV).to(BF16)
    check_forward(tb, x, None, None)
    del x
    for rows, cols in (((1 << 24) + 3, 1025), ((1 << 22) + 3, 4097)):
        torch.cuda.empty_cache()
        x = torch.empty(rows, cols, dtype=BF16, device=DEV)  # (what the other rows hold is their own)
        at = torch.tensor([0, 1, 4097, rows // 2, rows - 5, rows - 4, rows - 3, rows - 2, rows - 1], device=DEV)
        some = torch.randn(len(at), cols, generator=gen, device=DEV).to(BF16)
        x[at] = some
        want = tb.tropical_layer_norm_forward(some)
        got = tb.tropical_layer_norm_forward(x, y=x)
        assert all(torch.equal(a, b[at]) for a, b in zip(want, got))
        del x, got
    torch.cuda.empty_cache()


def test_more_columns_than_a_launch_holds(tb):
    """The column sums of 512 parts of 2^23 columns, and their sum over 2^27."""
    gen = torch.Generator(device=DEV).manual_seed(7)
    rows, cols = 515, (1 << 23) + 300
    x = torch.zeros(rows, cols, dtype=BF16, device=DEV)
    at = torch.tensor([0, 255, 4096, cols // 2, cols - 301, cols - 300, cols - 1], device=DEV)
    x[:, at] = torch.randn(rows, len(at), generator=gen, device=DEV).to(BF16)
    mean, rstd = torch.zeros(rows, device=DEV), torch.ones(rows, device=DEV)
    check = x[:, at].contiguous()
    _, dg, db = tb.tropical_layer_norm_backward(x, x, mean, rstd, dx=None)
    for got, terms in ((dg, check.double() ** 2), (db, check.double())):
        assert_within(got[at], terms.sum(0), (rows + 64) * U * terms.abs().sum(0), "column sums")
        got[at] = 0.0
        assert not got.any()
    del x
    torch.cuda.empty_cache()
    cols = (1 << 27) + 70
    x = torch.randn(1, cols, generator=gen, device=DEV).to(BF16)
    _, dg, db = tb.tropical_layer_norm_backward(x, x, mean[:1], rstd[:1], dx=None)
    assert torch.equal(db, x[0].float()) and torch.equal(dg, x[0].float() ** 2)
    del x, dg, db
    torch.cuda.empty_cache()
