"""Linear cross entropy on the GPU against its definition in 64 bits.

Tolerances, with u = 2^-24 and S_nv = sum_d |x_nd| |w_vd|:
  logits   width + 40 float32 roundings of a term at most (sums in any order,
           the float16 split of float32 operands: 12 u of each product):
           dl_nv = (width + 40) u S_nv
  lse      the largest dl of the row, and 200 u for the exponentials and the
           joined sums (a term e^-t of the sum carries a relative error t u)
  G        |g| p (dl + dlse + 60 u), then its rounding to 16 bits: 2^-8 of G
           for bfloat16 (8 significant bits), 2^-22 of G and 2^-38 of max |g|
           for float32 (two times 11 bits); an exponential below the smallest
           normal number, 2^-126, may be taken for zero
  grads    G's error times the other factor, (terms + 40) u of the terms'
           magnitudes for the sum, one rounding of the output (2^-8 of a
           bfloat16 value)
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


def case(tokens, width, vocab, dtype, seed=0, ignored=0.3, pad=(0, 0), scale=2.0, tdtype=torch.int64):
    """x, w (views of wider NaN-filled buffers), target, weights."""
    g = torch.Generator(device=DEV).manual_seed(seed * 7919 + tokens * 31 + width * 17 + vocab)

    def matrix(r, c, p, s):
        buf = torch.full((r, c + p), float("nan"), device=DEV, dtype=dtype)
        buf[:, :c] = (torch.randn(r, c, generator=g, device=DEV) * s).to(dtype)
        return buf[:, :c]

    x = matrix(tokens, width, pad[0], 1.0)
    w = matrix(vocab, width, pad[1], scale / width ** 0.5)
    t = torch.randint(0, vocab, (tokens,), generator=g, device=DEV).to(tdtype)
    t[torch.rand(tokens, generator=g, device=DEV) < ignored] = -100
    gl = torch.rand(tokens, generator=g, device=DEV) + 0.1
    return x, w, t, gl


def reference(x, w, t, gl=None, ignore_index=-100):
    """(loss, lse, grad_x, grad_w) in 64 bits and their tolerances."""
    n, d = x.shape
    v = w.shape[0]
    X, W, t = x.double(), w.double(), t.long()
    keep = (t != ignore_index) & (t >= 0) & (t < v)
    X = torch.where(keep[:, None], X, 0.0)
    l = X @ W.t()
    dl = (d + 40) * U * (X.abs() @ W.abs().t())
    lse = torch.logsumexp(l, 1)
    idx = torch.where(keep, t, 0)[:, None]
    tl = l.gather(1, idx)[:, 0]
    dlse = dl.amax(1) + 200 * U + 4 * U * lse.abs()
    out = [torch.where(keep, lse - tl, 0.0), torch.where(keep, lse, 0.0)]
    tol = [dlse + dl.gather(1, idx)[:, 0] + 4 * U * tl.abs(), dlse]
    if gl is None:
        return out, tol
    g = torch.where(keep, gl.double(), 0.0)[:, None]
    p = (l - lse[:, None]).exp()
    G = p.scatter_add(1, idx, torch.full_like(lse[:, None], -1.0)) * g
    half = 2.0 ** -8 if x.dtype == BF16 else 2.0 ** -22
    dG = g.abs() * p * (dl + dlse[:, None] + 60 * U) + half * G.abs() * 1.01 + 4 * U * G.abs() + 2.0 ** -126
    if x.dtype == F32:
        dG = dG + 2.0 ** -38 * g.abs().max()
    r = 2.0 ** -8 if x.dtype == BF16 else 4 * U
    gx, gw = G @ W, G.t() @ X
    tx = dG @ W.abs() + (v + 40) * U * (G.abs() @ W.abs())
    tw = dG.t() @ X.abs() + (n + 40) * U * (G.t().abs() @ X.abs())
    if x.dtype == F32:  # the planes' floor: 2^-38 of a matrix's largest element
        tx = tx + 2.0 ** -38 * G.abs().sum(1, keepdim=True) * W.abs().max()
        tw = tw + 2.0 ** -38 * G.abs().sum(0)[:, None] * X.abs().max()
    out += [gx, gw]
    tol += [tx + r * (gx.abs() + tx), tw + r * (gw.abs() + tw)]
    return out, tol


def assert_within(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    if bad.any():
        i = bad.nonzero()[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got {float(got[tuple(i)])}, "
                             f"want {float(want[tuple(i)])} within {float(tol[tuple(i)]):.3g}")


def check(tb, x, w, t, gl=None, ignore_index=-100, **kw):
    want, tol = reference(x, w, t, gl, ignore_index)
    loss, lse = tb.tropical_linear_cross_entropy_forward(x, w, t, ignore_index=ignore_index)
    got = [loss, lse]
    if gl is not None:
        got += tb.tropical_linear_cross_entropy_backward(x, w, t, lse, gl, ignore_index=ignore_index, **kw)
    for g, r, e, what in zip(got, want, tol, ("loss", "lse", "grad_x", "grad_w")):
        if g is not None:
            assert_within(g, r, e, what)
    return got


@pytest.mark.parametrize("tokens,width,vocab", [
    (1, 1, 1), (1, 8, 2), (3, 5, 7), (16, 40, 63), (17, 64, 129), (33, 100, 1000), (64, 72, 2050), (65, 64, 128),
    (65, 520, 255), (130, 33, 300), (128, 128, 128), (300, 200, 257), (257, 136, 4099), (1, 700, 70000)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad", [(0, 0), (8, 16), (1, 3)])
def test_small(tb, tokens, width, vocab, dtype, pad):
    x, w, t, gl = case(tokens, width, vocab, dtype, pad=pad, ignored=0.3 if tokens > 1 else 0.0)
    check(tb, x, w, t, gl)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens,width,vocab", [
    (300, 64, 24581),     # logits in 256 x 256 tiles
    (300, 72, 24581),     # the same, the width ending in the first half of 64 columns
    (300, 8, 24581),
    (700, 1096, 8300),    # grad_x in 256 x 256 tiles, split along the labels
    (200, 1000, 12345),   # grad_w in 256 x 256 tiles
    (60, 256, 66000),     # few tokens, two blocks of labels a wave
    (30, 1300, 33001),    # few tokens, four blocks of labels; odd column blocks
    (9, 2604, 1501),      # few tokens, several units of columns to a wave
    (16, 1030, 32777),
    (60, 130, 40001),
    (50, 1024, 12000),
    (50, 130, 5000),      # grad_w's columns in parts
    (66, 420, 30001),     # a large label matrix and few tiles of tokens
    (256, 2604, 4100),
    (130, 100, 120001),
    (70, 1000, 11011),
    (700, 264, 700),      # grad_w split along the tokens beside grad_x
    (40, 256, 9000)])
def test_tiles(tb, tokens, width, vocab, dtype):
    check(tb, *case(tokens, width, vocab, dtype, seed=1))


@pytest.mark.parametrize("tokens", [40, 70, 300])
@pytest.mark.parametrize("dtype,pad", [(F32, (3, 4)), (F32, (0, 1)), (BF16, (8, 8))])
def test_large_matrix_in_a_wider_buffer(tb, tokens, dtype, pad):
    check(tb, *case(tokens, 1000, 17001, dtype, seed=9, pad=pad))


@pytest.mark.parametrize("dtype,pad", [(F32, (0, 0)), (BF16, (0, 0)), (BF16, (1, 1))])
def test_pieces(tb, dtype, pad):
    """A label set of several pieces (of 256 MiB of its logits' gradient)."""
    check(tb, *case(4100, 72, 70001, dtype, seed=2, pad=pad))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens", [20, 200])
def test_masked_tokens_reach_nothing(tb, tokens, dtype):
    """NaN and infinities in the rows of tokens that do not count."""
    x, w, t, gl = case(tokens, 96, 500, dtype, seed=3)
    a = check(tb, x, w, t, gl)
    off = (t < 0).nonzero()[:, 0]
    assert len(off) >= 3
    x = x.clone()
    x[off[0]] = float("nan")
    x[off[1]] = float("inf")
    x[off[2]] = 1e30
    gl = gl.clone()
    gl[off] = float("nan")
    b = check(tb, x, w, t, gl)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert not b[2][off].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens", [5, 70, 300])
def test_all_masked(tb, tokens, dtype):
    x, w, t, gl = case(tokens, 64, 300, dtype)
    t.fill_(-100)
    for g in check(tb, x, w, t, gl):
        assert not g.any()


def test_targets(tb):
    """Targets outside the vocabulary, 32-bit targets, an ignore_index within it."""
    for tokens in (30, 100):
        x, w, t, gl = case(tokens, 48, 77, F32, ignored=0.0, tdtype=torch.int32)
        a = check(tb, x, w, t, gl, ignore_index=5)
        t[0], t[1], t[2] = 77, -1, 5
        b = check(tb, x, w, t, gl, ignore_index=5)
        assert not b[0][:3].any() and not b[2][:3].any() and torch.equal(a[0][3:], b[0][3:])
        t = t.long()
        t[1] = 2 ** 40
        c = check(tb, x, w, t, gl, ignore_index=5)
        assert all(torch.equal(p, q) for p, q in zip(b, c))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_logits(tb, dtype):
    """Logits in the hundreds: the maximum is taken out of the sums."""
    x, w, t, gl = case(90, 64, 700, dtype, seed=4, scale=120.0)
    check(tb, x, w, t, gl)
    check(tb, x[:9], w, t[:9], gl[:9])


def test_float32_scales(tb):
    """Operands far from 1: the planes are scaled to them."""
    for sx, sw in ((1e-20, 1e20), (1e12, 1e-12), (1e-3, 1e3)):
        x, w, t, gl = case(100, 64, 700, F32, seed=5)
        check(tb, x * sx, w * sw, t, gl)


def test_weights_of_tokens(tb):
    """Zero, equal, broadcast, strided and tiny weights."""
    x, w, t, gl = case(150, 64, 900, BF16, seed=6)
    check(tb, x, w, t, torch.zeros_like(gl))
    check(tb, x, w, t, gl * 1e-20)
    loss, lse = tb.tropical_linear_cross_entropy_forward(x, w, t)
    one = torch.full((), 0.125, device=DEV)
    a = tb.tropical_linear_cross_entropy_backward(x, w, t, lse, one)
    for g in (one.expand(150), torch.full((150, 3), 0.125, device=DEV)[:, 1]):
        b = tb.tropical_linear_cross_entropy_backward(x, w, t, lse, g)
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    check(tb, x, w, t, one.expand(150))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_single_gradients_and_strided_outputs(tb, dtype):
    x, w, t, gl = case(140, 90, 333, dtype, seed=7)
    loss, lse = tb.tropical_linear_cross_entropy_forward(x, w, t)
    gx, gw = tb.tropical_linear_cross_entropy_backward(x, w, t, lse, gl)
    a, none = tb.tropical_linear_cross_entropy_backward(x, w, t, lse, gl, grad_w=None)
    assert none is None and torch.equal(a, gx)
    none, b = tb.tropical_linear_cross_entropy_backward(x, w, t, lse, gl, grad_x=None)
    assert none is None and torch.equal(b, gw)
    bx, bw = torch.full((140, 101), 7.0, device=DEV, dtype=dtype), torch.full((333, 95), 7.0, device=DEV, dtype=dtype)
    tb.tropical_linear_cross_entropy_backward(x, w, t, lse, gl, grad_x=bx[:, 3:93], grad_w=bw[:, :90])
    assert torch.equal(bx[:, 3:93], gx) and torch.equal(bw[:, :90], gw)
    assert (bx[:, :3] == 7).all() and (bx[:, 93:] == 7).all() and (bw[:, 90:] == 7).all()


def test_gradients_against_differences(tb):
    """Against central differences of the loss in 64 bits (step 1e-5)."""
    for tokens in (10, 90):
        x, w, t, gl = case(tokens, 32, 150, F32, seed=8)
        _, lse = tb.tropical_linear_cross_entropy_forward(x, w, t)
        grads = tb.tropical_linear_cross_entropy_backward(x, w, t, lse, gl)

        def total(a, b):
            l = a @ b.t()
            keep = t >= 0
            per = torch.logsumexp(l, 1) - l.gather(1, t.clamp(min=0)[:, None])[:, 0]
            return (torch.where(keep, per, 0.0) * gl.double()).sum()

        g = torch.Generator(device=DEV).manual_seed(1)
        X, W = x.double(), w.double()
        for i, grad in enumerate(grads):
            for _ in range(3):
                d = torch.randn(grad.shape, generator=g, device=DEV).double()
                plus, minus = [X, W], [X, W]
                plus[i], minus[i] = plus[i] + 1e-5 * d, minus[i] - 1e-5 * d
                want = (total(*plus) - total(*minus)) / 2e-5
                got = (grad.double() * d).sum()
                assert abs(got - want) <= 2e-6 * (grad.double() * d).abs().sum() + 1e-7


def test_repeatable_other_stream_and_graph(tb):
    x, w, t, gl = case(333, 264, 3000, BF16, seed=9)
    want = check(tb, x, w, t, gl)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    loss, lse = tb.tropical_linear_cross_entropy_forward(x, w, t, stream=s)
    got = [loss, lse, *tb.tropical_linear_cross_entropy_backward(x, w, t, lse, gl, stream=s)]
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    n = max(tb.tropical_linear_cross_entropy_workspace_size(BF16, 333, 264, 3000, b) for b in (False, True))
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    out = [torch.empty_like(g) for g in want]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tb.tropical_linear_cross_entropy_forward(x, w, t, loss=out[0], lse=out[1], workspace=ws)
        tb.tropical_linear_cross_entropy_backward(x, w, t, out[1], gl, grad_x=out[2], grad_w=out[3], workspace=ws)
    for i in range(3):
        x.copy_(case(333, 264, 3000, BF16, seed=20 + i)[0])
        t.copy_(case(333, 264, 3000, BF16, seed=20 + i)[2])  # other tokens kept: the graph holds no count
        graph.replay()
        torch.cuda.synchronize()
        want = check(tb, x, w, t, gl)
        assert all(torch.equal(a, b) for a, b in zip(want, out)), i


def test_one_token_equals_many(tb):
    """A token's loss does not depend on the others beyond rounding."""
    x, w, t, gl = case(80, 128, 1500, F32, seed=10, ignored=0.0)
    many, _ = tb.tropical_linear_cross_entropy_forward(x, w, t)
    for i in (0, 41, 79):
        one, _ = tb.tropical_linear_cross_entropy_forward(x[i:i + 1], w, t[i:i + 1])
        assert abs(float(one) - float(many[i])) <= 400 * U * 16


def test_offsets_past_32_bits(tb):
    """Rows of w and grad_w spread over more than 2^32 bytes."""
    ld, vocab, width = 1 << 21, 1200, 64
    buf = torch.empty((vocab - 1) * ld + width, dtype=BF16, device=DEV)
    w = torch.as_strided(buf, (vocab, width), (ld, 1))
    for tokens in (10, 100):
        x, dense, t, gl = case(tokens, width, vocab, BF16, seed=11)
        w.copy_(dense)
        want = check(tb, x, dense, t, gl)
        loss, lse = tb.tropical_linear_cross_entropy_forward(x, w, t)
        gx, _ = tb.tropical_linear_cross_entropy_backward(x, w, t, lse, gl, grad_w=None)
        _, gw = tb.tropical_linear_cross_entropy_backward(x, dense, t, lse, gl, grad_x=None, grad_w=w)
        assert all(torch.equal(a, b) for a, b in zip(want, (loss, lse, gx, gw)))


def test_no_tokens(tb):
    x, w, t, gl = case(4, 64, 300, F32)
    loss, lse = tb.tropical_linear_cross_entropy_forward(x[:0], w, t[:0])
    gx, gw = tb.tropical_linear_cross_entropy_backward(x[:0], w, t[:0], lse, gl[:0])
    assert loss.shape == (0,) and gx.shape == (0, 64) and gw.shape == (300, 64) and not gw.any()


def test_refusals(tb):
    x, w, t, gl = case(100, 64, 300, F32)
    _, lse = tb.tropical_linear_cross_entropy_forward(x, w, t)
    small = torch.empty(1000, dtype=torch.uint8, device=DEV)
    for f in (lambda: tb.tropical_linear_cross_entropy_forward(x, w, t, workspace=small),
              lambda: tb.tropical_linear_cross_entropy_backward(x, w, t, lse, gl, workspace=small)):
        with pytest.raises(tb.TropicalError) as e:
            f()
        assert e.value.status == tb.WORKSPACE_TOO_SMALL
    with pytest.raises(tb.TropicalError) as e:
        tb.tropical_linear_cross_entropy_forward(x, w, t.cpu())
    assert e.value.status == tb.NOT_DEVICE_MEMORY
    with pytest.raises(TypeError):
        tb.tropical_linear_cross_entropy_forward(x, w.to(BF16), t)
    with pytest.raises(TypeError):
        tb.tropical_linear_cross_entropy_forward(x, w, t.float())
    with pytest.raises(ValueError):
        tb.tropical_linear_cross_entropy_forward(x, w[:, :63], t)
    with pytest.raises(ValueError):
        tb.tropical_linear_cross_entropy_forward(x, w, t[:99])
    with pytest.raises(ValueError):
        tb.tropical_linear_cross_entropy_forward(x.t(), w, t)
    with pytest.raises(ValueError):
        tb.tropical_linear_cross_entropy_backward(x, w, t, lse, gl[:50])
    with pytest.raises(ValueError):
        tb.tropical_linear_cross_entropy_backward(x, w, t, lse, gl, grad_w=torch.empty(300, 63, device=DEV))


def check_float32(tb, x, w, t, gl):
    """Float32 gradients where magnitudes differ within a matrix.

    As above, but what the planes keep of G is measured where it counts: an
    element's absolute error is 2^-38 of its own token's weight in grad_x and
    2^-38 of its own label's largest G in grad_w.  The planes of x and w keep
    2^-38 of their matrix's largest element (in the logits too)."""
    n, d = x.shape
    X, W, g = x.double(), w.double(), gl.double()[:, None]
    keep = t >= 0
    g, X = torch.where(keep[:, None], g, 0.0), torch.where(keep[:, None], X, 0.0)
    floor = 2.0 ** -38
    l = X @ W.t()
    dl = (d + 40) * U * (X.abs() @ W.abs().t())
    dl = dl + floor * (X.abs().max() * W.abs().sum(1) + W.abs().max() * X.abs().sum(1)[:, None])
    lse = torch.logsumexp(l, 1)
    dlse = dl.amax(1) + 200 * U + 4 * U * lse.abs()
    p = (l - lse[:, None]).exp()
    G = p.scatter_add(1, t.clamp(min=0)[:, None], torch.full_like(g, -1.0)) * g
    dG = g.abs() * p * (dl + dlse[:, None] + 60 * U) + (2.0 ** -22 * 1.01 + 4 * U) * G.abs() + 2.0 ** -126
    want = G @ W, G.t() @ X
    tol = [(dG + floor * g.abs()) @ W.abs() + (w.shape[0] + 40) * U * (G.abs() @ W.abs())
           + floor * G.abs().sum(1, keepdim=True) * W.abs().max(),
           (dG + floor * G.abs().amax(0)).t() @ X.abs() + (n + 40) * U * (G.t().abs() @ X.abs())
           + floor * G.abs().sum(0)[:, None] * X.abs().max()]
    loss, lse = tb.tropical_linear_cross_entropy_forward(x, w, t)
    got = tb.tropical_linear_cross_entropy_backward(x, w, t, lse, gl)
    for a, b, e, what in zip(got, want, tol, ("grad_x", "grad_w")):
        assert_within(a, b, e + 4 * U * (b.abs() + e), what)


# streaming, small tiles, w as it lies, grad_x / grad_w in 256 x 256 tiles, grad_w in parts along the tokens
F32_SHAPES = [(30, 64, 500), (100, 64, 500), (70, 1000, 11011), (700, 1096, 8300), (2100, 64, 300), (700, 264, 700)]


@pytest.mark.parametrize("tokens,width,vocab", F32_SHAPES)
def test_float32_weights_of_tokens_far_apart(tb, tokens, width, vocab):
    """A token's gradient keeps its digits beside tokens of 2^30 its weight."""
    x, w, t, gl = case(tokens, width, vocab, F32, seed=12)
    g = torch.Generator(device=DEV).manual_seed(tokens)
    check_float32(tb, x, w, t, torch.exp2(-30 * torch.rand(tokens, generator=g, device=DEV)))


@pytest.mark.parametrize("tokens,width,vocab", F32_SHAPES)
def test_float32_improbable_labels(tb, tokens, width, vocab):
    """Labels that every token finds improbable (1e-9 and down to 1e-20) keep
    the digits of their rows of grad_w."""
    x, w, t, gl = case(tokens, width, vocab, F32, seed=13)
    x[:, 0] = 4.0
    rare = torch.arange(vocab, device=DEV) % 7 == 3
    w[:, 0] = torch.where(rare, -4.0 - 0.05 * (torch.arange(vocab, device=DEV) % 80), 0.0)
    t[rare[t.clamp(min=0)]] = 0
    check_float32(tb, x, w, t, gl)


@pytest.mark.parametrize("tokens,width,vocab", F32_SHAPES)
def test_float32_mixed_magnitudes(tb, tokens, width, vocab):
    """Rows of x and w of 1 down to 2^-20."""
    x, w, t, gl = case(tokens, width, vocab, F32, seed=14)
    g = torch.Generator(device=DEV).manual_seed(tokens)
    for m in (x, w):
        m *= torch.exp2(-20 * torch.rand(len(m), 1, generator=g, device=DEV))
    check_float32(tb, x, w, t, gl)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens", [20, 90, 300])
def test_one_infinite_weight(tb, tokens, dtype):
    """An infinite weight reaches its own token's row of grad_x and no other."""
    x, w, t, gl = case(tokens, 64, 500, dtype, seed=15, ignored=0.1)
    gl = gl * 100
    at = int((t >= 0).nonzero()[3])
    gl[at] = 0.0
    want, tol = reference(x, w, t, gl)
    _, lse = tb.tropical_linear_cross_entropy_forward(x, w, t)
    for bad in (float("inf"), float("-inf"), float("nan")):
        gl[at] = bad
        gx, _ = tb.tropical_linear_cross_entropy_backward(x, w, t, lse, gl)
        assert not torch.isfinite(gx[at]).any()
        gx[at] = 0.0
        assert_within(gx, want[2], tol[2], f"grad_x beside a weight of {bad}")


@pytest.mark.parametrize("tokens", [10, 90])
def test_float32_largest_numbers(tb, tokens):
    """Elements of the largest float32 magnitude, logits of ordinary size."""
    x, w, t, gl = case(tokens, 32, 300, F32, seed=16)
    big = torch.finfo(F32).max
    x, w = torch.where(x < 0, -big, big), w * 2.0 ** -125  # (normal numbers but for a few)
    w[w.abs() < 2.0 ** -126] = 0.0
    gl = gl * 1e-4
    want, tol = reference(x, w, t, gl)
    loss, lse = tb.tropical_linear_cross_entropy_forward(x, w, t)
    gw = tb.tropical_linear_cross_entropy_backward(x, w, t, lse, gl, grad_x=None)[1]
    for a, b, e, what in zip((loss, lse, gw), (want[0], want[1], want[3]), (tol[0], tol[1], tol[3]), ("loss", "lse", "grad_w")):
        assert_within(a, b, e, what)


def few_of_many(tokens, width, vocab, dtype, seed):
    """x, target, weights of `tokens` tokens of which eight count, and those eight."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.empty(tokens, width, dtype=dtype, device=DEV)  # (what the others hold reaches nothing)
    t = torch.full((tokens,), -100, dtype=torch.int32, device=DEV)
    at = torch.tensor([0, 1, 300, tokens // 2, tokens - 70, tokens - 3, tokens - 2, tokens - 1], device=DEV)
    x[at] = torch.randn(8, width, generator=g, device=DEV).to(dtype)
    t[at] = torch.randint(0, vocab, (8,), generator=g, device=DEV).int()
    t[at[0]], t[at[1]] = vocab - 1, 0
    return x, t, torch.rand(tokens, generator=g, device=DEV) + 0.1, at


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_more_logits_than_a_launch_holds(tb, dtype):
    """2^22 tokens and 131372 labels: more than 2^23 tiles of 256 x 256."""
    x, t, _, at = few_of_many(1 << 22, 16, 131372, dtype, 17)
    w = torch.randn(131372, 16, device=DEV, generator=torch.Generator(device=DEV).manual_seed(17)).to(dtype)
    loss, lse = tb.tropical_linear_cross_entropy_forward(x, w, t)
    want, tol = reference(x[at], w, t[at])
    for got, b, e, what in zip((loss, lse), want, tol, ("loss", "lse")):
        assert_within(got[at], b, e, what)
        got[at] = 0.0
        assert not got.any()
    del x, loss, lse
    torch.cuda.empty_cache()


def test_more_labels_than_a_launch_holds(tb):
    """More than 2^29 labels with 32 to a workgroup of the streaming form."""
    vocab = (1 << 29) + 100
    g = torch.Generator(device=DEV).manual_seed(18)
    w = torch.randn(vocab, 1, generator=g, device=DEV).to(BF16)
    x = torch.randn(2, 1, generator=g, device=DEV).to(BF16)
    t = torch.tensor([vocab - 1, 5], device=DEV)
    got = tb.tropical_linear_cross_entropy_forward(x, w, t)
    for i in range(2):
        want, tol = reference(x[i:i + 1], w, t[i:i + 1])
        for a, b, e, what in zip(got, want, tol, ("loss", "lse")):
            assert_within(a[i:i + 1], b, e, what)
        del want, tol
    del w
    torch.cuda.empty_cache()


def test_more_rows_of_grad_x_than_a_launch_holds(tb):
    """2^22 tokens of more than three times 1024 columns."""
    tokens, width, vocab = 1 << 22, 3100, 16
    x, t, gl, at = few_of_many(tokens, width, vocab, BF16, 19)
    w = torch.randn(vocab, width, device=DEV, generator=torch.Generator(device=DEV).manual_seed(19)).to(BF16)
    _, lse = tb.tropical_linear_cross_entropy_forward(x, w, t)
    gx, gw = tb.tropical_linear_cross_entropy_backward(x, w, t, lse, gl)
    want, tol = reference(x[at], w, t[at], gl[at])
    del x
    assert_within(gx[at], want[2], tol[2], "grad_x")
    assert_within(gw, want[3], tol[3], "grad_w")
    gx[at] = 0.0
    assert not any(part.any() for part in gx.split(1 << 19))
    del gx
    torch.cuda.empty_cache()
