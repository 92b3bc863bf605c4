"""The norms, gate and sum between two residual blocks on the GPU, forward and
backward, against the formulas in 64 bits.

Tolerances, with u = 2^-24 (one float32 rounding, relative):
  - a sum over a row is a tree: at most 16 sequential terms per thread, 6
    steps across lanes, 16 waves; with the product and the factor 1 / cols
    fewer than 48 roundings touch a term (rows past the registers add cols /
    1024 sequential terms): n u sum |terms|;
  - a sum over rows in P <= rows parts has at most rows / P + P / 4 sequential
    terms, and fewer than 32 more in joining waves and parts: below rows + 64,
    so (rows + 64) u sum |terms|;
  - dgate is gamma A + beta B with A = sum H x^ and B = sum H over a gate row's
    rows, each off by (group + 64) u times its terms' magnitudes; two products,
    their sum and branch_scale add four roundings of |gamma A| + |beta B| at
    most: (group + 68) u sum |H| (|x^ gamma| + |beta|), and sum |H v| in place
    of the last without a post norm, where v is u;
  - elementwise errors are carried through the formulas to first order;
  - an output is rounded to its type once (torch.finfo(t).eps / 2).
"""
import math

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
    torch.cuda.synchronize()
    torch._C._cuda_clearCublasWorkspaces()
    torch.cuda.empty_cache()


def matrix(rows, cols, pad, dtype, gen, offset=0.0):
    """rows x cols view of a wider buffer whose other elements are NaN."""
    buf = torch.full((rows, cols + pad), float("nan"))
    buf[:, :cols] = torch.randn(rows, cols, generator=gen) + offset
    return buf.to(dtype).to(DEV)[:, :cols]


def assert_within(got, want, tol, what):
    tol = tol + torch.finfo(got.dtype).eps / 2 * (want.abs() + tol)
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, worst {float((err - tol).max()):.3g} over"


def f32(x):
    return float(torch.tensor(x, dtype=F32))


def rows_of(n, cols):
    return n + cols / 1024


class Problem:
    """Inputs of an operator, as its calls take them."""

    def __init__(self, rows, cols, dtype, ptype, post, pre, gates, pad=0, seed=0, residual=True, weights=True,
                 group=None, gate_dtype=None):
        g = torch.Generator().manual_seed(seed + rows * 100003 + cols)
        self.rows, self.cols, self.dtype = rows, cols, dtype
        self.u = matrix(rows, cols, pad, dtype, g, offset=0.7)
        self.r = matrix(rows, cols, (pad + 1) % 3, dtype, g, offset=-0.4) if residual else None
        self.dy = matrix(rows, cols, pad % 2, dtype, g) if pre else None
        self.dh = matrix(rows, cols, pad, dtype, g)

        def vector(mean, spread):
            return (mean + spread * torch.randn(cols, generator=g)).to(ptype).to(DEV)

        self.op = dict(post=post, pre=pre, residual_scale=1.1, branch_scale=0.7)
        if weights:
            if post:
                self.op.update(post_gamma=vector(1, 0.2), post_beta=vector(0, 0.5))
            if pre:
                self.op.update(pre_gamma=vector(1, 0.2), pre_beta=vector(0, 0.5))
        if gates:
            gate = matrix(gates, cols, pad, gate_dtype or ptype, g, offset=0.8)
            self.op["gate"] = gate if gates > 1 or rows == 1 else gate[0]
            if group:
                self.op["gate_group"] = group
        self.group = group or (max(1, rows // gates) if gates else max(rows, 1))

    def weight(self, name, other):
        w = self.op.get(name)
        return w.double() if w is not None else torch.full((self.cols,), other, dtype=torch.float64, device=DEV)

    def gate_rows(self):
        """branch_scale gate for every row."""
        gate = self.op.get("gate")
        gate = torch.ones(1, self.cols, dtype=torch.float64, device=DEV) if gate is None else gate.double().view(-1, self.cols)
        index = torch.arange(self.rows, device=DEV) // self.group
        return gate[index] * f32(self.op["branch_scale"])


def norm_reference(x, ex, kind, gamma, beta):
    """(normed, its error, mean, its error, rstd, its relative error) of rows x
    known up to ex."""
    n = rows_of(48, x.shape[1])
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    em = n * U * x.abs().mean(1, keepdim=True) + ex.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(mean)
    xc = x - mean
    rstd = 1 / ((xc * xc).mean(1, keepdim=True) + f32(1e-5)).sqrt()
    e = ex + em + U * xc.abs()  # of an element about the mean
    rel = n * U + rstd ** 2 * ((xc.abs() * ex).mean(1, keepdim=True) + (e * e).mean(1, keepdim=True))
    if kind == "rms":
        rel = rel + rstd ** 2 * (xc.abs() * ex).mean(1, keepdim=True)
    xh = xc * rstd
    exh = rstd * e + xh.abs() * (rel + 2 * U)
    y = xh * gamma + beta
    return y, exh * gamma.abs() + 2 * U * ((xh * gamma).abs() + y.abs()), mean[:, 0], em[:, 0], rstd[:, 0], rel[:, 0]


def forward_reference(q):
    op = q.op
    u = q.u.double()
    v, ev = u, torch.zeros_like(u)
    out = {}
    if op["post"]:
        v, ev, mean, em, rstd, rel = norm_reference(u, ev, op["post"], q.weight("post_gamma", 1.0), q.weight("post_beta", 0.0))
        out.update(post_mean=(mean, em), post_rstd=(rstd, rel * rstd))
    gs = q.gate_rows()
    h, eh = gs * v, gs.abs() * ev + 2 * U * (gs * v).abs()
    if q.r is not None:
        res = q.r.double() * f32(op["residual_scale"])
        h, eh = h + res, eh + U * (res.abs() + (h + res).abs())
    out["h"] = (h, eh)
    if op["pre"]:
        y, ey, mean, em, rstd, rel = norm_reference(h, eh, op["pre"], q.weight("pre_gamma", 1.0), q.weight("pre_beta", 0.0))
        out.update(pre_mean=(mean, em), pre_rstd=(rstd, rel * rstd), y=(y, ey))
    return out


def check_forward(tb, q, **kw):
    f = tb.tropical_residual_norm_forward(q.u, q.r, **q.op, **kw)
    want = forward_reference(q)
    for name in ("post_mean", "post_rstd", "pre_mean", "pre_rstd", "h", "y"):
        got = getattr(f, name)
        which = name.split("_")[0]
        there = name in want and not (name.endswith("mean") and q.op[which] != "layer")
        assert (got is not None) == there or kw.get(name, True) is None, name
        if got is not None:
            assert_within(got, *want[name], name)
    return f


def kept_of(tb, f, q, held):
    """u and h for a backward, and their values."""
    if held:
        u, h = (tb.tropical_act8_pack(x) for x in (q.u, f.h))
        return u, h, tb.tropical_act8_unpack(u).double(), tb.tropical_act8_unpack(h).double()
    return q.u, f.h, q.u.double(), f.h.double()


def backward_reference(q, f, u, h):
    """{name: (value, error)} with the statistics of f taken as they are."""
    op, out = q.op, {}
    cols = q.cols
    n = rows_of(50, cols)

    def standard(x, which):
        mean, rstd = getattr(f, which + "_mean"), getattr(f, which + "_rstd").double()[:, None]
        xh = (x if mean is None else x - mean.double()[:, None]) * rstd
        return xh, 3 * U * xh.abs(), rstd

    def through(d, ed, xh, exh, rstd, which):
        """A norm's Jacobian applied to d (known up to ed), before rstd."""
        g = q.weight(which + "_gamma", 1.0)
        w, ew = d * g, ed * g.abs() + U * (d * g).abs()
        layer = op[which] == "layer"
        c1 = w.mean(1, keepdim=True) if layer else torch.zeros_like(w[:, :1])
        e1 = (ew.mean(1, keepdim=True) + n * U * w.abs().mean(1, keepdim=True)) if layer else torch.zeros_like(c1)
        c2 = (w * xh).mean(1, keepdim=True)
        e2 = (ew * xh.abs() + w.abs() * exh).mean(1, keepdim=True) + n * U * (w * xh).abs().mean(1, keepdim=True)
        t = w - c1 - xh * c2
        et = ew + e1 + xh.abs() * e2 + c2.abs() * exh + 4 * U * (w.abs() + c1.abs() + (xh * c2).abs())
        return rstd * t, rstd * et + 2 * U * (rstd * t).abs()

    def column_sum(x, ex, count):
        return x.sum(0), ex.sum(0) + (count + 64) * U * x.abs().sum(0)

    zero = torch.zeros(q.rows, cols, dtype=torch.float64, device=DEV)
    H = zero if q.dh is None else q.dh.double()
    eH = zero
    if op["pre"]:
        dy = q.dy.double()
        xh, exh, rstd = standard(h, "pre")
        out["pre_gamma"] = column_sum(dy * xh, dy.abs() * exh, q.rows)
        out["pre_beta"] = column_sum(dy, zero, q.rows)
        t, et = through(dy, zero, xh, exh, rstd, "pre")
        H, eH = H + t, et + U * (H + t).abs()
    rs = f32(op["residual_scale"])
    out["r"] = (H * rs, eH * abs(rs) + U * (H * rs).abs())
    v, ev, av = u, zero, u.abs()
    if op["post"]:
        xu, exu, rstd_u = standard(u, "post")
        g, b = q.weight("post_gamma", 1.0), q.weight("post_beta", 0.0)
        v, ev, av = xu * g + b, exu * g.abs(), (xu * g).abs() + b.abs()
    gates = -(-q.rows // q.group) if q.rows else 0
    index = torch.arange(q.rows, device=DEV) // q.group

    def group_sum(x):
        return torch.zeros(gates, cols, dtype=torch.float64, device=DEV).index_add_(0, index, x)

    bs = f32(op["branch_scale"])
    eg = group_sum(eH * av + H.abs() * ev) + (q.group + 68) * U * group_sum(H.abs() * av)
    gate = group_sum(H * v) * bs
    out["gate"] = (gate, eg * abs(bs) + U * gate.abs())
    gs = q.gate_rows()
    dv, edv = H * gs, eH * gs.abs() + 2 * U * (H * gs).abs()
    if op["post"]:
        out["post_gamma"] = column_sum(dv * xu, edv * xu.abs() + dv.abs() * exu, q.rows)
        out["post_beta"] = column_sum(dv, edv, q.rows)
        dv, edv = through(dv, edv, xu, exu, rstd_u, "post")
    out["u"] = (dv, edv)
    return out


def check_backward(tb, q, f, held=False, **kw):
    u, h, uv, hv = kept_of(tb, f, q, held)
    stats = {k: getattr(f, k) for k in ("post_mean", "post_rstd", "pre_mean", "pre_rstd")}
    g = tb.tropical_residual_norm_backward(q.dy, q.dh, u, h, **stats, **q.op, **kw)
    want = backward_reference(q, f, uv, hv)
    for name, got in g._asdict().items():
        if got is not None:
            ref, tol = want[name]
            assert_within(got, ref.view(got.shape), tol.view(got.shape), name)
    return g


SHAPES = [(1, 1), (1, 64), (3, 7), (5, 8), (4, 512), (9, 513), (4, 1000), (6, 1025), (7, 2048), (6, 2049), (3, 4096),
          (3, 4097), (2, 8191), (3, 8192), (2, 8193), (2, 16384), (2, 16385), (1, 40001), (2049, 24), (700, 520)]
TYPES = [(F32, F32), (BF16, BF16), (BF16, F32)]
NORMS = [("layer", "layer"), ("rms", "rms"), (None, "rms"), ("layer", None), (None, None)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype,ptype", TYPES)
@pytest.mark.parametrize("held", [False, True])
def test_forward_and_backward(tb, rows, cols, dtype, ptype, held):
    post, pre = NORMS[(rows + cols) % 3]
    q = Problem(rows, cols, dtype, ptype, post, pre, gates=1, pad=(rows + cols) % 4)
    f = check_forward(tb, q)
    check_backward(tb, q, f, held)


@pytest.mark.parametrize("post,pre", NORMS + [("rms", "layer"), ("rms", None), (None, "layer"), ("layer", "rms")])
@pytest.mark.parametrize("rows,cols", [(37, 200), (20, 1500), (11, 3000), (13, 5000), (5, 9000)])
@pytest.mark.parametrize("residual,weights", [(True, True), (False, False)])
def test_norms(tb, post, pre, rows, cols, residual, weights):
    for dtype in (F32, BF16):
        q = Problem(rows, cols, dtype, F32, post, pre, gates=1, pad=1, residual=residual, weights=weights)
        f = check_forward(tb, q)
        check_backward(tb, q, f)
        q.op.pop("gate")
        f = check_forward(tb, q)
        check_backward(tb, q, f, held=True)
        if pre:
            q.dh = None
            check_backward(tb, q, f)


# (rows, gate rows, rows of one): one for all, for a few rows, ends inside a
# group, for every row, more gate rows than the backward has parts
GATES = [(60, 1, 60), (60, 4, 15), (62, 5, 15), (60, 60, 1), (700, 700, 1), (1400, 700, 2), (1399, 700, 2),
         (1600, 534, 3), (2000, 2, 1000), (600, 300, 2), (1, 1, 1)]


@pytest.mark.parametrize("rows,gates,group", GATES)
@pytest.mark.parametrize("cols", [40, 1100, 2100, 4200, 8200])
def test_gates(tb, rows, gates, group, cols):
    if rows * cols > 3000000:
        rows, gates = rows // 2, -(-(rows // 2) // group)
    for dtype, gate_dtype, post, held in ((F32, F32, "layer", True), (BF16, BF16, None, False), (BF16, F32, "rms", True)):
        q = Problem(rows, cols, dtype, F32, post, "layer", gates, pad=3, group=group, gate_dtype=gate_dtype)
        f = check_forward(tb, q)
        g = check_backward(tb, q, f, held)
        assert g.gate.shape == q.op["gate"].shape and g.gate.dtype == gate_dtype


@pytest.mark.parametrize("cols", [40, 700, 3000, 6000, 10000])
def test_each_gradient_alone(tb, cols):
    q = Problem(21, cols, F32, F32, "layer", "rms", gates=3, pad=1)
    f = check_forward(tb, q)
    everything = check_backward(tb, q, f)
    names = ["dr", "du", "dgate", "dpost_gamma", "dpost_beta", "dpre_gamma", "dpre_beta"]
    for k, name in enumerate(names):
        g = check_backward(tb, q, f, **{n: None for n in names if n != name})
        assert [x is not None for x in g] == [n == name for n in names]
        assert torch.equal(g[k], everything[k])
    g = check_backward(tb, q, f, **{n: None for n in names})
    assert all(x is None for x in g)


@pytest.mark.parametrize("cols", [40, 700, 3000, 6000, 10000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_held_is_the_same_as_its_values(tb, cols, dtype):
    """u and h in 8 bits give the bits that their values give."""
    q = Problem(40, cols, dtype, F32, "rms", "layer", gates=4, pad=1)
    f = tb.tropical_residual_norm_forward(q.u, q.r, **q.op)
    u8, h8 = tb.tropical_act8_pack(q.u), tb.tropical_act8_pack(f.h)
    stats = {k: getattr(f, k) for k in ("post_rstd", "pre_mean", "pre_rstd")}
    a = tb.tropical_residual_norm_backward(q.dy, q.dh, u8, h8, **stats, **q.op)
    b = tb.tropical_residual_norm_backward(q.dy, q.dh, tb.tropical_act8_unpack(u8, dtype),
                                           tb.tropical_act8_unpack(h8, dtype), **stats, **q.op)
    assert all(x is None and y is None or torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("rows,cols", [(3, 31), (5, 1000), (4, 1025), (3, 5000), (2, 17000)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("post", [None, "layer"])
def test_forward_leaves_8_bits(tb, rows, cols, dtype, post):
    """u8 is u packed.  h8 is h packed before its rounding: without a post norm
    that h is residual_scale r + (branch_scale gate) u, each operation one
    float32 operation; with one the codes are within a step and what h is off."""
    q = Problem(rows, cols, dtype, F32, post, "rms", gates=1, pad=1)
    f = tb.tropical_residual_norm_forward(q.u, q.r, **q.op, hold_u=True, hold_h=True)
    want = tb.tropical_act8_pack(q.u)
    assert torch.equal(f.u8.codes, want.codes) and torch.equal(f.u8.exponents, want.exponents)
    ref, eh = forward_reference(q)["h"]
    if post is None:
        h = q.r.float() * 1.1 + (q.op["gate"].view(1, -1) * 0.7) * q.u.float()
        want = tb.tropical_act8_pack(h)
        assert torch.equal(f.h8.codes, want.codes) and torch.equal(f.h8.exponents, want.exponents)
    v = tb.tropical_act8_unpack(f.h8).double()
    step = torch.exp2(f.h8.exponents.double() - 127).repeat_interleave(32, 1)[:, :cols]
    assert ((v - ref).abs() <= step / 2 + eh).all()
    plain = tb.tropical_residual_norm_forward(q.u, q.r, **q.op)
    assert torch.equal(f.h, plain.h) and torch.equal(f.y, plain.y)
    # given buffers are filled, and nothing beside them
    blocks = -(-cols // 32)
    buf = tb.Act8(torch.full((rows, cols + 5), 99, dtype=torch.int8, device=DEV)[:, :cols],
                  torch.full((rows, blocks + 5), 99, dtype=torch.uint8, device=DEV)[:, :blocks])
    tb.tropical_residual_norm_forward(q.u, q.r, **q.op, hold_h=buf)
    assert torch.equal(buf.codes, f.h8.codes) and torch.equal(buf.exponents, f.h8.exponents)
    assert (buf.codes._base[:, cols:] == 99).all() and (buf.exponents._base[:, blocks:] == 99).all()


@pytest.mark.parametrize("cols", [50, 3000, 9000, 20000])
def test_h_in_place_of_r(tb, cols):
    q = Problem(6, cols, BF16, BF16, "rms", "layer", gates=1, pad=2)
    want = tb.tropical_residual_norm_forward(q.u, q.r, **q.op)
    got = tb.tropical_residual_norm_forward(q.u, q.r, **q.op, h=q.r)
    assert got.h is q.r and torch.equal(got.h, want.h) and torch.equal(got.y, want.y)


@pytest.mark.parametrize("cols", [50, 3000, 9000, 20000])
def test_what_lies_beside_is_left(tb, cols):
    q = Problem(9, cols, F32, F32, "layer", "rms", gates=3, pad=1)

    def hole(rows):
        return torch.full((rows, cols + 3), 7.0, device=DEV)

    h, y, dr, du, dg = hole(9), hole(9), hole(9), hole(9), hole(3)
    f = check_forward(tb, q, h=h[:, :cols], y=y[:, :cols])
    check_backward(tb, q, f, dr=dr[:, :cols], du=du[:, :cols], dgate=dg[:, :cols])
    for t in (h, y, dr, du, dg):
        assert (t[:, cols:] == 7.0).all()


@pytest.mark.parametrize("cols", [50, 3000, 9000, 20000])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_non_finite_rows_stay_apart(tb, cols, bad):
    q = Problem(8, cols, F32, F32, "layer", "rms", gates=1)
    clean = tb.tropical_residual_norm_forward(q.u, q.r, **q.op)
    q.u[2, cols // 2] = bad
    q.r[5, 0] = bad
    f = tb.tropical_residual_norm_forward(q.u, q.r, **q.op, hold_h=True)
    good = [i for i in range(8) if i not in (2, 5)]
    assert torch.equal(f.y[good], clean.y[good]) and torch.equal(f.h[good], clean.h[good])
    assert f.y[2].isnan().all() and not torch.isfinite(f.pre_rstd[5]) or f.y[5].isnan().any()
    assert f.h[2].isnan().all() and (f.h8.exponents[2] == 255).all()
    q.u[2, cols // 2] = 0
    q.r[5, 0] = 0
    f = tb.tropical_residual_norm_forward(q.u, q.r, **q.op)
    stats = {k: getattr(f, k) for k in ("post_mean", "post_rstd", "pre_rstd")}
    clean = tb.tropical_residual_norm_backward(q.dy, q.dh, q.u, f.h, **stats, **q.op)
    q.dy[3, 1] = bad
    g = tb.tropical_residual_norm_backward(q.dy, q.dh, q.u, f.h, **stats, **q.op)
    good = [i for i in range(8) if i != 3]
    assert torch.equal(g.r[good], clean.r[good]) and torch.equal(g.u[good], clean.u[good])
    assert not torch.isfinite(g.r[3]).any() and not torch.isfinite(g.u[3]).any()
    only = torch.arange(cols, device=DEV) != 1
    assert torch.equal(g.pre_beta[only], clean.pre_beta[only]) and not torch.isfinite(g.pre_beta[1])


@pytest.mark.parametrize("cols", [50, 3000, 9000, 20000])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_non_finite_rows_whole(tb, cols, bad):
    """What a non-finite element makes of its own row.  In u before a layer norm
    it makes the mean and all of the row NaN.  In r before an RMS norm a NaN does
    so too; an infinity makes rstd 0, its own y NaN and the others beta."""
    q = Problem(8, cols, F32, F32, "layer", "rms", gates=1)
    clean = tb.tropical_residual_norm_forward(q.u, q.r, **q.op)
    q.u[2, cols // 2] = bad
    q.r[5, 0] = bad
    f = tb.tropical_residual_norm_forward(q.u, q.r, **q.op)
    for t in (f.h, f.y):
        assert t[2].isnan().all()
    assert f.post_rstd[2].isnan() and f.pre_rstd[2].isnan() and not torch.isfinite(f.post_mean[2])
    assert torch.equal(f.post_mean[5], clean.post_mean[5]) and torch.equal(f.post_rstd[5], clean.post_rstd[5])
    assert torch.equal(f.h[5, 1:], clean.h[5, 1:]) and not torch.isfinite(f.h[5, 0])
    if math.isnan(bad):
        assert f.pre_rstd[5].isnan() and f.y[5].isnan().all()
    else:
        assert f.pre_rstd[5] == 0 and f.y[5, 0].isnan() and torch.equal(f.y[5, 1:], q.op["pre_beta"][1:])


def test_no_rows(tb):
    for rows, cols in ((0, 40), (3, 0), (0, 9000)):
        q = Problem(rows, cols, F32, F32, "layer", "rms", gates=1)
        f = tb.tropical_residual_norm_forward(q.u, q.r, **q.op)
        assert f.h.shape == (rows, cols)
        stats = {k: getattr(f, k) for k in ("post_mean", "post_rstd", "pre_rstd")}
        out = [torch.full((cols,), 5.0, device=DEV) for _ in range(4)]
        g = tb.tropical_residual_norm_backward(q.dy, q.dh, q.u, f.h, **stats, **q.op, dpost_gamma=out[0],
                                               dpost_beta=out[1], dpre_gamma=out[2], dpre_beta=out[3])
        assert all((t == 0).all() for t in out) and g.r.shape == (rows, cols)


@pytest.mark.parametrize("cols", [5, 40, 9000])
@pytest.mark.parametrize("gates,group", [(1, None), (3, 7)])
@pytest.mark.parametrize("post", [None, "layer"])
def test_gate_gradient_without_rows(tb, cols, gates, group, post):
    """Zeros for every gate row that is there, as for the weights, asked for
    with them or alone, and on a stream of its own."""
    q = Problem(0, cols, F32, F32, post, "rms", gates=0)
    gate = torch.ones(gates, cols, device=DEV)
    q.op["gate"] = gate if group else gate[0]
    if group:
        q.op["gate_group"] = group
    f = tb.tropical_residual_norm_forward(q.u, q.r, **q.op)
    stats = {k: getattr(f, k) for k in ("post_mean", "post_rstd", "pre_rstd")}
    names = ["dr", "du", "dpost_gamma", "dpost_beta", "dpre_gamma", "dpre_beta"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for kw in ({}, {n: None for n in names}, dict(stream=side)):
        dgate = torch.full_like(q.op["gate"], math.nan)
        side.wait_stream(torch.cuda.current_stream())
        g = tb.tropical_residual_norm_backward(q.dy, q.dh, q.u, f.h, **stats, **q.op, dgate=dgate, **kw)
        side.synchronize()
        assert g.gate is dgate and (dgate == 0).all()
        assert all(x is None or (x == 0).all() for x in g[3:])
    # allocated by the call, in memory that held something else
    torch.full_like(q.op["gate"], math.nan)
    g = tb.tropical_residual_norm_backward(q.dy, q.dh, q.u, f.h, **stats, **q.op)
    assert g.gate.shape == q.op["gate"].shape and (g.gate == 0).all()


@pytest.mark.parametrize("gates", [1, 3])
def test_gate_rows_without_rows(tb, gates):
    """Gate rows whose batch is empty: outputs of no rows, gradients of zeros."""
    q = Problem(0, 40, F32, F32, "layer", "rms", gates=0)
    q.op["gate"] = torch.ones(gates, 40, device=DEV)
    f = tb.tropical_residual_norm_forward(q.u, q.r, **q.op)
    assert f.h.shape == f.y.shape == (0, 40)
    stats = {k: getattr(f, k) for k in ("post_mean", "post_rstd", "pre_rstd")}
    g = tb.tropical_residual_norm_backward(q.dy, q.dh, q.u, f.h, **stats, **q.op,
                                           dgate=torch.full((gates, 40), math.nan, device=DEV))
    assert g.r.shape == (0, 40) and all((x == 0).all() for x in g[2:] if x is not None)


@pytest.mark.parametrize("cols", [33, 1001, 9000])
def test_vectors_changed_in_place(tb, cols):
    """Statistics and weight gradients are tensors of their own: one changed in
    place, by what needs a gradient too, leaves the others and what autograd
    kept of them."""
    q = Problem(12, cols, F32, F32, "layer", "layer", gates=1)
    f = check_forward(tb, q)
    g = check_backward(tb, q, f)
    for vectors in (f[2:6], g[3:]):
        want = [t.clone() for t in vectors]
        a = torch.ones_like(vectors[1], requires_grad=True)
        out = (a * vectors[1]).sum()
        vectors[0].add_(torch.ones_like(vectors[0], requires_grad=True))
        vectors[2].zero_()
        out.backward()
        assert torch.equal(a.grad, want[1]) and torch.equal(vectors[1], want[1]) and torch.equal(vectors[3], want[3])
        assert torch.equal(vectors[0], want[0] + 1) and (vectors[2] == 0).all()
        assert [t.requires_grad for t in vectors] == [True, False, False, False]


@pytest.mark.parametrize("rows,cols,gates", [(2049, 24, 1), (700, 520, 700), (300, 4096, 3), (90, 8192, 1), (50, 9000, 5)])
def test_the_same_bits_every_time(tb, rows, cols, gates):
    q = Problem(rows, cols, BF16, F32, "rms", "rms", gates)
    f = tb.tropical_residual_norm_forward(q.u, q.r, **q.op)
    stats = {k: getattr(f, k) for k in ("post_rstd", "pre_rstd")}
    a, b = (tb.tropical_residual_norm_backward(q.dy, q.dh, q.u, f.h, **stats, **q.op) for _ in range(2))
    assert all(x is None or torch.equal(x, y) for x, y in zip(a, b))


def reference_loss(q, u, r, gate, weights, gy, gh):
    """sum(gy y + gh h) in 64 bits."""
    op = q.op

    def norm(x, which):
        if not op[which]:
            return x
        xc = x - x.mean(1, keepdim=True) if op[which] == "layer" else x
        return (xc / ((xc * xc).mean(1, keepdim=True) + f32(1e-5)).sqrt()) * weights[which + "_gamma"] + weights[which + "_beta"]

    index = torch.arange(q.rows, device=DEV) // q.group
    h = norm(u, "post") * gate[index] * f32(op["branch_scale"]) + f32(op["residual_scale"]) * r
    return float((norm(h, "pre") * gy).sum() + (h * gh).sum())


@pytest.mark.parametrize("post,pre", [("layer", "layer"), ("rms", "rms"), (None, "layer")])
@pytest.mark.parametrize("rows,cols", [(12, 48), (6, 700), (3, 9000)])
def test_gradients_against_differences(tb, post, pre, rows, cols):
    """Along a random direction in every input at once: the kernels' gradients
    against a central difference of the loss in 64 bits.  The difference is off
    by t^2 times its third derivative, the gradients by a few hundred float32
    roundings of their terms: 1e-4 of the sum of |gradient direction| has room
    for both at t = 1e-4."""
    q = Problem(rows, cols, F32, F32, post, pre, gates=3, pad=0)
    f = tb.tropical_residual_norm_forward(q.u, q.r, **q.op)
    stats = {k: getattr(f, k) for k in ("post_mean", "post_rstd", "pre_mean", "pre_rstd")}
    g = tb.tropical_residual_norm_backward(q.dy, q.dh, q.u, f.h, **stats, **q.op)
    gen = torch.Generator(device=DEV).manual_seed(rows)
    names = [w + p for w in ("post", "pre") if q.op[w] for p in ("_gamma", "_beta")]
    base = dict(u=q.u, r=q.r, gate=q.op["gate"], **{n: q.op[n] for n in names})
    base = {k: v.double() for k, v in base.items()}
    move = {k: torch.randn(v.shape, generator=gen, device=DEV, dtype=torch.float64) for k, v in base.items()}
    gy, gh = q.dy.double(), q.dh.double()

    def loss(t):
        at = {k: v + t * move[k] for k, v in base.items()}
        return reference_loss(q, at["u"], at["r"], at["gate"], at, gy, gh)

    t = 1e-4
    diff = (loss(t) - loss(-t)) / (2 * t)
    along = [getattr(g, k).double() * m for k, m in move.items()]
    total, size = sum(float(x.sum()) for x in along), sum(float(x.abs().sum()) for x in along)
    assert abs(total - diff) <= 1e-4 * size, (total, diff, size)


@pytest.mark.parametrize("cols", [300, 3000, 9000])
def test_graph_and_streams(tb, cols):
    """A captured forward and backward, replayed between eager work, and the
    same on a second stream."""
    q = Problem(64, cols, BF16, F32, "rms", "layer", gates=2)
    h, y = torch.empty_like(q.u), torch.empty_like(q.u)
    u8, h8 = tb.tropical_act8_pack(q.u), tb.tropical_act8_pack(q.u)
    ws = torch.empty(tb.tropical_residual_norm_backward_workspace_size(BF16, 64, cols, "rms", "layer", 32), dtype=torch.uint8,
                     device=DEV)

    def step(**kw):
        f = tb.tropical_residual_norm_forward(q.u, q.r, **q.op, h=h, y=y, hold_u=u8, hold_h=h8)
        stats = {k: getattr(f, k) for k in ("post_rstd", "pre_mean", "pre_rstd")}
        return tb.tropical_residual_norm_backward(q.dy, q.dh, u8, h8, **stats, **q.op, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    gen = torch.Generator(device=DEV).manual_seed(1)
    for k in range(3):
        for t in (q.u, q.r, q.dy, q.dh):
            t.copy_(torch.randn(t.shape, generator=gen, device=DEV))
        want = [x.clone() for x in step() if x is not None] + [h.clone(), y.clone()]
        torch.cuda.synchronize()
        h.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [x for x in out if x is not None] + [h, y]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    side.wait_stream(torch.cuda.current_stream())
    f = tb.tropical_residual_norm_forward(q.u, q.r, **q.op, stream=side)
    stats = {k: getattr(f, k) for k in ("post_rstd", "pre_mean", "pre_rstd")}
    g = tb.tropical_residual_norm_backward(q.dy, q.dh, u8, h8, **stats, **q.op, stream=side)
    side.synchronize()
    assert torch.equal(f.y, y) and all(torch.equal(a, b) for a, b in zip([x for x in g if x is not None], want))


@pytest.mark.parametrize("cols", [300, 2000, 9000])
def test_calls_at_once_on_two_streams(tb, cols):
    """Forward, backward and weight gradient of different inputs, issued in turn
    to two streams without a wait between them, against one after another."""
    problems = [Problem(200, cols, BF16, F32, "rms", "layer", gates=g, seed=g) for g in (2, 200)]

    def step(q):
        f = tb.tropical_residual_norm_forward(q.u, q.r, **q.op, hold_u=True, hold_h=True)
        stats = {k: getattr(f, k) for k in ("post_rstd", "pre_mean", "pre_rstd")}
        g = tb.tropical_residual_norm_backward(q.dy, q.dh, f.u8, f.h8, **stats, **q.op)
        return [f.h, f.y, *(x for x in g if x is not None), tb.tropical_act8_linear_grad_w(q.dy, f.u8)]

    want = [step(q) for q in problems]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for k, q in enumerate(problems):
            with torch.cuda.stream(streams[k]):
                got[k].append(step(q))
    for s in streams:
        s.synchronize()
    for k in range(2):
        for out in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[k]))


def test_offsets_past_32_bits(tb):
    """Rows that lie more than 2^31 elements apart."""
    ld = (1 << 31) + 64
    q = Problem(2, 300, BF16, F32, "layer", "rms", gates=1)
    f = tb.tropical_residual_norm_forward(q.u, q.r, **q.op)
    stats = {k: getattr(f, k) for k in ("post_mean", "post_rstd", "pre_rstd")}
    want = tb.tropical_residual_norm_backward(q.dy, q.dh, q.u, f.h, **stats, **q.op)
    buf = torch.empty(ld + 8 * 512, dtype=BF16, device=DEV)
    far = [buf[512 * i:].as_strided((2, 300), (ld, 1)) for i in range(8)]
    for t, s in zip(far, (q.u, q.r, q.dy, q.dh)):
        t.copy_(s)
    got = tb.tropical_residual_norm_forward(far[0], far[1], **q.op, h=far[4], y=far[5])
    assert torch.equal(got.h, f.h) and torch.equal(got.y, f.y)
    g = tb.tropical_residual_norm_backward(far[2], far[3], far[0], far[4], **stats, **q.op, dr=far[6], du=far[7])
    assert all(a is None or torch.equal(a, b) for a, b in zip(g, want))


def test_refusals(tb):
    q = Problem(6, 64, F32, F32, "layer", "rms", gates=2)
    f = tb.tropical_residual_norm_forward(q.u, q.r, **q.op)
    stats = {k: getattr(f, k) for k in ("post_mean", "post_rstd", "pre_rstd")}

    def backward(dy=q.dy, dh=q.dh, u=q.u, h=f.h, **kw):
        return tb.tropical_residual_norm_backward(dy, dh, u, h, **{**stats, **q.op, **kw})

    def status(call, *a, **kw):
        with pytest.raises(tb.TropicalError) as e:
            call(*a, **kw)
        return e.value.status

    u8 = tb.tropical_act8_pack(q.u)
    assert status(backward, u=u8) == tb.INVALID_ARGUMENT  # one in 8 bits, one not
    assert status(backward, h=u8) == tb.INVALID_ARGUMENT
    assert status(backward, u=None) == tb.NOT_DEVICE_MEMORY
    assert status(backward, h=None) == tb.NOT_DEVICE_MEMORY
    assert status(backward, dy=None) == tb.NOT_DEVICE_MEMORY
    assert status(backward, pre_rstd=None) == tb.NOT_DEVICE_MEMORY
    assert status(backward, post_mean=None) == tb.NOT_DEVICE_MEMORY
    assert status(backward, workspace=torch.empty(16, dtype=torch.uint8, device=DEV)) == tb.WORKSPACE_TOO_SMALL
    assert status(tb.tropical_residual_norm_forward, q.u.cpu(), q.r, **q.op) == tb.NOT_DEVICE_MEMORY
    wide = torch.zeros(6, 70, device=DEV)
    assert status(tb.tropical_residual_norm_forward, q.u, wide[:, :64], **q.op, h=wide.view(-1)[:384].view(6, 64)) == \
        tb.INVALID_ARGUMENT  # h is r with another stride
    assert status(tb.tropical_residual_norm_forward, q.u, q.r, **{**q.op, "pre_eps": -1.0}) == tb.INVALID_ARGUMENT
    assert status(tb.tropical_residual_norm_forward, q.u, q.r, **{**q.op, "branch_scale": math.inf}) == tb.INVALID_ARGUMENT
    # what is not needed may be left out
    names = dict(dgate=None, dpost_gamma=None, dpost_beta=None)
    g = backward(u=None, du=None, **names)
    assert g.u is None and torch.equal(g.r, backward().r)
    torch.cuda.synchronize()
