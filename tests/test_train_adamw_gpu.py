"""AdamW on the GPU against the formulas in 64 bits, and bit for bit against
the same float32 operations done one at a time on the CPU (the root by numpy,
whose float32 root is the correctly rounded one; torch's CPU root is not).

Tolerances against 64 bits, u = 2^-24: m is two products and a sum of float32
factors (5 u of its terms), v one product more (6 u); the update divides m by
a root and a sum (16 u of its size) and joins q in two more roundings (4 u);
a bfloat16 parameter is rounded once (2^-8 of it).
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
BLOCK = 256


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


def tensors(sizes, dtype, seed, odd_offsets=False):
    """CPU (params, grads, m, v); m and v as after a few steps."""
    g = torch.Generator().manual_seed(seed)
    ps, gs, ms, vs = [], [], [], []
    for i, s in enumerate(sizes):
        ps.append(torch.randn(s, generator=g).to(dtype))
        gs.append((torch.randn(s, generator=g) * 10.0 ** -(i % 5)).to(dtype))
        ms.append(torch.randn(s, generator=g) * 10.0 ** -(i % 5))
        vs.append(torch.rand(s, generator=g) * 100.0 ** -(i % 5))
    return ps, gs, ms, vs


def place(ts, shift):
    """Device copies, each `shift` elements past an allocation's start."""
    out = []
    for t in ts:
        buf = torch.empty(t.numel() + shift, dtype=t.dtype, device=DEV)
        buf[shift:].copy_(t.view(-1))
        out.append(buf[shift:])
    return out


def factors(step, h=HYPER):
    return (h["lr"] / (1 - h["beta1"] ** step), 1 / math.sqrt(1 - h["beta2"] ** step),
            1 - h["lr"] * h["weight_decay"])


def same_operations(q, g, m, v, step, h=HYPER):
    """The header's float32 operations in their order (CPU)."""
    size, root, keep = factors(step, h)
    m = m * h["beta1"] + g * (1 - h["beta1"])
    v = v * h["beta2"] + (g * g) * (1 - h["beta2"])
    denom = torch.from_numpy(np.sqrt(v.numpy())) * root + h["eps"]
    return q * keep - (m / denom) * size, m, v


def check64(q0, g, m0, v0, q, m, v, step, dtype=F32, param=None):
    h = HYPER
    q0, g, m0, v0 = (t.double() for t in (q0, g, m0, v0))
    rm = h["beta1"] * m0 + (1 - h["beta1"]) * g
    rv = h["beta2"] * v0 + (1 - h["beta2"]) * g * g
    tm = 5 * U * (h["beta1"] * m0.abs() + (1 - h["beta1"]) * g.abs())
    tv = 6 * U * rv
    up = h["lr"] * (rm / (1 - h["beta1"] ** step)) / ((rv / (1 - h["beta2"] ** step)).sqrt() + h["eps"])
    rq = (1 - h["lr"] * h["weight_decay"]) * q0 - up
    tq = 16 * U * up.abs() + tm / rm.abs().clamp(min=1e-300) * up.abs() + 4 * U * (q0.abs() + up.abs())
    if m is not None:
        assert ((m.double() - rm).abs() <= tm).all()
        assert ((v.double() - rv).abs() <= tv).all()
    if q is not None:
        assert ((q.double() - rq).abs() <= tq).all()
    if param is not None and dtype == BF16:
        assert ((param.double() - rq).abs() <= tq + 2.0 ** -8 * (rq.abs() + tq)).all()


SIZES = [[1], [0, 5, 0], [4096, 4097, 255, 256, 257], [100003, 3, 1], [2 + 37 * i for i in range(200)]]


@pytest.mark.parametrize("sizes", SIZES, ids=["one", "empty", "edges", "odd", "many"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("shift", [0, 1])
def test_step(tb, sizes, dtype, master, shift):
    ps, gs, ms, vs = tensors(sizes, dtype, len(sizes))
    qs = [p.float() + (1e-3 if master else 0.0) for p in ps]
    P, G, M, V = (place(t, shift) for t in (ps, gs, ms, vs))
    Q = place(qs, shift) if master else None
    tb.tropical_adamw_step(P, G, M, V, step=7, masters=Q, **HYPER)
    torch.cuda.synchronize()
    for i in range(len(sizes)):
        q, m, v = same_operations(qs[i], gs[i].float(), ms[i], vs[i], 7)
        assert torch.equal(M[i].cpu(), m) and torch.equal(V[i].cpu(), v)
        assert torch.equal(P[i].cpu(), q.to(dtype))
        if master:
            assert torch.equal(Q[i].cpu(), q)
        exact32 = Q[i].cpu() if master else (P[i].cpu() if dtype == F32 else None)
        check64(qs[i], gs[i].float(), ms[i], vs[i], exact32, M[i].cpu(), V[i].cpu(), 7, dtype, P[i].cpu())


def codes_m(m):
    """Codes, scales and the real numbers that were rounded, in 64 bits."""
    n = m.numel()
    pad = -n % BLOCK
    b = torch.nn.functional.pad(m.double(), (0, pad)).view(-1, BLOCK)
    a = b.abs().amax(1)
    r = 127 * (b.abs() / torch.where(a > 0, a, 1.0)[:, None]).sqrt()
    return r.view(-1)[:n], a


def codes_v(v):
    n = v.numel()
    pad = -n % BLOCK
    b = torch.nn.functional.pad(v.double(), (0, pad)).view(-1, BLOCK)
    a = b.amax(1)
    r = 255 * (b / torch.where(a > 0, a, 1.0)[:, None]) ** 0.25
    return r.view(-1)[:n], a


def value_m(c, a):
    t = c.double() / 127
    return a.double().repeat_interleave(BLOCK)[:c.numel()] * t * t.abs()


def value_v(c, a):
    return a.double().repeat_interleave(BLOCK)[:c.numel()] * (c.double() / 255) ** 4


@pytest.mark.parametrize("sizes", SIZES, ids=["one", "empty", "edges", "odd", "many"])
@pytest.mark.parametrize("dtype,master", [(F32, False), (F32, True), (BF16, True), (BF16, False)])
@pytest.mark.parametrize("shift", [0, 1])
def test_step_8bit(tb, sizes, dtype, master, shift):
    """Three steps from zero states.  After each, the codes are the rounding
    of the real codes of m and v computed in 64 bits from the codes before:
    equal unless the real code is within 1e-4 of a rounding boundary (its
    float32 evaluation has a relative error below 8 u, 255 * 8 u < 1.3e-4 / 1)."""
    P, G, _, _ = (place(t, shift) for t in tensors(sizes, dtype, 50 + len(sizes)))
    Q = [p.float() for p in P] if master else None
    nb = [-(-s // BLOCK) for s in sizes]
    M = place([torch.zeros(s, dtype=torch.int8) for s in sizes], shift)
    V = place([torch.zeros(s, dtype=torch.uint8) for s in sizes], shift)
    MS = [torch.zeros(n, device=DEV) for n in nb]
    VS = [torch.zeros(n, device=DEV) for n in nb]
    for step in (1, 2, 3):
        before = [(p.cpu().clone(), g.cpu(), m.cpu().clone(), a.cpu().clone(), v.cpu().clone(), b.cpu().clone())
                  for p, g, m, a, v, b in zip(Q if master else P, G, M, MS, V, VS)]
        tb.tropical_adamw8_step(P, G, M, MS, V, VS, step=step, masters=Q, **HYPER)
        mv, vv = tb.tropical_adamw8_unpack(M, MS, V, VS)
        torch.cuda.synchronize()
        for i, (q0, g, m0, a0, v0, b0) in enumerate(before):
            if not sizes[i]:
                continue
            om, ov = value_m(m0, a0), value_v(v0, b0)
            g = g.float()
            q = (Q if master else P)[i].cpu()
            # (states start from codes' float32 values: 4 u more in m and v)
            check64(q0.float(), g, om, ov, q if q.dtype == F32 else None, None, None, step, dtype, P[i].cpu())
            m = HYPER["beta1"] * om + (1 - HYPER["beta1"]) * g.double()
            v = HYPER["beta2"] * ov + (1 - HYPER["beta2"]) * g.double() ** 2
            cm, am = codes_m(m)
            cv, av = codes_v(v)
            assert ((MS[i].cpu().double() - am).abs() <= 12 * U * am).all()
            assert ((VS[i].cpu().double() - av).abs() <= 12 * U * av).all()
            gm, gv = M[i].cpu().double(), V[i].cpu().double()
            # m is a sum of two terms: its own rounding moves the real code too
            slack = 2e-4 + 127 * 0.5 * (12 * U * (om.abs() + g.double().abs())) / m.abs().clamp(min=1e-300)
            assert ((gm.abs() - cm).abs() <= 0.5 + slack.clamp(max=127)).all()
            assert ((gm == 0) | (gm.sign() == m.sign())).all()
            want = torch.where(v > 0, cv.clamp(min=1.0), 0.0)
            assert ((gv - want).abs() <= 0.5 + 2e-4).all() and ((gv > 0) == (v > 0)).all()
            assert ((mv[i].cpu().double() - value_m(M[i].cpu(), MS[i].cpu())).abs() <= 6 * U * am.max()).all()
            assert ((vv[i].cpu().double() - value_v(V[i].cpu(), VS[i].cpu())).abs() <= 8 * U * av.max()).all()


def test_8bit_zero_gradients_and_nonfinite(tb):
    n = 1000
    p = torch.ones(n, device=DEV)
    g = torch.zeros(n, device=DEV)
    m, v = torch.zeros(n, dtype=torch.int8, device=DEV), torch.zeros(n, dtype=torch.uint8, device=DEV)
    ms, vs = torch.zeros(4, device=DEV), torch.zeros(4, device=DEV)
    tb.tropical_adamw8_step([p], [g], [m], [ms], [v], [vs], lr=0.1, step=1)
    assert torch.equal(p, torch.ones_like(p)) and not m.any() and not v.any() and not ms.any() and not vs.any()
    # a NaN gradient spoils its own block and no other
    g.fill_(0.5)
    g[300] = float("nan")
    tb.tropical_adamw8_step([p], [g], [m], [ms], [v], [vs], lr=0.1, step=1)
    mv, vv = tb.tropical_adamw8_unpack([m], [ms], [v], [vs])
    bad = torch.zeros(n, dtype=torch.bool, device=DEV)
    bad[256:512] = True
    assert torch.equal(mv[0].isnan(), bad) and torch.equal(vv[0].isnan(), bad)
    assert p[300].isnan() and torch.isfinite(p[~bad]).all()


def test_8bit_keeps_small_second_moments(tb):
    """A v far below its block's largest keeps a positive code, so that its
    element is never divided by eps alone."""
    g = torch.full((256,), 1e-6, device=DEV)
    g[0] = 1.0
    p = torch.zeros(256, device=DEV)
    m, v = torch.zeros(256, dtype=torch.int8, device=DEV), torch.zeros(256, dtype=torch.uint8, device=DEV)
    ms, vs = torch.zeros(1, device=DEV), torch.zeros(1, device=DEV)
    for step in (1, 2, 3, 4):
        tb.tropical_adamw8_step([p], [g], [m], [ms], [v], [vs], lr=1e-2, step=step)
    assert (v > 0).all() and torch.isfinite(p).all() and p.abs().max() <= 4.5e-2


def test_step_is_repeatable_and_on_another_stream(tb):
    ps, gs, ms, vs = tensors([70001, 33, 4096], F32, 3)
    outs = []
    for stream in (None, torch.cuda.Stream()):
        P, G, M, V = (place(t, 0) for t in (ps, gs, ms, vs))
        torch.cuda.synchronize()
        for step in (1, 2, 3):
            tb.tropical_adamw_step(P, G, M, V, step=step, stream=stream, **HYPER)
        torch.cuda.synchronize()
        outs.append(P + M + V)
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_launches(tb):
    ps, gs, ms, vs = (place(t, 0) for t in tensors([10] * 150, F32, 4))
    tb.tropical_reset_stats()
    tb.tropical_adamw_step(ps, gs, ms, vs, step=1, **HYPER)
    assert tb.tropical_get_train_stats()["launches"]["adamw"] == 3  # 72 tensors a launch
    tb.tropical_adamw_step([], [], [], [], step=1, **HYPER)
    assert tb.tropical_get_train_stats()["launches_total"] == 3


def test_refusals(tb):
    P, G, M, V = (place(t, 0) for t in tensors([64], F32, 1))
    for bad in (dict(beta1=1.0), dict(beta2=-0.1), dict(step=0), dict(lr=float("nan")), dict(eps=-1.0),
                dict(weight_decay=float("inf"))):
        with pytest.raises(tb.TropicalError) as e:
            tb.tropical_adamw_step(P, G, M, V, **{**HYPER, "step": 1, **bad})
        assert e.value.status == tb.INVALID_ARGUMENT
    with pytest.raises(ValueError):
        tb.tropical_adamw_step(P, G, M, [], step=1, **HYPER)
    with pytest.raises(ValueError):
        tb.tropical_adamw_step(P, G, M, [V[0][:63]], step=1, **HYPER)
    with pytest.raises(ValueError):
        tb.tropical_adamw_step(P, [G[0].to(BF16)], M, V, step=1, **HYPER)
    with pytest.raises(tb.TropicalError) as e:
        tb.tropical_adamw_step(P, [G[0].cpu()], M, V, step=1, **HYPER)
    assert e.value.status == tb.NOT_DEVICE_MEMORY and "grad of tensor 0" in str(e.value)
    before = P[0].clone()
    table = (tb.trop_adamw_tensor * 2)()
    table[0] = tb.trop_adamw_tensor(P[0].data_ptr(), G[0].data_ptr(), M[0].data_ptr(), V[0].data_ptr(), None, 64)
    table[1] = tb.trop_adamw_tensor(P[0].data_ptr(), G[0].data_ptr(), M[0].data_ptr(), V[0].data_ptr(), None, -1)
    import ctypes
    h = tb.trop_adamw_hyper(1e-3, 0.9, 0.99, 1e-8, 0.0, 1)
    assert tb.lib().tropical_adamw_step(0, table, 2, ctypes.byref(h), None) == tb.INVALID_ARGUMENT
    table[1].elements = 1 << 36  # past its allocation
    assert tb.lib().tropical_adamw_step(0, table, 2, ctypes.byref(h), None) == tb.INVALID_ARGUMENT
    # master weights for one of two tensors
    table[1].elements = 64
    table[1].master = M[0].data_ptr()
    assert tb.lib().tropical_adamw_step(0, table, 2, ctypes.byref(h), None) == tb.INVALID_ARGUMENT
    torch.cuda.synchronize()
    assert torch.equal(P[0], before)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan"), 1e25])
def test_8bit_infinite_state(tb, bad):
    """An infinite gradient spoils its own block's m and v and no other's; one
    whose square alone overflows spoils v."""
    n = 1000
    g = torch.linspace(-1, 1, n, device=DEV)
    g[400] = 0.0
    g[300] = bad
    p = torch.ones(n, device=DEV)
    m, v = torch.zeros(n, dtype=torch.int8, device=DEV), torch.zeros(n, dtype=torch.uint8, device=DEV)
    ms, vs = torch.zeros(4, device=DEV), torch.zeros(4, device=DEV)
    tb.tropical_adamw8_step([p], [g], [m], [ms], [v], [vs], lr=0.1, step=1)
    mv, vv = tb.tropical_adamw8_unpack([m], [ms], [v], [vs])
    block = torch.zeros(n, dtype=torch.bool, device=DEV)
    block[256:512] = True
    assert torch.equal(vv[0].isnan(), block) and torch.isfinite(vv[0][~block]).all()
    if bad == 1e25:
        assert torch.isfinite(mv[0]).all()
    else:
        assert torch.equal(mv[0].isnan(), block) and torch.isfinite(mv[0][~block]).all()
    assert torch.isfinite(p[~block]).all()
