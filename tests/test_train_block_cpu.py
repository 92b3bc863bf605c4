"""The operators around a residual block on the CPU: argument checks that
precede any device call, workspace sizes, and the binding's own checks.  No
kernel runs."""
import ctypes
import math

import pytest
import torch

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def tb():
    import os

    from tropical_semiring_tensor_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from tropical_semiring_tensor_amd.csrc import build
        build.build()
    binding.lib()
    return binding


def test_act8_argument_errors(tb):
    L = tb.lib()
    a = tb.trop_act8(None, None, 64, 2)
    for f in (lambda dt=0, rows=4, cols=64, a=a: L.tropical_act8_pack(dt, None, 64, a, rows, cols, None),
              lambda dt=0, rows=4, cols=64, a=a: L.tropical_act8_unpack(a, dt, None, 64, rows, cols, None)):
        assert f(dt=1) == tb.INVALID_ARGUMENT and "float32 or bfloat16" in tb.tropical_last_error()
        assert f(rows=-1) == tb.INVALID_ARGUMENT and f(cols=-1) == tb.INVALID_ARGUMENT
        assert f(a=None) == tb.INVALID_ARGUMENT and "NULL" in tb.tropical_last_error()
        # nothing to do: before any pointer or device is looked at
        assert f(rows=0) == tb.OK and f(cols=0) == tb.OK and tb.tropical_last_error() == ""


def test_grad_w_argument_errors(tb):
    L = tb.lib()
    a = tb.trop_act8(None, None, 64, 2)

    def f(dt=0, tokens=4, cols=64, outs=8, x=a):
        return L.tropical_act8_linear_grad_w(dt, None, 8, x, None, 64, tokens, cols, outs, None, 0, None)

    assert f(dt=1) == tb.INVALID_ARGUMENT and f(x=None) == tb.INVALID_ARGUMENT
    assert f(tokens=-1) == tb.INVALID_ARGUMENT and f(cols=-1) == tb.INVALID_ARGUMENT and f(outs=-1) == tb.INVALID_ARGUMENT
    assert f(tokens=2 ** 22 + 1) == tb.UNSUPPORTED and f(cols=2 ** 23) == tb.UNSUPPORTED
    assert f(outs=2 ** 23) == tb.UNSUPPORTED
    assert f(cols=0) == tb.OK and f(outs=0) == tb.OK


def test_grad_w_workspace(tb):
    ws = tb.tropical_act8_linear_grad_w_workspace_size
    # x as bfloat16 at least, dz packed once (bfloat16) or in three parts
    assert ws(BF16, 64, 64, 64) >= 2 * 64 * 64 * 2
    assert ws(F32, 64, 64, 64) >= 64 * 64 * 2 + 64 * 64 * 6
    assert ws(F32, 0, 64, 64) == 0 and ws(F32, 64, 0, 64) == 0 and ws(F32, 64, 64, 0) == 0
    # pieces: bounded however wide the layer is
    assert ws(BF16, 8192, 2 ** 20, 2 ** 20) < 2 ** 31
    assert ws(F32, 8192, 2 ** 20, 2 ** 20) < 2 ** 31
    with pytest.raises(TypeError):
        ws(torch.int32, 4, 4, 4)
    with pytest.raises(tb.TropicalError):
        ws(F32, -1, 4, 4)
    L = tb.lib()
    assert L.tropical_act8_linear_grad_w_workspace_size(0, 4, 4, 4, None) == tb.INVALID_ARGUMENT
    nb = ctypes.c_size_t(0)
    for t in (1, 64, 65, 2 ** 22):
        for c in (1, 2 ** 22):
            for o in (1, 2 ** 22):
                for d in (0, 2):
                    st = L.tropical_act8_linear_grad_w_workspace_size(d, t, c, o, ctypes.byref(nb))
                    assert st == tb.OK and 0 < nb.value < 2 ** 62


def op(tb, **kw):
    o = tb.trop_residual_norm(0, 0, 0, 1, 2, 1.0, 1.0, 1e-5, 1e-5, 4, 64, None, 0, 0)
    for k, v in kw.items():
        setattr(o, k, v)
    return o


def bad_ops(tb):
    return [op(tb, dtype=1), op(tb, param_dtype=2), op(tb, post=3), op(tb, pre=-1), op(tb, rows=-1), op(tb, cols=-1),
            op(tb, residual_scale=math.inf), op(tb, branch_scale=math.nan), op(tb, post_eps=-1.0),
            op(tb, pre_eps=math.inf), op(tb, gate=4096, gate_group=0), op(tb, gate=4096, gate_group=1, gate_dtype=2)]


def test_residual_norm_argument_errors(tb):
    L = tb.lib()
    none = (ctypes.c_uint64 * 14)()
    grads = (ctypes.c_uint64 * 10)()
    for o in bad_ops(tb):
        assert L.tropical_residual_norm_forward(o, none, None) == tb.INVALID_ARGUMENT
        assert L.tropical_residual_norm_backward(o, none, grads, None, 0, None) == tb.INVALID_ARGUMENT
    good = op(tb)
    assert L.tropical_residual_norm_forward(None, none, None) == tb.INVALID_ARGUMENT
    assert L.tropical_residual_norm_forward(good, None, None) == tb.INVALID_ARGUMENT
    assert L.tropical_residual_norm_backward(good, None, grads, None, 0, None) == tb.INVALID_ARGUMENT
    assert L.tropical_residual_norm_backward(good, none, None, None, 0, None) == tb.INVALID_ARGUMENT
    # nothing to do
    assert L.tropical_residual_norm_forward(op(tb, rows=0), none, None) == tb.OK
    assert L.tropical_residual_norm_forward(op(tb, cols=0), none, None) == tb.OK
    assert L.tropical_residual_norm_backward(good, none, grads, None, 0, None) == tb.OK  # no gradient asked for
    # a y, gradients or a dy of a norm that is not there
    y = (ctypes.c_uint64 * 14)(0, 0, 0, 0, 0, 0, 4096, 64)
    assert L.tropical_residual_norm_forward(op(tb, pre=0), y, None) == tb.INVALID_ARGUMENT
    for field, norm in ((6, "post"), (7, "post"), (8, "pre"), (9, "pre")):
        g = (ctypes.c_uint64 * 10)()
        g[field] = 4096
        assert L.tropical_residual_norm_backward(op(tb, **{norm: 0}), none, g, None, 0, None) == tb.INVALID_ARGUMENT
    g = (ctypes.c_uint64 * 10)()
    g[4] = 4096  # a gate's gradient without a gate
    assert L.tropical_residual_norm_backward(good, none, g, None, 0, None) == tb.INVALID_ARGUMENT
    dy = (ctypes.c_uint64 * 14)(*[0] * 10, 4096, 64)
    assert L.tropical_residual_norm_backward(op(tb, pre=0), dy, grads, None, 0, None) == tb.INVALID_ARGUMENT
    a = tb.trop_act8(4096, 4096, 64, 2)
    both = (ctypes.c_uint64 * 14)(4096, 64, 0, 0, ctypes.addressof(a))
    assert L.tropical_residual_norm_backward(good, both, grads, None, 0, None) == tb.INVALID_ARGUMENT


def test_residual_norm_workspace(tb):
    ws = tb.tropical_residual_norm_backward_workspace_size
    assert ws(F32, 0, 64) == 0 and ws(F32, 100, 64, None, None) == 0
    # two sums for each norm, one for the gate, in parts of four rows at least
    assert ws(BF16, 100, 64) == 25 * 2 * 64 * 4
    assert ws(BF16, 100, 64, "rms", "rms") == 25 * 4 * 64 * 4
    assert ws(BF16, 100, 64, "rms", "rms", gate_group=100) == 25 * 5 * 64 * 4
    assert ws(BF16, 100, 64, "rms", "rms", gate_group=10) == 10 * 3 * 5 * 64 * 4  # three parts to a gate row
    # more gate rows than parts: the parts write their gradients themselves
    assert ws(F32, 4096, 64, "rms", "rms", gate_group=1) == 512 * 4 * 64 * 4
    assert ws(F32, 10 ** 6, 4096, "layer", "layer") == 512 * 4 * 4096 * 4
    # rows too wide for the registers also keep two means each
    assert ws(F32, 1000, 20000) == 125 * 2 * 20000 * 4 + 1000 * 8
    for bad in (dict(rows=-1), dict(cols=-1), dict(gate_group=0)):
        with pytest.raises(tb.TropicalError) as e:
            ws(**{**dict(dtype=F32, rows=4, cols=4), **bad})
        assert e.value.status == tb.INVALID_ARGUMENT
    with pytest.raises(tb.TropicalError):
        ws(F32, 10 ** 6, 2 ** 60)
    with pytest.raises(TypeError):
        ws(torch.float16, 4, 4)
    with pytest.raises(ValueError):
        ws(F32, 4, 4, "batch")
    L = tb.lib()
    assert L.tropical_residual_norm_backward_workspace_size(op(tb), None) == tb.INVALID_ARGUMENT
    nb = ctypes.c_size_t(0)
    assert L.tropical_residual_norm_backward_workspace_size(None, ctypes.byref(nb)) == tb.INVALID_ARGUMENT
    # any size is answered without overflow
    for rows in (1, 5, 513, 10 ** 9):
        for cols in (1, 8, 8192, 8193, 2 ** 31):
            for group in (None, 1, 3, 2 ** 62):
                assert 0 < ws(BF16, rows, cols, "layer", "rms", gate_group=group) < 2 ** 62


def test_binding_checks(tb):
    x = torch.zeros(6, 64)
    fwd, bwd = tb.tropical_residual_norm_forward, tb.tropical_residual_norm_backward
    v = torch.zeros(64)
    for kw in (dict(post="batch"), dict(pre="l2"), dict(post_gamma=v), dict(pre=None, pre_beta=v),
               dict(pre_gamma=v[:63]), dict(pre_gamma=torch.zeros(128)[::2]), dict(gate=v[:5]),
               dict(gate=torch.zeros(4, 64)), dict(gate=torch.zeros(2, 64), gate_group=2),
               dict(gate=torch.zeros(2, 63)), dict(r=x[:5]), dict(r=x.bfloat16()), dict(h=x[:5]),
               dict(pre=None, y=x), dict(hold_u=tb.Act8(x, x))):
        with pytest.raises(ValueError):
            fwd(x, **kw)
    with pytest.raises(ValueError):  # weights of two types
        fwd(x.bfloat16(), pre_gamma=v, pre_beta=v.bfloat16())
    for bad in (x.int(), x.half()):
        with pytest.raises(TypeError):
            fwd(bad)
    with pytest.raises(TypeError):
        fwd(x, gate=v.half())
    with pytest.raises(ValueError):
        fwd(torch.zeros(64))
    with pytest.raises(ValueError):
        fwd(x.t())
    with pytest.raises(ValueError):
        bwd(None, None, x, x)
    for kw in (dict(u=x[:5]), dict(h=x.bfloat16()), dict(dh=x[:, :63]), dict(pre_rstd=v), dict(dgate=v),
               dict(dr=x[:5]), dict(gate=v, dgate=v[:5]), dict(dpre_gamma=v[:5])):
        with pytest.raises(ValueError):
            bwd(**{**dict(dy=x, dh=x, u=x, h=x), **kw})
    codes, exps = torch.zeros(6, 64, dtype=torch.int8), torch.zeros(6, 2, dtype=torch.uint8)
    for a in (tb.Act8(codes.int(), exps), tb.Act8(codes, exps.int()), tb.Act8(codes[:5], exps), tb.Act8(codes, exps[:, :1]),
              tb.Act8(codes.t().contiguous().t(), exps)):
        with pytest.raises(ValueError):
            tb.tropical_act8_pack(x, a)
    with pytest.raises(TypeError):
        tb.tropical_act8_pack(x.half())
    with pytest.raises(TypeError):
        tb.tropical_act8_unpack(tb.Act8(codes, exps), torch.float16)
    with pytest.raises(ValueError):
        tb.tropical_act8_linear_grad_w(torch.zeros(5, 3), tb.Act8(codes, exps))
    with pytest.raises(ValueError):
        tb.tropical_act8_linear_grad_w(x, tb.Act8(codes, exps), grad_w=torch.zeros(64, 63))
    with pytest.raises(TypeError):
        tb.tropical_act8_linear_grad_w(x.half(), tb.Act8(codes, exps))


@pytest.mark.parametrize("shape,kw", [((64,), {}), ((3, 64), dict(gate_group=5)), ((0, 64), {})])
def test_gate_gradient_without_rows(tb, monkeypatch, shape, kw):
    """An empty batch: the library has no gate row to write, the gradient of a
    gate that is there all the same is zero.  Asked for alone, which needs no
    device."""
    monkeypatch.setattr(tb, "_stream_ptr", lambda stream, t: None)
    x, gate = torch.zeros(0, 64), torch.ones(shape)
    others = dict(dr=None, du=None, dpost_gamma=None, dpost_beta=None, dpre_gamma=None, dpre_beta=None)
    for dgate in (torch.full(shape, 5.0), torch.full(shape, math.nan)):
        g = tb.tropical_residual_norm_backward(x, x, x, x, gate=gate, dgate=dgate, **others, **kw)
        assert g.gate is dgate and bool((dgate == 0).all())
    g = tb.tropical_residual_norm_backward(x, x, x, x, gate=gate, **others, **kw)
    assert g.gate.shape == gate.shape and bool((g.gate == 0).all())


@pytest.mark.parametrize("gates", [1, 3])
def test_gate_rows_without_rows(tb, monkeypatch, gates):
    """Gate rows whose batch is empty are taken as a gate vector is: each is for
    none of the rows."""
    monkeypatch.setattr(tb, "_stream_ptr", lambda stream, t: None)
    x, gate = torch.zeros(0, 64), torch.ones(gates, 64)
    f = tb.tropical_residual_norm_forward(x, x, gate=gate, post="rms")
    assert f.h.shape == f.y.shape == x.shape
    others = dict(dr=None, du=None, dpost_gamma=None, dpost_beta=None, dpre_gamma=None, dpre_beta=None)
    g = tb.tropical_residual_norm_backward(x, x, x, x, gate=gate, dgate=torch.full((gates, 64), 5.0), **others)
    assert bool((g.gate == 0).all())
    # a width or a group that no batch has is refused all the same
    for kw in (dict(gate=torch.ones(gates, 63)), dict(gate=gate, gate_group=0)):
        with pytest.raises(ValueError):
            tb.tropical_residual_norm_forward(x, x, **kw)
    # and so are gate rows that do not divide the rows there are
    with pytest.raises(ValueError):
        tb.tropical_residual_norm_forward(torch.zeros(gates + 1, 64), gate=torch.ones(gates + 2, 64))


@pytest.mark.parametrize("n", [0, 1, 5, 64])
@pytest.mark.parametrize("there", [(True, True, True, True), (True, False, True, True), (False, True, False, True)])
def test_new_vectors_are_tensors_of_their_own(tb, there, n):
    """Vectors that a call allocates together: no views of one another's matrix,
    so each may be changed in place, by what needs a gradient too, while
    another is kept for a backward."""
    v = tb._new_flats(there, n, F32, torch.device("cpu"))
    assert [t is not None for t in v] == list(there)
    v = [t for t in v if t is not None]
    for k, t in enumerate(v):
        assert t.shape == (n,) and t.is_contiguous() and t.dtype == F32 and not t._is_view()
        t.fill_(float(k))
    assert all(bool((t == k).all()) for k, t in enumerate(v))
    a = torch.ones(n, requires_grad=True)
    kept = v[0].clone()
    out = (a * v[0]).sum()
    for t in v[1:]:
        t.zero_()
    out.backward()
    assert torch.equal(a.grad, kept)
    v[1].add_(torch.ones(n, requires_grad=True))
    assert v[1].requires_grad and not v[0].requires_grad


def test_code_object_is_gfx950_only():
    import os

    from tropical_semiring_tensor_amd.csrc import build
    co = os.path.join(build.BUILD, "block_kernels.co")
    if not os.path.exists(co):
        build.build()
    data = open(co, "rb").read()
    assert data[:4] == b"\x7fELF" and b"gfx950" in data
    for other in (b"gfx90a", b"gfx942", b"gfx1100"):
        assert other not in data
