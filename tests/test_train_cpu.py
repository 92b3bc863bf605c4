"""The training operators on the CPU: argument checks that precede any device
call, workspace sizes, and the binding's own checks.  No kernel runs."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def tb():
    import os

    from tropical_semiring_tensor_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from tropical_semiring_tensor_amd.csrc import build
        build.build()
    binding.lib()
    return binding


def test_layer_norm_argument_errors(tb):
    L = tb.lib()
    fwd = L.tropical_layer_norm_forward
    ok = [0, 0, None, 8, None, None, 1e-5, None, 8, None, None, 4, 8, None]

    def call(**kw):
        names = ["dtype", "pdtype", "x", "ldx", "gamma", "beta", "eps", "y", "ldy", "mean", "rstd", "rows", "cols",
                 "stream"]
        args = list(ok)
        for k, v in kw.items():
            args[names.index(k)] = v
        return fwd(*args)

    assert call(dtype=1) == tb.INVALID_ARGUMENT and "float32 or bfloat16" in tb.tropical_last_error()
    assert call(dtype=7) == tb.INVALID_ARGUMENT
    assert call(pdtype=2) == tb.INVALID_ARGUMENT  # float32 rows, bfloat16 weights
    assert call(rows=-1) == tb.INVALID_ARGUMENT and call(cols=-1) == tb.INVALID_ARGUMENT
    for eps in (-1.0, float("nan"), float("inf")):
        assert call(eps=eps) == tb.INVALID_ARGUMENT and "eps" in tb.tropical_last_error()
    # nothing to do: before any pointer or device is looked at
    assert call(rows=0) == tb.OK and call(cols=0) == tb.OK and tb.tropical_last_error() == ""
    bwd = L.tropical_layer_norm_backward
    assert bwd(0, 0, None, 8, None, 8, None, None, None, None, 8, None, None, 4, 8, None, 0, None) == tb.OK
    assert bwd(1, 0, None, 8, None, 8, None, None, None, None, 8, None, None, 4, 8, None, 0, None) == tb.INVALID_ARGUMENT


def test_layer_norm_workspace(tb):
    ws = tb.tropical_layer_norm_backward_workspace_size
    assert ws(100, 64, with_params=False) == 0
    assert ws(0, 64) == 0
    assert ws(100, 64) == 25 * 2 * 64 * 4        # four rows to a workgroup up to 1024 columns
    assert ws(100, 1025) == 100 * 2 * 1025 * 4   # one
    assert ws(10 ** 6, 4096) == 512 * 2 * 4096 * 4
    with pytest.raises(tb.TropicalError) as e:
        ws(-1, 4)
    assert e.value.status == tb.INVALID_ARGUMENT
    with pytest.raises(tb.TropicalError):
        ws(10 ** 6, 2 ** 60)
    assert tb.lib().tropical_layer_norm_backward_workspace_size(4, 4, 1, None) == tb.INVALID_ARGUMENT


def test_cross_entropy_argument_errors(tb):
    L = tb.lib()

    def fwd(dtype=0, tbytes=8, tokens=4, width=8, vocab=16):
        return L.tropical_linear_cross_entropy_forward(dtype, None, width, None, width, None, tbytes, -100, None, None,
                                                       tokens, width, vocab, None, 0, None)

    def bwd(dtype=0, tbytes=8, tokens=4, width=8, vocab=16, gstride=1):
        return L.tropical_linear_cross_entropy_backward(dtype, None, width, None, width, None, tbytes, -100, None,
                                                        None, gstride, None, width, None, width, tokens, width, vocab,
                                                        None, 0, None)

    for f in (fwd, bwd):
        assert f(dtype=1) == tb.INVALID_ARGUMENT
        assert f(tbytes=2) == tb.INVALID_ARGUMENT and "4 or 8" in tb.tropical_last_error()
        assert f(tokens=-1) == tb.INVALID_ARGUMENT and f(vocab=-1) == tb.INVALID_ARGUMENT
        assert f(vocab=0) == tb.INVALID_ARGUMENT and f(width=0) == tb.INVALID_ARGUMENT
        assert f(tokens=2 ** 23) == tb.UNSUPPORTED and f(width=2 ** 23) == tb.UNSUPPORTED
        assert f(vocab=2 ** 31) == tb.UNSUPPORTED
        assert f(tokens=0, vocab=0) == tb.OK
    assert bwd(gstride=-1) == tb.INVALID_ARGUMENT
    assert bwd() == tb.OK  # neither gradient asked for


def test_cross_entropy_workspace(tb):
    ws = tb.tropical_linear_cross_entropy_workspace_size
    f32, bf16 = torch.float32, torch.bfloat16
    # few tokens: statistics per 16 or 32 labels, the targets' logits; 256 bytes to align
    assert ws(bf16, 1, 4096, 65536) == 256 + 2048 * 8 + 256
    assert ws(f32, 3, 64, 100) == 256 + 256 + 256
    assert ws(f32, 0, 64, 100) == 0
    assert ws(f32, 0, 64, 100, backward=True) > 0  # grad_w is zeroed
    # bounded by pieces of the label set: far below the logits
    for dt, size in ((f32, 4), (bf16, 2)):
        n = ws(dt, 8192, 4096, 262144, backward=True)
        assert n < 2 ** 31 < 8192 * 262144 * size
    # more labels cost no more than a piece (statistics aside)
    assert ws(bf16, 8192, 4096, 2 ** 20, backward=True) <= ws(bf16, 8192, 4096, 2 ** 18, backward=True) + 2 ** 26
    with pytest.raises(TypeError):
        ws(torch.int32, 4, 4, 4)
    with pytest.raises(tb.TropicalError):
        ws(f32, -1, 4, 4)
    L = tb.lib()
    assert L.tropical_linear_cross_entropy_workspace_size(0, 4, 4, 4, 0, None) == tb.INVALID_ARGUMENT
    # any size is answered without overflow
    nb = ctypes.c_size_t(0)
    for t in (1, 64, 65, 2 ** 22):
        for w in (1, 2 ** 22):
            for v in (1, 2 ** 31 - 600):
                for d in (0, 2):
                    for b in (0, 1):
                        st = L.tropical_linear_cross_entropy_workspace_size(d, t, w, v, b, ctypes.byref(nb))
                        assert st == tb.OK and 0 < nb.value < 2 ** 62


def test_adamw_argument_errors(tb):
    L = tb.lib()

    def hyper(**kw):
        h = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1)
        h.update(kw)
        return tb.trop_adamw_hyper(**h)

    for fn, kind in ((L.tropical_adamw_step, tb.trop_adamw_tensor), (L.tropical_adamw8_step, tb.trop_adamw8_tensor)):
        t = (kind * 2)()
        h = hyper()
        assert fn(0, None, 0, ctypes.byref(h), None) == tb.OK
        assert fn(0, t, 2, ctypes.byref(h), None) == tb.OK  # no elements
        assert fn(1, t, 2, ctypes.byref(h), None) == tb.INVALID_ARGUMENT
        assert fn(0, None, 2, ctypes.byref(h), None) == tb.INVALID_ARGUMENT
        assert fn(0, t, -1, ctypes.byref(h), None) == tb.INVALID_ARGUMENT
        assert fn(0, t, 2, None, None) == tb.INVALID_ARGUMENT
        for bad in (dict(step=0), dict(beta1=1.0), dict(beta2=-1e-3), dict(beta1=float("nan")), dict(lr=-1.0),
                    dict(lr=float("inf")), dict(eps=float("nan")), dict(weight_decay=-0.1)):
            b = hyper(**bad)
            assert fn(0, t, 2, ctypes.byref(b), None) == tb.INVALID_ARGUMENT, bad
        t[1].elements = -5
        assert fn(0, t, 2, ctypes.byref(h), None) == tb.INVALID_ARGUMENT
        assert "tensor 1" in tb.tropical_last_error()
        t[1].elements = 2 ** 50
        assert fn(0, t, 2, ctypes.byref(h), None) == tb.INVALID_ARGUMENT
    assert L.tropical_adamw8_unpack(None, 0, None, None, None) == tb.OK
    assert L.tropical_adamw8_unpack(None, 3, None, None, None) == tb.INVALID_ARGUMENT


def test_binding_checks(tb):
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        tb.tropical_layer_norm_forward(x.int())
    with pytest.raises(ValueError):
        tb.tropical_layer_norm_forward(torch.zeros(8))
    with pytest.raises(ValueError):
        tb.tropical_adamw_step([x], [x], [x], [x[:2]], lr=1e-3)
    with pytest.raises(ValueError):
        tb.tropical_adamw_step([x], [x, x], [x], [x], lr=1e-3)
    with pytest.raises(ValueError):
        tb.tropical_adamw8_step([x], [x], [x], [x], [x], [x], lr=1e-3)
    with pytest.raises(ValueError):  # not contiguous
        tb.tropical_adamw_step([x.t()], [x.t()], [x], [x], lr=1e-3)
    assert tb.tropical_adamw8_unpack([], [], [], []) == ([], [])
    s = tb.tropical_get_train_stats()
    assert set(s["launches"]) == set(tb.TRAIN_FAMILIES) and s["launches_total"] == sum(s["launches"].values())


def test_contraction_calls_refuse_bfloat16(tb):
    L = tb.lib()
    s = tb.trop_strides(1, 1, 1)
    assert L.tropical_gemm_strided_batched(0, 2, None, s, None, s, None, s, None, 1, 1, 1, 1, None) == tb.INVALID_ARGUMENT
    assert L.tropical_tree_plan_create(0, 2, 0, None, None, None, 0, None, None) != tb.OK
    with pytest.raises(TypeError):
        tb.tropical_gemm_strided_batched("max_plus", torch.zeros(2, 2, dtype=torch.bfloat16),
                                         torch.zeros(2, 2, dtype=torch.bfloat16), torch.zeros(2, 2))


def test_training_code_object_is_gfx950_only():
    import os

    from tropical_semiring_tensor_amd.csrc import build
    co = os.path.join(build.BUILD, "train_kernels.co")
    if not os.path.exists(co):
        build.build()
    data = open(co, "rb").read()
    assert data[:4] == b"\x7fELF" and b"gfx950" in data
    for other in (b"gfx90a", b"gfx942", b"gfx1100"):
        assert other not in data
