"""Activations in 8 bits and the weight gradient from them on the GPU.

The 8-bit form is compared bit for bit: codes, exponents and values follow
from the elements alone.  The weight gradient's products are exact (a code has
7 bits, float32 gradients are cut into three bfloat16 values), so only sums
round.  With u = 2^-24: a matrix instruction adds 32 terms to its sum, float32
tokens pass three times, parts of the sum join at the end, so a term meets at
most 3 tokens / 32 + 32 + 32 roundings, each at most 2 u (the instruction's
own sums may truncate); the result's rounding to its type follows.
"""
import math
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda:0"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
BLOCK = 32


@pytest.fixture(scope="module")
def tb():
    from tropical_semiring_tensor_amd import binding
    binding.tropical_train_init(0)
    yield binding
    torch.cuda.synchronize()
    torch._C._cuda_clearCublasWorkspaces()
    torch.cuda.empty_cache()


def reference_pack(x):
    """(codes, exponents, values) of a CPU matrix, block by block in 64 bits."""
    rows, cols = x.shape
    n = -(-cols // BLOCK)
    x = torch.nn.functional.pad(x.double(), (0, n * BLOCK - cols)).view(rows, n, BLOCK)
    bad = ~torch.isfinite(x).all(2)
    a = torch.where(bad, 0.0, x.abs().amax(2))
    _, e = torch.frexp(a)  # a = m 2^e, m in [1/2, 1)
    e = torch.where(a > 0, e, -1000) - 7 + 127
    e = torch.where(torch.round(a * torch.exp2((127 - e).clamp(max=900).double())) > 127, e + 1, e).clamp(1, 248)
    step = torch.exp2((e - 127).double())[:, :, None]
    c = torch.where(bad[:, :, None], 0.0, torch.round(x / step).clamp(-127, 127))
    v = torch.where(bad[:, :, None], math.nan, c * step)
    e = torch.where(bad, 255, e)
    flat = lambda t: t.reshape(rows, n * BLOCK)[:, :cols]  # noqa: E731
    return flat(c).to(torch.int8), e.to(torch.uint8), flat(v)


def same(a, b):
    return a.shape == b.shape and bool(((a == b) | (a.isnan() & b.isnan())).all())


def padded(x, pad, fill):
    """x as a view of a wider device buffer."""
    buf = torch.full((x.shape[0], x.shape[1] + pad), fill, dtype=x.dtype)
    buf[:, :x.shape[1]] = x
    return buf.to(DEV)[:, :x.shape[1]]


SHAPES = [(1, 1), (3, 31), (2, 32), (5, 33), (7, 64), (4, 1000), (3, 1024), (2, 1025), (33, 4096), (2, 20001),
          (2049, 24), (1, 100000)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad", [0, 3])
def test_pack_and_unpack(tb, rows, cols, dtype, pad):
    g = torch.Generator().manual_seed(rows * 1009 + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-30, 30, (rows, 1), generator=g).float())
    x[0] *= torch.linspace(0, 1, cols) ** 8  # blocks of every magnitude
    x = x.to(dtype)
    codes, exps, values = reference_pack(x)
    out = tb.Act8(torch.full((rows, cols + pad), 77, dtype=torch.int8, device=DEV)[:, :cols],
                  torch.full((rows, exps.shape[1] + pad), 77, dtype=torch.uint8, device=DEV)[:, :exps.shape[1]])
    got = tb.tropical_act8_pack(padded(x, pad, math.nan), out if pad else None)
    assert torch.equal(got.codes.cpu(), codes) and torch.equal(got.exponents.cpu(), exps)
    for ty in (F32, BF16):
        buf = torch.full((rows, cols + pad), 5.0, dtype=ty, device=DEV)
        tb.tropical_act8_unpack(got, out=buf[:, :cols])
        assert same(buf[:, :cols].cpu().double(), values)
        assert (buf[:, cols:] == 5.0).all()
    assert same(tb.tropical_act8_unpack(got).cpu().double(), values)
    if pad:  # nothing beside the rows is touched
        assert (out.codes._base[:, cols:] == 77).all() and (out.exponents._base[:, exps.shape[1]:] == 77).all()


def test_pack_borders(tb):
    """Ties, the magnitudes where the exponent changes, the ends of the range,
    zeros, infinities and NaN."""
    f = torch.finfo(F32)
    rows = []
    for a in (127.0, 127.49, 127.5, 127.51, 128.0, 63.75, 64.0, 1.0, 2.0 ** -120, 2.0 ** -126, 2.0 ** -140, f.max,
              f.tiny, 0.0):
        step = a / 127 if a else 0.0
        rows.append(torch.tensor([a, -a, a / 2, -a / 3, 0.0, -0.0] + [step * (i + 0.5) for i in range(26)]))
    for bad in (math.inf, -math.inf, math.nan):
        rows.append(torch.tensor([1.0] * 31 + [bad]))
    rows.append(torch.tensor([0.5 + i for i in range(31)] + [100.0]))  # halves between codes at a step of 1
    x = torch.stack(rows).float()
    codes, exps, values = reference_pack(x)
    got = tb.tropical_act8_pack(x.to(DEV))
    assert torch.equal(got.exponents.cpu(), exps)
    assert torch.equal(got.codes.cpu(), codes)
    assert same(tb.tropical_act8_unpack(got).cpu().double(), values)
    # a block's NaN stays in its block
    x = torch.ones(1, 96)
    x[0, 40] = math.nan
    v = tb.tropical_act8_unpack(tb.tropical_act8_pack(x.to(DEV)))
    assert v[0, 32:64].isnan().all() and (v[0, :32] == 1).all() and (v[0, 64:] == 1).all()


def test_values_are_within_their_bound(tb):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(64, 640, generator=g).to(DEV)
    v = tb.tropical_act8_unpack(tb.tropical_act8_pack(x))
    a = x.view(64, 20, 32).abs().amax(2, keepdim=True)
    assert ((v - x).abs().view(64, 20, 32) <= a / 127).all()
    # packing the values again changes nothing
    again = tb.tropical_act8_pack(v)
    assert torch.equal(tb.tropical_act8_unpack(again), v)


def held(tb, x):
    return tb.tropical_act8_pack(x.to(DEV))


def check_grad_w(tb, dz, x8, grad_w=None, **kw):
    got = tb.tropical_act8_linear_grad_w(dz, x8, grad_w, **kw)
    d, x = dz.double(), tb.tropical_act8_unpack(x8).double()
    want, scale = d.t().mm(x), d.abs().t().mm(x.abs())
    n = dz.shape[0]
    tol = (3 * n / 32 + 64) * 2 * U * scale
    tol = tol + torch.finfo(dz.dtype).eps / 2 * (want.abs() + tol)
    err = (got.double() - want).abs()
    assert not (~(err <= tol)).any(), f"{int((~(err <= tol)).sum())} of {err.numel()}, worst {float((err - tol).max())}"
    return got


GRAD_SHAPES = [
    (1, 1, 1), (1, 40, 7), (2, 64, 64), (63, 33, 65), (64, 100, 256), (65, 256, 100), (300, 130, 70),
    (1000, 1001, 777), (129, 2000, 8), (700, 300, 1000), (5000, 64, 64), (20000, 72, 40), (256, 4100, 2000),
]


@pytest.mark.parametrize("tokens,cols,outs", GRAD_SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad", [0, 5])
def test_grad_w(tb, tokens, cols, outs, dtype, pad):
    g = torch.Generator().manual_seed(tokens * 31 + cols * 7 + outs)
    x8 = held(tb, torch.randn(tokens, cols, generator=g) * (1 + 9 * (torch.rand(1, cols, generator=g) > 0.95)))
    # gradients of very unequal tokens and features
    dz = torch.randn(tokens, outs, generator=g) * torch.exp(torch.randn(tokens, 1, generator=g))
    dz *= torch.exp2(torch.randint(-20, 20, (1, outs), generator=g).float())
    dz = padded(dz.to(dtype), pad, math.nan)
    out = torch.full((outs, cols + pad), 5.0, dtype=dtype, device=DEV)
    check_grad_w(tb, dz, x8, out[:, :cols])
    assert (out[:, cols:] == 5.0).all()
    # the same bits again, and from a workspace of any alignment
    need = tb.tropical_act8_linear_grad_w_workspace_size(dtype, tokens, cols, outs)
    ws = torch.full((need + 1,), 255, dtype=torch.uint8, device=DEV)[1:]
    assert torch.equal(tb.tropical_act8_linear_grad_w(dz, x8, workspace=ws), out[:, :cols])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_grad_w_in_pieces(tb, dtype):
    """More tokens than a piece of 256 MiB holds of all columns, and more
    output features than one holds of float32."""
    g = torch.Generator(device=DEV).manual_seed(9)
    tokens, cols, outs = (300000, 600, 40) if dtype == BF16 else (100000, 72, 600)
    x8 = tb.tropical_act8_pack(torch.randn(tokens, cols, generator=g, device=DEV))
    dz = torch.randn(tokens, outs, generator=g, device=DEV).to(dtype)
    check_grad_w(tb, dz, x8)


def test_grad_w_of_nothing(tb):
    x8 = held(tb, torch.zeros(0, 40))
    out = torch.full((7, 40), 3.0, device=DEV)
    tb.tropical_act8_linear_grad_w(torch.zeros(0, 7, device=DEV), x8, out)
    assert (out == 0).all()
    assert tb.tropical_act8_linear_grad_w(torch.zeros(4, 0, device=DEV), held(tb, torch.zeros(4, 8))).shape == (0, 8)
    assert tb.tropical_act8_linear_grad_w(torch.zeros(4, 3, device=DEV), held(tb, torch.zeros(4, 0))).shape == (3, 0)
    assert tb.tropical_act8_pack(torch.zeros(0, 8, device=DEV)).exponents.shape == (0, 1)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_grad_w_float_range(tb, dtype):
    """Gradients next to the ends of float32's range, and x in tiny steps."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(40, 64, generator=g)
    for scale_x, scale_d in ((1e-4, 1e38), (1e30, 1e-30), (1.0, 1e-30)):
        dz = (torch.rand(40, 16, generator=g) * 3).to(dtype) * scale_d
        check_grad_w(tb, dz.to(DEV), held(tb, x * scale_x))


def test_grad_w_non_finite_stays_in_its_place(tb):
    g = torch.Generator().manual_seed(2)
    for dtype, tokens in ((F32, 70), (BF16, 70), (BF16, 64)):
        dz = torch.randn(tokens, 24, generator=g).to(dtype)
        x = torch.randn(tokens, 96, generator=g)
        dz[tokens - 1, 5] = math.inf
        dz[3, 6] = math.nan
        x[10, 40] = math.nan
        got = tb.tropical_act8_linear_grad_w(dz.to(DEV), held(tb, x))
        bad = torch.zeros(24, 96, dtype=torch.bool)
        bad[5] = bad[6] = True
        bad[:, 32:64] = True
        assert torch.equal(~torch.isfinite(got).cpu(), bad)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_grad_w_against_differences(tb, dtype):
    """The gradient of sum(dz z), z = x w^T, along a direction in w: linear in
    w, so the difference quotient is the product itself in 64 bits."""
    g = torch.Generator().manual_seed(4)
    x8 = held(tb, torch.randn(90, 50, generator=g))
    dz = torch.randn(90, 30, generator=g).to(dtype).to(DEV)
    got = tb.tropical_act8_linear_grad_w(dz, x8).double()
    x, d = tb.tropical_act8_unpack(x8).double(), dz.double()
    w = torch.randn(30, 50, generator=g).double().to(DEV)
    step = torch.randn(30, 50, generator=g).double().to(DEV)
    f = lambda m: float((d * (x @ m.t().contiguous())).sum())  # noqa: E731
    diff = (f(w + 0.5 * step) - f(w - 0.5 * step))
    bound = (d.abs().t().mm(x.abs()) * step.abs()).sum() * (64 * 2 * U) + (got.abs() * step.abs()).sum() * (
        torch.finfo(dtype).eps / 2 + 1e-12)
    assert abs(float((got * step).sum()) - diff) <= float(bound)


def test_graph_and_streams(tb):
    """A captured pack, gradient and unpack, replayed between eager work, and
    calls on a second stream."""
    g = torch.Generator(device=DEV).manual_seed(6)
    x = torch.randn(500, 300, generator=g, device=DEV)
    dz = torch.randn(500, 200, generator=g, device=DEV)
    x8 = tb.tropical_act8_pack(x)
    gw, values = torch.empty(200, 300, device=DEV), torch.empty_like(x)
    ws = torch.empty(tb.tropical_act8_linear_grad_w_workspace_size(F32, 500, 300, 200), dtype=torch.uint8, device=DEV)

    def step():
        tb.tropical_act8_pack(x, x8)
        tb.tropical_act8_linear_grad_w(dz, x8, gw, workspace=ws)
        tb.tropical_act8_unpack(x8, out=values)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        x.copy_(torch.randn(500, 300, generator=g, device=DEV))
        dz.copy_(torch.randn(500, 200, generator=g, device=DEV))
        want8 = tb.tropical_act8_pack(x)
        want = tb.tropical_act8_linear_grad_w(dz, want8)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(gw, want) and torch.equal(values, tb.tropical_act8_unpack(want8))
    side.wait_stream(torch.cuda.current_stream())
    out8 = tb.tropical_act8_pack(x, stream=side)
    out = tb.tropical_act8_linear_grad_w(dz, out8, stream=side)
    side.synchronize()
    assert torch.equal(out, gw)


def test_each_code_object_is_loaded_by_its_first_call():
    """A layer norm loads its own code object, 8-bit activations theirs."""
    program = """
import torch
from tropical_semiring_tensor_amd import binding as tb
x = torch.randn(4, 64, device="cuda:0")
loads = [tb.tropical_get_train_stats()["module_loads"]]
tb.tropical_layer_norm_forward(x)
loads.append(tb.tropical_get_train_stats()["module_loads"])
for _ in range(2):
    tb.tropical_act8_pack(x)
    loads.append(tb.tropical_get_train_stats()["module_loads"])
tb.tropical_train_init(0)
loads.append(tb.tropical_get_train_stats()["module_loads"])
torch.cuda.synchronize()
print("LOADS", *loads)
"""
    out = subprocess.run([sys.executable, "-c", program], capture_output=True, text=True, timeout=110, cwd=ROOT)
    assert out.returncode == 0 and "LOADS 0 1 2 2 2" in out.stdout, out.stdout + out.stderr


def test_offsets_past_32_bits(tb):
    """Rows that lie more than 2^32 elements apart."""
    ld = (1 << 32) + 64
    buf = torch.empty(ld + 100, dtype=BF16, device=DEV)
    x = buf.as_strided((2, 100), (ld, 1))
    x.copy_(torch.randn(2, 100, device=DEV))
    codes = torch.empty(ld + 100, dtype=torch.int8, device=DEV).as_strided((2, 100), (ld, 1))
    exps = torch.empty((2, 4), dtype=torch.uint8, device=DEV)
    got = tb.tropical_act8_pack(x, tb.Act8(codes, exps))
    want = tb.tropical_act8_pack(x.contiguous())
    assert torch.equal(got.codes.contiguous(), want.codes) and torch.equal(exps, want.exponents)
    gw = tb.tropical_act8_linear_grad_w(x, got)  # (a row stride that the product cannot take: dz is packed)
    assert torch.equal(gw, tb.tropical_act8_linear_grad_w(x.contiguous(), want))


def test_refusals(tb):
    x = torch.zeros(8, 64, device=DEV)
    x8 = tb.tropical_act8_pack(x)
    with pytest.raises(tb.TropicalError) as e:
        tb.tropical_act8_pack(torch.zeros(8, 64))
    assert e.value.status == tb.NOT_DEVICE_MEMORY
    with pytest.raises(ValueError):
        tb.tropical_act8_pack(x, tb.Act8(x8.codes[:, :63], x8.exponents))
    with pytest.raises(ValueError):
        tb.tropical_act8_pack(x, tb.Act8(x8.codes, x8.exponents[:, :1]))
    with pytest.raises(ValueError):
        tb.tropical_act8_pack(x.t())
    with pytest.raises(TypeError):
        tb.tropical_act8_unpack(x8, torch.float16)
    with pytest.raises(ValueError):
        tb.tropical_act8_linear_grad_w(torch.zeros(7, 4, device=DEV), x8)
    with pytest.raises(tb.TropicalError) as e:
        tb.tropical_act8_linear_grad_w(torch.zeros(8, 4, device=DEV), x8,
                                       workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
    assert e.value.status == tb.WORKSPACE_TOO_SMALL
    # rows that reach past the end of their allocation (a stated stride too large)
    big = torch.zeros(1 << 22, dtype=torch.uint8, device=DEV)
    a = tb.trop_act8(big.data_ptr(), x8.exponents.data_ptr(), 1 << 40, 2)
    assert tb.lib().tropical_act8_pack(0, x.data_ptr(), 64, a, 8, 64, None) == tb.INVALID_ARGUMENT
    a = tb.trop_act8(x8.codes.data_ptr(), x8.exponents.data_ptr(), 64, 1)
    assert tb.lib().tropical_act8_pack(0, x.data_ptr(), 64, a, 8, 64, None) == tb.INVALID_ARGUMENT
    torch.cuda.synchronize()
