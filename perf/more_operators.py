"""The operators around a residual block and its saved activations, as their
users call them: the norms after and before a block fused with its gate and
the residual sum, forward and backward; activations held in 8 bits; the weight
gradient of a linear layer whose input was held so.

``listed`` and ``draw`` give cases, ``prepare`` makes what a program holds
before the call, ``run`` is one call of the operator: in elementary torch
operations when ``own`` is false, through the library when it is true.
``exact`` is the same from the definitions in 64 bits.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "bf16": 2}
_BLOCK = 32  # elements of a row that share an exponent
_EPS = 1e-5


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token between two blocks while serving: the smallest call
        dict(name="rn_forward_1x4096_bf16", op="rn", rows=1, cols=4096, pad=0, dtype="bf16", post="rms", pre="rms",
             group=1, held8=False, backward=False),
        # a batch of 29 conditioned samples of 53 rows, a gate vector each, odd widths inside wider buffers
        dict(name="rn_forward_1537x1001_f32", op="rn", rows=1537, cols=1001, pad=7, dtype="f32", post="layer",
             pre="layer", group=53, held8=False, backward=False),
        # a large training batch that leaves its 8-bit activations for the backward
        dict(name="rn_forward_16384x4096_bf16_held8", op="rn", rows=16384, cols=4096, pad=0, dtype="bf16", post="none",
             pre="rms", group=16384, held8=True, backward=False),
        # a training step of a small model that keeps its activations as they are
        dict(name="rn_backward_64x512_f32", op="rn", rows=64, cols=512, pad=0, dtype="f32", post="none", pre="layer",
             group=64, held8=False, backward=True),
        # the conditioned batch's way back, from activations in 8 bits
        dict(name="rn_backward_1537x1001_f32_held8", op="rn", rows=1537, cols=1001, pad=7, dtype="f32", post="layer",
             pre="layer", group=53, held8=True, backward=True),
        # the large training batch's way back with both norms, from activations in 8 bits
        dict(name="rn_backward_16384x4096_bf16_held8", op="rn", rows=16384, cols=4096, pad=0, dtype="bf16", post="rms",
             pre="rms", group=16384, held8=True, backward=True),
        # a small activation put away and taken out again
        dict(name="act8_33x1000_f32", op="act8", rows=33, cols=1000, pad=3, dtype="f32"),
        # the hidden states of a large training batch
        dict(name="act8_16384x4096_bf16", op="act8", rows=16384, cols=4096, pad=0, dtype="bf16"),
        # the weight gradient of a small layer held in 32 bits
        dict(name="grad_w_256x512x512_f32", op="grad_w", tokens=256, cols=512, out=512, pad=0, dtype="f32"),
        # odd sizes throughout
        dict(name="grad_w_1000x1001x777_bf16", op="grad_w", tokens=1000, cols=1001, out=777, pad=3, dtype="bf16"),
        # an ordinary layer in 32 bits
        dict(name="grad_w_4096x1024x4096_f32", op="grad_w", tokens=4096, cols=1024, out=4096, pad=0, dtype="f32"),
        # the widening layer of a large block
        dict(name="grad_w_8192x4096x16384_bf16", op="grad_w", tokens=8192, cols=4096, out=16384, pad=0, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rn", "rn", "rn", "act8", "grad_w", "grad_w"])
    dtype = rng.choice(["f32", "bf16"])
    pad = rng.choice([0, 0, 3, 8])
    if op == "grad_w":
        while True:
            tokens, cols, out = _log_int(rng, 1, 16384), _log_int(rng, 64, 8192), _log_int(rng, 64, 16384)
            if rng.random() < 0.6:
                cols, out = (cols + 63) // 64 * 64, (out + 63) // 64 * 64
            if tokens * cols * out <= 8192 * 4096 * 16384 // (8 if dtype == "f32" else 1):
                break
        return dict(op="grad_w", tokens=tokens, cols=cols, out=out, pad=pad, dtype=dtype)
    most = 16384 * 4096 // (2 if dtype == "f32" else 1)
    while True:
        rows, cols = _log_int(rng, 1, 16384), _log_int(rng, 64, 16384)
        if rng.random() < 0.5:
            cols = (cols + 7) // 8 * 8
        if rows * cols <= most:
            break
    if op == "act8":
        return dict(op="act8", rows=rows, cols=cols, pad=pad, dtype=dtype)
    gates = _log_int(rng, 1, rows)  # from one gate vector for all rows to one for each
    group = max(1, rows // gates)
    rows = rows // group * group
    return dict(op="rn", rows=rows, cols=cols, pad=pad, dtype=dtype, post=rng.choice(["none", "layer", "rms"]),
                pre=rng.choice(["layer", "rms"]), group=group, held8=rng.random() < 0.5, backward=rng.random() < 0.6)


# ---------------------------------------------------------------------------
# 8-bit activations: int8 codes and, for each 32 elements of a row, a power
# of two 2^(e - 127).  The exponent is the smallest with which no magnitude
# rounds past 127.  A block with a NaN or an infinity has e = 255.
# ---------------------------------------------------------------------------

def _power(e):
    """2^(e - 127) as float32, for e in [1, 254]."""
    return (e.int() << 23).view(torch.float32)


def _blocks(x):
    rows, cols = x.shape
    n = -(-cols // _BLOCK)
    if n * _BLOCK != cols:
        x = torch.cat([x, x.new_zeros(rows, n * _BLOCK - cols)], 1)
    return x.view(rows, n, _BLOCK)


def _pack(x):
    """(codes, exponents) of float32 rows."""
    b = _blocks(x)
    bits = b.abs().amax(2).view(torch.int32)
    # a mantissa of 127.5 / 64 or more would round to 128
    e = (((bits + 0x10000) >> 23) - 6).clamp(min=1)
    c = torch.round(b * _power(254 - e)[:, :, None])
    codes = c.reshape(x.shape[0], -1)[:, :x.shape[1]].to(torch.int8)
    return codes.contiguous(), e.to(torch.uint8)


def _values(codes, e):
    """float32; every value is exact in bfloat16 too."""
    v = _blocks(codes.float()) * _power(e)[:, :, None]
    return v.reshape(codes.shape[0], -1)[:, :codes.shape[1]]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def prepare(case, seed):
    g = _gen(seed)
    dev, dt = "cuda", _DT[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    def matrix(rows, cols, offset=0.0, spread=1.0):
        """Rows of a buffer that may be wider."""
        x = randn(rows, cols + case["pad"]) * spread
        if offset:
            x += offset * randn(rows, 1)
        return x.to(dt)[:, :cols]

    def outliers(x):
        """A few channels are much larger than the others, as hidden states have them."""
        scale = torch.ones(x.shape[1], device=dev)
        scale[torch.randint(x.shape[1], (1 + x.shape[1] // 256,), generator=g, device=dev)] = 20.0
        return (x.float() * scale).to(dt)

    if case["op"] == "act8":
        return dict(case=case, x=matrix(case["rows"], case["cols"], 0.5))
    if case["op"] == "grad_w":
        n, c, o = case["tokens"], case["cols"], case["out"]
        # the layer's input, a normed hidden state; gradients of a mean, unequal from token to token
        dz = randn(n, o + case["pad"]) * (randn(n, 1).exp() / n)
        st = dict(case=case, dz=dz.to(dt)[:, :o])
        st["codes"], st["exponents"] = _pack(outliers(randn(n, c)).float())
        return st
    rows, cols = case["rows"], case["cols"]
    par = torch.float32  # weights and gates
    st = dict(case=case, u=matrix(rows, cols, 0.3), residual_scale=1.1, branch_scale=0.5,
              gate=(0.8 + 0.3 * randn(rows // case["group"], cols)).to(par))
    for which in ("post", "pre"):
        if case[which] != "none":
            st[which + "_gamma"] = (1 + 0.1 * randn(cols)).to(par)
            st[which + "_beta"] = (0.1 * randn(cols)).to(par) if case[which] == "layer" else None
    if not case["backward"]:
        st["r"] = matrix(rows, cols, 0.5, 2.0)
        return st
    # what the forward left: h, the statistics of both norms; the gradients that come back
    st["h"] = matrix(rows, cols, 0.5, 2.0)
    for which, x in (("post", st["u"]), ("pre", st["h"])):
        if case[which] != "none":
            _, mean, rstd = _norm(x.float(), case[which])
            if mean is not None:
                st[which + "_mean"] = mean[:, 0].contiguous()
            st[which + "_rstd"] = rstd[:, 0].contiguous()
    st["dy"], st["dh"] = matrix(rows, cols), matrix(rows, cols)
    if case["held8"]:
        st["u8"], st["h8"] = _pack(st.pop("u").float()), _pack(st.pop("h").float())
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _norm(x, kind):
    """(normalised rows, mean or None, rstd)."""
    inv = 1.0 / x.shape[1]
    mean = x.sum(1, keepdim=True) * inv if kind == "layer" else None
    xc = x if mean is None else x - mean
    rstd = 1.0 / ((xc * xc).sum(1, keepdim=True) * inv + _EPS).sqrt()
    return xc * rstd, mean, rstd


def _affine(x, gamma, beta):
    return x * gamma if beta is None else x * gamma + beta


def _plain_forward(st):
    case, dt = st["case"], st["u"].dtype
    rows, cols = st["u"].shape
    out = {}
    u = st["u"].float()
    v = u
    if case["post"] != "none":
        v, mean, rstd = _norm(u, case["post"])
        v = _affine(v, st["post_gamma"], st["post_beta"])
        if mean is not None:
            out["post_mean"] = mean[:, 0]
        out["post_rstd"] = rstd[:, 0]
    gate = (st["gate"] * st["branch_scale"])[:, None, :]
    h = st["r"].float() * st["residual_scale"] + (gate * v.view(-1, case["group"], cols)).view(rows, cols)
    y, mean, rstd = _norm(h, case["pre"])
    if mean is not None:
        out["pre_mean"] = mean[:, 0]
    out["pre_rstd"] = rstd[:, 0]
    out["h"], out["y"] = h.to(dt), _affine(y, st["pre_gamma"], st["pre_beta"]).to(dt)
    if case["held8"]:
        out["u8"] = _values(*_pack(u)).to(torch.bfloat16)
        out["h8"] = _values(*_pack(h)).to(torch.bfloat16)
    return out


def _norm_backward(dy, x, mean, rstd, gamma):
    """(gradient of the norm's input, of gamma, of beta)."""
    inv = 1.0 / x.shape[1]
    xh = (x if mean is None else x - mean[:, None]) * rstd[:, None]
    w = dy * gamma
    c2 = (w * xh).sum(1, keepdim=True) * inv
    dx = w - xh * c2
    if mean is not None:
        dx = dx - w.sum(1, keepdim=True) * inv
    return dx * rstd[:, None], (dy * xh).sum(0), dy.sum(0)


def _plain_backward(st):
    case, dt = st["case"], st["dy"].dtype
    rows, cols = st["dy"].shape
    group = case["group"]
    u = _values(*st["u8"]) if case["held8"] else st["u"].float()
    h = _values(*st["h8"]) if case["held8"] else st["h"].float()
    out = {}
    dh, dgamma, dbeta = _norm_backward(st["dy"].float(), h, st.get("pre_mean"), st["pre_rstd"], st["pre_gamma"])
    dh = dh + st["dh"].float()
    out["pre_gamma"] = dgamma
    if st["pre_beta"] is not None:
        out["pre_beta"] = dbeta
    out["r"] = (dh * st["residual_scale"]).to(dt)
    v = u
    if case["post"] != "none":
        mean, rstd = st.get("post_mean"), st["post_rstd"]
        v = _affine((u if mean is None else u - mean[:, None]) * rstd[:, None], st["post_gamma"], st["post_beta"])
    out["gate"] = (dh * v).view(-1, group, cols).sum(1) * st["branch_scale"]
    dv = (dh.view(-1, group, cols) * (st["gate"] * st["branch_scale"])[:, None, :]).view(rows, cols)
    if case["post"] != "none":
        dv, dgamma, dbeta = _norm_backward(dv, u, mean, rstd, st["post_gamma"])
        out["post_gamma"] = dgamma
        if st["post_beta"] is not None:
            out["post_beta"] = dbeta
    out["u"] = dv.to(dt)
    return out


def _plain_act8(st):
    return dict(values=_values(*_pack(st["x"].float())).to(st["x"].dtype))


def _plain_grad_w(st):
    return dict(grad_w=(st["dz"].float().t() @ _values(st["codes"], st["exponents"])).to(st["dz"].dtype))


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _own_args(st):
    case = st["case"]
    return dict(gate=st["gate"], post=None if case["post"] == "none" else case["post"], pre=case["pre"],
                post_gamma=st.get("post_gamma"), post_beta=st.get("post_beta"), pre_gamma=st["pre_gamma"],
                pre_beta=st["pre_beta"], residual_scale=st["residual_scale"], branch_scale=st["branch_scale"])


def _own_forward(st):
    from tropical_semiring_tensor_amd import binding as tb
    f = tb.tropical_residual_norm_forward(st["u"], st["r"], post_eps=_EPS, pre_eps=_EPS, hold_u=st["case"]["held8"],
                                          hold_h=st["case"]["held8"], **_own_args(st))
    out = {}
    for name in ("post_mean", "post_rstd", "pre_mean", "pre_rstd", "h", "y"):
        if getattr(f, name) is not None:
            out[name] = getattr(f, name)
    if f.u8 is not None:
        out["u8"] = tb.tropical_act8_unpack(f.u8, torch.bfloat16)
        out["h8"] = tb.tropical_act8_unpack(f.h8, torch.bfloat16)
    return out


def _own_backward(st):
    from tropical_semiring_tensor_amd import binding as tb
    case = st["case"]
    u, h = (tb.Act8(*st["u8"]), tb.Act8(*st["h8"])) if case["held8"] else (st["u"], st["h"])
    f = tb.tropical_residual_norm_backward(
        st["dy"], st["dh"], u, h, post_mean=st.get("post_mean"), post_rstd=st.get("post_rstd"),
        pre_mean=st.get("pre_mean"), pre_rstd=st["pre_rstd"], **_own_args(st))
    out = dict(pre_gamma=f.pre_gamma)
    if st["pre_beta"] is not None:
        out["pre_beta"] = f.pre_beta
    out.update(r=f.r, gate=f.gate)
    if case["post"] != "none":
        out["post_gamma"] = f.post_gamma
        if st["post_beta"] is not None:
            out["post_beta"] = f.post_beta
    out["u"] = f.u
    return out


def _own_act8(st):
    from tropical_semiring_tensor_amd import binding as tb
    return dict(values=tb.tropical_act8_unpack(tb.tropical_act8_pack(st["x"]), st["x"].dtype))


def _own_grad_w(st):
    from tropical_semiring_tensor_amd import binding as tb
    return dict(grad_w=tb.tropical_act8_linear_grad_w(st["dz"], tb.Act8(st["codes"], st["exponents"])))


def run(state):
    case = state["case"]
    what = {"rn": "backward" if case.get("backward") else "forward"}.get(case["op"], case["op"])
    if own:
        return {"forward": _own_forward, "backward": _own_backward, "act8": _own_act8,
                "grad_w": _own_grad_w}[what](state)
    return {"forward": _plain_forward, "backward": _plain_backward, "act8": _plain_act8,
            "grad_w": _plain_grad_w}[what](state)


# ---------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------

def work(case):
    s = _BYTES[case["dtype"]]
    held = 1 + 1 / _BLOCK  # bytes of an element in 8 bits
    if case["op"] == "grad_w":
        n, c, o = case["tokens"], case["cols"], case["out"]
        return {"bytes": int(n * o * s + n * c * held + o * c * s), "flops": 2 * n * c * o}
    e = case["rows"] * case["cols"]
    if case["op"] == "act8":  # rows read, held, and written again as values
        return {"bytes": int(e * (2 * s + 2 * held)), "flops": 6 * e}
    norms = (case["post"] != "none") + (case["pre"] != "none")
    vectors = 4 * case["cols"] * (2 * norms + case["rows"] // case["group"]) + 8 * case["rows"] * norms
    if not case["backward"]:
        # r and u read, h and y written; held activations written, and returned as 16-bit values
        return {"bytes": int(e * (4 * s + (2 * (held + held + 2) if case["held8"] else 0)) + vectors),
                "flops": (4 + 6 * norms) * e}
    # the gradients of y and h read, those of r and u written, u and h read; vectors and their gradients
    return {"bytes": int(e * (4 * s + 2 * (held if case["held8"] else s)) + 2 * vectors), "flops": (8 + 12 * norms) * e}


def _exact_values(packed):
    codes, e = packed
    scale = torch.ldexp(torch.ones((), dtype=torch.float64, device=codes.device), e.int() - 127)
    return codes.to(torch.float64) * scale.repeat_interleave(_BLOCK, 1)[:, :codes.shape[1]]


def _exact_hold(x):
    """64-bit rows rounded to their 8-bit values: the block's step is the
    smallest power of two that keeps round(x / step) within 127."""
    n = -(-x.shape[1] // _BLOCK)
    a = torch.nn.functional.pad(x, (0, n * _BLOCK - x.shape[1])).view(x.shape[0], n, _BLOCK).abs().amax(2)
    e = torch.ceil(torch.log2(torch.where(a > 0, a, 1.0) / 127.5))
    e = torch.where(a * torch.exp2(-e) >= 127.5, e + 1, e)  # (a tie rounds to 128)
    step = torch.exp2(e.clamp(min=-126)).repeat_interleave(_BLOCK, 1)[:, :x.shape[1]]
    return torch.round(x / step) * step


def exact(case, seed):
    st = prepare(case, seed)
    f8 = torch.float64
    if case["op"] == "act8":
        return dict(values=_exact_hold(st["x"].to(f8)))
    if case["op"] == "grad_w":
        return dict(grad_w=torch.mm(st["dz"].to(f8).t(), _exact_values((st["codes"], st["exponents"]))))
    cols = case["cols"]
    gate = st["branch_scale"] * st["gate"].to(f8).repeat_interleave(case["group"], 0)

    def weights(which):
        g, b = st[which + "_gamma"].to(f8), st[which + "_beta"]
        return g, torch.zeros_like(g) if b is None else b.to(f8)

    if not case["backward"]:
        out = {}

        def normed(x, which):
            mean = x.mean(1) if case[which] == "layer" else None
            xc = x if mean is None else x - mean[:, None]
            rstd = (torch.linalg.vecdot(xc, xc) / cols + _EPS) ** -0.5
            if mean is not None:
                out[which + "_mean"] = mean
            out[which + "_rstd"] = rstd
            g, b = weights(which)
            return torch.addcmul(b, xc * rstd[:, None], g)

        u = st["u"].to(f8)
        v = u if case["post"] == "none" else normed(u, "post")
        h = torch.addcmul(st["residual_scale"] * st["r"].to(f8), gate, v)
        y = normed(h, "pre")
        out["h"], out["y"] = h, y
        if case["held8"]:
            out["u8"], out["h8"] = _exact_hold(u), _exact_hold(h)
        return out
    u, h = (_exact_values(st[k + "8"]) if case["held8"] else st[k].to(f8) for k in ("u", "h"))

    def standard(x, which):
        m = st.get(which + "_mean")
        return (x if m is None else x - m.to(f8)[:, None]) * st[which + "_rstd"].to(f8)[:, None]

    def through(dy, xh, which):
        """The Jacobian of the norm's row applied to its output's gradient."""
        w = dy * weights(which)[0]
        if case[which] == "layer":
            w = w - w.mean(1, keepdim=True) - xh * (torch.linalg.vecdot(dy * weights(which)[0], xh)[:, None] / cols)
        else:
            w = w - xh * (torch.linalg.vecdot(w, xh)[:, None] / cols)
        return w * st[which + "_rstd"].to(f8)[:, None]

    dy = st["dy"].to(f8)
    hh = standard(h, "pre")
    out = dict(pre_gamma=torch.linalg.vecdot(dy, hh, dim=0))
    if st["pre_beta"] is not None:
        out["pre_beta"] = dy.sum(0)
    dh = through(dy, hh, "pre") + st["dh"].to(f8)
    out["r"] = st["residual_scale"] * dh
    uh = v = u
    if case["post"] != "none":
        uh = standard(u, "post")
        g, b = weights("post")
        v = torch.addcmul(b, uh, g)
    out["gate"] = st["branch_scale"] * (dh * v).unflatten(0, (-1, case["group"])).sum(1)
    dv = dh * gate
    if case["post"] != "none":
        out["post_gamma"] = torch.linalg.vecdot(dv, uh, dim=0)
        if st["post_beta"] is not None:
            out["post_beta"] = dv.sum(0)
        dv = through(dv, uh, "post")
    out["u"] = dv
    return out
