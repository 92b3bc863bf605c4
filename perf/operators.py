"""The training-step operators as their users call them: layer norm, softmax
cross entropy over a large label set, AdamW over many tensors.

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
_BLOCK = 256  # elements that share a scale of the 8-bit optimiser state


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token on its way through a norm while serving: the smallest call
        dict(name="ln_forward_1x4096_bf16", op="ln", rows=1, cols=4096, pad=0, dtype="bf16", train=False),
        # a training batch whose width is odd and whose rows lie in a wider buffer
        dict(name="ln_train_1537x1001_f32", op="ln", rows=1537, cols=1001, pad=7, dtype="f32", train=True),
        # the norm of a large training batch
        dict(name="ln_train_16384x4096_bf16", op="ln", rows=16384, cols=4096, pad=0, dtype="bf16", train=True),
        # scoring one token over a large vocabulary: one read of the weight
        dict(name="ce_score_1x4096x65536_bf16", op="ce", tokens=1, width=4096, vocab=65536, dtype="bf16",
             ignored=0.0, train=False),
        # scoring a few tokens over a small label set
        dict(name="ce_score_48x512x4099_f32", op="ce", tokens=48, width=512, vocab=4099, dtype="f32",
             ignored=0.0, train=False),
        # a training step of a small classifier held in 32 bits
        dict(name="ce_train_256x512x8000_f32", op="ce", tokens=256, width=512, vocab=8000, dtype="f32",
             ignored=0.0, train=True),
        # odd sizes throughout, a third of the tokens masked out of the loss
        dict(name="ce_train_1000x1000x50001_bf16", op="ce", tokens=1000, width=1000, vocab=50001, dtype="bf16",
             ignored=0.33, train=True),
        # an ordinary training step in 32 bits
        dict(name="ce_train_4096x1024x32768_f32", op="ce", tokens=4096, width=1024, vocab=32768, dtype="f32",
             ignored=0.05, train=True),
        # the largest training step
        dict(name="ce_train_8192x4096x65536_bf16", op="ce", tokens=8192, width=4096, vocab=65536, dtype="bf16",
             ignored=0.05, train=True),
        # the site tensors of the 5 x 5 lattice network with bonds of 16: 25 tensors of 256 to 65536 elements
        dict(name="adamw_lattice_25_f32", op="adamw", tensors=25, largest=65536, dtype="f32", state="f32"),
        # a model in 16 bits with 32-bit master weights: matrices and small vectors, 170 million elements or so
        dict(name="adamw_96_bf16_master", op="adamw", tensors=96, largest=16777216, dtype="bf16", state="f32"),
        # the same in 32 bits with the state held in 8
        dict(name="adamw_96_f32_state8", op="adamw", tensors=96, largest=16777216, dtype="f32", state="8bit"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ln", "ce", "ce", "adamw"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "ln":
        while True:
            rows, cols = _log_int(rng, 1, 16384), _log_int(rng, 64, 8192)
            if rng.random() < 0.5:
                cols = (cols + 7) // 8 * 8
            if rows * cols <= 16384 * 4096:
                break
        return dict(op="ln", rows=rows, cols=cols, pad=rng.choice([0, 0, 3, 8]), dtype=dtype,
                    train=rng.random() < 0.7)
    if op == "ce":
        while True:
            tokens, width, vocab = _log_int(rng, 1, 8192), _log_int(rng, 64, 4096), _log_int(rng, 256, 65536)
            if rng.random() < 0.6:
                width = (width + 63) // 64 * 64
            flops = tokens * width * vocab
            if flops <= 4096 * 1024 * 32768 * (1 if dtype == "f32" else 8):
                break
        return dict(op="ce", tokens=tokens, width=width, vocab=vocab, dtype=dtype,
                    ignored=rng.choice([0.0, 0.05, 0.4]), train=rng.random() < 0.7)
    state = rng.choice(["f32", "8bit"])
    return dict(op="adamw", tensors=_log_int(rng, 1, 96), largest=_log_int(rng, 4096, 16777216), dtype=dtype,
                state=state)


def _sizes(case):
    """Element counts of an AdamW case's tensors: from `largest` down in
    powers of two and back, every third a vector, every fifth odd; the
    lattice's own for 25 tensors up to 65536."""
    n, big = case["tensors"], case["largest"]
    if n == 25 and big == 65536:  # 5 x 5 sites: two bonds in a corner, three on an edge, four inside
        bonds = [4 - (r in (0, 4)) - (c in (0, 4)) for r in range(5) for c in range(5)]
        return [16 ** b for b in bonds]
    out = []
    for i in range(n):
        s = max(1, big >> (i * 5 % 7))
        if i % 3 == 2:
            s = max(1, math.isqrt(s))
        if i % 5 == 4:
            s = s - s // 9 | 1
        out.append(s)
    return out


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def prepare(case, seed):
    g = _gen(seed)
    dev = "cuda"
    dt = _DT.get(case["dtype"])
    if case["op"] == "ln":
        rows, cols, ld = case["rows"], case["cols"], case["cols"] + case["pad"]
        # hidden states: unit spread about an offset of their own per row
        x = torch.randn(rows, ld, generator=g, device=dev)
        x += torch.randn(rows, 1, generator=g, device=dev)
        st = dict(case=case, x=x.to(dt)[:, :cols],
                  gamma=(1 + 0.1 * torch.randn(cols, generator=g, device=dev)).to(dt),
                  beta=(0.1 * torch.randn(cols, generator=g, device=dev)).to(dt))
        if case["train"]:
            st["dy"] = torch.randn(rows, ld, generator=g, device=dev).to(dt)[:, :cols]
        return st
    if case["op"] == "ce":
        n, d, v = case["tokens"], case["width"], case["vocab"]
        # normalised hidden states, logits with a spread of about 2
        x = torch.randn(n, d, generator=g, device=dev).to(dt)
        w = (torch.randn(v, d, generator=g, device=dev) * (2 / math.sqrt(d))).to(dt)
        # small labels are more frequent than large ones
        t = (v * torch.rand(n, generator=g, device=dev) ** 3).long().clamp_(max=v - 1)
        if case["ignored"]:
            t[torch.rand(n, generator=g, device=dev) < case["ignored"]] = -100
        st = dict(case=case, x=x, w=w, target=t)
        if case["train"]:  # the gradient of the mean over the tokens that count
            count = (t >= 0).sum().clamp(min=1)
            st["grad_loss"] = torch.ones(n, device=dev) / count
        return st
    # parameters, gradients and state live in one buffer each, as programs that bucket them keep them
    sizes = _sizes(case)
    st = dict(case=case, step=100, flat={}, masters=None,
              hyper=dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01))

    def hold(name, dtype):
        st["flat"][name], st[name] = _buffer(sizes, dtype)

    eight = case["state"] == "8bit"
    for name in ("params", "grads"):
        hold(name, dt)
    if dt != torch.float32:
        hold("masters", torch.float32)
    hold("m_value" if eight else "m", torch.float32)
    hold("v_value" if eight else "v", torch.float32)
    if eight:
        hold("m", torch.int8)
        hold("v", torch.uint8)
        st["m_scale"] = [torch.empty(-(-s // _BLOCK), device=dev) for s in sizes]
        st["v_scale"] = [torch.empty(-(-s // _BLOCK), device=dev) for s in sizes]
    for i, s in enumerate(sizes):
        spread = 10.0 ** -(2 + i % 4)  # gradients of layers at different depths
        p = 0.05 * torch.randn(s, generator=g, device=dev)
        grad = torch.randn(s, generator=g, device=dev) * spread
        m = 0.3 * grad + 0.1 * torch.randn(s, generator=g, device=dev) * spread
        v = grad * grad * 0.5 + 0.5 * spread ** 2 * torch.rand(s, generator=g, device=dev)
        st["params"][i].copy_(p)
        st["grads"][i].copy_(grad)
        if st["masters"] is not None:
            st["masters"][i].copy_(p)
        if eight:
            for name, (c, a) in (("m", _quantise_m(m)), ("v", _quantise_v(v))):
                st[name][i].copy_(c)
                st[name + "_scale"][i].copy_(a)
        else:
            st["m"][i].copy_(m)
            st["v"][i].copy_(v)
    return st


def _buffer(sizes, dtype):
    """One buffer for tensors of these sizes, each at a multiple of a block."""
    starts = [0]
    for s in sizes:
        starts.append(starts[-1] + -(-s // _BLOCK) * _BLOCK)
    flat = torch.zeros(starts[-1], dtype=dtype, device="cuda")
    return flat, [flat[o:o + s] for o, s in zip(starts, sizes)]


def _adamw_outputs(st, flat):
    """The buffers that a step has changed; 8-bit states as their values."""
    names = ["params"] + (["masters"] if st["masters"] is not None else [])
    names += ["m_value", "v_value"] if st["case"]["state"] == "8bit" else ["m", "v"]
    return {name: flat[name] for name in names}


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _blocks(t):
    """t as rows of one block each, the last one filled up with zeros."""
    n = t.numel()
    nb = (n + _BLOCK - 1) // _BLOCK
    if nb * _BLOCK != n:
        t = torch.cat([t, t.new_zeros(nb * _BLOCK - n)])
    return t.view(nb, _BLOCK)


def _quantise_m(m):
    """Signed 8-bit codes c with m about a (c / 127) |c / 127|, a the block's
    largest magnitude."""
    b = _blocks(m)
    a = b.abs().amax(1)
    ratio = b.abs() / torch.where(a > 0, a, 1.0)[:, None]
    c = torch.round(ratio.sqrt() * 127.0) * b.sign()
    return c.view(-1)[:m.numel()].to(torch.int8), a


def _value_m(c, a):
    t = _blocks(c.to(a.dtype)) * torch.tensor(1 / 127, dtype=torch.float32).item()
    return ((a[:, None] * t) * t.abs()).view(-1)[:c.numel()]


def _quantise_v(v):
    """Unsigned 8-bit codes c with v about a (c / 255)^4, a the block's
    largest; a positive value keeps a positive code."""
    b = _blocks(v)
    a = b.amax(1)
    ratio = b / torch.where(a > 0, a, 1.0)[:, None]
    c = torch.round(ratio.sqrt().sqrt() * 255.0)
    c = torch.where(b > 0, c.clamp(min=1.0), 0.0)
    return c.view(-1)[:v.numel()].to(torch.uint8), a


def _value_v(c, a):
    t = _blocks(c.to(a.dtype)) * torch.tensor(1 / 255, dtype=torch.float32).item()
    t2 = t * t
    return (a[:, None] * (t2 * t2)).view(-1)[:c.numel()]


def _plain_ln(st):
    x, gamma, beta = st["x"].float(), st["gamma"].float(), st["beta"].float()
    inv = 1.0 / x.shape[1]
    mean = x.sum(1) * inv
    xc = x - mean[:, None]
    rstd = 1.0 / ((xc * xc).sum(1) * inv + 1e-5).sqrt()
    xh = xc * rstd[:, None]
    y = xh * gamma + beta
    out = dict(y=y.to(st["x"].dtype), mean=mean, rstd=rstd)
    if "dy" in st:
        dy = st["dy"].float()
        w = dy * gamma
        c1 = w.sum(1, keepdim=True) * inv
        c2 = (w * xh).sum(1, keepdim=True) * inv
        out["dx"] = ((w - c1 - xh * c2) * rstd[:, None]).to(st["x"].dtype)
        out["dgamma"] = (dy * xh).sum(0).to(st["gamma"].dtype)
        out["dbeta"] = dy.sum(0).to(st["beta"].dtype)
    return out


def _plain_ce(st):
    x, w, t = st["x"].float(), st["w"].float(), st["target"]
    valid = (t >= 0) & (t < w.shape[0])
    idx = torch.where(valid, t, 0)[:, None]
    logits = x @ w.t()
    top = logits.amax(1, keepdim=True)
    lse = top + (logits - top).exp().sum(1, keepdim=True).log()
    loss = torch.where(valid, (lse - logits.gather(1, idx))[:, 0], 0.0)
    out = dict(loss=loss, lse=torch.where(valid, lse[:, 0], 0.0))
    if "grad_loss" in st:
        p = (logits - lse).exp()
        p.scatter_add_(1, idx, torch.full_like(lse, -1.0))
        p = p * torch.where(valid, st["grad_loss"], 0.0)[:, None]
        out["grad_x"] = (p @ w).to(st["x"].dtype)
        out["grad_w"] = (p.t() @ torch.where(valid[:, None], x, 0.0)).to(st["w"].dtype)
    return out


def _plain_adamw(st):
    h, step = st["hyper"], st["step"]
    b1, b2 = h["beta1"], h["beta2"]
    step_size = h["lr"] / (1 - b1 ** step)
    root = 1 / math.sqrt(1 - b2 ** step)
    keep = 1 - h["lr"] * h["weight_decay"]
    eight = st["case"]["state"] == "8bit"
    for i, (p, g) in enumerate(zip(st["params"], st["grads"])):
        q = p if st["masters"] is None else st["masters"][i]
        g = g.float()
        m = _value_m(st["m"][i], st["m_scale"][i]) if eight else st["m"][i]
        v = _value_v(st["v"][i], st["v_scale"][i]) if eight else st["v"][i]
        m = m * b1 + g * (1 - b1)
        v = v * b2 + (g * g) * (1 - b2)
        q.copy_(q * keep - (m / (v.sqrt() * root + h["eps"])) * step_size)
        if q is not p:
            p.copy_(q)
        if eight:
            for name, (c, a), value in (("m", _quantise_m(m), _value_m), ("v", _quantise_v(v), _value_v)):
                st[name][i].copy_(c)
                st[name + "_scale"][i].copy_(a)
                st[name + "_value"][i].copy_(value(c, a))
        else:
            st["m"][i].copy_(m)
            st["v"][i].copy_(v)
    return _adamw_outputs(st, st["flat"])


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _own_ln(st):
    from tropical_semiring_tensor_amd import binding as tb
    y, mean, rstd = tb.tropical_layer_norm_forward(st["x"], st["gamma"], st["beta"], eps=1e-5)
    out = dict(y=y, mean=mean, rstd=rstd)
    if "dy" in st:
        out["dx"], out["dgamma"], out["dbeta"] = tb.tropical_layer_norm_backward(
            st["dy"], st["x"], mean, rstd, st["gamma"])
    return out


def _own_ce(st):
    from tropical_semiring_tensor_amd import binding as tb
    loss, lse = tb.tropical_linear_cross_entropy_forward(st["x"], st["w"], st["target"])
    out = dict(loss=loss, lse=lse)
    if "grad_loss" in st:
        out["grad_x"], out["grad_w"] = tb.tropical_linear_cross_entropy_backward(
            st["x"], st["w"], st["target"], lse, st["grad_loss"])
    return out


def _own_adamw(st):
    from tropical_semiring_tensor_amd import binding as tb
    if st["case"]["state"] == "8bit":
        tb.tropical_adamw8_step(st["params"], st["grads"], st["m"], st["m_scale"], st["v"], st["v_scale"],
                                step=st["step"], masters=st["masters"], **st["hyper"])
        tb.tropical_adamw8_unpack(st["m"], st["m_scale"], st["v"], st["v_scale"], st["m_value"], st["v_value"])
    else:
        tb.tropical_adamw_step(st["params"], st["grads"], st["m"], st["v"], step=st["step"],
                               masters=st["masters"], **st["hyper"])
    return _adamw_outputs(st, st["flat"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"ln": _own_ln, "ce": _own_ce, "adamw": _own_adamw}[op](state)
    return {"ln": _plain_ln, "ce": _plain_ce, "adamw": _plain_adamw}[op](state)


# ---------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------

def work(case):
    s = _BYTES[case["dtype"]]
    if case["op"] == "ln":
        r, c = case["rows"], case["cols"]
        if not case["train"]:
            return {"bytes": 2 * r * c * s + 8 * r + 2 * c * s, "flops": 8 * r * c}
        # x and dy read, y and dx written; the statistics and the weights' gradients
        return {"bytes": 4 * r * c * s + 8 * r + 4 * c * s, "flops": 22 * r * c}
    if case["op"] == "ce":
        n, d, v = case["tokens"], case["width"], case["vocab"]
        if not case["train"]:
            return {"bytes": (n * d + v * d) * s + 16 * n, "flops": 2 * n * d * v}
        # the tokens that count; logits, the gradient of x and that of the weight: one product each
        kept = n * (1 - case["ignored"])
        return {"bytes": 2 * (n * d + v * d) * s + 20 * n, "flops": 6 * kept * d * v}
    e = sum(_sizes(case))
    per = 2 * s + s  # parameter read (or its 16-bit copy written) and written, gradient read
    if case["dtype"] == "bf16":
        per = 2 * s + 8  # gradient read, parameter written; the master weight read and written
    # the state read and written; 8-bit states are also returned as values
    per += 16 if case["state"] == "f32" else 4 + 8
    return {"bytes": per * e, "flops": 15 * e}


def exact(case, seed):
    st = prepare(case, seed)
    f8 = torch.float64
    if case["op"] == "ln":
        x, gamma, beta = st["x"].to(f8), st["gamma"].to(f8), st["beta"].to(f8)
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + 1e-5) ** -0.5
        xh = (x - mean[:, None]) * rstd[:, None]
        out = dict(y=torch.addcmul(beta, xh, gamma), mean=mean, rstd=rstd)
        if case["train"]:
            dy = st["dy"].to(f8)
            # the Jacobian of the normalised row applied to gamma dy
            w = gamma * dy
            proj = torch.linalg.vecdot(w, xh)[:, None] / x.shape[1]
            out["dx"] = rstd[:, None] * (w - w.mean(1, keepdim=True) - proj * xh)
            out["dgamma"] = torch.linalg.vecdot(dy, xh, dim=0)
            out["dbeta"] = dy.sum(0)
        return out
    if case["op"] == "ce":
        x, w, t = st["x"].to(f8), st["w"].to(f8), st["target"]
        n = x.shape[0]
        rows = torch.nonzero(t >= 0)[:, 0]  # the tokens that count
        labels = t[rows]
        logits = torch.mm(x[rows], w.t())
        lse = torch.logsumexp(logits, 1)
        out = dict(loss=x.new_zeros(n).index_copy(0, rows, lse - logits[torch.arange(len(rows), device=rows.device), labels]),
                   lse=x.new_zeros(n).index_copy(0, rows, lse))
        if case["train"]:
            logits.sub_(lse[:, None]).exp_()
            logits[torch.arange(len(rows), device=rows.device), labels] -= 1.0
            logits.mul_(st["grad_loss"].to(f8)[rows, None])
            out["grad_x"] = torch.zeros_like(x).index_copy(0, rows, torch.mm(logits, w))
            out["grad_w"] = torch.mm(logits.t(), x[rows])
        return out
    h, step = st["hyper"], st["step"]
    sizes = _sizes(case)
    flat, views = {}, {}
    for name in ("params", "masters", "m", "v"):
        flat[name], views[name] = _buffer(sizes, f8)
    flat["m_value"], flat["v_value"] = flat["m"], flat["v"]

    def spread(scale, like):  # each block's scale at its elements
        return scale.to(f8).repeat_interleave(_BLOCK)[:like.numel()]

    for i, p in enumerate(st["params"]):
        g = st["grads"][i].to(f8)
        q = (p if st["masters"] is None else st["masters"][i]).to(f8)
        m, v = st["m"][i].to(f8), st["v"][i].to(f8)
        if case["state"] == "8bit":
            m = spread(st["m_scale"][i], m) * m.sign() * (m / 127) ** 2
            v = spread(st["v_scale"][i], v) * (v / 255) ** 4
        m = torch.lerp(g, m, h["beta1"])
        v = torch.lerp(g * g, v, h["beta2"])
        m_hat = m / (1 - h["beta1"] ** step)
        v_hat = v / (1 - h["beta2"] ** step)
        q = q - h["lr"] * (h["weight_decay"] * q + m_hat / (v_hat.sqrt() + h["eps"]))
        views["params"][i].copy_(q)
        views["masters"][i].copy_(q)
        if case["state"] == "8bit":
            nb = (m.numel() + _BLOCK - 1) // _BLOCK
            pad = nb * _BLOCK - m.numel()
            am = torch.nn.functional.pad(m, (0, pad)).view(nb, _BLOCK).abs().amax(1)
            av = torch.nn.functional.pad(v, (0, pad)).view(nb, _BLOCK).amax(1)
            am, av = spread(am, m), spread(av, v)
            cm = torch.round(127 * (m.abs() / am).nan_to_num() ** 0.5)
            cv = torch.round(255 * (v / av).nan_to_num() ** 0.25)
            cv = torch.maximum(cv, (v > 0).to(f8))
            m, v = m.sign() * am * (cm / 127) ** 2, av * (cv / 255) ** 4
        views["m"][i].copy_(m)
        views["v"][i].copy_(v)
    return _adamw_outputs(st, flat)
