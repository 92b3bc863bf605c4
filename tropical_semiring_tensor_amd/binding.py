"""Thin ctypes binding of libtropical.so (see include/tropical.h).

Each function has the name of the C entry point it calls and only marshals
arguments: torch tensors become data pointers, element strides and sizes,
the stream defaults to torch's current stream.  All computation happens in
the library's gfx950 kernels.  There is no fallback: if the library was not
built, the first call raises ``TropicalLibraryMissing``.

Output tensors are allocated with torch when the caller passes none; torch
is used only for device memory and streams.
"""
import collections
import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libtropical.so")

OK, INVALID_ARGUMENT, UNSUPPORTED, NOT_DEVICE_MEMORY, WORKSPACE_TOO_SMALL, HIP_ERROR = range(6)
STATUS_NAMES = {0: "TROP_OK", 1: "TROP_ERR_INVALID_ARGUMENT", 2: "TROP_ERR_UNSUPPORTED",
                3: "TROP_ERR_NOT_DEVICE_MEMORY", 4: "TROP_ERR_WORKSPACE_TOO_SMALL",
                5: "TROP_ERR_HIP"}
SEMIRINGS = {"max_plus": 0, "min_plus": 1, "max_mul": 2}
F32, I32, BF16 = 0, 1, 2
KERNEL_FAMILIES = ["gemm_tiled", "gemm_simple", "fill", "gather_copy", "gather_tiled",
                   "gather_naive", "gather_reduce", "gemm_backward", "gemm_splitk_merge",
                   "argmax_compose", "gemm_domain"]
TRAIN_FAMILIES = ["layer_norm_forward", "layer_norm_backward", "ce_pack", "ce_logits", "ce_merge", "ce_grad",
                  "adamw", "act8", "act8_grad_w", "residual_forward", "residual_backward"]
MAX_DIMS = 8


class TropicalLibraryMissing(RuntimeError):
    pass


class TropicalError(RuntimeError):
    def __init__(self, status, message):
        self.status = status
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")


class trop_strides(ctypes.Structure):
    _fields_ = [("row", ctypes.c_int64), ("col", ctypes.c_int64), ("batch", ctypes.c_int64)]


class trop_tree_step(ctypes.Structure):
    _fields_ = [("lhs", ctypes.c_int32), ("rhs", ctypes.c_int32), ("out", ctypes.c_char_p)]


class trop_stats(ctypes.Structure):
    _fields_ = [("module_loads", ctypes.c_uint64), ("launches_total", ctypes.c_uint64),
                ("launches", ctypes.c_uint64 * 11)]


class trop_adamw_tensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "exp_avg", "exp_avg_sq", "master")] + [
        ("elements", ctypes.c_int64)]


class trop_adamw8_tensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "exp_avg", "exp_avg_scale", "exp_avg_sq",
                                               "exp_avg_sq_scale", "master")] + [("elements", ctypes.c_int64)]


class trop_adamw_hyper(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay")] + [
        ("step", ctypes.c_int64)]


class trop_train_stats(ctypes.Structure):
    _fields_ = [("module_loads", ctypes.c_uint64), ("launches_total", ctypes.c_uint64),
                ("launches", ctypes.c_uint64 * 11)]


class trop_act8(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("exponents", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("ld_exponents", ctypes.c_int64)]


class trop_residual_norm(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int) for n in ("dtype", "param_dtype", "gate_dtype", "post", "pre")] +
                [(n, ctypes.c_float) for n in ("residual_scale", "branch_scale", "post_eps", "pre_eps")] +
                [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("gate", ctypes.c_void_p),
                 ("ldgate", ctypes.c_int64), ("gate_group", ctypes.c_int64)] +
                [(n, ctypes.c_void_p) for n in ("post_gamma", "post_beta", "pre_gamma", "pre_beta")])


# trop_residual_norm_rows, trop_residual_norm_kept, trop_residual_norm_grads:
# every field is 8 bytes, so a call fills them as flat arrays
_rows_fields, _kept_fields, _grads_fields = ctypes.c_uint64 * 14, ctypes.c_uint64 * 14, ctypes.c_uint64 * 10


_lib = None


def lib():
    """The loaded library (loaded on first use; raises if not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise TropicalLibraryMissing(
            f"{LIB_PATH} is not built; run __graft_entry__.build() "
            "(python tropical_semiring_tensor_amd/csrc/build.py)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    I64P = ctypes.POINTER(ctypes.c_int64)
    I32P = ctypes.POINTER(ctypes.c_int32)
    L.tropical_init.argtypes = [i32]
    L.tropical_gemm_strided_batched.argtypes = [i32, i32, vp, trop_strides, vp, trop_strides, vp,
                                                trop_strides, vp, i64, i64, i64, i64, vp]
    L.tropical_gemm_strided_batched_ws.argtypes = [i32, i32, vp, trop_strides, vp, trop_strides, vp,
                                                   trop_strides, vp, i64, i64, i64, i64, vp, sz, vp]
    L.tropical_gemm_workspace_size.argtypes = [i64, i64, i64, i64, ctypes.POINTER(sz)]
    L.tropical_gemm_workspace_size_strided.argtypes = [trop_strides, trop_strides, i32, i64, i64, i64, i64,
                                                       ctypes.POINTER(sz)]
    L.tropical_gemm_backward.argtypes = [i32, i32, vp, trop_strides, vp, trop_strides, vp, vp,
                                         trop_strides, vp, trop_strides, vp, trop_strides,
                                         i64, i64, i64, i64, vp]
    L.tropical_permute.argtypes = [sz, i32, I64P, I64P, I32P, i32, ctypes.POINTER(vp),
                                   ctypes.POINTER(vp), vp]
    L.tropical_diag_gather.argtypes = [i32, i32, i32, I64P, I64P, I32P, i32, I32P, vp, vp, vp]
    L.tropical_contract_pair_workspace_size.argtypes = [ctypes.c_char_p, I64P, I64P,
                                                        ctypes.POINTER(sz)]
    L.tropical_contract_pair.argtypes = [ctypes.c_char_p, i32, i32, vp, I64P, I64P, vp, I64P, I64P,
                                         vp, vp, vp, sz, vp]
    L.tropical_contract_pair_describe.argtypes = [ctypes.c_char_p, I64P, I64P, I64P, I64P,
                                                  ctypes.c_char_p, sz]
    L.tropical_contract_pair_noalloc.argtypes = [ctypes.c_char_p, i32, i32, vp, I64P, I64P, vp, I64P, I64P,
                                                 vp, vp, vp]
    PP = ctypes.POINTER
    L.tropical_tree_plan_create.argtypes = [i32, i32, i32, PP(ctypes.c_char_p), PP(I64P), PP(I64P), i32,
                                            PP(trop_tree_step), PP(vp)]
    L.tropical_tree_plan_destroy.argtypes = [vp]
    L.tropical_tree_plan_destroy.restype = None
    L.tropical_tree_workspace_size.argtypes = [vp, PP(sz)]
    L.tropical_tree_step_info.argtypes = [vp, i32, ctypes.c_char_p, I64P, I64P]
    L.tropical_tree_run.argtypes = [vp, PP(vp), vp, PP(vp), vp, sz, vp]
    L.tropical_tree_describe.argtypes = [vp, ctypes.c_char_p, sz]
    L.tropical_last_error.restype = ctypes.c_char_p
    L.tropical_get_stats.argtypes = [ctypes.POINTER(trop_stats)]
    L.tropical_reset_stats.restype = None
    for fn in ("tropical_init", "tropical_gemm_strided_batched", "tropical_gemm_backward", "tropical_permute",
               "tropical_gemm_strided_batched_ws", "tropical_gemm_workspace_size",
               "tropical_gemm_workspace_size_strided",
               "tropical_diag_gather", "tropical_contract_pair_workspace_size",
               "tropical_contract_pair", "tropical_contract_pair_describe", "tropical_get_stats",
               "tropical_contract_pair_noalloc",
               "tropical_tree_plan_create", "tropical_tree_workspace_size", "tropical_tree_step_info",
               "tropical_tree_run", "tropical_tree_describe"):
        getattr(L, fn).restype = ctypes.c_int
    # declared argument types: ctypes then converts plain ints (data
    # pointers, sizes) without inspecting each argument's type per call
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    L.tropical_gemm_strided_batched.argtypes = [ctypes.c_int, ctypes.c_int, vp, trop_strides, vp, trop_strides,
                                                vp, trop_strides, vp, i64, i64, i64, i64, vp]
    f32 = ctypes.c_float
    L.tropical_train_init.argtypes = [i32]
    L.tropical_layer_norm_forward.argtypes = [i32, i32, vp, i64, vp, vp, f32, vp, i64, vp, vp, i64, i64, vp]
    L.tropical_layer_norm_backward_workspace_size.argtypes = [i64, i64, i32, PP(sz)]
    L.tropical_layer_norm_backward.argtypes = [i32, i32, vp, i64, vp, i64, vp, vp, vp, vp, i64, vp, vp, i64, i64,
                                               vp, sz, vp]
    L.tropical_linear_cross_entropy_forward.argtypes = [i32, vp, i64, vp, i64, vp, i32, i64, vp, vp, i64, i64, i64,
                                                        vp, sz, vp]
    L.tropical_linear_cross_entropy_workspace_size.argtypes = [i32, i64, i64, i64, i32, PP(sz)]
    L.tropical_linear_cross_entropy_backward.argtypes = [i32, vp, i64, vp, i64, vp, i32, i64, vp, vp, i64, vp, i64,
                                                         vp, i64, i64, i64, i64, vp, sz, vp]
    L.tropical_adamw_step.argtypes = [i32, PP(trop_adamw_tensor), i64, PP(trop_adamw_hyper), vp]
    L.tropical_adamw8_step.argtypes = [i32, PP(trop_adamw8_tensor), i64, PP(trop_adamw_hyper), vp]
    L.tropical_adamw8_unpack.argtypes = [PP(trop_adamw8_tensor), i64, PP(vp), PP(vp), vp]
    L.tropical_act8_pack.argtypes = [i32, vp, i64, PP(trop_act8), i64, i64, vp]
    L.tropical_act8_unpack.argtypes = [PP(trop_act8), i32, vp, i64, i64, i64, vp]
    L.tropical_act8_linear_grad_w.argtypes = [i32, vp, i64, PP(trop_act8), vp, i64, i64, i64, i64, vp, sz, vp]
    L.tropical_act8_linear_grad_w_workspace_size.argtypes = [i32, i64, i64, i64, PP(sz)]
    L.tropical_residual_norm_forward.argtypes = [PP(trop_residual_norm), PP(ctypes.c_uint64), vp]
    L.tropical_residual_norm_backward.argtypes = [PP(trop_residual_norm), PP(ctypes.c_uint64), PP(ctypes.c_uint64), vp,
                                                  sz, vp]
    L.tropical_residual_norm_backward_workspace_size.argtypes = [PP(trop_residual_norm), PP(sz)]
    L.tropical_get_train_stats.argtypes = [PP(trop_train_stats)]
    for fn in ("tropical_train_init", "tropical_layer_norm_forward", "tropical_layer_norm_backward_workspace_size",
               "tropical_layer_norm_backward", "tropical_linear_cross_entropy_forward",
               "tropical_linear_cross_entropy_workspace_size", "tropical_linear_cross_entropy_backward",
               "tropical_adamw_step", "tropical_adamw8_step", "tropical_adamw8_unpack", "tropical_act8_pack",
               "tropical_act8_unpack", "tropical_act8_linear_grad_w", "tropical_act8_linear_grad_w_workspace_size",
               "tropical_residual_norm_forward", "tropical_residual_norm_backward",
               "tropical_residual_norm_backward_workspace_size", "tropical_get_train_stats"):
        getattr(L, fn).restype = ctypes.c_int
    _lib = L
    return L


def _check(status, what):
    if status != OK:
        msg = lib().tropical_last_error().decode(errors="replace")
        raise TropicalError(status, f"{what}: {msg}")


def _sr(semiring):
    return SEMIRINGS[semiring] if isinstance(semiring, str) else int(semiring)


def _dt(t):
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.int32:
        return I32
    raise TypeError(f"float32 or int32 tensors only, got {t.dtype}")


# torch's current stream as a raw pointer, without building a Stream object
# per call (the public call below is the fallback)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_ptr(stream, t):
    """Raw stream pointer (int) for a call on tensor t's device."""
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(t.device.index if t.device.index is not None else torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return ctypes.c_void_p(_raw_stream(torch.cuda.current_device()))
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _i64(vals):
    return (ctypes.c_int64 * max(1, len(vals)))(*[int(v) for v in vals])


def _i32(vals):
    return (ctypes.c_int32 * max(1, len(vals)))(*[int(v) for v in vals])


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _as3(t):
    return t.unsqueeze(0) if t.dim() == 2 else t


# ---------------------------------------------------------------------------

def tropical_init(device=0):
    _check(lib().tropical_init(int(device)), "tropical_init")


def tropical_gemm_strided_batched(semiring, A, B, C, argmax=None, stream=None):
    """C[b,i,j] = (+)_k A[b,i,k] (x) B[b,k,j] and argmax[b,i,j] = first winning k.

    A: (batch, m, k), B: (batch, k, n), C and argmax: (batch, m, n) views
    (2-d tensors are batch 1).  Any non-negative strides; argmax must share
    C's strides.  Enqueued on `stream` (default: torch's current stream).
    """
    A3, B3, C3 = _as3(A), _as3(B), _as3(C)
    batch, m, k = A3.shape
    n = B3.shape[2]
    a, b, c = A3.stride(), B3.stride(), C3.stride()
    if argmax is not None and _as3(argmax).stride() != c:
        raise ValueError("argmax must have the strides of C")
    st = lib().tropical_gemm_strided_batched(_sr(semiring), _dt(A3), A3.data_ptr(), trop_strides(a[1], a[2], a[0]),
                                             B3.data_ptr(), trop_strides(b[1], b[2], b[0]), C3.data_ptr(),
                                             trop_strides(c[1], c[2], c[0]),
                                             argmax.data_ptr() if argmax is not None else None,
                                             m, n, k, batch, _stream_ptr(stream, A3))
    _check(st, "tropical_gemm_strided_batched")
    return C, argmax


def tropical_gemm_workspace_size(m, n, k, batch=1):
    nb = ctypes.c_size_t(0)
    _check(lib().tropical_gemm_workspace_size(int(m), int(n), int(k), int(batch), ctypes.byref(nb)),
           "tropical_gemm_workspace_size")
    return nb.value


def tropical_gemm_workspace_size_strided(A, B, with_argmax=True):
    """Workspace bytes for tropical_gemm_strided_batched_ws with the shapes
    and strides of the (batch, m, k) and (batch, k, n) tensors A and B."""
    A3, B3 = _as3(A), _as3(B)
    batch, m, k = A3.shape
    n = B3.shape[2]
    sA = trop_strides(A3.stride(1), A3.stride(2), A3.stride(0))
    sB = trop_strides(B3.stride(1), B3.stride(2), B3.stride(0))
    nb = ctypes.c_size_t(0)
    _check(lib().tropical_gemm_workspace_size_strided(sA, sB, 1 if with_argmax else 0, m, n, k, batch,
                                                      ctypes.byref(nb)), "tropical_gemm_workspace_size_strided")
    return nb.value


def tropical_gemm_strided_batched_ws(semiring, A, B, C, argmax=None, workspace=None, stream=None):
    """tropical_gemm_strided_batched with a workspace (split along K when
    the product has few output tiles and a long K; a transposed copy of a
    row-major B for a long-K argmax product).  workspace: None to allocate
    tropical_gemm_workspace_size_strided bytes with torch, or a uint8
    device tensor."""
    A3, B3, C3 = _as3(A), _as3(B), _as3(C)
    batch, m, k = A3.shape
    n = B3.shape[2]
    if argmax is not None and _as3(argmax).stride() != C3.stride():
        raise ValueError("argmax must have the strides of C")
    if workspace is None:
        nb = tropical_gemm_workspace_size_strided(A3, B3, argmax is not None)
        workspace = torch.empty(nb, dtype=torch.uint8, device=A3.device) if nb else None
    sA = trop_strides(A3.stride(1), A3.stride(2), A3.stride(0))
    sB = trop_strides(B3.stride(1), B3.stride(2), B3.stride(0))
    sC = trop_strides(C3.stride(1), C3.stride(2), C3.stride(0))
    st = lib().tropical_gemm_strided_batched_ws(_sr(semiring), _dt(A3), _ptr(A3), sA, _ptr(B3), sB,
                                                _ptr(C3), sC, _ptr(argmax), m, n, k, batch, _ptr(workspace),
                                                workspace.numel() if workspace is not None else 0,
                                                _stream(stream))
    _check(st, "tropical_gemm_strided_batched_ws")
    return C, argmax


def tropical_gemm_backward(semiring, argmax, grad_c, A=None, B=None, k=None, grad_a=True,
                           grad_b=True, stream=None):
    """Gradients of sum(grad_c * C) routed along the forward's argmax.

    argmax (int32) and grad_c (float32): (batch, m, n) with equal strides.
    A (batch, m, k) and B (batch, k, n) are read for max-mul only.  k is the
    contracted size (from A or B when omitted).  grad_a / grad_b: True to
    allocate (float32, contiguous), a tensor to fill, or None to skip.
    Returns (grad_a, grad_b).
    """
    I3, G3 = _as3(argmax), _as3(grad_c)
    if I3.stride() != G3.stride() or I3.shape != G3.shape:
        raise ValueError("argmax and grad_c must share shape and strides")
    batch, m, n = I3.shape
    A3 = _as3(A) if A is not None else None
    B3 = _as3(B) if B is not None else None
    if k is None:
        k = A3.shape[2] if A3 is not None else B3.shape[1]
    dev = I3.device
    if grad_a is True:
        grad_a = torch.empty(batch, m, k, dtype=torch.float32, device=dev)
    if grad_b is True:
        grad_b = torch.empty(batch, k, n, dtype=torch.float32, device=dev)
    ga3 = _as3(grad_a) if grad_a is not None else None
    gb3 = _as3(grad_b) if grad_b is not None else None

    def strides(t):
        return trop_strides(t.stride(1), t.stride(2), t.stride(0)) if t is not None else trop_strides(0, 0, 0)

    dt = _dt(A3) if A3 is not None else (_dt(B3) if B3 is not None else F32)
    st = lib().tropical_gemm_backward(_sr(semiring), dt, _ptr(A3), strides(A3), _ptr(B3), strides(B3),
                                      _ptr(I3), _ptr(G3), strides(I3), _ptr(ga3), strides(ga3),
                                      _ptr(gb3), strides(gb3), m, n, int(k), batch, _stream(stream))
    _check(st, "tropical_gemm_backward")
    return grad_a, grad_b


def tropical_permute(x, perm, out=None, x2=None, out2=None, stream=None):
    """out = x.permute(perm) made contiguous; x2 -> out2 with the same mapping."""
    perm = [int(p) for p in perm]
    shape = [x.shape[p] for p in perm]
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
    n = 1
    ins = [x.data_ptr()]
    outs = [out.data_ptr()]
    if x2 is not None:
        if x2.shape != x.shape or x2.stride() != x.stride():
            raise ValueError("x2 must have the shape and strides of x")
        if out2 is None:
            out2 = torch.empty(shape, dtype=x2.dtype, device=x2.device)
        ins.append(x2.data_ptr())
        outs.append(out2.data_ptr())
        n = 2
    in_arr = (ctypes.c_void_p * 2)(*ins, *([0] * (2 - n)))
    out_arr = (ctypes.c_void_p * 2)(*outs, *([0] * (2 - n)))
    st = lib().tropical_permute(x.element_size(), x.dim(), _i64(x.shape), _i64(x.stride()),
                                _i32(perm), n, in_arr, out_arr, _stream(stream))
    _check(st, "tropical_permute")
    return (out, out2) if x2 is not None else out


def _label_ids(labels):
    return [ord(c) if isinstance(c, str) else int(c) for c in labels]


def tropical_diag_gather(semiring, x, in_labels, out_labels, out=None, stream=None):
    """Repeated-label diagonal (and (+)-reduction of labels absent from out)."""
    il, ol = _label_ids(in_labels), _label_ids(out_labels)
    if len(il) != x.dim():
        raise ValueError("one label per input axis")
    ext = {}
    for lab, e in zip(il, x.shape):
        ext.setdefault(lab, e)
    if out is None:
        out = torch.empty([ext.get(lab, 0) for lab in ol], dtype=x.dtype, device=x.device)
    st = lib().tropical_diag_gather(_sr(semiring), _dt(x), x.dim(), _i64(x.shape), _i64(x.stride()),
                                    _i32(il), len(ol), _i32(ol), _ptr(x), _ptr(out),
                                    _stream(stream))
    _check(st, "tropical_diag_gather")
    return out


def tropical_contract_pair_workspace_size(spec, shapeA, shapeB):
    n = ctypes.c_size_t(0)
    st = lib().tropical_contract_pair_workspace_size(spec.encode(), _i64(shapeA), _i64(shapeB),
                                                     ctypes.byref(n))
    _check(st, "tropical_contract_pair_workspace_size")
    return n.value


def tropical_contract_pair_describe(spec, shapeA, shapeB, stridesA=None, stridesB=None):
    buf = ctypes.create_string_buffer(1024)
    st = lib().tropical_contract_pair_describe(
        spec.encode(), _i64(shapeA), _i64(stridesA) if stridesA is not None else None,
        _i64(shapeB), _i64(stridesB) if stridesB is not None else None, buf, len(buf))
    _check(st, "tropical_contract_pair_describe")
    return buf.value.decode()


def _out_shape(spec, A, B):
    lhs, out = spec.replace(" ", "").split("->")
    la, lb = lhs.split(",")
    ext = {}
    for sub, t in ((la, A), (lb, B)):
        for c, e in zip(sub, t.shape):
            ext.setdefault(c, e)
    return [ext.get(c, 0) for c in out]


def tropical_contract_pair(spec, semiring, A, B, C=None, argmax=True, workspace=None, stream=None):
    """Pairwise tropical einsum; returns (C, argmax) (argmax None if not asked).

    argmax=True allocates the int32 argmax; pass a tensor to reuse one, or
    None / False to skip it.  The workspace is allocated with torch when
    not given.
    """
    shape = _out_shape(spec, A, B)
    if C is None:
        C = torch.empty(shape, dtype=A.dtype, device=A.device)
    if argmax is True:
        argmax = torch.empty(shape, dtype=torch.int32, device=A.device)
    elif argmax is False:
        argmax = None
    if workspace is None:
        nbytes = tropical_contract_pair_workspace_size(spec, A.shape, B.shape)
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=A.device)
    st = lib().tropical_contract_pair(spec.encode(), _sr(semiring), _dt(A), _ptr(A), _i64(A.shape),
                                      _i64(A.stride()), _ptr(B), _i64(B.shape), _i64(B.stride()),
                                      _ptr(C), _ptr(argmax), _ptr(workspace), workspace.numel(),
                                      _stream(stream))
    _check(st, "tropical_contract_pair")
    return C, argmax


NOALLOC_SCRATCH_BYTES = 32 << 20  # TROP_NOALLOC_SCRATCH_BYTES in include/tropical.h


def tropical_contract_pair_noalloc(spec, semiring, A, B, C, argmax=None, stream=None):
    """Pairwise tropical einsum into the caller's C (and argmax, or None)
    with the library's own scratch: the call allocates nothing, so C (and
    argmax) must be given."""
    st = lib().tropical_contract_pair_noalloc(spec.encode(), _sr(semiring), _dt(A), _ptr(A), _i64(A.shape),
                                              _i64(A.stride()), _ptr(B), _i64(B.shape), _i64(B.stride()),
                                              _ptr(C), _ptr(argmax), _stream(stream))
    _check(st, "tropical_contract_pair_noalloc")
    return C, argmax


class TreePlan:
    """Handle of a planned contraction tree (owns the library's plan)."""

    def __init__(self, handle, n_inputs, n_steps, dtype):
        self.handle = handle
        self.n_inputs = n_inputs
        self.n_steps = n_steps
        self.dtype = dtype

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.tropical_tree_plan_destroy(self.handle)
            self.handle = None


def tropical_tree_plan_create(semiring, dtype, subs, shapes, steps, strides=None):
    """Plan a tree.  subs / shapes: per input; strides: None, or per input
    None (contiguous) or its element strides; steps: (lhs_slot, rhs_slot,
    out_subscript) with slots 0..n-1 the inputs and n + s step s's result.
    dtype: torch.float32 or torch.int32."""
    n, m = len(subs), len(steps)
    dt = F32 if dtype == torch.float32 else (I32 if dtype == torch.int32 else None)
    if dt is None:
        raise TypeError(f"float32 or int32 only, got {dtype}")
    sub_arr = (ctypes.c_char_p * n)(*[x.encode() for x in subs])
    shape_keep = [_i64(sh) for sh in shapes]
    I64P = ctypes.POINTER(ctypes.c_int64)
    shape_arr = (I64P * n)(*[ctypes.cast(a, I64P) for a in shape_keep])
    stride_arr = None
    if strides is not None:
        stride_keep = [_i64(st) if st is not None else None for st in strides]
        stride_arr = (I64P * n)(*[ctypes.cast(a, I64P) if a is not None else I64P() for a in stride_keep])
    out_keep = [o.encode() for _, _, o in steps]
    step_arr = (trop_tree_step * m)(*[trop_tree_step(int(a), int(b), o) for (a, b, _), o in zip(steps, out_keep)])
    h = ctypes.c_void_p(0)
    st = lib().tropical_tree_plan_create(_sr(semiring), dt, n, sub_arr, shape_arr, stride_arr, m, step_arr,
                                         ctypes.byref(h))
    _check(st, "tropical_tree_plan_create")
    return TreePlan(h.value, n, m, dtype)


def tropical_tree_plan_destroy(plan):
    if plan.handle:
        lib().tropical_tree_plan_destroy(plan.handle)
        plan.handle = None


def tropical_tree_workspace_size(plan):
    n = ctypes.c_size_t(0)
    _check(lib().tropical_tree_workspace_size(plan.handle, ctypes.byref(n)), "tropical_tree_workspace_size")
    return n.value


def tropical_tree_step_info(plan, step):
    """(subscript, shape) of step `step`'s output."""
    sub = ctypes.create_string_buffer(16)
    shape = (ctypes.c_int64 * 8)()
    _check(lib().tropical_tree_step_info(plan.handle, int(step), sub, shape, None), "tropical_tree_step_info")
    s = sub.value.decode()
    return s, [shape[d] for d in range(len(s))]


def tropical_tree_describe(plan):
    buf = ctypes.create_string_buffer(64 * 1024)
    _check(lib().tropical_tree_describe(plan.handle, buf, len(buf)), "tropical_tree_describe")
    return buf.value.decode()


def tropical_tree_run(plan, inputs, out=None, argmax=False, workspace=None, stream=None):
    """Run a planned tree; returns (out, [argmax of each step or None]).

    argmax: False (none), True (every step) or one flag / tensor / None per
    step; requested ones are allocated as contiguous int32 tensors.  The
    workspace is allocated with torch when not given.
    """
    if len(inputs) != plan.n_inputs:
        raise ValueError(f"the plan has {plan.n_inputs} inputs")
    dev = inputs[0].device
    if out is None:
        _, shape = tropical_tree_step_info(plan, plan.n_steps - 1)
        out = torch.empty(shape, dtype=plan.dtype, device=dev)
    flags = [argmax] * plan.n_steps if isinstance(argmax, bool) else list(argmax)
    if len(flags) != plan.n_steps:
        raise ValueError("one argmax entry per step")
    ams = []
    for s, f in enumerate(flags):
        if f is True:
            ams.append(torch.empty(tropical_tree_step_info(plan, s)[1], dtype=torch.int32, device=dev))
        elif f is False or f is None:
            ams.append(None)
        else:
            ams.append(f)
    if workspace is None:
        workspace = torch.empty(max(tropical_tree_workspace_size(plan), 1), dtype=torch.uint8, device=dev)
    in_arr = (ctypes.c_void_p * len(inputs))(*[t.data_ptr() for t in inputs])
    am_arr = (ctypes.c_void_p * plan.n_steps)(*[a.data_ptr() if a is not None else 0 for a in ams])
    st = lib().tropical_tree_run(plan.handle, in_arr, _ptr(out), am_arr, _ptr(workspace), workspace.numel(),
                                 _stream(stream))
    _check(st, "tropical_tree_run")
    return out, ams


# ---------------------------------------------------------------------------
# training operators

_TRAIN_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}


def _tdt(t, what):
    dt = _TRAIN_DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError(f"{what} must be float32 or bfloat16, got {t.dtype}")
    return dt


def _row_stride(t, what):
    """Row stride of a 2-d tensor with unit stride along its rows."""
    strides = t.stride()
    if len(strides) != 2:
        raise ValueError(f"{what} must be 2-d, got {t.dim()}-d")
    ld, inner = strides
    rows, cols = t.shape
    if inner != 1 and cols > 1:
        raise ValueError(f"{what} must have unit stride along its rows")
    return ld if rows > 1 else max(ld, cols)


def _flat(t, what, n, dtype):
    if t.shape != (n,) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous 1-d {dtype} tensor of {n} elements")
    return t.data_ptr()


def _new_matrix(rows, cols, dtype, device):
    # (empty_strided reads its arguments in half of empty's time)
    return torch.empty_strided((rows, cols), (max(cols, 1), 1), dtype=dtype, device=device)


def _out_matrix(t, rows, cols, dtype, device, what):
    """(tensor, pointer, row stride) of the caller's output matrix, checked,
    or of a new one for True / None."""
    if t is None or t is True:
        t = _new_matrix(rows, cols, dtype, device)
        return t, t.data_ptr(), cols
    if tuple(t.shape) != (rows, cols) or t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype} of shape {(rows, cols)}")
    return t, t.data_ptr(), _row_stride(t, what)


def _out_flat(t, n, dtype, device, what):
    """(tensor, pointer) of a 1-d output, likewise."""
    if t is None or t is True:
        t = torch.empty_strided((n,), (1,), dtype=dtype, device=device)
        return t, t.data_ptr()
    return t, _flat(t, what, n, dtype)


def _new_flats(there, n, dtype, device):
    """A new vector of n elements for each that is there, None for the others;
    of several one after another in one allocation (four vectors 3.2 us of host
    time against 5.0).  unsafe_chunk makes them tensors of their own: views of
    one matrix would share its version, and refuse some changes in place."""
    count = sum(there)
    if count > 2:
        parts = iter(torch.unsafe_chunk(torch.empty_strided((count * n,), (1,), dtype=dtype, device=device), count))
        return [next(parts) if t else None for t in there]
    return [torch.empty_strided((n,), (1,), dtype=dtype, device=device) if t else None for t in there]


def _workspace(workspace, nbytes, device):
    """(tensor to keep alive, pointer, bytes) of a workspace given or made."""
    if workspace is None:
        if not nbytes:
            return None, None, 0
        workspace = torch.empty_strided((nbytes,), (1,), dtype=torch.uint8, device=device)
        return workspace, workspace.data_ptr(), nbytes
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _on_stream(fn):
    """With a `stream` argument, run the call with that stream current, so
    that the outputs and the workspace it allocates belong to that stream."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream))
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def tropical_train_init(device=0):
    _check(lib().tropical_train_init(int(device)), "tropical_train_init")


@_on_stream
def tropical_layer_norm_forward(x, gamma=None, beta=None, eps=1e-5, y=None, mean=None, rstd=None):
    """Layer norm of the rows of x (rows, cols): (y, mean, rstd).

    x: float32 or bfloat16, unit stride along the rows, any row stride.
    gamma, beta: cols elements, float32 or x's type (one type), or None.
    mean, rstd: float32 statistics for the backward.  Outputs are allocated
    when not given; y may be x.
    """
    dt = _tdt(x, "x")
    ldx = _row_stride(x, "x")
    rows, cols = x.shape
    par = gamma if gamma is not None else beta
    pdt = _tdt(par, "gamma and beta") if par is not None else F32
    pg = _flat(gamma, "gamma", cols, par.dtype) if gamma is not None else None
    pb = _flat(beta, "beta", cols, par.dtype) if beta is not None else None
    dev = x.device
    y, py, ldy = _out_matrix(y, rows, cols, x.dtype, dev, "y")
    mean, pm = _out_flat(mean, rows, torch.float32, dev, "mean")
    rstd, pr = _out_flat(rstd, rows, torch.float32, dev, "rstd")
    st = lib().tropical_layer_norm_forward(dt, pdt, x.data_ptr(), ldx, pg, pb, eps, py, ldy, pm, pr, rows, cols,
                                           _stream_ptr(None, x))
    if st != OK:
        _check(st, "tropical_layer_norm_forward")
    return y, mean, rstd


def tropical_layer_norm_backward_workspace_size(rows, cols, with_params=True):
    nb = ctypes.c_size_t(0)
    _check(lib().tropical_layer_norm_backward_workspace_size(int(rows), int(cols), 1 if with_params else 0,
                                                             ctypes.byref(nb)),
           "tropical_layer_norm_backward_workspace_size")
    return nb.value


@_on_stream
def tropical_layer_norm_backward(dy, x, mean, rstd, gamma=None, dx=True, dgamma=True, dbeta=True, workspace=None):
    """Gradients of a layer norm: (dx, dgamma, dbeta).

    x, mean, rstd: the forward's.  dx (x's type), dgamma and dbeta (gamma's
    type, float32 without gamma): True to allocate, a tensor to fill, or None
    to skip.  dx may be dy.  The workspace is allocated with torch when not
    given.
    """
    dt = _tdt(x, "x")
    rows, cols = x.shape
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError("dy must have the shape and type of x")
    ptype = gamma.dtype if gamma is not None else torch.float32
    pdt = _tdt(gamma, "gamma") if gamma is not None else F32
    pg = _flat(gamma, "gamma", cols, ptype) if gamma is not None else None
    dev = x.device
    px, ldx, pdg, pdb = None, 0, None, None
    if dx is not None:
        dx, px, ldx = _out_matrix(dx, rows, cols, x.dtype, dev, "dx")
    if dgamma is not None:
        dgamma, pdg = _out_flat(dgamma, cols, ptype, dev, "dgamma")
    if dbeta is not None:
        dbeta, pdb = _out_flat(dbeta, cols, ptype, dev, "dbeta")
    need = 0
    if workspace is None and (dgamma is not None or dbeta is not None):
        need = tropical_layer_norm_backward_workspace_size(rows, cols)
    workspace, wp, wn = _workspace(workspace, need, dev)
    st = lib().tropical_layer_norm_backward(
        dt, pdt, dy.data_ptr(), _row_stride(dy, "dy"), x.data_ptr(), _row_stride(x, "x"),
        _flat(mean, "mean", rows, torch.float32), _flat(rstd, "rstd", rows, torch.float32), pg, px, ldx, pdg, pdb,
        rows, cols, wp, wn, _stream_ptr(None, x))
    if st != OK:
        _check(st, "tropical_layer_norm_backward")
    return dx, dgamma, dbeta


def tropical_linear_cross_entropy_workspace_size(dtype, tokens, width, vocab, backward=False):
    """Workspace bytes of a cross entropy call (dtype: torch.float32 or
    torch.bfloat16)."""
    if dtype not in _TRAIN_DTYPES:
        raise TypeError(f"float32 or bfloat16 only, got {dtype}")
    nb = ctypes.c_size_t(0)
    _check(lib().tropical_linear_cross_entropy_workspace_size(_TRAIN_DTYPES[dtype], int(tokens), int(width),
                                                              int(vocab), 1 if backward else 0, ctypes.byref(nb)),
           "tropical_linear_cross_entropy_workspace_size")
    return nb.value


def _ce_operands(x, w, target):
    dt = _tdt(x, "x")
    if w.dtype != x.dtype:
        raise TypeError("w must have the type of x")
    ldx, ldw = _row_stride(x, "x"), _row_stride(w, "w")
    tokens, width = x.shape
    if w.shape[1] != width:
        raise ValueError(f"x has a width of {width}, w of {w.shape[1]}")
    if target.dtype not in (torch.int64, torch.int32):
        raise TypeError(f"target must be int32 or int64, got {target.dtype}")
    pt = _flat(target, "target", tokens, target.dtype)
    return dt, ldx, ldw, tokens, width, w.shape[0], pt, target.element_size()


@_on_stream
def tropical_linear_cross_entropy_forward(x, w, target, ignore_index=-100, loss=None, lse=None, workspace=None):
    """Softmax cross entropy of tokens over a label set: (loss, lse), float32
    per token, with logits x @ w.T that are never kept.

    x (tokens, width), w (vocab, width): float32 or bfloat16, unit stride
    along the rows.  target: int32 or int64; a token whose target is
    ignore_index or outside the vocabulary does not count (loss and lse 0).
    The workspace is allocated with torch when not given.
    """
    dt, ldx, ldw, tokens, width, vocab, pt, tbytes = _ce_operands(x, w, target)
    dev = x.device
    loss, pl = _out_flat(loss, tokens, torch.float32, dev, "loss")
    lse, ps = _out_flat(lse, tokens, torch.float32, dev, "lse")
    need = 0
    if workspace is None:
        need = tropical_linear_cross_entropy_workspace_size(x.dtype, tokens, width, vocab)
    workspace, wp, wn = _workspace(workspace, need, dev)
    st = lib().tropical_linear_cross_entropy_forward(dt, x.data_ptr(), ldx, w.data_ptr(), ldw, pt, tbytes,
                                                     ignore_index, pl, ps, tokens, width, vocab, wp, wn,
                                                     _stream_ptr(None, x))
    if st != OK:
        _check(st, "tropical_linear_cross_entropy_forward")
    return loss, lse


@_on_stream
def tropical_linear_cross_entropy_backward(x, w, target, lse, grad_loss, ignore_index=-100, grad_x=True, grad_w=True,
                                           workspace=None):
    """Gradients of sum(grad_loss * loss): (grad_x, grad_w) in x's type.

    lse: the forward's.  grad_loss: float32, one per token (any stride, an
    expanded scalar too) or a 0-d tensor for all.  grad_x, grad_w: True to
    allocate, a tensor to fill, or None to skip.
    """
    dt, ldx, ldw, tokens, width, vocab, pt, tbytes = _ce_operands(x, w, target)
    dev = x.device
    if grad_loss.dtype != torch.float32 or grad_loss.dim() > 1 or (grad_loss.dim() == 1 and
                                                                   grad_loss.shape[0] != tokens):
        raise ValueError(f"grad_loss must be float32, 0-d or of {tokens} elements")
    gstride = grad_loss.stride(0) if grad_loss.dim() == 1 and tokens > 1 else 0
    px, ldgx, pw, ldgw = None, 0, None, 0
    if grad_x is not None:
        grad_x, px, ldgx = _out_matrix(grad_x, tokens, width, x.dtype, dev, "grad_x")
    if grad_w is not None:
        grad_w, pw, ldgw = _out_matrix(grad_w, vocab, width, x.dtype, dev, "grad_w")
    need = 0
    if workspace is None:
        need = tropical_linear_cross_entropy_workspace_size(x.dtype, tokens, width, vocab, backward=True)
    workspace, wp, wn = _workspace(workspace, need, dev)
    st = lib().tropical_linear_cross_entropy_backward(
        dt, x.data_ptr(), ldx, w.data_ptr(), ldw, pt, tbytes, ignore_index, _flat(lse, "lse", tokens, torch.float32),
        grad_loss.data_ptr(), gstride, px, ldgx, pw, ldgw, tokens, width, vocab, wp, wn, _stream_ptr(None, x))
    if st != OK:
        _check(st, "tropical_linear_cross_entropy_backward")
    return grad_x, grad_w


def _adamw_table(kind, columns, params, grads, masters):
    """The ctypes table of `kind` and the elements' type.  columns: (field,
    tensors, type, elements per scale or 0)."""
    n = len(params)
    if not n:
        return None, F32
    dtype = params[0].dtype
    dt = _tdt(params[0], "params")
    columns = [("param", params, dtype, 0), ("grad", grads, dtype, 0)] + columns
    if masters is not None:
        columns = columns + [("master", masters, torch.float32, 0)]
    for name, ts, ty, block in columns:
        if len(ts) != n:
            raise ValueError(f"{name}: {len(ts)} tensors for {n} parameters")
    counts = [p.numel() for p in params]
    ptrs = {}
    for name, ts, ty, block in columns:
        want = [(e + block - 1) // block for e in counts] if block else counts
        if not all([t.dtype is ty and t.numel() == e and t.is_contiguous() for t, e in zip(ts, want)]):
            raise ValueError(f"{name} must be contiguous {ty} tensors of the parameters' sizes")
        ptrs[name] = [t.data_ptr() for t in ts]
    none = [0] * n
    # (every field is 8 bytes: the table as one flat array)
    rows = zip(*(ptrs.get(f[0], none) for f in kind._fields_[:-1]), counts)
    flat = [x for row in rows for x in row]
    return ctypes.cast((ctypes.c_uint64 * len(flat))(*flat), ctypes.POINTER(kind)), dt


def _adamw_hyper(lr, beta1, beta2, eps, weight_decay, step):
    return trop_adamw_hyper(lr, beta1, beta2, eps, weight_decay, step)


@_on_stream
def tropical_adamw_step(params, grads, exp_avgs, exp_avg_sqs, lr, beta1=0.9, beta2=0.999, eps=1e-8,
                        weight_decay=0.0, step=1, masters=None):
    """One AdamW step over lists of tensors, in place (see
    include/tropical.h).  params and grads: float32 or bfloat16, one type;
    states and masters float32; all contiguous.  step counts from 1."""
    f = torch.float32
    table, dt = _adamw_table(trop_adamw_tensor, [("exp_avg", exp_avgs, f, 0), ("exp_avg_sq", exp_avg_sqs, f, 0)],
                             params, grads, masters)
    h = _adamw_hyper(lr, beta1, beta2, eps, weight_decay, step)
    st = lib().tropical_adamw_step(dt, table, len(params), ctypes.byref(h),
                                   _stream_ptr(None, params[0]) if params else None)
    if st != OK:
        _check(st, "tropical_adamw_step")


ADAMW_BLOCK = 256  # TROP_ADAMW_BLOCK in include/tropical.h


def _adamw8_columns(m, m_scales, v, v_scales):
    f = torch.float32
    return [("exp_avg", m, torch.int8, 0), ("exp_avg_scale", m_scales, f, ADAMW_BLOCK),
            ("exp_avg_sq", v, torch.uint8, 0), ("exp_avg_sq_scale", v_scales, f, ADAMW_BLOCK)]


@_on_stream
def tropical_adamw8_step(params, grads, exp_avgs, exp_avg_scales, exp_avg_sqs, exp_avg_sq_scales, lr, beta1=0.9,
                         beta2=0.999, eps=1e-8, weight_decay=0.0, step=1, masters=None):
    """tropical_adamw_step with 8-bit states: int8 exp_avgs and uint8
    exp_avg_sqs with a float32 scale for each ADAMW_BLOCK elements (zeros
    everywhere are the state before the first step)."""
    table, dt = _adamw_table(trop_adamw8_tensor, _adamw8_columns(exp_avgs, exp_avg_scales, exp_avg_sqs,
                                                                 exp_avg_sq_scales), params, grads, masters)
    h = _adamw_hyper(lr, beta1, beta2, eps, weight_decay, step)
    st = lib().tropical_adamw8_step(dt, table, len(params), ctypes.byref(h),
                                    _stream_ptr(None, params[0]) if params else None)
    if st != OK:
        _check(st, "tropical_adamw8_step")


@_on_stream
def tropical_adamw8_unpack(exp_avgs, exp_avg_scales, exp_avg_sqs, exp_avg_sq_scales, exp_avg_values=None,
                           exp_avg_sq_values=None):
    """The float32 values that 8-bit states stand for: two lists of tensors
    (allocated when not given)."""
    n = len(exp_avgs)
    if exp_avg_values is None:
        exp_avg_values = [torch.empty(t.shape, dtype=torch.float32, device=t.device) for t in exp_avgs]
    if exp_avg_sq_values is None:
        exp_avg_sq_values = [torch.empty(t.shape, dtype=torch.float32, device=t.device) for t in exp_avg_sqs]
    if not n:
        return exp_avg_values, exp_avg_sq_values
    # the values' tensors stand where a step's float32 parameters would
    table, _ = _adamw_table(trop_adamw8_tensor, _adamw8_columns(exp_avgs, exp_avg_scales, exp_avg_sqs,
                                                                exp_avg_sq_scales), exp_avg_values,
                            exp_avg_sq_values, None)
    mv = (ctypes.c_void_p * n)(*[t.data_ptr() for t in exp_avg_values])
    vv = (ctypes.c_void_p * n)(*[t.data_ptr() for t in exp_avg_sq_values])
    st = lib().tropical_adamw8_unpack(table, n, mv, vv, _stream_ptr(None, exp_avgs[0]))
    if st != OK:
        _check(st, "tropical_adamw8_unpack")
    return exp_avg_values, exp_avg_sq_values


ACT8_BLOCK = 32  # TROP_ACT8_BLOCK in include/tropical.h

# A matrix held in 8 bits: int8 codes (rows, cols) and uint8 exponents
# (rows, ceil(cols / ACT8_BLOCK)).
Act8 = collections.namedtuple("Act8", ["codes", "exponents"])


def _act8(a, rows, cols, what):
    """The C structure of an Act8 of this shape."""
    codes, exponents = a
    if codes.dtype != torch.int8 or codes.shape != (rows, cols):
        raise ValueError(f"{what}: codes must be int8 of shape {(rows, cols)}")
    if exponents.dtype != torch.uint8 or exponents.shape != (rows, (cols + ACT8_BLOCK - 1) // ACT8_BLOCK):
        raise ValueError(f"{what}: exponents must be uint8, one for each {ACT8_BLOCK} elements of a row")
    return trop_act8(codes.data_ptr(), exponents.data_ptr(), _row_stride(codes, what), _row_stride(exponents, what))


def _new_act8(rows, cols, device):
    return Act8(_new_matrix(rows, cols, torch.int8, device),
                _new_matrix(rows, (cols + ACT8_BLOCK - 1) // ACT8_BLOCK, torch.uint8, device))


@_on_stream
def tropical_act8_pack(x, out=None):
    """The rows of x (float32 or bfloat16) in 8 bits: an Act8 (allocated when
    not given).  Each value is off by 1/127 of its block's largest magnitude at
    most; see include/tropical.h."""
    dt = _tdt(x, "x")
    ldx = _row_stride(x, "x")
    rows, cols = x.shape
    if out is None:
        out = _new_act8(rows, cols, x.device)
    st = lib().tropical_act8_pack(dt, x.data_ptr(), ldx, _act8(out, rows, cols, "out"), rows, cols,
                                  _stream_ptr(None, x))
    if st != OK:
        _check(st, "tropical_act8_pack")
    return out


@_on_stream
def tropical_act8_unpack(x8, dtype=torch.float32, out=None):
    """The values of an Act8 as float32 or bfloat16 (exact in both)."""
    rows, cols = x8[0].shape
    if out is not None:
        dtype = out.dtype
    if dtype not in _TRAIN_DTYPES:
        raise TypeError(f"out must be float32 or bfloat16, got {dtype}")
    out, po, ldo = _out_matrix(out, rows, cols, dtype, x8[0].device, "out")
    st = lib().tropical_act8_unpack(_act8(x8, rows, cols, "x8"), _TRAIN_DTYPES[dtype], po, ldo, rows, cols,
                                    _stream_ptr(None, out))
    if st != OK:
        _check(st, "tropical_act8_unpack")
    return out


@functools.lru_cache(maxsize=4096)
def _grad_w_workspace(dt, tokens, cols, out_features):
    nb = ctypes.c_size_t(0)
    _check(lib().tropical_act8_linear_grad_w_workspace_size(dt, tokens, cols, out_features, ctypes.byref(nb)),
           "tropical_act8_linear_grad_w_workspace_size")
    return nb.value


def tropical_act8_linear_grad_w_workspace_size(dtype, tokens, cols, out_features):
    """Workspace bytes of the weight gradient (dtype: torch.float32 or
    torch.bfloat16)."""
    if dtype not in _TRAIN_DTYPES:
        raise TypeError(f"float32 or bfloat16 only, got {dtype}")
    return _grad_w_workspace(_TRAIN_DTYPES[dtype], int(tokens), int(cols), int(out_features))


@_on_stream
def tropical_act8_linear_grad_w(dz, x8, grad_w=None, workspace=None):
    """dz.T @ x for a linear layer's input held in 8 bits.

    dz (tokens, out_features): float32 or bfloat16, unit stride along the
    rows.  x8: Act8 of (tokens, cols).  grad_w (out_features, cols) has dz's
    type; it and the workspace are allocated with torch when not given.
    """
    dt = _tdt(dz, "dz")
    lddz = _row_stride(dz, "dz")
    tokens, outs = dz.shape
    if x8[0].dim() != 2 or x8[0].shape[0] != tokens:
        raise ValueError(f"x8 must have dz's {tokens} rows")
    cols = x8[0].shape[1]
    x = _act8(x8, tokens, cols, "x8")
    grad_w, pw, ldw = _out_matrix(grad_w, outs, cols, dz.dtype, dz.device, "grad_w")
    need = 0
    if workspace is None:
        need = _grad_w_workspace(dt, tokens, cols, outs)
    workspace, wp, wn = _workspace(workspace, need, dz.device)
    st = lib().tropical_act8_linear_grad_w(dt, dz.data_ptr(), lddz, x, pw, ldw, tokens, cols, outs, wp, wn,
                                           _stream_ptr(None, dz))
    if st != OK:
        _check(st, "tropical_act8_linear_grad_w")
    return grad_w


_NORMS = {None: 0, "layer": 1, "rms": 2}
_WEIGHTS = ("post_gamma", "post_beta", "pre_gamma", "pre_beta")
_STATISTICS = ("post_mean", "post_rstd", "pre_mean", "pre_rstd")

ResidualNorm = collections.namedtuple("ResidualNorm", ["h", "y", "post_mean", "post_rstd", "pre_mean", "pre_rstd",
                                                       "u8", "h8"])
ResidualNormGrads = collections.namedtuple("ResidualNormGrads", ["r", "u", "gate", "post_gamma", "post_beta",
                                                                 "pre_gamma", "pre_beta"])


def _residual_op(dt, rows, cols, gate, gate_group, post, post_gamma, post_beta, post_eps, pre, pre_gamma, pre_beta,
                 pre_eps, residual_scale, branch_scale):
    """(C structure, weights' type)."""
    if post not in _NORMS or pre not in _NORMS:
        raise ValueError("norms are None, 'layer' or 'rms'")
    pdt, gdt, ptype = F32, F32, None
    weights = [None, None, None, None]
    i = 0
    for w in (post_gamma, post_beta, pre_gamma, pre_beta):
        if w is not None:
            name = _WEIGHTS[i]
            if (pre if i > 1 else post) is None:
                raise ValueError(f"{name} without its norm")
            if ptype is None:
                ptype = w.dtype
                pdt = _tdt(w, "gamma and beta")
            weights[i] = _flat(w, name, cols, ptype)
        i += 1
    pg, ldg, group = None, 0, 0
    if gate is not None:
        gdt = _tdt(gate, "gate")
        if gate.dim() == 1:
            pg, ldg, group = _flat(gate, "gate", cols, gate.dtype), cols, max(rows, 1)
        else:
            pg, ldg, group = gate.data_ptr(), _row_stride(gate, "gate"), gate_group
            gates, width = gate.shape
            if group is None:
                group = rows // gates if rows and gates else 1
                if rows and gates * group != rows:
                    raise ValueError(f"{gates} gate rows do not divide {rows} rows: give gate_group")
            if group < 1 or width != cols or (rows and gates != -(-rows // group)):
                raise ValueError(f"gate must have a row of {cols} for each {group} of {rows} rows")
    op = trop_residual_norm(dt, pdt, gdt, _NORMS[post], _NORMS[pre], residual_scale, branch_scale, post_eps, pre_eps,
                            rows, cols, pg, ldg, group, *weights)
    return op, ptype or torch.float32


@_on_stream
def tropical_residual_norm_forward(u, r=None, gate=None, post=None, post_gamma=None, post_beta=None, post_eps=1e-5,
                                   pre="layer", pre_gamma=None, pre_beta=None, pre_eps=1e-5, residual_scale=1.0,
                                   branch_scale=1.0, gate_group=None, h=True, y=True, hold_u=False, hold_h=False):
    """Between two residual blocks, in one pass:

        h = residual_scale r + branch_scale gate post_norm(u),  y = pre_norm(h)

    u (rows, cols), the block's output, and r, its input (None: left out):
    float32 or bfloat16, unit stride along the rows.  post, pre: None, 'layer'
    or 'rms', with weights of cols elements (float32 or u's type) or None.
    gate: cols elements for all rows, or (gates, cols) with a gate row for each
    gate_group consecutive rows (rows / gates when not given), float32 or u's
    type.  h, y: True to allocate, a tensor to fill (h may be r), None to skip.
    hold_u, hold_h: also leave u and h in 8 bits (True, or an Act8 to fill).
    Returns a ResidualNorm; what there is none of is None.  Statistics that the
    call allocates lie one after another in one allocation, which lives as long
    as any of them.
    """
    dt = _tdt(u, "u")
    ldu = _row_stride(u, "u")
    rows, cols = u.shape
    dev, dtype = u.device, u.dtype
    op, _ = _residual_op(dt, rows, cols, gate, gate_group, post, post_gamma, post_beta, post_eps, pre, pre_gamma,
                         pre_beta, pre_eps, residual_scale, branch_scale)
    pr = ldr = ph = ldh = py = ldy = 0
    if r is not None:
        if r.shape != u.shape or r.dtype != dtype:
            raise ValueError("r must have the shape and type of u")
        pr, ldr = r.data_ptr(), _row_stride(r, "r")
    if h is not None:
        h, ph, ldh = _out_matrix(h, rows, cols, dtype, dev, "h")
    if pre is None:
        if y is not None and y is not True:
            raise ValueError("y without a norm before the next block")
        y = None
    if y is not None:
        y, py, ldy = _out_matrix(y, rows, cols, dtype, dev, "y")
    io = [pr, ldr, u.data_ptr(), ldu, ph, ldh, py, ldy]
    stats = _new_flats((post == "layer", post is not None, pre == "layer", pre is not None), rows, torch.float32, dev)
    for t in stats:
        io.append(0 if t is None else t.data_ptr())
    held, alive = [None, None], []
    if hold_u is not None and hold_u is not False:
        held[0] = x = _new_act8(rows, cols, dev) if hold_u is True else hold_u
        alive.append(_act8(x, rows, cols, "hold_u"))
        io.append(ctypes.addressof(alive[-1]))
    else:
        io.append(0)
    if hold_h is not None and hold_h is not False:
        held[1] = x = _new_act8(rows, cols, dev) if hold_h is True else hold_h
        alive.append(_act8(x, rows, cols, "hold_h"))
        io.append(ctypes.addressof(alive[-1]))
    else:
        io.append(0)
    st = lib().tropical_residual_norm_forward(op, _rows_fields(*io), _stream_ptr(None, u))
    if st != OK:
        _check(st, "tropical_residual_norm_forward")
    return ResidualNorm(h, y, *stats, *held)


@_on_stream
def tropical_residual_norm_backward(dy, dh, u, h, post_mean=None, post_rstd=None, pre_mean=None, pre_rstd=None,
                                    gate=None, post=None, post_gamma=None, post_beta=None, post_eps=1e-5, pre="layer",
                                    pre_gamma=None, pre_beta=None, pre_eps=1e-5, residual_scale=1.0, branch_scale=1.0,
                                    gate_group=None, dr=True, du=True, dgate=True, dpost_gamma=True, dpost_beta=True,
                                    dpre_gamma=True, dpre_beta=True, workspace=None):
    """Gradients of tropical_residual_norm_forward, from dy and dh, those of y
    and h (dy is None without a pre norm; dh may be None with one).

    u, h: the forward's, both as they were (u's type) or both held in 8 bits
    (Act8), each None where it is not needed.  The statistics, weights, gate
    and scales are the forward's.  dr, du: True to allocate, a tensor to fill,
    None to skip; the others likewise, True meaning where the forward had that
    weight or gate.  Without rows the gradients of weights and gate are zeros.
    Gradients of gamma and beta that the call allocates lie one after another in
    one allocation, which lives as long as any of them.  The workspace is
    allocated with torch when not given.
    Returns a ResidualNormGrads.
    """
    lead = dy if dy is not None else dh
    if lead is None:
        raise ValueError("neither dy nor dh")
    dt = _tdt(lead, "dy and dh")
    lead_ld = _row_stride(lead, "dy" if dy is not None else "dh")
    shape, dtype, dev = lead.shape, lead.dtype, lead.device
    rows, cols = shape
    op, ptype = _residual_op(dt, rows, cols, gate, gate_group, post, post_gamma, post_beta, post_eps, pre, pre_gamma,
                             pre_beta, pre_eps, residual_scale, branch_scale)

    def matrix(t, what):
        if t.shape != shape or t.dtype != dtype:
            raise ValueError(f"{what} must be {dtype} of shape {(rows, cols)}")
        return t.data_ptr(), _row_stride(t, what)

    alive = []
    kept = [0, 0, 0, 0, 0, 0]  # u, h, u8, h8
    for i, t in ((0, u), (1, h)):
        if isinstance(t, torch.Tensor):
            kept[2 * i], kept[2 * i + 1] = matrix(t, "uh"[i])
        elif t is not None:
            alive.append(_act8(t, rows, cols, "uh"[i]))
            kept[4 + i] = ctypes.addressof(alive[-1])
    i = 0
    for t in (post_mean, post_rstd, pre_mean, pre_rstd):
        kept.append(0 if t is None else _flat(t, _STATISTICS[i], rows, torch.float32))
        i += 1
    if dy is not None:
        kept += (dy.data_ptr(), lead_ld)
        kept += matrix(dh, "dh") if dh is not None else (0, 0)
    else:
        kept += (0, 0, dh.data_ptr(), lead_ld)
    grads = [0] * 10
    if dr is not None:
        dr, grads[0], grads[1] = _out_matrix(dr, rows, cols, dtype, dev, "dr")
    if du is not None:
        du, grads[2], grads[3] = _out_matrix(du, rows, cols, dtype, dev, "du")
    if dgate is True:
        dgate = None
        if gate is not None:
            dgate = (torch.empty_strided((cols,), (1,), dtype=gate.dtype, device=dev) if gate.dim() == 1 else
                     _new_matrix(*gate.shape, gate.dtype, dev))
    if dgate is not None:
        if gate is None:
            raise ValueError("dgate without a gate")
        if dgate.shape != gate.shape or dgate.dtype != gate.dtype:
            raise ValueError("dgate must have the gate's shape and type")
        flat = dgate.dim() == 1
        grads[4] = _flat(dgate, "dgate", cols, gate.dtype) if flat else dgate.data_ptr()
        grads[5] = cols if flat else _row_stride(dgate, "dgate")
    given = (dpost_gamma, dpost_beta, dpre_gamma, dpre_beta)
    weights = _new_flats([g is True and w is not None for g, w in
                          zip(given, (post_gamma, post_beta, pre_gamma, pre_beta))], cols, ptype, dev)
    sums = dgate is not None
    for i in range(4):
        g = weights[i]
        if g is not None:
            grads[6 + i] = g.data_ptr()
        elif given[i] is not None and given[i] is not True:
            weights[i], grads[6 + i] = given[i], _flat(given[i], "d" + _WEIGHTS[i], cols, ptype)
        else:
            continue
        sums = True
    need = 0
    if workspace is None and sums:
        need = _residual_workspace(dt, rows, cols, op.post, op.pre, op.gate_group if gate is not None else None)
    workspace, wp, wn = _workspace(workspace, need, dev)
    st = lib().tropical_residual_norm_backward(op, _kept_fields(*kept), _grads_fields(*grads), wp, wn,
                                               _stream_ptr(None, lead))
    if st != OK:
        _check(st, "tropical_residual_norm_backward")
    if rows == 0 and dgate is not None:
        # (no row has a gate row: the call wrote none of those that are there)
        dgate.detach().zero_()
    return ResidualNormGrads(dr, du, dgate, *weights)


@functools.lru_cache(maxsize=4096)
def _residual_workspace(dt, rows, cols, post, pre, gate_group):
    op = trop_residual_norm(dtype=dt, post=post, pre=pre, rows=rows, cols=cols)
    if gate_group is not None:
        op.gate, op.gate_group = 1, gate_group
    nb = ctypes.c_size_t(0)
    _check(lib().tropical_residual_norm_backward_workspace_size(op, ctypes.byref(nb)),
           "tropical_residual_norm_backward_workspace_size")
    return nb.value


def tropical_residual_norm_backward_workspace_size(dtype, rows, cols, post=None, pre="layer", gate_group=None):
    """Workspace bytes of a backward (dtype: torch.float32 or torch.bfloat16;
    gate_group: None without a gate)."""
    if dtype not in _TRAIN_DTYPES:
        raise TypeError(f"float32 or bfloat16 only, got {dtype}")
    if post not in _NORMS or pre not in _NORMS:
        raise ValueError("norms are None, 'layer' or 'rms'")
    return _residual_workspace(_TRAIN_DTYPES[dtype], int(rows), int(cols), _NORMS[post], _NORMS[pre],
                               None if gate_group is None else int(gate_group))


def tropical_get_train_stats():
    s = trop_train_stats()
    _check(lib().tropical_get_train_stats(ctypes.byref(s)), "tropical_get_train_stats")
    return {"module_loads": s.module_loads, "launches_total": s.launches_total,
            "launches": {name: s.launches[i] for i, name in enumerate(TRAIN_FAMILIES)}}


def tropical_get_stats():
    s = trop_stats()
    _check(lib().tropical_get_stats(ctypes.byref(s)), "tropical_get_stats")
    return {"module_loads": s.module_loads, "launches_total": s.launches_total,
            "launches": {name: s.launches[i] for i, name in enumerate(KERNEL_FAMILIES)}}


def tropical_reset_stats():
    lib().tropical_reset_stats()


def tropical_last_error():
    return lib().tropical_last_error().decode(errors="replace")
