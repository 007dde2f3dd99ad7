"""Thin ctypes binding of libmhc_seam.so (C ABI in include/mhc_seam.h).

Argument marshalling only: every step of the seam runs in the library's HIP
kernels.  PyTorch supplies device memory and the stream.  The library is
loaded on first use; if it is missing this raises instead of computing
anything another way.
"""
from __future__ import annotations

import ctypes
import functools
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("MHC_SEAM_LIB") or os.path.join(HERE, "libmhc_seam.so")

OK, INVALID_ARG, UNSUPPORTED_DEVICE, OUT_OF_MEMORY, HIP_ERROR, CAPTURE_ALLOC = range(6)
FORMS = {"post": 0, "no_post": 1}
OUT_DTYPES = {"bf16": 0, "fp8_grid": 1, "mxfp8": 2, "mxfp8_g128": 3}

DTYPES = {"bf16": 0, "f16": 1, "f32": 2}
GATE_NONE, GATE_TOKEN, GATE_CHANNEL, GATE_ELEMENT = range(4)
SCORINGS = {"softmax": 0, "sigmoid": 1}

_P = ctypes.c_void_p


class Desc(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("n", ctypes.c_int32), ("eps", ctypes.c_float),
                ("sinkhorn_iters", ctypes.c_int32), ("fn", _P), ("gamma", _P), ("bias", _P),
                ("max_tokens", ctypes.c_int64), ("device", ctypes.c_int32),
                ("ksplit", ctypes.c_int32), ("spin_polls", ctypes.c_int32),
                ("reserved", ctypes.c_int32 * 6)]


class Args(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("form", ctypes.c_int32),
                ("identity_pre", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("unshifted", ctypes.c_int32),
                ("x", _P), ("y", _P), ("pre", _P), ("post", _P), ("res", _P),
                ("residual_out", _P), ("norm", _P), ("grid", _P), ("codes", _P),
                ("scales", _P), ("pre_out", _P), ("post_out", _P), ("res_out", _P)]


class Plan(ctypes.Structure):
    _fields_ = [("blocks", ctypes.c_int32), ("ksplit", ctypes.c_int32),
                ("segs_per_split", ctypes.c_int32), ("grid", ctypes.c_int32),
                ("row_segs", ctypes.c_int32), ("rows_blocks", ctypes.c_int32),
                ("reserved", ctypes.c_int32 * 2)]


class BlockNormArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("x_dtype", ctypes.c_int32), ("gate_kind", ctypes.c_int32),
                ("eps", ctypes.c_float), ("residual_scale", ctypes.c_float),
                ("branch_scale", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("x", _P), ("y", _P), ("gamma_post", _P), ("gate", _P), ("gamma", _P),
                ("residual_out", _P), ("norm", _P), ("codes", _P), ("scales", _P)]


class RouteArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scoring", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32),
                ("group_top", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("scale", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("logits", _P), ("bias", _P), ("weights", _P), ("ids", _P)]


class RopeArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("q_heads", ctypes.c_int32), ("k_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("rotary", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("position_bytes", ctypes.c_int32),
                ("axes", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("inverse", ctypes.c_int32), ("scale", ctypes.c_float),
                ("position_axis", ctypes.c_int64),
                ("q_token", ctypes.c_int64), ("q_head", ctypes.c_int64),
                ("k_token", ctypes.c_int64), ("k_head", ctypes.c_int64),
                ("q_out_token", ctypes.c_int64), ("q_out_head", ctypes.c_int64),
                ("k_out_token", ctypes.c_int64), ("k_out_head", ctypes.c_int64),
                ("q", _P), ("k", _P), ("positions", _P), ("inv_freq", _P), ("pair_axis", _P),
                ("q_out", _P), ("k_out", _P)]


class CacheArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("slot_bytes", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("k_token", ctypes.c_int64),
                ("k_head", ctypes.c_int64), ("v_token", ctypes.c_int64),
                ("v_head", ctypes.c_int64), ("cache", _P), ("slots", _P), ("k", _P), ("v", _P)]


class CacheAttentionArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("max_len", ctypes.c_int64), ("pages", ctypes.c_int64),
                ("q_token", ctypes.c_int64), ("q_head", ctypes.c_int64),
                ("table_stride", ctypes.c_int64), ("B", ctypes.c_int32),
                ("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("table_width", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("window", ctypes.c_int32), ("scale", ctypes.c_float),
                ("softcap", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("q", _P), ("cache", _P), ("tables", _P), ("lens", _P), ("q_starts", _P),
                ("out", _P), ("lse", _P), ("workspace", _P), ("workspace_bytes", ctypes.c_uint64)]


EXPORTS = ("mhc_seam_create", "mhc_seam_run", "mhc_seam_run_noalloc", "mhc_seam_destroy",
           "mhc_seam_validate",
           "mhc_seam_plan_for", "mhc_seam_status_string", "mhc_seam_last_error",
           "mhc_seam_copy", "mhc_stream_mix", "mhc_seam_quantize", "mhc_head_reduce",
           "mhc_mxfp8_gemm", "mhc_mxfp8_gemm_blocks", "mhc_block_norm", "mhc_int8_quantize",
           "mhc_int8_gemm", "mhc_int8_gemm_blocks", "mhc_route", "mhc_rope", "mhc_cache_write",
           "mhc_cache_read", "mhc_cache_attention", "mhc_cache_attention_workspace")

_lib = None


class SeamError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"mhc_seam status {status}: {message}")
        self.status = status


def lib():
    """Load libmhc_seam.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m layer_mhc_seam_amd.build` (hipcc, gfx950)")
    L = ctypes.CDLL(LIB_PATH)
    L.mhc_seam_create.argtypes = [ctypes.POINTER(Desc), ctypes.POINTER(_P)]
    L.mhc_seam_run.argtypes = [_P, ctypes.POINTER(Args), _P]
    L.mhc_seam_run_noalloc.argtypes = [_P, ctypes.POINTER(Args), _P]
    L.mhc_seam_destroy.argtypes = [_P]
    L.mhc_seam_validate.argtypes = [ctypes.POINTER(Desc), ctypes.POINTER(Args)]
    L.mhc_seam_plan_for.argtypes = [ctypes.c_int32, ctypes.c_int64, ctypes.c_int32,
                                    ctypes.c_int32, ctypes.POINTER(Plan)]
    L.mhc_seam_status_string.argtypes = [ctypes.c_int]
    L.mhc_seam_status_string.restype = ctypes.c_char_p
    L.mhc_seam_last_error.restype = ctypes.c_char_p
    L.mhc_seam_copy.argtypes = [_P, _P, ctypes.c_size_t, _P]
    L.mhc_stream_mix.argtypes = [_P, ctypes.c_size_t, _P, ctypes.c_size_t, _P]
    L.mhc_head_reduce.argtypes = [_P, _P, ctypes.c_int64, ctypes.c_int32, _P, _P]
    L.mhc_mxfp8_gemm.argtypes = [_P, _P, _P, _P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                 _P, _P]
    L.mhc_seam_quantize.argtypes = [_P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                    _P, _P, _P, _P]
    L.mhc_mxfp8_gemm_blocks.argtypes = [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                        ctypes.POINTER(ctypes.c_int32),
                                        ctypes.POINTER(ctypes.c_int32),
                                        ctypes.POINTER(ctypes.c_int32)]
    L.mhc_block_norm.argtypes = [ctypes.POINTER(BlockNormArgs), _P]
    L.mhc_int8_quantize.argtypes = [_P, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, _P, _P, _P]
    L.mhc_int8_gemm.argtypes = [_P, _P, _P, _P, _P, ctypes.c_int64, ctypes.c_int32,
                                ctypes.c_int32, ctypes.c_int32, _P, _P]
    L.mhc_route.argtypes = [ctypes.POINTER(RouteArgs), _P]
    L.mhc_int8_gemm_blocks.argtypes = [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                       ctypes.POINTER(ctypes.c_int32),
                                       ctypes.POINTER(ctypes.c_int32)]
    L.mhc_rope.argtypes = [ctypes.POINTER(RopeArgs), _P]
    L.mhc_cache_write.argtypes = [ctypes.POINTER(CacheArgs), _P]
    L.mhc_cache_read.argtypes = [ctypes.POINTER(CacheArgs), _P]
    L.mhc_cache_attention.argtypes = [ctypes.POINTER(CacheAttentionArgs), _P]
    L.mhc_cache_attention_workspace.argtypes = [ctypes.c_int64, *[ctypes.c_int32] * 5,
                                                ctypes.c_int64, ctypes.POINTER(ctypes.c_uint64)]
    for name in ("mhc_block_norm", "mhc_int8_quantize", "mhc_int8_gemm", "mhc_int8_gemm_blocks",
                 "mhc_route", "mhc_rope", "mhc_cache_write", "mhc_cache_read",
                 "mhc_cache_attention", "mhc_cache_attention_workspace"):
        getattr(L, name).restype = ctypes.c_int
    for name in ("mhc_seam_create", "mhc_seam_run", "mhc_seam_run_noalloc", "mhc_seam_destroy",
                 "mhc_seam_validate",
                 "mhc_seam_plan_for", "mhc_seam_copy", "mhc_stream_mix", "mhc_seam_quantize",
                 "mhc_mxfp8_gemm_blocks"):
        getattr(L, name).restype = ctypes.c_int
    _lib = L
    return L


def _check(status):
    if status != OK:
        raise SeamError(status, lib().mhc_seam_last_error().decode())


def plan(H, T, cu_count=256, ksplit=0):
    """Launch plan the library would use (host only)."""
    p = Plan()
    _check(lib().mhc_seam_plan_for(H, T, cu_count, ksplit, ctypes.byref(p)))
    return dict(blocks=p.blocks, ksplit=p.ksplit, segs_per_split=p.segs_per_split,
                grid=p.grid, row_segs=p.row_segs, rows_blocks=p.rows_blocks)


def gemm_blocks(T, N, cu_count=256):
    """Output blocks (TM, TN) and LDS stages mhc_mxfp8_gemm launches for
    T x N on cu_count CUs (host only)."""
    tm, tn, st = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(lib().mhc_mxfp8_gemm_blocks(T, N, cu_count, ctypes.byref(tm), ctypes.byref(tn),
                                       ctypes.byref(st)))
    return tm.value, tn.value, st.value


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


class Seam:
    """A seam handle: packed fn, gamma and bias for one width H.

    fn f32 [4H,24], gamma bf16 [H], bias f32 [24]: device tensors, copied by
    the library at creation.
    """

    def __init__(self, fn, gamma, bias, *, max_tokens, eps=1e-6, sinkhorn_iters=20,
                 ksplit=0, spin_polls=0):
        import torch
        H = gamma.shape[0]
        self._check_tensor("fn", fn, torch.float32, (4 * H, 24))
        self._check_tensor("gamma", gamma, torch.bfloat16, (H,))
        self._check_tensor("bias", bias, torch.float32, (24,))
        d = Desc()
        d.H, d.n, d.eps, d.sinkhorn_iters = H, 4, eps, sinkhorn_iters
        d.fn, d.gamma, d.bias = fn.data_ptr(), gamma.data_ptr(), bias.data_ptr()
        d.max_tokens = max_tokens
        d.device = fn.device.index if fn.device.index is not None else torch.cuda.current_device()
        d.ksplit = ksplit
        d.spin_polls = spin_polls
        h = _P()
        _check(lib().mhc_seam_create(ctypes.byref(d), ctypes.byref(h)))
        self._h = h
        self.H, self.max_tokens, self.device = H, max_tokens, fn.device

    @staticmethod
    def _check_tensor(name, t, dtype, shape):
        if t is None:
            raise ValueError(f"{name} is required")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")

    def run(self, x, y=None, pre=None, post=None, res=None, *, form="post",
            identity_pre=False, out_dtype="bf16", unshifted=False, out=None, stream=None,
            noalloc=False):
        """Enqueue one seam on `stream` (default: torch's current stream).

        noalloc: call mhc_seam_run_noalloc, whose split-mode scratch is the
        library's fixed per-GPU array (pass every output in `out` to keep
        the call free of allocations).

        unshifted: gates from x' first, then the collapse with the fresh pre
        (pre_out) instead of a carried one; takes no pre.
        Returns a dict of output tensors (allocated unless given in `out`):
        residual_out (post form), norm, grid (fp8_grid), codes and scales
        (mxfp8, uint8), pre_out, post_out, res_out.
        """
        import torch
        T, H = x.shape[0], self.H
        dev = x.device
        post_form = form == "post"
        self._check_tensor("x", x, torch.bfloat16, (T, 4, H))
        if post_form:
            self._check_tensor("y", y, torch.bfloat16, (T, H))
            self._check_tensor("post", post, torch.float32, (T, 4))
            self._check_tensor("res", res, torch.float32, (T, 4, 4))
        elif any(v is not None for v in (y, post, res)):
            raise ValueError("no_post form takes no y, post or res")
        if unshifted:
            if pre is not None or identity_pre:
                raise ValueError("unshifted takes no pre and no identity_pre")
        elif not identity_pre:
            self._check_tensor("pre", pre, torch.float32, (T, 4))
        elif pre is not None:
            raise ValueError("identity_pre takes no pre")
        o = dict(out or {})

        def want(name, shape, dtype):
            if name not in o:
                o[name] = torch.empty(shape, dtype=dtype, device=dev)
            self._check_tensor(name, o[name], dtype, shape)

        if post_form:
            want("residual_out", (T, 4, H), torch.bfloat16)
        want("norm", (T, H), torch.bfloat16)
        if out_dtype == "fp8_grid":
            want("grid", (T, H), torch.bfloat16)
        if out_dtype in ("mxfp8", "mxfp8_g128"):
            want("codes", (T, H), torch.uint8)
            want("scales", (T, H // (128 if out_dtype == "mxfp8_g128" else 32)), torch.uint8)
        want("pre_out", (T, 4), torch.float32)
        want("post_out", (T, 4), torch.float32)
        want("res_out", (T, 4, 4), torch.float32)
        a = Args()
        a.T, a.form, a.identity_pre = T, FORMS[form], int(bool(identity_pre))
        a.out_dtype = OUT_DTYPES[out_dtype]
        a.unshifted = int(bool(unshifted))
        a.x, a.y, a.pre, a.post, a.res = (_ptr(x), _ptr(y), _ptr(pre), _ptr(post), _ptr(res))
        a.residual_out = _ptr(o.get("residual_out"))
        a.norm, a.grid = _ptr(o["norm"]), _ptr(o.get("grid"))
        a.codes, a.scales = _ptr(o.get("codes")), _ptr(o.get("scales"))
        a.pre_out, a.post_out = _ptr(o["pre_out"]), _ptr(o["post_out"])
        a.res_out = _ptr(o["res_out"])
        entry = lib().mhc_seam_run_noalloc if noalloc else lib().mhc_seam_run
        _check(entry(self._h, ctypes.byref(a), _stream_handle(stream)))
        return o

    def close(self):
        if getattr(self, "_h", None):
            _check(lib().mhc_seam_destroy(self._h))
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def quantize(src, *, group=32, codes=True, grid=True, stream=None):
    """MXFP8 quantisation of a bf16 [rows, H] device tensor in groups of
    `group` (32 or 128) elements with the seam's device quantiser.  Returns
    (codes u8, scales u8 [rows, H/group], grid bf16); the parts not asked for
    are None."""
    import torch
    rows, H = src.shape
    if src.dtype != torch.bfloat16 or not src.is_cuda or not src.is_contiguous():
        raise ValueError("src must be a contiguous bf16 device tensor")
    c = torch.empty((rows, H), dtype=torch.uint8, device=src.device) if codes else None
    sc = torch.empty((rows, H // group), dtype=torch.uint8, device=src.device) if codes else None
    g = torch.empty_like(src) if grid else None
    _check(lib().mhc_seam_quantize(_ptr(src), rows, H, group, _ptr(c), _ptr(sc), _ptr(g),
                                   _stream_handle(stream)))
    return c, sc, g


def copy(dst, src, nbytes, stream=None):
    """The library's 16-byte non-temporal device copy (bandwidth ceiling)."""
    _check(lib().mhc_seam_copy(_ptr(dst), _ptr(src), nbytes, _stream_handle(stream)))


def stream_mix(dst, dst_bytes, src, src_bytes, stream=None):
    """The library's read-src_bytes / write-dst_bytes streaming kernel (the
    copy ceiling at another read/write mix)."""
    _check(lib().mhc_stream_mix(_ptr(dst), dst_bytes, _ptr(src), src_bytes,
                                _stream_handle(stream)))


def head_reduce(x, w=None, *, out=None, stream=None):
    """n -> 1 reduction of the streams, stored: out[t, h] = bf16(sum_i
    w[t, i] * x[t, i, h]) (the seam's collapse chain) on the device.
    x bf16 [T, 4, H], w f32 [T, 4] or None for weights of 1/4.  Returns
    out bf16 [T, H] (allocated unless given)."""
    import torch
    if x.dtype != torch.bfloat16 or not x.is_cuda or not x.is_contiguous() or x.dim() != 3 \
            or x.shape[1] != 4:
        raise ValueError("x must be a contiguous bf16 [T, 4, H] device tensor")
    T, _, H = x.shape
    if w is not None and (w.dtype != torch.float32 or tuple(w.shape) != (T, 4)
                          or not w.is_contiguous() or w.device != x.device):
        raise ValueError("w must be a contiguous f32 [T, 4] tensor on x's device")
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=x.device)
    elif out.dtype != torch.bfloat16 or tuple(out.shape) != (T, H) or not out.is_contiguous() \
            or out.device != x.device:
        raise ValueError("out must be a contiguous bf16 [T, H] tensor on x's device")
    _check(lib().mhc_head_reduce(_ptr(x), _ptr(w), T, H, _ptr(out), _stream_handle(stream)))
    return out


def mxfp8_gemm(a, a_scales, b, b_scales, *, out=None, stream=None):
    """Consumer GEMM of MXFP8 operands along K on the device: out[t, n] =
    bf16(sum_k a(t, k) b(n, k)).  a u8 [T, K] e4m3fn codes with a_scales u8
    [T, K/32] ue8m0 (the seam's mxfp8 output as it is), b u8 [N, K] and
    b_scales u8 [N, K/32] (weights).  Returns out bf16 [T, N]."""
    import torch
    T, K = a.shape
    N = b.shape[0]
    for name, t, shape in (("a", a, (T, K)), ("a_scales", a_scales, (T, K // 32)),
                           ("b", b, (N, K)), ("b_scales", b_scales, (N, K // 32))):
        if t.dtype != torch.uint8 or tuple(t.shape) != shape or not t.is_contiguous() \
                or t.device != a.device or not t.is_cuda:
            raise ValueError(f"{name} must be a contiguous u8 {shape} device tensor")
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=a.device)
    elif out.dtype != torch.bfloat16 or tuple(out.shape) != (T, N) or not out.is_contiguous() \
            or out.device != a.device:
        raise ValueError("out must be a contiguous bf16 [T, N] tensor on a's device")
    _check(lib().mhc_mxfp8_gemm(_ptr(a), _ptr(a_scales), _ptr(b), _ptr(b_scales), T, N, K,
                                _ptr(out), _stream_handle(stream)))
    return out


# ------------------------------------------------ one-stream block boundary --
#
# Unlike the calls above, these run on the device their tensors are on,
# whichever is current, and on that device's current stream.  A `stream` of
# their own has to come after what made the tensors, as ever; it gets the
# outputs' memory too.  Tensors are dense and start on 16 bytes (route's, and
# scales and biases, on their elements): a slice that does not is refused.

@functools.lru_cache(maxsize=None)
def _types():
    """torch's types by the names of DTYPES, and their codes by type."""
    import torch
    types = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
    return types, {t: DTYPES[n] for n, t in types.items()}


def _need(name, t, dtype, shape, index):
    """t is a dense tensor of that type and shape on that device."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == index >= 0 \
            and t.is_contiguous():
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} must be a tensor on cuda:{index}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _new(rows, cols, dtype, device):
    """An uninitialised dense [rows, cols] (the cheapest way to one: 1.3 us
    against torch.empty's 1.7)."""
    import torch
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _enqueue(index, call, *args):
    """call(*args, stream) on that device and its current stream.  (Stream
    handle and device are asked for as they are: a Stream object takes 2 us,
    as long as a small kernel's whole launch.)"""
    import torch
    handle = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        status = call(*args, handle)
    else:
        with torch.cuda.device(index):
            status = call(*args, handle)
    if status != OK:
        _check(status)


def _tensors(v):
    """The tensors in v: itself, or what a dict, tuple or list holds."""
    import torch
    if isinstance(v, torch.Tensor):
        return (v,)
    if isinstance(v, dict):
        v = v.values()
    elif not isinstance(v, (tuple, list)):
        return ()
    return tuple(t for t in v if isinstance(t, torch.Tensor))


def _on_stream(stream, op, *args, **kw):
    """op(*args, **kw) with `stream` current, so that its outputs are allocated
    there.  The memory of the tensors given is not handed on by the allocator
    before the stream is done with them: of the inputs, and of the outputs,
    which the result holds whatever `out` gave them in."""
    import torch
    if stream.device != args[0].device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {args[0].device}")
    with torch.cuda.stream(stream):
        result = op(*args, **kw)
    used = {id(t): t for v in (*args, *kw.values(), result) for t in _tensors(v)}
    for t in used.values():
        t.record_stream(stream)
    return result


def _fits(bits):
    """Sizes, or'ed together, that the library takes: ctypes would cut longer
    ones to their low 32 bits."""
    if bits >> 31 not in (0, -1):
        raise ValueError("a size is out of range")


def _address(t):
    return None if t is None else t.data_ptr()


def block_norm(x, gamma=None, y=None, *, gamma_post=None, gate=None, residual_scale=1.0,
               branch_scale=1.0, eps=1e-6, norm=True, int8=False, out=None, stream=None):
    """Norms before and after a sub-layer with its gate and residual scale:
    r = residual_scale x + branch_scale gate p with p = rmsnorm(y) gamma_post
    (or y), stored as residual_out, and norm = rmsnorm(r) gamma.

    x [T, H] (bf16 or f16, or f32 beside either), y [T, H], gamma and
    gamma_post [H] bf16 or f16.  gate: f32 [T, 1] (token), f32 [H] (channel)
    or y's type [T, H] (element).  Without y: the norm of x alone.  Without
    gamma: residual_out alone.  int8: also the norm's codes (int8 [T, H]) and
    scales (f32 [T]), the operand of int8_gemm; norm=False then leaves the
    norm itself out.
    H up to 32768, or 32752 if no multiple of 8.  eps in [0, 1]; 0 selects
    1e-6.
    Returns a dict of outputs (allocated unless given in `out`, a dict too;
    residual_out may be x)."""
    import torch
    if stream is not None:
        return _on_stream(stream, block_norm, x, gamma, y, gamma_post=gamma_post, gate=gate,
                          residual_scale=residual_scale, branch_scale=branch_scale, eps=eps,
                          norm=norm, int8=int8, out=out)
    if x.dim() != 2:
        raise ValueError("x must be [T, H]")
    T, H = shape = x.shape
    _fits(H)
    index = x.get_device()
    codes = _types()[1]
    dt = gamma.dtype if gamma is not None else None if y is None else y.dtype
    if dt is None:
        raise ValueError("block_norm needs y, gamma or both")
    if dt is not torch.bfloat16 and dt is not torch.float16:
        raise ValueError(f"gamma and y must be bfloat16 or float16, got {dt}")
    x_dt = torch.float32 if x.dtype is torch.float32 else dt
    _need("x", x, x_dt, shape, index)
    y_at = post_at = gate_at = gamma_at = r_at = n_at = c_at = s_at = None
    o = {} if out is None else dict(out)
    given, writes = len(o), 0
    if y is not None:
        _need("y", y, dt, shape, index)
        y_at = y.data_ptr()
        r = o.get("residual_out")
        if r is None:
            r = o["residual_out"] = torch.empty_like(x)   # x is dense
        else:
            _need("residual_out", r, x_dt, shape, index)
            writes += 1
        r_at = r.data_ptr()
    if gamma is not None:
        _need("gamma", gamma, dt, (H,), index)
        gamma_at = gamma.data_ptr()
        if norm:
            n = o.get("norm")
            if n is None:
                n = o["norm"] = torch.empty_like(x, dtype=dt)
            else:
                _need("norm", n, dt, shape, index)
                writes += 1
            n_at = n.data_ptr()
    if int8:
        if gamma is None:
            raise ValueError("int8 codes are those of the norm: give gamma")
        c, s = o.get("codes"), o.get("scales")
        if c is None:
            c = o["codes"] = torch.empty_like(x, dtype=torch.int8)
        else:
            _need("codes", c, torch.int8, shape, index)
            writes += 1
        if s is None:
            s = o["scales"] = torch.empty((T,), dtype=torch.float32, device=x.device)
        else:
            _need("scales", s, torch.float32, (T,), index)
            writes += 1
        c_at, s_at = c.data_ptr(), s.data_ptr()
    if writes != given:
        raise ValueError(f"out holds more than this call writes: {', '.join(out)}")
    if gamma_post is not None:
        _need("gamma_post", gamma_post, dt, (H,), index)
        post_at = gamma_post.data_ptr()
    kind = GATE_NONE
    if gate is not None:
        if gate.dtype is not torch.float32:
            kind = GATE_ELEMENT
            _need("gate", gate, dt, shape, index)
        elif gate.dim() == 1:
            kind = GATE_CHANNEL
            _need("gate", gate, torch.float32, (H,), index)
        else:
            kind = GATE_TOKEN
            _need("gate", gate, torch.float32, (T, 1), index)
        gate_at = gate.data_ptr()
    a = BlockNormArgs(T, H, codes[dt], codes[x_dt], kind, eps, residual_scale, branch_scale, 0,
                      x.data_ptr(), y_at, post_at, gate_at, gamma_at, r_at, n_at, c_at, s_at)
    _enqueue(index, lib().mhc_block_norm, ctypes.byref(a))
    return o


def int8_quantize(src, *, out=None, stream=None):
    """int8 codes [rows, H] and f32 scales [rows] of a bf16 or f16 [rows, H]
    device tensor, one scale a row: the operands of int8_gemm, which takes
    widths that are multiples of 16.  H up to 32768, or 32752 if no multiple of
    8.  out: the pair to write to."""
    import torch
    if stream is not None:
        return _on_stream(stream, int8_quantize, src, out=out)
    if src.dim() != 2:
        raise ValueError("src must be [rows, H]")
    if src.dtype is not torch.bfloat16 and src.dtype is not torch.float16:
        raise ValueError(f"src must be bfloat16 or float16, got {src.dtype}")
    rows, H = src.shape
    _fits(H)
    index = src.get_device()
    _need("src", src, src.dtype, (rows, H), index)
    if out is None:
        codes = torch.empty_like(src, dtype=torch.int8)
        scales = torch.empty((rows,), dtype=torch.float32, device=src.device)
    else:
        codes, scales = out
        _need("codes", codes, torch.int8, (rows, H), index)
        _need("scales", scales, torch.float32, (rows,), index)
    _enqueue(index, lib().mhc_int8_quantize, src.data_ptr(), _types()[1][src.dtype],
             rows, H, codes.data_ptr(), scales.data_ptr())
    return codes, scales


def int8_gemm(a, a_scales, b, b_scales, bias=None, *, out_dtype="bf16", out=None, stream=None):
    """Product of int8 codes with a scale for each token and channel:
    out[t, n] = sum_k a[t, k] b[n, k] * a_scales[t] * b_scales[n] (+ bias[n]).
    a int8 [T, K], a_scales f32 [T] (block_norm's or int8_quantize's), b int8
    [N, K], b_scales and bias f32 [N]; out_dtype bf16, f16 or f32.  K a
    multiple of 16, up to 131056; any N."""
    import torch
    if stream is not None:
        return _on_stream(stream, int8_gemm, a, a_scales, b, b_scales, bias, out_dtype=out_dtype,
                          out=out)
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError("a must be [T, K] and b [N, K]")
    T, K = a.shape
    N = b.shape[0]
    _fits(N | K)
    index = a.get_device()
    if out_dtype not in DTYPES:
        raise ValueError(f"out_dtype must be one of {', '.join(DTYPES)}")
    dt = _types()[0][out_dtype]
    _need("a", a, torch.int8, (T, K), index)
    _need("a_scales", a_scales, torch.float32, (T,), index)
    _need("b", b, torch.int8, (N, K), index)
    _need("b_scales", b_scales, torch.float32, (N,), index)
    if bias is not None:
        _need("bias", bias, torch.float32, (N,), index)
    if out is None:
        out = _new(T, N, dt, a.device)
    else:
        _need("out", out, dt, (T, N), index)
    _enqueue(index, lib().mhc_int8_gemm, a.data_ptr(), a_scales.data_ptr(), b.data_ptr(),
             b_scales.data_ptr(), _address(bias), T, N, K, DTYPES[out_dtype], out.data_ptr())
    return out


def int8_gemm_blocks(T, N, cu_count=256):
    """Output blocks (TM, TN) int8_gemm launches for T x N on cu_count CUs
    (host only)."""
    _fits(N | cu_count)
    tm, tn = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().mhc_int8_gemm_blocks(T, N, cu_count, ctypes.byref(tm), ctypes.byref(tn)))
    return tm.value, tn.value


def route(logits, k, *, scoring="softmax", bias=None, groups=1, topk_groups=1, group_top=1,
          renormalize=True, scale=1.0, out=None, stream=None):
    """Routing of tokens to experts: of logits [T, E] (f32, bf16 or f16) the k
    experts of the highest score + bias in the topk_groups best groups, and
    their scores (softmax or sigmoid), renormalized and times scale.  bias f32
    [E].  A group's score is the sum of its group_top (1 or 2) highest keys.
    Returns (weights f32 [T, k], ids int32 [T, k]), highest first; id -1 and
    weight 0 where masks (-inf) leave fewer than k experts.  E up to 1024, k
    and groups up to 64.  out: the pair to write to."""
    import torch
    if stream is not None:
        return _on_stream(stream, route, logits, k, scoring=scoring, bias=bias, groups=groups,
                          topk_groups=topk_groups, group_top=group_top, renormalize=renormalize,
                          scale=scale, out=out)
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    if logits.dtype not in _types()[1]:
        raise ValueError(f"logits must be float32, bfloat16 or float16, got {logits.dtype}")
    if scoring not in SCORINGS:
        raise ValueError(f"scoring must be one of {', '.join(SCORINGS)}")
    T, E = logits.shape
    _fits(E | k | groups | topk_groups | group_top)
    index = logits.get_device()
    _need("logits", logits, logits.dtype, (T, E), index)
    if bias is not None:
        _need("bias", bias, torch.float32, (E,), index)
    if out is None:
        dev = logits.device
        weights = _new(T, k, torch.float32, dev)
        ids = _new(T, k, torch.int32, dev)
    else:
        weights, ids = out
        _need("weights", weights, torch.float32, (T, k), index)
        _need("ids", ids, torch.int32, (T, k), index)
    a = RouteArgs(T, E, k, _types()[1][logits.dtype], SCORINGS[scoring], groups, topk_groups,
                  group_top, int(bool(renormalize)), scale, 0, logits.data_ptr(), _address(bias),
                  weights.data_ptr(), ids.data_ptr())
    _enqueue(index, lib().mhc_route, ctypes.byref(a))
    return weights, ids


# ------------------------------------------- attention over a 4-bit cache --
#
# Streams and devices as above.  q, k and v may be slices of wider rows, a
# qkv product's say: their channels are dense, strides else are free.

def _head_strides(name, t, dtype, shape, index):
    """(token, head) strides of t, [T, heads, D] of that type and shape on that
    device with dense channels.  An axis of one takes the stride it would have."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or index < 0:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a device tensor")
        if t.get_device() != index:
            raise ValueError(f"{name} must be a tensor on cuda:{index}")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    token, head, channel = t.stride()
    if channel != 1 and shape[2] > 1:
        raise ValueError(f"{name}'s channels must be dense")
    if shape[1] == 1:
        head = shape[2]
    if shape[0] <= 1:
        token = head * shape[1]
    return token, head


def _dense_like(t):
    """An uninitialised dense tensor of t's type and [T, heads, D] shape."""
    import torch
    if t.is_contiguous():
        return torch.empty_like(t)
    T, H, D = t.shape
    return torch.empty_strided((T, H, D), (H * D, D, 1), dtype=t.dtype, device=t.device)


@functools.lru_cache(maxsize=64)
def _pair_axes(axes, pairs, most):
    """axes, one for each pair, as the library's bytes."""
    if len(axes) != pairs or any(type(a) is not int or not 0 <= a < most for a in axes):
        raise ValueError(f"axes must be {pairs} whole numbers from 0 to {most - 1}")
    return (ctypes.c_uint8 * pairs)(*axes)


_WHOLE = {}


def _whole_bytes(name, t):
    """Bytes of int32 or int64 elements."""
    if not _WHOLE:
        import torch
        _WHOLE.update({torch.int32: 4, torch.int64: 8})
    size = _WHOLE.get(t.dtype)
    if size is None:
        raise ValueError(f"{name} must be int32 or int64, got {t.dtype}")
    return size


def rope(q, k, positions, inv_freq, *, axes=None, interleaved=False, inverse=False, scale=1.0,
         out=None, stream=None):
    """Rotary positions: pair i of the first 2 len(inv_freq) channels of q
    [T, Hq, D] and k [T, Hk, D] (bf16 or f16; k may be None) turns by
    positions * inv_freq[i] and is multiplied with scale; pairs are channels i
    and i + len(inv_freq), or 2 i and 2 i + 1 if interleaved.  positions [T],
    or [A, T] for up to four axes (time, height, width), of which axes[i] is
    pair i's: [0] * 16 + [1] * 24 + [2] * 24, or 0, 1, 2 in turn.  int32 or
    int64, any size: theta is taken in 64 bits.  inv_freq f32 [R / 2].
    inverse turns the other way: rope(dq, dk, ..., inverse=True) is the
    gradient.
    Returns (q', k'), dense, or written to the pair given in `out`, (q, k)
    itself for one."""
    import torch
    if stream is not None:
        return _on_stream(stream, rope, q, k, positions, inv_freq, axes=axes,
                          interleaved=interleaved, inverse=inverse, scale=scale, out=out)
    if q.dim() != 3 or (k is not None and k.dim() != 3):
        raise ValueError("q and k must be [T, heads, D]")
    if q.dtype is not torch.bfloat16 and q.dtype is not torch.float16:
        raise ValueError(f"q must be bfloat16 or float16, got {q.dtype}")
    T, Hq, D = q.shape
    Hk = 0 if k is None else k.shape[1]
    pairs = inv_freq.numel()
    _fits(Hq | Hk | D | pairs * 2)
    index = q.get_device()
    dt = q.dtype
    qs = _head_strides("q", q, dt, q.shape, index)
    _need("inv_freq", inv_freq, torch.float32, (pairs,), index)
    if positions.dim() not in (1, 2) or positions.shape[-1] != T:
        raise ValueError(f"positions must be [{T}] or [axes, {T}], got {tuple(positions.shape)}")
    if positions.get_device() != index:
        raise ValueError(f"positions must be a tensor on cuda:{index}")
    most = positions.shape[0] if positions.dim() == 2 else 1
    if T > 1 and positions.stride(-1) != 1:
        raise ValueError("each axis of positions must be dense")
    of_axis = positions.stride(0) if most > 1 else T
    table = None if axes is None else _pair_axes(tuple(axes), pairs, most)
    ks = (0, 0)
    if k is not None:
        ks = _head_strides("k", k, dt, (T, Hk, D), index)
        if Hk == 0:
            raise ValueError("k has no heads: give None")
    if out is None:
        qo, ko = _dense_like(q), None if k is None else _dense_like(k)
        qos, kos = (Hq * D, D), (Hk * D, D)
    else:
        qo, ko = out
        if (ko is None) != (k is None):
            raise ValueError("out must be a pair (q, k), k None exactly where k is")
        qos = _head_strides("out's q", qo, dt, (T, Hq, D), index)
        kos = (0, 0) if ko is None else _head_strides("out's k", ko, dt, (T, Hk, D), index)
    a = RopeArgs(T, Hq, Hk, D, 2 * pairs, _types()[1][dt], _whole_bytes("positions", positions), most,
                 bool(interleaved), bool(inverse), scale, of_axis, *qs, *ks, *qos, *kos,
                 q.data_ptr(), _address(k), positions.data_ptr(), inv_freq.data_ptr(),
                 None if table is None else ctypes.addressof(table), qo.data_ptr(), _address(ko))
    _enqueue(index, lib().mhc_rope, ctypes.byref(a))
    return qo, ko


def kv_cache(pages, heads, head_dim, page_size=64, *, device="cuda"):
    """An empty 4-bit cache: u8 [pages, heads, page_size * (head_dim +
    head_dim / 16)] of zeros, codes and scales of keys and values.  Slot
    page * page_size + i is place i of a page.  head_dim 64, 128 or 256,
    page_size a multiple of 16 up to 512."""
    import torch
    if head_dim not in (64, 128, 256) or page_size not in range(16, 513, 16):
        raise ValueError("head_dim must be 64, 128 or 256, page_size a multiple of 16 up to 512")
    return torch.zeros((pages, heads, page_size * (head_dim + head_dim // 16)), dtype=torch.uint8,
                       device=device)


@functools.lru_cache(maxsize=256)
def _pages_of(shape, heads, D):
    """(pages, page_size) of a cache of that shape for those heads."""
    if len(shape) != 3:
        raise ValueError("cache must be [pages, heads, bytes of a page]")
    pages, H, each = shape
    token = D + D // 16
    if H != heads or D < 1 or each == 0 or each % (16 * token):     # pages of whole 16 tokens
        raise ValueError(f"cache {tuple(shape)} does not hold {heads} heads of {D} channels")
    return pages, each // token


def _cache_sizes(cache, heads, D, index):
    """(pages, page_size) of a cache for those heads, on that device."""
    import torch
    sizes = _pages_of(cache.shape, heads, D)
    if cache.dtype is not torch.uint8 or cache.get_device() != index or not cache.is_contiguous():
        _need("cache", cache, torch.uint8, cache.shape, index)
    return sizes


def cache_write(cache, k, v, slots, *, stream=None):
    """Quantises k and v [T, H, D] (bf16 or f16) into slots [T] (int32 or
    int64) of the cache: 4-bit codes, one power of two for 32 channels.  A slot
    below 0 or past the cache writes nothing; the others must differ.  Returns
    the cache."""
    import torch
    if stream is not None:
        return _on_stream(stream, cache_write, cache, k, v, slots)
    if k.dim() != 3:
        raise ValueError("k and v must be [T, heads, D]")
    dt = k.dtype
    if dt is not torch.bfloat16 and dt is not torch.float16:
        raise ValueError(f"k and v must be bfloat16 or float16, got {dt}")
    T, H, D = shape = k.shape
    _fits(H | D)
    index = k.get_device()
    ks, vs = _head_strides("k", k, dt, shape, index), _head_strides("v", v, dt, shape, index)
    pages, ps = _cache_sizes(cache, H, D, index)
    _need("slots", slots, slots.dtype, (T,), index)
    a = CacheArgs(T, pages, ps, H, D, _types()[1][dt], _whole_bytes("slots", slots), 0, *ks, *vs,
                  cache.data_ptr(), slots.data_ptr(), k.data_ptr(), v.data_ptr())
    _enqueue(index, lib().mhc_cache_write, ctypes.byref(a))
    return cache


def cache_read(cache, slots, head_dim, *, dtype="bf16", out=None, stream=None):
    """k and v [T, H, head_dim] of the cache's slots [T] (int32 or int64), in
    bf16 or f16.  A slot below 0 or past the cache reads as zeros.  out: the
    pair to write to."""
    import torch
    if stream is not None:
        return _on_stream(stream, cache_read, cache, slots, head_dim, dtype=dtype, out=out)
    if slots.dim() != 1 or cache.dim() != 3:
        raise ValueError("slots must be [T] and cache [pages, heads, bytes of a page]")
    if dtype not in ("bf16", "f16"):
        raise ValueError("dtype must be bf16 or f16")
    T, H = slots.shape[0], cache.shape[1]
    _fits(H | head_dim)
    index = cache.get_device()
    pages, ps = _cache_sizes(cache, H, head_dim, index)
    _need("slots", slots, slots.dtype, (T,), index)
    dt, shape = _types()[0][dtype], (T, H, head_dim)
    if out is None:
        ks = vs = (H * head_dim, head_dim)
        where = cache.device
        k = torch.empty_strided(shape, (*ks, 1), dtype=dt, device=where)
        v = torch.empty_strided(shape, (*ks, 1), dtype=dt, device=where)
    else:
        k, v = out
        ks, vs = _head_strides("k", k, dt, shape, index), _head_strides("v", v, dt, shape, index)
    a = CacheArgs(T, pages, ps, H, head_dim, DTYPES[dtype], _whole_bytes("slots", slots), 0, *ks, *vs,
                  cache.data_ptr(), slots.data_ptr(), k.data_ptr(), v.data_ptr())
    _enqueue(index, lib().mhc_cache_read, ctypes.byref(a))
    return k, v


@functools.lru_cache(maxsize=None)
def _compute_units(index):
    import torch
    return torch.cuda.get_device_properties(index).multi_processor_count


@functools.lru_cache(maxsize=4096)
def cache_attention_workspace(T, B, q_heads, kv_heads, head_dim, cu_count=256, max_len=1 << 30):
    """Bytes of workspace that cache_attention takes for T query rows in B
    sequences of up to max_len tokens (host only)."""
    _fits(B | q_heads | kv_heads | head_dim | cu_count)
    n = ctypes.c_uint64()
    _check(lib().mhc_cache_attention_workspace(T, B, q_heads, kv_heads, head_dim, cu_count, max_len,
                                               ctypes.byref(n)))
    return n.value


def cache_attention(q, cache, tables, lens, *, q_starts=None, scale=None, causal=True, window=0,
                    softcap=0.0, lse=False, max_len=None, out=None, stream=None):
    """Attention of q [T, Hq, D] (bf16 or f16) over the 4-bit cache.  Sequence b
    has lens[b] tokens (int32 [B]), token t on page tables[b, t // page_size]
    (int32 [B, pages a sequence may have]), and the query rows q_starts[b] ..
    q_starts[b + 1] (int32 [B + 1]), which are its last tokens; without
    q_starts one row each.  Query head h reads kv head h // (Hq / Hkv).  A row
    sees the tokens up to its own (causal) or all, the last `window` of them
    if window > 0; scores are q . k * scale (D ** -0.5), capped by softcap *
    tanh(s / softcap) if softcap > 0.  Rows that see nothing are 0.
    max_len: no sequence is longer, or is cut there; past what the tables hold
    it says nothing.
    Returns out [T, Hq, D] in q's type, and with lse the logarithms of the sums
    too (f32 [T, Hq]), by which parts over different tokens can be joined.  out:
    the tensor, or with lse the pair, to write to; rows that belong to no
    sequence are left as they are."""
    import torch
    if stream is not None:
        return _on_stream(stream, cache_attention, q, cache, tables, lens, q_starts=q_starts,
                          scale=scale, causal=causal, window=window, softcap=softcap, lse=lse,
                          max_len=max_len, out=out)
    if q.dim() != 3 or cache.dim() != 3 or tables.dim() != 2:
        raise ValueError("q must be [T, heads, D], cache [pages, heads, bytes], tables [B, pages]")
    dt = q.dtype
    if dt is not torch.bfloat16 and dt is not torch.float16:
        raise ValueError(f"q must be bfloat16 or float16, got {dt}")
    T, Hq, D = shape = q.shape
    B, width = tables.shape
    Hk = cache.shape[1]
    _fits(Hq | D | B | width | window)
    index = q.get_device()
    qs = _head_strides("q", q, dt, shape, index)
    pages, ps = _cache_sizes(cache, Hk, D, index)
    if tables.dtype is not torch.int32 or tables.get_device() != index \
            or (width > 1 and tables.stride(1) != 1):
        raise ValueError(f"tables must be int32 with dense rows on cuda:{index}")
    _need("lens", lens, torch.int32, (B,), index)
    if q_starts is not None:
        _need("q_starts", q_starts, torch.int32, (B + 1,), index)
    if max_len is not None and max_len < 1:
        raise ValueError("max_len must be positive")
    sums = None
    if out is None:
        out = _dense_like(q)
        if lse:
            sums = _new(T, Hq, torch.float32, q.device)
    else:
        if lse:
            out, sums = out
            _need("lse", sums, torch.float32, (T, Hq), index)
        _need("out", out, dt, shape, index)
    most = width * ps if max_len is None else min(max_len, width * ps)
    size = cache_attention_workspace(T, B, Hq, Hk, D, _compute_units(index), most)
    space = torch.empty_strided((size,), (1,), dtype=torch.uint8, device=q.device) if size else None
    a = CacheAttentionArgs(T, most, pages, *qs, tables.stride(0) if B > 1 else width, B, Hq, Hk, D, ps,
                           width, _types()[1][dt], bool(causal), window,
                           D ** -0.5 if scale is None else scale, softcap, 0, q.data_ptr(),
                           cache.data_ptr(), tables.data_ptr(), lens.data_ptr(), _address(q_starts),
                           out.data_ptr(), _address(sums), _address(space), size)
    _enqueue(index, lib().mhc_cache_attention, ctypes.byref(a))
    return (out, sums) if lse else out
