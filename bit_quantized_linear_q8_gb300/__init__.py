"""GB300 (sm_103a) quantized-weight linear projection.

Python binding of libbq8's C ABI (``include/bq8.h``).  Each function here only marshals
torch tensors into device pointers, sizes and the current CUDA stream, calls the C entry
point of the same name and raises on a nonzero status; every step of the computation runs
in the library's CUDA kernels.  PyTorch is used for device memory and streams only.

The projection contract is ``out[m, n] = input[m, k] @ W^T`` (the serving stack's
init_q2.rs `qkvz_q2_prefill_gemm`, q4k_mmq.rs `q4k_mmq_gemm`).  BF16 tensors are
``torch.bfloat16``; packed weights and q8_1 buffers are ``torch.uint8``.
"""
import ctypes
import functools
from dataclasses import dataclass

from . import _abi
from ._abi import BQ8Error, LibraryNotBuilt, check, lib  # noqa: F401

__all__ = [
    "Q2Weight", "q2_pack", "quantize_weight_q4k", "quantize_act_q8_1", "q2_gemv", "q2_gemv_batchm",
    "silu_mul_bf16", "ffn_q2_km", "ffn_q2_km_noalloc", "q2_mmq_gemm", "q4k_mmq_gemm", "dequant_q2_to_bf16",
    "dense_gemm_bf16", "dequant_nvfp4_to_bf16", "q2_prefill_proj",
    "rms_norm_int8", "rms_norm_q8_1", "quantize_int8", "dequant_int8_to_bf16", "int8_gemm", "int8_gemm_scratch_bytes",
    "gated_delta_decode", "gated_delta_prefill", "gated_delta_prefill_scratch_bytes",
    "q2_weight_bytes", "q8_1_bytes", "q4k_weight_bytes", "BQ8Error", "LibraryNotBuilt",
]


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t):
    # the C signatures declare void*, so ctypes converts the int (None is NULL)
    return t.data_ptr() if t is not None else None


_raw_stream = None


def _stream():
    """The current CUDA stream of the current device, as a handle for the C ABI."""
    global _raw_stream
    if _raw_stream is None:
        torch = _torch()
        get_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        get_dev = getattr(torch._C, "_cuda_getDevice", None)
        if get_raw is not None and get_dev is not None:
            _raw_stream = lambda: get_raw(get_dev())  # noqa: E731  (no Stream object per call)
        else:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return _raw_stream()


def _need(t, dtype, name, shape=None):
    try:  # all is well, in one pass: the calls of single tokens are bound by the host
        if t.dtype is dtype and t.is_cuda and t.is_contiguous() and (shape is None or t.shape == shape):
            return t
    except AttributeError:
        pass
    if not isinstance(t, _torch().Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (the library has no CPU path)" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    return t


def _need_bytes(t, nbytes, name, device=None):
    """A uint8 CUDA buffer of at least `nbytes` bytes, on `device` where one is given."""
    _need(t, _torch().uint8, name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, the call's tensors on %s" % (name, t.device, device))
    if t.numel() < nbytes:
        raise ValueError("%s holds %d bytes, needs %d" % (name, t.numel(), nbytes))
    return t


@functools.lru_cache(maxsize=256)
def q2_weight_bytes(n: int, k: int, group: int = 128) -> int:
    return int(lib().bq_q2_weight_bytes(n, k, group))


@functools.lru_cache(maxsize=256)
def q8_1_bytes(m: int, k: int) -> int:
    return int(lib().bq_q8_1_bytes(m, k))


def q4k_weight_bytes(n: int, k: int) -> int:
    return int(lib().bq_q4k_weight_bytes(n, k))


@dataclass
class Q2Weight:
    """A packed Q2_0 weight (init_q2.rs `PackedQ2Weight { weight, n, k, group }`)."""
    data: object  # torch.uint8 CUDA tensor of q2_weight_bytes(n, k, group) bytes
    n: int
    k: int
    group: int = 128

    def desc(self):
        """The C struct for this weight; checked and built again whenever the tensor or the
        shape fields change."""
        t = self.data
        key = (id(t), t.data_ptr() if hasattr(t, "data_ptr") else None, getattr(t, "dtype", None),
               getattr(t, "shape", None), self.n, self.k, self.group)
        cached = self.__dict__.get("_desc")
        if cached is not None and cached[0] == key:
            return cached[1]
        _need_bytes(t, q2_weight_bytes(self.n, self.k, self.group), "Q2Weight.data")
        d = _abi.Q2WeightDesc(t.data_ptr(), self.n, self.k, self.group)
        self.__dict__["_desc"] = (key, d)
        return d


def q2_pack(codes, scales, group: int = 128) -> Q2Weight:
    """codes [n, k] uint8 (0..3), scales [n, k/group] bf16 -> packed Q2Weight."""
    torch = _torch()
    n, k = codes.shape
    _need(codes, torch.uint8, "codes")
    _need(scales, torch.bfloat16, "scales", (n, k // group))
    out = torch.empty(q2_weight_bytes(n, k, group), dtype=torch.uint8, device=codes.device)
    check(lib().bq_q2_pack(_ptr(codes), _ptr(scales), _ptr(out), n, k, group, _stream()))
    return Q2Weight(out, n, k, group)


def quantize_weight_q4k(w):
    """w [n, k] bf16 -> block_q4_K bytes (n * k/256 * 144)."""
    torch = _torch()
    n, k = w.shape
    _need(w, torch.bfloat16, "w")
    out = torch.empty(q4k_weight_bytes(n, k), dtype=torch.uint8, device=w.device)
    check(lib().quantize_weight_q4k(_ptr(w), _ptr(out), n, k, _stream()))
    return out


def quantize_act_q8_1(x, out=None):
    """x [m, k] bf16 -> q8_1 buffer (q8_1_bytes(m, k) uint8)."""
    torch = _torch()
    m, k = x.shape
    _need(x, torch.bfloat16, "x")
    if out is None:
        out = torch.empty(q8_1_bytes(m, k), dtype=torch.uint8, device=x.device)
    _need_bytes(out, q8_1_bytes(m, k), "out")
    check(lib().quantize_act_q8_1(_ptr(x), _ptr(out), m, k, _stream()))
    return out


def q2_gemv(x, w: Q2Weight, out=None):
    """x [1, k] bf16 -> y [1, n] bf16."""
    torch = _torch()
    _need(x, torch.bfloat16, "x", (1, w.k))
    if out is None:
        out = torch.empty((1, w.n), dtype=torch.bfloat16, device=x.device)
    _need(out, torch.bfloat16, "out", (1, w.n))
    d = w.desc()
    check(lib().q2_gemv(_ptr(x), ctypes.byref(d), _ptr(out), _stream()))
    return out


def q2_gemv_batchm(x, w: Q2Weight, out=None):
    """x [m, k] bf16 (1 <= m <= 8) -> y [m, n] bf16."""
    torch = _torch()
    m = x.shape[0]
    _need(x, torch.bfloat16, "x", (m, w.k))
    if out is None:
        out = torch.empty((m, w.n), dtype=torch.bfloat16, device=x.device)
    _need(out, torch.bfloat16, "out", (m, w.n))
    d = w.desc()
    check(lib().q2_gemv_batchm(_ptr(x), ctypes.byref(d), _ptr(out), m, _stream()))
    return out


def silu_mul_bf16(gate, up, out=None):
    torch = _torch()
    _need(gate, torch.bfloat16, "gate")
    _need(up, torch.bfloat16, "up", tuple(gate.shape))
    if out is None:
        out = torch.empty_like(gate)
    _need(out, torch.bfloat16, "out", tuple(gate.shape))
    check(lib().silu_mul_bf16(_ptr(gate), _ptr(up), _ptr(out), gate.numel(), _stream()))
    return out


def ffn_q2_km(x, gate: Q2Weight, up: Q2Weight, down: Q2Weight, gate_scratch=None, up_scratch=None, out=None):
    """Packed-Q2 FFN decode for m = x.shape[0] rows; returns (out, gate_scratch=h, up_scratch=u)."""
    torch = _torch()
    m = x.shape[0]
    _need(x, torch.bfloat16, "x", (m, gate.k))
    inter, hidden = gate.n, gate.k
    if gate_scratch is None:
        gate_scratch = torch.empty((m, inter), dtype=torch.bfloat16, device=x.device)
    if up_scratch is None:
        up_scratch = torch.empty((m, inter), dtype=torch.bfloat16, device=x.device)
    if out is None:
        out = torch.empty((m, hidden), dtype=torch.bfloat16, device=x.device)
    _need(gate_scratch, torch.bfloat16, "gate_scratch", (m, inter))
    _need(up_scratch, torch.bfloat16, "up_scratch", (m, inter))
    _need(out, torch.bfloat16, "out", (m, down.n))
    dg, du, dd = gate.desc(), up.desc(), down.desc()
    check(lib().ffn_q2_km(_ptr(x), ctypes.byref(dg), ctypes.byref(du), ctypes.byref(dd), _ptr(gate_scratch),
                          _ptr(up_scratch), _ptr(out), m, _stream()))
    return out, gate_scratch, up_scratch


def ffn_q2_km_noalloc(x, gate: Q2Weight, up: Q2Weight, down: Q2Weight, out=None):
    """ffn_q2_km with its two intermediates in the library's built-in device array (for
    callers that cannot allocate; m * inter <= 262144).  Calls that overlap on the GPU race
    on that array.  Returns out [m, hidden]."""
    torch = _torch()
    m = x.shape[0]
    _need(x, torch.bfloat16, "x", (m, gate.k))
    if out is None:
        out = torch.empty((m, gate.k), dtype=torch.bfloat16, device=x.device)
    _need(out, torch.bfloat16, "out", (m, gate.k))
    dg, du, dd = gate.desc(), up.desc(), down.desc()
    check(lib().ffn_q2_km_noalloc(_ptr(x), ctypes.byref(dg), ctypes.byref(du), ctypes.byref(dd), _ptr(out), m,
                                  _stream()))
    return out


def q2_mmq_gemm(act_q8, w: Q2Weight, m: int, out=None):
    """q8_1 activations for [m, w.k] -> out [m, n] bf16 (group must be 128)."""
    torch = _torch()
    _need_bytes(act_q8, q8_1_bytes(m, w.k), "act_q8")
    if out is None:
        out = torch.empty((m, w.n), dtype=torch.bfloat16, device=act_q8.device)
    _need(out, torch.bfloat16, "out", (m, w.n))
    d = w.desc()
    check(lib().q2_mmq_gemm(_ptr(act_q8), ctypes.byref(d), _ptr(out), m, _stream()))
    return out


def q4k_mmq_gemm(act_q8, w_q4k, m: int, n: int, k: int, out=None):
    torch = _torch()
    _need_bytes(act_q8, q8_1_bytes(m, k), "act_q8")
    _need_bytes(w_q4k, q4k_weight_bytes(n, k), "w_q4k")
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=act_q8.device)
    _need(out, torch.bfloat16, "out", (m, n))
    check(lib().q4k_mmq_gemm(_ptr(act_q8), _ptr(w_q4k), _ptr(out), m, n, k, _stream()))
    return out


def dequant_q2_to_bf16(w: Q2Weight, out=None):
    torch = _torch()
    if out is None:
        out = torch.empty((w.n, w.k), dtype=torch.bfloat16, device=w.data.device)
    _need(out, torch.bfloat16, "out", (w.n, w.k))
    d = w.desc()
    check(lib().dequant_q2_to_bf16(ctypes.byref(d), _ptr(out), _stream()))
    return out


def dense_gemm_bf16(a, w, out=None):
    """out [m, n] = a [m, k] @ w [n, k]^T, BF16 in and out, fp32 accumulation (the fallback
    route's dense GEMM, init_q2.rs `dense_gemm_bf16_pipelined`); k a multiple of 64."""
    torch = _torch()
    m, k = a.shape
    n = w.shape[0]
    _need(a, torch.bfloat16, "a", (m, k))
    _need(w, torch.bfloat16, "w", (n, k))
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=a.device)
    _need(out, torch.bfloat16, "out", (m, n))
    check(lib().dense_gemm_bf16(_ptr(a), _ptr(w), _ptr(out), m, n, k, _stream()))
    return out


def dequant_nvfp4_to_bf16(packed, scales, scale2: float, n: int, k: int, out=None):
    """NVFP4 [n, k] -> BF16 [n, k]: packed E2M1 codes [n, k/2] (uint8), E4M3 scale bytes
    [n, k/16] (uint8) and the per-tensor fp32 scale2 (q4k_mmq.rs, `dequant_nvfp4_to_bf16`)."""
    torch = _torch()
    _need(packed, torch.uint8, "packed")
    _need(scales, torch.uint8, "scales")
    if packed.numel() != n * (k // 2) or scales.numel() != n * (k // 16):
        raise ValueError("packed must hold n*k/2 bytes and scales n*k/16 bytes")
    if out is None:
        out = torch.empty((n, k), dtype=torch.bfloat16, device=packed.device)
    _need(out, torch.bfloat16, "out", (n, k))
    check(lib().dequant_nvfp4_to_bf16(_ptr(packed), _ptr(scales), _ptr(out), ctypes.c_float(scale2), n, k,
                                      _stream()))
    return out


def q2_prefill_proj(x, w: Q2Weight, mode: str = "mmq", act_q8=None, scratch=None, out=None):
    """The prefill projection out = x @ W^T by either route of init_q2.rs
    `qkvz_q2_prefill_gemm`: "mmq" (q8_1 quantisation + Q2 MMQ, group 128 only) or
    "dequant" (dequantise to BF16 into `scratch` [n, k], then this library's tcgen05 BF16
    GEMM).  Returns (out, mode_used)."""
    torch = _torch()
    m = x.shape[0]
    if mode == "mmq":
        if w.group != 128:
            raise ValueError("the MMQ route needs group size 128")
        act_q8 = quantize_act_q8_1(x, out=act_q8)
        return q2_mmq_gemm(act_q8, w, m, out=out), "mmq"
    if mode == "dequant":
        _need(x, torch.bfloat16, "x", (m, w.k))
        wd = dequant_q2_to_bf16(w, out=scratch)
        return dense_gemm_bf16(x, wd, out=out), "dequant"
    raise ValueError("mode must be 'mmq' or 'dequant'")


def _norm_args(x, weight, residual, residual_out, y_out):
    """Checks the tensors that both norms share; returns (m, k, residual_out)."""
    torch = _torch()
    _need(x, torch.bfloat16, "x")
    if x.dim() != 2:
        raise ValueError("x must have shape [m, k], got %s" % (tuple(x.shape),))
    m, k = x.shape
    _need(weight, torch.bfloat16, "weight", (k,))
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out needs a residual")
    else:
        _need(residual, torch.bfloat16, "residual", (m, k))
        if residual_out is None:
            residual_out = torch.empty_like(x)
        else:
            _need(residual_out, torch.bfloat16, "residual_out", (m, k))
    if y_out is not None:
        _need(y_out, torch.bfloat16, "y_out", (m, k))
    return m, k, residual_out


def rms_norm_int8(x, weight, residual=None, eps: float = 1e-6, residual_out=None, y_out=None, codes=None, scales=None):
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight; int8 codes of y with one scale a
    row.  x, residual [m, k] and weight [k] bf16.  Returns (codes [m, k] int8, scales [m] fp32, h [m, k]
    bf16 or None without a residual); residual_out may be residual or x itself.  y_out: also BF16(y)."""
    torch = _torch()
    m, k, residual_out = _norm_args(x, weight, residual, residual_out, y_out)
    if codes is None:
        codes = torch.empty((m, k), dtype=torch.int8, device=x.device)
    else:
        _need(codes, torch.int8, "codes", (m, k))
    if scales is None:
        scales = torch.empty((m,), dtype=torch.float32, device=x.device)
    else:
        _need(scales, torch.float32, "scales", (m,))
    check(lib().rms_norm_int8(_ptr(x), _ptr(residual), _ptr(weight), eps, _ptr(residual_out), _ptr(y_out), _ptr(codes),
                              _ptr(scales), m, k, _stream()))
    return codes, scales, residual_out


def rms_norm_q8_1(x, weight, residual=None, eps: float = 1e-6, residual_out=None, y_out=None, out=None):
    """The norm of rms_norm_int8 with a q8_1 output (q8_1_bytes(m, k) uint8), the activations of
    q2_mmq_gemm and q4k_mmq_gemm.  Returns (act_q8, h or None)."""
    torch = _torch()
    m, k, residual_out = _norm_args(x, weight, residual, residual_out, y_out)
    if out is None:
        out = torch.empty(q8_1_bytes(m, k), dtype=torch.uint8, device=x.device)
    else:
        _need_bytes(out, q8_1_bytes(m, k), "out")
    check(lib().rms_norm_q8_1(_ptr(x), _ptr(residual), _ptr(weight), eps, _ptr(residual_out), _ptr(y_out), _ptr(out),
                              m, k, _stream()))
    return out, residual_out


def quantize_int8(x, codes=None, scales=None):
    """x [m, k] bf16 -> (codes [m, k] int8, scales [m] fp32): activations by token, weights by
    output channel."""
    torch = _torch()
    m, k = x.shape
    _need(x, torch.bfloat16, "x")
    if codes is None:
        codes = torch.empty((m, k), dtype=torch.int8, device=x.device)
    else:
        _need(codes, torch.int8, "codes", (m, k))
    if scales is None:
        scales = torch.empty((m,), dtype=torch.float32, device=x.device)
    else:
        _need(scales, torch.float32, "scales", (m,))
    check(lib().quantize_int8(_ptr(x), _ptr(codes), _ptr(scales), m, k, _stream()))
    return codes, scales


def dequant_int8_to_bf16(codes, scales, out=None):
    """codes [rows, k] int8, scales [rows] fp32 -> BF16(codes * scales) [rows, k]."""
    torch = _torch()
    rows, k = codes.shape
    _need(codes, torch.int8, "codes")
    _need(scales, torch.float32, "scales", (rows,))
    if out is None:
        out = torch.empty((rows, k), dtype=torch.bfloat16, device=codes.device)
    else:
        _need(out, torch.bfloat16, "out", (rows, k))
    check(lib().dequant_int8_to_bf16(_ptr(codes), _ptr(scales), _ptr(out), rows, k, _stream()))
    return out


@functools.lru_cache(maxsize=256)
def int8_gemm_scratch_bytes(m: int, n: int, k: int) -> int:
    return int(lib().bq_int8_gemm_scratch_bytes(m, n, k))


def int8_gemm(a, a_scales, w, w_scales, out=None, scratch=None):
    """W8A8 product: out [m, n] bf16 = (a [m, k] @ w [n, k]^T) * a_scales [m] * w_scales [n], int8 codes and
    fp32 scales; k a multiple of 16.  scratch: int8_gemm_scratch_bytes(m, n, k) uint8 (taken from
    torch's allocator where it is needed and not given)."""
    torch = _torch()
    m, k = a.shape
    n = w.shape[0]
    _need(a, torch.int8, "a")
    _need(w, torch.int8, "w", (n, k))
    _need(a_scales, torch.float32, "a_scales", (m,))
    _need(w_scales, torch.float32, "w_scales", (n,))
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=a.device)
    else:
        _need(out, torch.bfloat16, "out", (m, n))
    need = int8_gemm_scratch_bytes(m, n, k)
    if need:
        if scratch is None:
            scratch = torch.empty(need, dtype=torch.uint8, device=a.device)
        else:
            _need_bytes(scratch, need, "scratch", a.device)
    check(lib().int8_gemm(_ptr(a), _ptr(a_scales), _ptr(w), _ptr(w_scales), _ptr(out), _ptr(scratch) if need else None,
                          m, n, k, _stream()))
    return out


def _heads(t, dtype, name, tokens, heads, dim=None):
    """The C descriptor of a [tokens, heads(, dim)] tensor with any token and head stride."""
    shape = (tokens, heads) if dim is None else (tokens, heads, dim)
    try:
        well = t.dtype is dtype and t.is_cuda and t.shape == shape
    except AttributeError:
        well = False
    if not well:
        if not isinstance(t, _torch().Tensor):
            raise TypeError("%s must be a torch.Tensor" % name)
        if not t.is_cuda:
            raise ValueError("%s must be a CUDA tensor (the library has no CPU path)" % name)
        if t.dtype != dtype:
            raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
        raise ValueError("%s must have shape %s, got %s" % (name, shape, tuple(t.shape)))
    s = t.stride()
    if dim is not None and s[2] != 1:
        raise ValueError("the last dimension of %s must be contiguous" % name)
    # the stride of a dimension of one means nothing
    return _abi.HeadsDesc(t.data_ptr(), s[0] if tokens > 1 else 0, s[1] if heads > 1 else 0)


def _gated_delta_args(q, k, v, g, beta, state, state_idx, seqs, out):
    torch = _torch()
    if not (isinstance(q, torch.Tensor) and isinstance(v, torch.Tensor) and q.dim() == 3 and v.dim() == 3):
        raise ValueError("q and v must be tensors of shape [tokens, heads, head_dim]")
    tokens, hk, dim = q.shape
    hv = v.shape[1]
    desc = (_heads(q, torch.bfloat16, "q", tokens, hk, dim), _heads(k, torch.bfloat16, "k", tokens, hk, dim),
            _heads(v, torch.bfloat16, "v", tokens, hv, dim), _heads(g, torch.float32, "g", tokens, hv),
            _heads(beta, torch.float32, "beta", tokens, hv))
    _need(state, torch.float32, "state")
    slots = state.shape[0] if state.dim() else 0
    if state.shape != (slots, hv, dim, dim):
        raise ValueError("state must have shape [slots, %d, %d, %d], got %s" % (hv, dim, dim, tuple(state.shape)))
    if state_idx is not None:
        _need(state_idx, torch.int32, "state_idx", (seqs,))
    elif slots < seqs:
        raise ValueError("state has %d slots for %d sequences" % (slots, seqs))
    if out is None:
        out = torch.empty((tokens, hv, dim), dtype=torch.bfloat16, device=q.device)
    else:
        _need(out, torch.bfloat16, "out", (tokens, hv, dim))
    return desc, tokens, hk, hv, dim, out


def gated_delta_decode(q, k, v, g, beta, state, tokens: int = 1, state_idx=None, scale=None, l2norm: bool = False,
                       out=None):
    """The gated delta rule for single tokens (or the few of a verify batch) of every sequence.

    q, k [T, heads_k, 128], v [T, heads_v, 128] bf16 and g (log decay), beta [T, heads_v] fp32, any token
    and head strides; state [slots, heads_v, 128, 128] fp32, updated in place.  Sequence s owns rows
    s*tokens .. s*tokens + tokens - 1 and slot state_idx[s] (default s; a negative slot is skipped, its
    outputs are zero).  scale: default 128^-0.5.  Returns out [T, heads_v, 128] bf16."""
    total = q.shape[0]
    if tokens < 1 or total % tokens != 0:
        raise ValueError("%d token rows are not a multiple of tokens = %d" % (total, tokens))
    seqs = total // tokens
    d, total, hk, hv, dim, out = _gated_delta_args(q, k, v, g, beta, state, state_idx, seqs, out)
    b = ctypes.byref
    check(lib().gated_delta_decode(b(d[0]), b(d[1]), b(d[2]), b(d[3]), b(d[4]), _ptr(state), _ptr(state_idx), _ptr(out),
                                   seqs, tokens, hk, hv, dim, state.shape[0], dim ** -0.5 if scale is None else scale,
                                   int(l2norm), _stream()))
    return out


@functools.lru_cache(maxsize=256)
def gated_delta_prefill_scratch_bytes(seqs: int, total: int, heads_k: int, heads_v: int) -> int:
    return int(lib().bq_gated_delta_prefill_scratch_bytes(seqs, total, heads_k, heads_v))


def gated_delta_prefill(q, k, v, g, beta, state, cu_seqlens=None, state_idx=None, scale=None, l2norm: bool = False,
                        out=None, scratch=None):
    """The gated delta rule over whole prompts: tensors as in gated_delta_decode, the sequences'
    tokens one after the other.  cu_seqlens: int32 CUDA tensor [sequences + 1] of row bounds (default:
    one sequence); sequences may be empty.  scratch: gated_delta_prefill_scratch_bytes(sequences, T,
    heads_k, heads_v) uint8 (taken from torch's allocator when not given).  Returns out [T, heads_v, 128]
    bf16 (rows of no sequence are left as they are)."""
    torch = _torch()
    seqs = 1
    if cu_seqlens is not None:
        _need(cu_seqlens, torch.int32, "cu_seqlens")
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must have shape [sequences + 1]")
        seqs = cu_seqlens.numel() - 1
    d, total, hk, hv, dim, out = _gated_delta_args(q, k, v, g, beta, state, state_idx, seqs, out)
    need = gated_delta_prefill_scratch_bytes(seqs, total, hk, hv)
    if scratch is None:
        scratch = torch.empty(need, dtype=torch.uint8, device=q.device)
    else:
        _need_bytes(scratch, need, "scratch", q.device)
    b = ctypes.byref
    check(lib().gated_delta_prefill(b(d[0]), b(d[1]), b(d[2]), b(d[3]), b(d[4]), _ptr(state), _ptr(cu_seqlens),
                                    _ptr(state_idx), _ptr(out), _ptr(scratch), seqs, total, hk, hv, dim, state.shape[0],
                                    dim ** -0.5 if scale is None else scale, int(l2norm), _stream()))
    return out
