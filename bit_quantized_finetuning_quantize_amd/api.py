"""Thin Python binding over the C ABI (argument marshalling only).

Every computation runs in libqlora.so on the caller's current HIP stream;
torch is used only to hold device memory and to name the stream. Function
names match include/qlora.h.
"""

import ctypes

import torch

from ._lib import LIB

BLOCK = 64
GROUP = 256
# store types (include/qlora.h): bit flags
STORE_NF4 = 0
STORE_FP4 = 1
STORE_DQ_FP8 = 2
# code formats of the 8-bit blocks (include/qlora.h)
ACT8_E4M3 = 0
ACT8_E5M2 = 1


class QloraError(RuntimeError):
    pass


def _check(status):
    if status != 0:
        msg = LIB.qlora_status_string(status).decode()
        hip = LIB.qlora_last_hip_error() if status == -4 else 0
        raise QloraError(f"qlora status {status}: {msg}" + (f" (hipError {hip})" if hip else ""))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream():
    """The caller's stream on the current device, as an address. The raw
    accessors take 0.2 us where building a Stream object takes 3."""
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


_HIP = None


def _state_ptr(t, name):
    """Device-side address of an optimizer-state tensor: a contiguous GPU
    tensor, or a contiguous pinned host tensor (hipHostMalloc, e.g. torch's
    pin_memory=True), which the kernel then reads and writes over the host
    link; its device address comes from hipHostGetDevicePointer."""
    global _HIP
    if not t.is_contiguous():
        raise QloraError(f"{name} must be contiguous")
    if t.is_cuda:
        return ctypes.c_void_p(t.data_ptr())
    if not t.is_pinned():
        raise QloraError(f"{name} on the host must be pinned memory (pin_memory=True)")
    if _HIP is None:
        _HIP = ctypes.CDLL("libamdhip64.so")
        _HIP.hipHostGetDevicePointer.argtypes = [ctypes.POINTER(ctypes.c_void_p), ctypes.c_void_p,
                                                 ctypes.c_uint]
        _HIP.hipHostGetDevicePointer.restype = ctypes.c_int
    dptr = ctypes.c_void_p()
    rc = _HIP.hipHostGetDevicePointer(ctypes.byref(dptr), ctypes.c_void_p(t.data_ptr()), 0)
    if rc != 0 or not dptr.value:
        raise QloraError(f"{name}: hipHostGetDevicePointer failed ({rc})")
    return dptr


def _need(t, dtype, name):
    if t.dtype is not dtype or not t.is_cuda or not t.is_contiguous():
        raise QloraError(f"{name} must be a contiguous {dtype} tensor on the GPU")


def qlora_nf4_codes_bytes(numel):
    return int(LIB.qlora_nf4_codes_bytes(numel))


def qlora_nf4_num_blocks(numel):
    return int(LIB.qlora_nf4_num_blocks(numel))


def qlora_nf4_num_groups(numel):
    return int(LIB.qlora_nf4_num_groups(numel))


def qlora_nf4_codebook():
    buf = (ctypes.c_float * 16)()
    LIB.qlora_nf4_codebook(ctypes.cast(buf, ctypes.c_void_p))
    return list(buf)


class Nf4Store:
    """The device buffers of one 4-bit tensor (owned by torch). Without
    double quantization `absmax_q` is None and `absmax_s2` holds one float32
    constant per 64-block. `store_type`: STORE_NF4 (0), or the flags
    STORE_FP4 (FP4 levels) and STORE_DQ_FP8 (E4M3 constant code)."""

    def __init__(self, codes, absmax_q, absmax_s2, numel, shape=None, store_type=STORE_NF4):
        self.codes, self.absmax_q, self.absmax_s2 = codes, absmax_q, absmax_s2
        self.numel = int(numel)
        self.shape = tuple(shape) if shape is not None else (self.numel,)
        self.store_type = int(store_type)

    @property
    def double_quant(self):
        return self.absmax_q is not None

    def nbytes(self):
        q8 = self.absmax_q.numel() if self.absmax_q is not None else 0
        return self.codes.numel() + q8 + 4 * self.absmax_s2.numel()


def empty_store(numel, device, shape=None, double_quant=True, store_type=STORE_NF4):
    codes = torch.empty(qlora_nf4_codes_bytes(numel), dtype=torch.uint8, device=device)
    if double_quant:
        q8 = torch.empty(qlora_nf4_num_blocks(numel), dtype=torch.uint8, device=device)
        s2 = torch.empty(qlora_nf4_num_groups(numel), dtype=torch.float32, device=device)
    else:
        q8 = None
        s2 = torch.empty(qlora_nf4_num_blocks(numel), dtype=torch.float32, device=device)
    return Nf4Store(codes, q8, s2, numel, shape, store_type)


def qlora_nf4_quantize(w, out=None, double_quant=True, store_type=STORE_NF4):
    """Quantize a bf16 tensor (any shape, flattened row-major); with
    double_quant=False the store keeps the float32 block constants;
    store_type selects FP4 levels and / or the E4M3 constant code."""
    _need(w, torch.bfloat16, "w")
    if out is None:
        st = empty_store(w.numel(), w.device, w.shape, double_quant, store_type)
    else:
        st = out
        st.store_type = int(store_type)
    _check(LIB.qlora_nf4_quantize_ex(_ptr(w), w.numel(), _ptr(st.codes), _ptr(st.absmax_q),
                                     _ptr(st.absmax_s2), st.store_type, _stream()))
    return st


def qlora_nf4_dequantize(st, out=None):
    out = out if out is not None else torch.empty(st.numel, dtype=torch.float32,
                                                  device=st.codes.device)
    _check(LIB.qlora_nf4_dequantize_ex(_ptr(st.codes), _ptr(st.absmax_q), _ptr(st.absmax_s2),
                                       st.numel, st.store_type, _ptr(out), _stream()))
    return out


def qlora_nf4_dequantize_bf16(st, out=None):
    out = out if out is not None else torch.empty(st.numel, dtype=torch.bfloat16,
                                                  device=st.codes.device)
    _check(LIB.qlora_nf4_dequantize_bf16_ex(_ptr(st.codes), _ptr(st.absmax_q),
                                            _ptr(st.absmax_s2), st.numel, st.store_type,
                                            _ptr(out), _stream()))
    return out


def qlora_nf4_merge(st, A, B, scale, out=None):
    """bf16(w' + scale (A B)^T) for a store of W [N x K]: the adapter folded
    into a 16-bit copy of the frozen weight; returns bf16 [N x K]."""
    N, K = st.shape
    r = A.shape[1]
    out = out if out is not None else torch.empty(N, K, dtype=torch.bfloat16,
                                                  device=st.codes.device)
    _check(LIB.qlora_nf4_merge_ex(_ptr(st.codes), _ptr(st.absmax_q), _ptr(st.absmax_s2), N, K,
                                  _ptr(A), _ptr(B), r, float(scale), st.store_type, _ptr(out),
                                  _stream()))
    return out


def qlora_adamw_step(p, m, v, g, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0,
                     step=1, p_bf16=None):
    """One AdamW step in place on float32 p, m, v with gradient g (same
    number of elements); writes bf16(p) into p_bf16 when given."""
    n = p.numel()
    for t in (m, v, g):
        if t.numel() != n or t.dtype != torch.float32:
            raise QloraError("p, m, v, g must be float32 tensors of one size")
    if p_bf16 is not None and p_bf16.numel() != n:
        raise QloraError("p_bf16 must have as many elements as p")
    _check(LIB.qlora_adamw_step(_ptr(p), _state_ptr(m, "m"), _state_ptr(v, "v"), _ptr(g), n,
                                float(lr), float(beta1),
                                float(beta2), float(eps), float(weight_decay), int(step),
                                _ptr(p_bf16) if p_bf16 is not None else None, _stream()))


def adamw_state(n, device, host=False):
    """Zero float32 AdamW moments (m, v) for n parameters, on the GPU or
    (host=True) in pinned host memory."""
    if host:
        return tuple(torch.zeros(n, dtype=torch.float32, pin_memory=True) for _ in range(2))
    return tuple(torch.zeros(n, dtype=torch.float32, device=device) for _ in range(2))


def adamw8_state(n, device, host=False):
    """Zero 8-bit AdamW state for n parameters: (m8, m_scale, v8, v_scale),
    on the GPU or (host=True) in pinned host memory."""
    nb = (n + 255) // 256
    kw = dict(pin_memory=True) if host else dict(device=device)
    return (torch.zeros(n, dtype=torch.uint8, **kw),
            torch.zeros(nb, dtype=torch.float32, **kw),
            torch.zeros(n, dtype=torch.uint8, **kw),
            torch.zeros(nb, dtype=torch.float32, **kw))


def qlora_adamw8_step(p, m8, m_scale, v8, v_scale, g, lr, beta1=0.9, beta2=0.999, eps=1e-8,
                      weight_decay=0.0, step=1, p_bf16=None):
    """One AdamW step with 8-bit moments (all tensors updated in place)."""
    n = p.numel()
    _need(p, torch.float32, "p")
    _need(g, torch.float32, "g")
    for t, dt, name in ((m_scale, torch.float32, "m_scale"), (v_scale, torch.float32, "v_scale"),
                        (m8, torch.uint8, "m8"), (v8, torch.uint8, "v8")):
        if t.dtype != dt:
            raise QloraError(f"{name} must be a {dt} tensor")
    if g.numel() != n or m8.numel() != n or v8.numel() != n:
        raise QloraError("p, g, m8 and v8 must have the same number of elements")
    if m_scale.numel() != (n + 255) // 256 or v_scale.numel() != (n + 255) // 256:
        raise QloraError("one scale per block of 256 parameters")
    if p_bf16 is not None:
        _need(p_bf16, torch.bfloat16, "p_bf16")
    _check(LIB.qlora_adamw8_step(_ptr(p), _state_ptr(m8, "m8"), _state_ptr(m_scale, "m_scale"),
                                 _state_ptr(v8, "v8"), _state_ptr(v_scale, "v_scale"),
                                 _ptr(g), n, float(lr), float(beta1), float(beta2), float(eps),
                                 float(weight_decay), int(step),
                                 _ptr(p_bf16) if p_bf16 is not None else None, _stream()))


def qlora_linear_workspace_bytes(M, N, K, r):
    return int(LIB.qlora_linear_workspace_bytes(M, N, K, r))


def qlora_gemv_wait_limit(microseconds):
    _check(LIB.qlora_gemv_wait_limit(int(microseconds)))


def workspace(M, N, K, r, device):
    n = qlora_linear_workspace_bytes(M, N, K, r)
    if n == 0:
        raise QloraError(f"unsupported linear shape M={M} N={N} K={K} r={r}")
    return torch.empty(n, dtype=torch.uint8, device=device)


def qlora_linear_fwd(X, W, A, B, scale, want_T=True, Y=None, T=None, ws=None, events=None):
    """Y = X bf16(W')^T + scale (X A) B; returns (Y, T) with T fp32 or None.

    `events`: optional (begin, end) raw hipEvent_t handles recorded around
    the dominant kernel (profiling)."""
    M, K = X.shape
    N = W.shape[0]
    r = A.shape[1]
    for t, name in ((X, "X"), (A, "A"), (B, "B")):
        _need(t, torch.bfloat16, name)
    Y = Y if Y is not None else torch.empty(M, N, dtype=torch.bfloat16, device=X.device)
    if want_T and T is None:
        T = torch.empty(M, r, dtype=torch.float32, device=X.device)
    ws = ws if ws is not None else workspace(M, N, K, r, X.device)
    if W.store_type != STORE_NF4:
        if events is not None:
            raise QloraError("profiling events are taken on NF4 stores only")
        _check(LIB.qlora_linear_fwd_ex(_ptr(X), _ptr(W.codes), _ptr(W.absmax_q),
                                       _ptr(W.absmax_s2), _ptr(A), _ptr(B), M, N, K, r,
                                       float(scale), _ptr(Y), _ptr(T) if want_T else None,
                                       _ptr(ws), ws.numel(), W.store_type, _stream()))
        return Y, (T if want_T else None)
    ev = events if events is not None else (None, None)
    _check(LIB.qlora_linear_fwd_profiled(_ptr(X), _ptr(W.codes), _ptr(W.absmax_q),
                                         _ptr(W.absmax_s2), _ptr(A), _ptr(B), M, N, K, r,
                                         float(scale), _ptr(Y), _ptr(T) if want_T else None,
                                         _ptr(ws), ws.numel(), _stream(), ev[0], ev[1]))
    return Y, (T if want_T else None)


def qlora_linear_fwd_noalloc(X, W, A, B, scale, want_T=True, Y=None, T=None):
    """qlora_linear_fwd without a workspace: the library's fixed per-device
    scratch array serves as one (calls that overlap on one GPU race)."""
    M, K = X.shape
    N = W.shape[0]
    r = A.shape[1]
    for t, name in ((X, "X"), (A, "A"), (B, "B")):
        _need(t, torch.bfloat16, name)
    Y = Y if Y is not None else torch.empty(M, N, dtype=torch.bfloat16, device=X.device)
    if want_T and T is None:
        T = torch.empty(M, r, dtype=torch.float32, device=X.device)
    _check(LIB.qlora_linear_fwd_noalloc(_ptr(X), _ptr(W.codes), _ptr(W.absmax_q),
                                        _ptr(W.absmax_s2), _ptr(A), _ptr(B), M, N, K, r,
                                        float(scale), _ptr(Y), _ptr(T) if want_T else None,
                                        _stream()))
    return Y, (T if want_T else None)


def qlora_linear_bwd(dY, X, T, W, A, B, scale, want_dX=True, dX=None, dA=None, dB=None, ws=None,
                     events=None):
    """Returns (dX or None, dA fp32 [K x r], dB fp32 [r x N]).

    `events`: optional (begin, end) raw hipEvent_t handles recorded around
    the input-gradient kernel (profiling)."""
    M, N = dY.shape
    K = X.shape[1]
    r = A.shape[1]
    for t, name in ((dY, "dY"), (X, "X"), (A, "A"), (B, "B")):
        _need(t, torch.bfloat16, name)
    if want_dX and dX is None:
        dX = torch.empty(M, K, dtype=torch.bfloat16, device=X.device)
    dA = dA if dA is not None else torch.empty(K, r, dtype=torch.float32, device=X.device)
    dB = dB if dB is not None else torch.empty(r, N, dtype=torch.float32, device=X.device)
    ws = ws if ws is not None else workspace(M, N, K, r, X.device)
    if W.store_type != STORE_NF4:
        if events is not None:
            raise QloraError("profiling events are taken on NF4 stores only")
        _check(LIB.qlora_linear_bwd_ex(_ptr(dY), _ptr(X), _ptr(T), _ptr(W.codes),
                                       _ptr(W.absmax_q), _ptr(W.absmax_s2), _ptr(A), _ptr(B),
                                       M, N, K, r, float(scale), _ptr(dX) if want_dX else None,
                                       _ptr(dA), _ptr(dB), _ptr(ws), ws.numel(), W.store_type,
                                       _stream()))
        return (dX if want_dX else None), dA, dB
    ev = events if events is not None else (None, None)
    _check(LIB.qlora_linear_bwd_profiled(_ptr(dY), _ptr(X), _ptr(T), _ptr(W.codes),
                                         _ptr(W.absmax_q), _ptr(W.absmax_s2), _ptr(A), _ptr(B),
                                         M, N, K, r, float(scale), _ptr(dX) if want_dX else None,
                                         _ptr(dA), _ptr(dB), _ptr(ws), ws.numel(), _stream(),
                                         ev[0], ev[1]))
    return (dX if want_dX else None), dA, dB


def qlora_dropout_mask(M, K, p, seed, offset=0, out=None, device=None):
    """Keep mask of LoRA dropout over an [M x K] adapter input: int32 tensor
    [M, K // 32] holding the uint32 bit words (bit j of word w of row m keeps
    element (m, 32 w + j))."""
    if out is None:
        dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
        out = torch.empty(M, K // 32, dtype=torch.int32, device=dev)
    _need(out, torch.int32, "mask")
    _check(LIB.qlora_dropout_mask(M, K, float(p), int(seed) & (2**64 - 1),
                                  int(offset) & (2**64 - 1), _ptr(out), _stream()))
    return out


def qlora_linear_fwd_dropout(X, W, A, B, scale, keep_mask, p, want_T=True, Y=None, T=None,
                             ws=None):
    """qlora_linear_fwd with LoRA dropout on the adapter input; returns
    (Y, T) with T = D(X) A (fp32) or None."""
    M, K = X.shape
    N = W.shape[0]
    r = A.shape[1]
    for t, name in ((X, "X"), (A, "A"), (B, "B")):
        _need(t, torch.bfloat16, name)
    _need(keep_mask, torch.int32, "keep_mask")
    Y = Y if Y is not None else torch.empty(M, N, dtype=torch.bfloat16, device=X.device)
    if want_T and T is None:
        T = torch.empty(M, r, dtype=torch.float32, device=X.device)
    ws = ws if ws is not None else workspace(M, N, K, r, X.device)
    _check(LIB.qlora_linear_fwd_dropout(_ptr(X), _ptr(W.codes), _ptr(W.absmax_q),
                                        _ptr(W.absmax_s2), _ptr(A), _ptr(B), M, N, K, r,
                                        float(scale), _ptr(keep_mask), float(p), _ptr(Y),
                                        _ptr(T) if want_T else None, _ptr(ws), ws.numel(),
                                        _stream()))
    return Y, (T if want_T else None)


def qlora_linear_bwd_dropout(dY, X, T, W, A, B, scale, keep_mask, p, want_dX=True, dX=None,
                             dA=None, dB=None, ws=None):
    """qlora_linear_bwd with LoRA dropout; returns (dX or None, dA, dB)."""
    M, N = dY.shape
    K = X.shape[1]
    r = A.shape[1]
    for t, name in ((dY, "dY"), (X, "X"), (A, "A"), (B, "B")):
        _need(t, torch.bfloat16, name)
    _need(keep_mask, torch.int32, "keep_mask")
    if want_dX and dX is None:
        dX = torch.empty(M, K, dtype=torch.bfloat16, device=X.device)
    dA = dA if dA is not None else torch.empty(K, r, dtype=torch.float32, device=X.device)
    dB = dB if dB is not None else torch.empty(r, N, dtype=torch.float32, device=X.device)
    ws = ws if ws is not None else workspace(M, N, K, r, X.device)
    _check(LIB.qlora_linear_bwd_dropout(_ptr(dY), _ptr(X), _ptr(T), _ptr(W.codes),
                                        _ptr(W.absmax_q), _ptr(W.absmax_s2), _ptr(A), _ptr(B),
                                        M, N, K, r, float(scale), _ptr(keep_mask), float(p),
                                        _ptr(dX) if want_dX else None, _ptr(dA), _ptr(dB),
                                        _ptr(ws), ws.numel(), _stream()))
    return (dX if want_dX else None), dA, dB


# ---- 8-bit blocks ------------------------------------------------------------


class Act8:
    """A matrix [M x K] in 8-bit blocks: uint8 codes [M, row bytes] and scale
    bytes [M, scale row bytes] (include/qlora.h), `fmt` ACT8_E4M3 or ACT8_E5M2."""

    __slots__ = ("codes", "scales", "shape", "fmt")

    def __init__(self, codes, scales, shape, fmt=ACT8_E4M3):
        self.codes, self.scales = codes, scales
        self.shape = tuple(shape)
        self.fmt = int(fmt)

    def nbytes(self):
        return self.codes.numel() + self.scales.numel()


class Fp8Weight:
    """A frozen weight [N x K] in 128 x 128 blocks of E4M3 codes; `codes_t`
    and `scales_t` hold it transposed (for the input gradient) or are None."""

    __slots__ = ("codes", "scales", "codes_t", "scales_t", "shape")

    def __init__(self, codes, scales, codes_t, scales_t, shape):
        self.codes, self.scales = codes, scales
        self.codes_t, self.scales_t = codes_t, scales_t
        self.shape = tuple(shape)

    def nbytes(self):
        return sum(t.numel() for t in (self.codes, self.scales, self.codes_t, self.scales_t)
                   if t is not None)


def act8_row_bytes(K):
    return (K + 127) // 128 * 128


def act8_scale_row_bytes(K):
    return ((K + 127) // 128 + 3) // 4 * 4


def empty_act8(M, K, device, fmt=ACT8_E4M3):
    return Act8(torch.empty(M, act8_row_bytes(K), dtype=torch.uint8, device=device),
                torch.empty(M, act8_scale_row_bytes(K), dtype=torch.uint8, device=device),
                (M, K), fmt)


def _rows(t, shape, name):
    """Leading dimension of a bf16 matrix of `shape` on the GPU whose rows are contiguous."""
    if t.dtype is not torch.bfloat16 or t.shape != shape or not t.is_cuda:
        raise QloraError(f"{name} must be a bfloat16 tensor of shape {shape} on the GPU")
    M, K = shape
    ld, step = t.stride()
    if K > 1 and step != 1:
        raise QloraError(f"{name} must have contiguous rows")
    if M == 1:  # one row: the stride has no meaning
        return max(ld, K)
    if ld < K:
        raise QloraError(f"{name} must not have overlapping rows")
    return ld


def _bytes(t, shape, name, part):
    if (t.dtype is not torch.uint8 or t.shape != shape or not t.is_contiguous()
            or not t.is_cuda):
        raise QloraError(f"{name}{part} must be a contiguous uint8 tensor of shape {shape} on the GPU")


def _need_act8(a, name):
    M, K = a.shape
    _bytes(a.codes, (M, act8_row_bytes(K)), name, ".codes")
    _bytes(a.scales, (M, act8_scale_row_bytes(K)), name, ".scales")


def _need_weight(codes, scales, N, K, name):
    if codes is None or scales is None:
        raise QloraError(f"{name}: the weight does not hold this order")
    _bytes(codes, (N, act8_row_bytes(K)), name, " codes")
    _bytes(scales, ((N + 127) // 128, act8_scale_row_bytes(K)), name, " scales")


def qlora_act8_quantize(X, fmt=ACT8_E4M3, out=None):
    """The 8-bit blocks of a bf16 matrix [M x K] (rows may be strided)."""
    if X.dim() != 2:
        raise QloraError("X must be a matrix")
    M, K = X.shape
    ld = _rows(X, (M, K), "X")
    a = out if out is not None else empty_act8(M, K, X.device, fmt)
    if out is not None:
        if a.shape != (M, K):
            raise QloraError("out must have the shape of X")
        _need_act8(a, "out")
        a.fmt = int(fmt)
    _check(LIB.qlora_act8_quantize(_ptr(X), M, K, ld, a.fmt, _ptr(a.codes), _ptr(a.scales),
                                   _stream()))
    return a


def qlora_act8_dequantize(a, out=None):
    """bf16 [M x K] of 8-bit blocks (exact)."""
    _need_act8(a, "a")
    M, K = a.shape
    out = out if out is not None else torch.empty(M, K, dtype=torch.bfloat16, device=a.codes.device)
    ld = _rows(out, (M, K), "out")
    _check(LIB.qlora_act8_dequantize(_ptr(a.codes), _ptr(a.scales), M, K, a.fmt, _ptr(out), ld,
                                     _stream()))
    return out


def qlora_swiglu_act8_fwd(G, U, fmt=ACT8_E4M3, want_h=True, want_h8=True, want_checkpoint=True,
                          H=None, h8=None, g8=None, u8=None):
    """H = bf16(G sigmoid(G) U) with its 8-bit blocks and those of G and U in
    one pass; returns (H, h8, g8, u8), each None where not wanted."""
    if G.dim() != 2:
        raise QloraError("G must be a matrix")
    M, F = G.shape
    ldg, ldu = _rows(G, (M, F), "G"), _rows(U, (M, F), "U")
    if want_h and H is None:
        H = torch.empty(M, F, dtype=torch.bfloat16, device=G.device)
    ldh = _rows(H, (M, F), "H") if H is not None else 0

    def blocks(a, want, name):
        if a is None:
            return empty_act8(M, F, G.device, fmt) if want else None
        if a.shape != (M, F):
            raise QloraError(f"{name} must have the shape of G")
        _need_act8(a, name)
        a.fmt = int(fmt)
        return a

    h8 = blocks(h8, want_h8, "h8")
    g8 = blocks(g8, want_checkpoint, "g8")
    u8 = blocks(u8, want_checkpoint, "u8")
    args = []
    for a in (h8, g8, u8):
        args += [_ptr(a.codes), _ptr(a.scales)] if a is not None else [None, None]
    _check(LIB.qlora_swiglu_act8_fwd(_ptr(G), ldg, _ptr(U), ldu, M, F, int(fmt), _ptr(H), ldh, *args,
                                     _stream()))
    return H, h8, g8, u8


def qlora_swiglu_act8_bwd(dH, g8, u8, dG=None, dU=None):
    """(dG, dU) of the gated activation from the 8-bit blocks of G and U."""
    _need_act8(g8, "g8")
    _need_act8(u8, "u8")
    if g8.shape != u8.shape or g8.fmt != u8.fmt:
        raise QloraError("g8 and u8 must have one shape and one format")
    M, F = g8.shape
    lddh = _rows(dH, (M, F), "dH")
    dG = dG if dG is not None else torch.empty(M, F, dtype=torch.bfloat16, device=dH.device)
    dU = dU if dU is not None else torch.empty(M, F, dtype=torch.bfloat16, device=dH.device)
    lddg, lddu = _rows(dG, (M, F), "dG"), _rows(dU, (M, F), "dU")
    _check(LIB.qlora_swiglu_act8_bwd(_ptr(dH), lddh, _ptr(g8.codes), _ptr(g8.scales),
                                     _ptr(u8.codes), _ptr(u8.scales), M, F, g8.fmt, _ptr(dG), lddg,
                                     _ptr(dU), lddu, _stream()))
    return dG, dU


def qlora_act8_workspace_bytes(M, N, K, r):
    return int(LIB.qlora_act8_workspace_bytes(M, N, K, r))


def qlora_fp8_workspace_bytes(M, N, K, r, backward=True):
    return int(LIB.qlora_fp8_workspace_bytes(M, N, K, r, int(backward)))


def _ws(n, M, N, K, r, device):
    if n == 0:
        raise QloraError(f"unsupported linear shape M={M} N={N} K={K} r={r}")
    return torch.empty(n, dtype=torch.uint8, device=device)


def act8_workspace(M, N, K, r, device):
    """Workspace of qlora_linear_bwd_act8, with room for its bf16 copy of the
    weight; it serves the 8-bit weight's linear calls too (r = 0 without an adapter)."""
    return _ws(qlora_act8_workspace_bytes(M, N, K, r), M, N, K, r, device)


def fp8_workspace(M, N, K, r, device, backward=True):
    """Workspace of the 8-bit weight's linear calls (r = 0 without an adapter);
    without `backward` of the forward alone, and of a backward pass without dX."""
    return _ws(qlora_fp8_workspace_bytes(M, N, K, r, backward), M, N, K, r, device)


def _given_ws(ws):
    _need(ws, torch.uint8, "ws")
    return ws


def _adapter(A, B, N, K):
    """Rank of an adapter, checked; 0 without one."""
    if A is None and B is None:
        return 0
    if A is None or B is None:
        raise QloraError("A and B come together")
    _need(A, torch.bfloat16, "A")
    _need(B, torch.bfloat16, "B")
    r = A.shape[1] if A.dim() == 2 else -1
    if A.shape != (K, r) or B.shape != (r, N):
        raise QloraError("A must be [K x r] and B [r x N]")
    return r


def _out(t, shape, dtype, device, name):
    if t is None:
        return torch.empty(*shape, dtype=dtype, device=device)  # 0.4 us less than of a tuple
    _need(t, dtype, name)
    if t.shape != shape:
        raise QloraError(f"{name} must have shape {shape}")
    return t


def _given(t, shape, dtype, name):
    if t is not None:
        _need(t, dtype, name)
        if t.shape != shape:
            raise QloraError(f"{name} must have shape {shape}")


def qlora_linear_bwd_act8(dY, X8, T, W, A, B, scale, want_dX=True, keep_mask=None, p=0.0, dX=None,
                          dA=None, dB=None, ws=None):
    """qlora_linear_bwd from the 8-bit blocks of X (keep_mask and p: the
    forward's LoRA dropout); returns (dX or None, dA, dB)."""
    _need_act8(X8, "X8")
    M, K = X8.shape
    N = W.shape[0]
    if tuple(W.shape) != (N, K):
        raise QloraError("W must be [N x K] with the K of X8")
    r = _adapter(A, B, N, K)
    if r == 0:
        raise QloraError("the backward of the NF4 layer needs its adapter")
    _given(dY, (M, N), torch.bfloat16, "dY")
    _given(T, (M, r), torch.float32, "T")
    _given(keep_mask, (M, K // 32), torch.int32, "keep_mask")
    dev = dY.device
    dX = _out(dX, (M, K), torch.bfloat16, dev, "dX") if want_dX else None
    dA = _out(dA, (K, r), torch.float32, dev, "dA")
    dB = _out(dB, (r, N), torch.float32, dev, "dB")
    ws = (_given_ws(ws) if ws is not None else act8_workspace(M, N, K, r, dev) if want_dX
          else fp8_workspace(M, N, K, r, dev, False))
    _check(LIB.qlora_linear_bwd_act8(_ptr(dY), _ptr(X8.codes), _ptr(X8.scales), X8.fmt, _ptr(T),
                                     _ptr(W.codes), _ptr(W.absmax_q), _ptr(W.absmax_s2), _ptr(A),
                                     _ptr(B), M, N, K, r, float(scale), _ptr(keep_mask), float(p),
                                     _ptr(dX), _ptr(dA), _ptr(dB), _ptr(ws), ws.numel(),
                                     W.store_type, _stream()))
    return dX, dA, dB


def qlora_fp8_weight_quantize(W, transposed=True):
    """A bf16 weight [N x K] in 128 x 128 blocks of E4M3 codes; `transposed`
    keeps the other order too, which the input gradient reads."""
    if W.dim() != 2:
        raise QloraError("W must be a matrix")
    _need(W, torch.bfloat16, "W")
    N, K = W.shape

    def pair(rows, cols):
        return (torch.empty(rows, act8_row_bytes(cols), dtype=torch.uint8, device=W.device),
                torch.empty((rows + 127) // 128, act8_scale_row_bytes(cols), dtype=torch.uint8,
                            device=W.device))

    codes, scales = pair(N, K)
    codes_t, scales_t = pair(K, N) if transposed else (None, None)
    _check(LIB.qlora_fp8_weight_quantize(_ptr(W), N, K, _ptr(codes), _ptr(scales), _ptr(codes_t),
                                         _ptr(scales_t), _stream()))
    return Fp8Weight(codes, scales, codes_t, scales_t, (N, K))


def qlora_fp8_linear_fwd(X8, W, A=None, B=None, scale=1.0, want_T=True, Y=None, T=None, ws=None):
    """Y = dec(X8) dec(W)^T + scale (dec(X8) A) B; returns (Y, T), T fp32 or
    None. Without A and B it is the plain product."""
    _need_act8(X8, "X8")
    M, K = X8.shape
    N = W.shape[0]
    if W.shape != (N, K):
        raise QloraError("W must be [N x K] with the K of X8")
    _need_weight(W.codes, W.scales, N, K, "W")
    r = _adapter(A, B, N, K)
    dev = X8.codes.device
    Y = _out(Y, (M, N), torch.bfloat16, dev, "Y")
    T = _out(T, (M, r), torch.float32, dev, "T") if want_T and r else None
    ws = _given_ws(ws) if ws is not None else fp8_workspace(M, N, K, r, dev, False)
    _check(LIB.qlora_fp8_linear_fwd(_ptr(X8.codes), _ptr(X8.scales), X8.fmt, _ptr(W.codes),
                                    _ptr(W.scales), _ptr(A), _ptr(B), M, N, K, r, float(scale),
                                    _ptr(Y), _ptr(T), _ptr(ws), ws.numel(), _stream()))
    return Y, T


def qlora_fp8_linear_bwd(dY, X8, T, W, A=None, B=None, scale=1.0, fmt=ACT8_E4M3, want_dX=True,
                         dX=None, dA=None, dB=None, ws=None):
    """Backward of qlora_fp8_linear_fwd; dY enters dX in 8-bit blocks of
    `fmt`. Returns (dX or None, dA, dB); without an adapter (dX, None, None),
    and X8 may then be None."""
    N, K = W.shape
    r = _adapter(A, B, N, K)
    if dY.dim() != 2:
        raise QloraError("dY must be a matrix")
    M = dY.shape[0]
    _given(dY, (M, N), torch.bfloat16, "dY")
    dev = dY.device
    if r:
        _need_act8(X8, "X8")
        if X8.shape != (M, K):
            raise QloraError("X8 must be [M x K]")
        _given(T, (M, r), torch.float32, "T")
        dA = _out(dA, (K, r), torch.float32, dev, "dA")
        dB = _out(dB, (r, N), torch.float32, dev, "dB")
    elif T is not None or dA is not None or dB is not None or not want_dX:
        raise QloraError("without an adapter only dX is formed")
    if want_dX:
        _need_weight(W.codes_t, W.scales_t, K, N, "W transposed")
        dX = _out(dX, (M, K), torch.bfloat16, dev, "dX")
    else:
        dX = None
    x = (_ptr(X8.codes), _ptr(X8.scales), X8.fmt) if r else (None, None, ACT8_E4M3)
    ws = _given_ws(ws) if ws is not None else fp8_workspace(M, N, K, r, dev, want_dX)
    _check(LIB.qlora_fp8_linear_bwd(_ptr(dY), int(fmt), *x, _ptr(T), _ptr(W.codes_t),
                                    _ptr(W.scales_t), _ptr(A), _ptr(B), M, N, K, r, float(scale),
                                    _ptr(dX), _ptr(dA), _ptr(dB), _ptr(ws), ws.numel(), _stream()))
    return dX, dA, dB


# ---- 4 bits in groups ----------------------------------------------------------

_FLOATS = {torch.bfloat16: 0, torch.float32: 1}  # QLORA_LOGITS_BF16, QLORA_LOGITS_F32


def _matrix(t, name, dtypes=_FLOATS):
    """(rows, columns, leading dimension, device) of a matrix on the current
    device whose rows are contiguous."""
    if t.dim() != 2 or t.dtype not in dtypes or not t.is_cuda:
        raise QloraError(f"{name} must be a matrix of {' or '.join(map(str, dtypes))} on the GPU")
    if t.get_device() != torch._C._cuda_getDevice():
        raise QloraError(f"{name} must be on the current device")
    M, K = t.shape
    ld, step = t.stride()
    if step != 1 and K > 1:
        raise QloraError(f"{name} must have contiguous rows")
    if M <= 1:  # one row: the stride has no meaning
        return M, K, K, t.device
    if ld < K:
        raise QloraError(f"{name} must not have overlapping rows")
    return M, K, ld, t.device


class Int4Weight:
    """A weight [N x K] in 4 bits with a bf16 scale and a zero point (`zeros`
    uint8, or None for 8) for each group of 32, 64 or 128 columns of a row
    (include/qlora.h): codes uint8 [N, K / 2], scales and zeros [N, groups]."""

    __slots__ = ("codes", "scales", "zeros", "shape", "group")

    def __init__(self, codes, scales, zeros, shape, group):
        self.codes, self.scales, self.zeros = codes, scales, zeros
        self.shape = tuple(shape)
        self.group = int(group)

    def nbytes(self):
        return self.codes.numel() + 2 * self.scales.numel() + (0 if self.zeros is None else self.zeros.numel())


def _need_int4(w, dev):
    """(N, K) of a weight whose tensors are checked, one condition to each."""
    N, K = w.shape
    c, s, z = w.codes, w.scales, w.zeros
    groups = -(-K // w.group) if w.group > 0 else -1
    if c.dtype is not torch.uint8 or c.shape != (N, K // 2) or c.device != dev or not c.is_contiguous():
        raise QloraError(f"the weight's codes must be a contiguous uint8 tensor of shape {(N, K // 2)} on {dev}")
    if s.dtype is not torch.bfloat16 or s.shape != (N, groups) or s.device != dev or not s.is_contiguous():
        raise QloraError(f"the weight's scales must be a contiguous bfloat16 tensor of shape {(N, groups)} on {dev}")
    if z is not None and (z.dtype is not torch.uint8 or z.shape != (N, groups) or z.device != dev
                          or not z.is_contiguous()):
        raise QloraError(f"the weight's zeros must be a contiguous uint8 tensor of shape {(N, groups)} on {dev}")
    return N, K


def qlora_int4_quantize(W, group=128, symmetric=False):
    """A bf16 weight [N x K] (rows may be strided) in 4 bits with a scale, and
    unless `symmetric` a zero point, for each `group` columns of a row."""
    N, K, ld, dev = _matrix(W, "W", (torch.bfloat16,))
    if group not in (32, 64, 128) or K % 32:
        raise QloraError("groups of 32, 64 or 128 columns, and a multiple of 32 of them")
    ng = -(-K // group)
    w = Int4Weight(torch.empty(N, K // 2, dtype=torch.uint8, device=dev),
                   torch.empty(N, ng, dtype=torch.bfloat16, device=dev),
                   None if symmetric else torch.empty(N, ng, dtype=torch.uint8, device=dev), (N, K), group)
    _check(LIB.qlora_int4_quantize(_ptr(W), N, K, ld, w.group, _ptr(w.codes), _ptr(w.scales),
                                   _ptr(w.zeros), _stream()))
    return w


def qlora_int4_dequantize(w, out=None):
    """bf16 [N x K] of a weight in groups of 4-bit codes."""
    dev = w.codes.device
    N, K = _need_int4(w, dev)
    out = out if out is not None else torch.empty(N, K, dtype=torch.bfloat16, device=dev)
    n, k, ld, on = _matrix(out, "out", (torch.bfloat16,))
    if (n, k) != (N, K) or on != dev:
        raise QloraError(f"out must have shape {(N, K)}, on {dev}")
    _check(LIB.qlora_int4_dequantize(_ptr(w.codes), _ptr(w.scales), _ptr(w.zeros), N, K, w.group,
                                     _ptr(out), ld, _stream()))
    return out


def qlora_int4_linear_fwd(X, w, dtype=torch.bfloat16, Y=None):
    """Y = X W^T of few tokens X bf16 [M x K] (rows may be strided), in `dtype`
    bfloat16 or float32 (or that of a given Y)."""
    M, K, ldx, dev = _matrix(X, "X", (torch.bfloat16,))
    N, k = _need_int4(w, dev)
    if k != K:
        raise QloraError("W must be [N x K] with the K of X")
    if Y is None:
        if dtype not in _FLOATS:
            raise QloraError("dtype must be bfloat16 or float32")
        Y, ldy = torch.empty(M, N, dtype=dtype, device=dev), N
    else:
        m, n, ldy, on = _matrix(Y, "Y")
        if (m, n) != (M, N) or on != dev:
            raise QloraError(f"Y must have shape {(M, N)}, on {dev}")
    _check(LIB.qlora_int4_linear_fwd(_ptr(X), M, ldx, _ptr(w.codes), _ptr(w.scales), _ptr(w.zeros), N, K,
                                     w.group, _ptr(Y), _FLOATS[Y.dtype], ldy, _stream()))
    return Y


# ---- rows of logits ------------------------------------------------------------


def _logits(Z, name="Z"):
    """(dtype code, T, V, leading dimension, device) of rows of logits."""
    T, V, ld, dev = _matrix(Z, name)
    return _FLOATS[Z.dtype], T, V, ld, dev


def _row(t, shape, dtype, dev, name):
    """A given tensor of one number (or list) per row, or None."""
    if t is not None and (t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous()):
        raise QloraError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on {dev}")
    return t


def _dlogits(Z, dZ, T, V, dev):
    """(dZ, its leading dimension)."""
    if dZ is None:
        return torch.empty(T, V, dtype=Z.dtype, device=dev), V
    if dZ.shape != Z.shape or dZ.dtype is not Z.dtype:
        raise QloraError("dZ must have the shape and type of Z")
    return dZ, _logits(dZ, "dZ")[3]


def qlora_logits_workspace_bytes(T, V, n_top=0):
    return int(LIB.qlora_logits_workspace_bytes(T, V, n_top))


def logits_workspace(T, V, n_top, device):
    """Workspace of qlora_logprobs_fwd (n_top alternatives) and of
    qlora_distill_fwd (n_top = 0)."""
    n = qlora_logits_workspace_bytes(T, V, n_top)
    if n == 0:
        raise QloraError(f"unsupported rows of logits T={T} V={V} n_top={n_top}")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _logits_ws(ws, T, V, n_top, dev):
    if ws is None:
        return logits_workspace(T, V, n_top, dev)
    if ws.dtype is not torch.uint8 or ws.device != dev or not ws.is_contiguous():
        raise QloraError(f"ws must be a contiguous uint8 tensor on {dev}")
    return ws


def qlora_logprobs_fwd(Z, target=None, temperature=1.0, n_top=0, want_entropy=True, want_stats=True,
                       ws=None):
    """Of rows of logits Z [T x V] at a temperature: (logp of target, entropy,
    top_ids, top_logp, stats), each None where not asked for. `target` int64
    [T], outside [0, V) where a row has none (logp 0); the n_top most likely
    entries of each row in descending order, of equal ones the lowest id
    first; `stats` float32 [T x 3] is what the backward pass takes."""
    dt, T, V, ld, dev = _logits(Z)
    _row(target, (T,), torch.int64, dev, "target")
    f32 = torch.float32
    logp = torch.empty(T, dtype=f32, device=dev) if target is not None else None
    ent = torch.empty(T, dtype=f32, device=dev) if want_entropy else None
    stats = torch.empty(T, 3, dtype=f32, device=dev) if want_stats else None
    ids = top = None
    if n_top:
        ids = torch.empty(T, n_top, dtype=torch.int64, device=dev)
        top = torch.empty(T, n_top, dtype=f32, device=dev)
    ws = _logits_ws(ws, T, V, n_top, dev)
    _check(LIB.qlora_logprobs_fwd(_ptr(Z), dt, T, V, ld, _ptr(target), float(temperature), _ptr(logp),
                                  _ptr(ent), int(n_top), _ptr(ids), _ptr(top), _ptr(stats), _ptr(ws),
                                  ws.numel(), _stream()))
    return logp, ent, ids, top, stats


def qlora_logprobs_bwd(Z, target, stats, g_logp=None, g_entropy=None, temperature=1.0, dZ=None):
    """The gradient of the logits from those of the targets' log-probabilities
    and of the entropies (float32 [T], either may be None), with the forward's
    stats. dZ may be Z."""
    dt, T, V, ld, dev = _logits(Z)
    _row(target, (T,), torch.int64, dev, "target")
    _row(stats, (T, 3), torch.float32, dev, "stats")
    _row(g_logp, (T,), torch.float32, dev, "g_logp")
    _row(g_entropy, (T,), torch.float32, dev, "g_entropy")
    dZ, ldd = _dlogits(Z, dZ, T, V, dev)
    _check(LIB.qlora_logprobs_bwd(_ptr(Z), dt, T, V, ld, _ptr(target), float(temperature), _ptr(stats),
                                  _ptr(g_logp), _ptr(g_entropy), _ptr(dZ), ldd, _stream()))
    return dZ


def _teacher(ids, values, T, dev):
    """(values' dtype code, k) of a teacher's top logits."""
    if ids.dim() != 2 or values.dtype not in _FLOATS:
        raise QloraError("ids must be [T x k] and values bfloat16 or float32")
    k = ids.shape[1]
    _row(ids, (T, k), torch.int64, dev, "ids")
    _row(values, (T, k), values.dtype, dev, "values")
    return _FLOATS[values.dtype], k


def qlora_distill_fwd(Z, ids, values, teacher_lse=None, temperature=1.0, want_stats=True, loss=None,
                      ws=None):
    """Divergence of the rows of the student's logits Z [T x V] from a teacher
    known by k logits of each row (ids int64 and values [T x k]; ids outside
    [0, V) are left out) and, optionally, its log sum exp (at the temperature)
    float32 [T]: the rest of its mass is then one more class, otherwise the
    list alone is the distribution. Returns (loss float32 [T], stats [T x 6] or
    None)."""
    dt, T, V, ld, dev = _logits(Z)
    vt, k = _teacher(ids, values, T, dev)
    _row(teacher_lse, (T,), torch.float32, dev, "teacher_lse")
    loss = _out(loss, (T,), torch.float32, dev, "loss")
    stats = torch.empty(T, 6, dtype=torch.float32, device=dev) if want_stats else None
    ws = _logits_ws(ws, T, V, 0, dev)
    _check(LIB.qlora_distill_fwd(_ptr(Z), dt, T, V, ld, _ptr(ids), _ptr(values), vt, k,
                                 _ptr(teacher_lse), float(temperature), _ptr(loss), _ptr(stats),
                                 _ptr(ws), ws.numel(), _stream()))
    return loss, stats


def qlora_distill_bwd(Z, ids, values, stats, g, temperature=1.0, dZ=None):
    """The gradient of the logits from that of qlora_distill_fwd's loss (g
    float32 [T]), with the forward's stats. dZ may be Z."""
    dt, T, V, ld, dev = _logits(Z)
    vt, k = _teacher(ids, values, T, dev)
    _row(stats, (T, 6), torch.float32, dev, "stats")
    _row(g, (T,), torch.float32, dev, "g")
    dZ, ldd = _dlogits(Z, dZ, T, V, dev)
    _check(LIB.qlora_distill_bwd(_ptr(Z), dt, T, V, ld, _ptr(ids), _ptr(values), vt, k,
                                 float(temperature), _ptr(stats), _ptr(g), _ptr(dZ), ldd, _stream()))
    return dZ
