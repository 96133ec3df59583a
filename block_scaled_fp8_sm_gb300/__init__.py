"""Python binding of libbsfp8 (block-scaled E4M3 GEMM, bf16 out, sm_103a).

Argument marshalling only: torch tensors are turned into device pointers and
the current CUDA stream, and the C entry points of include/bsfp8.h are called
by the same names.  Every step of the computation runs in the library's CUDA
kernels; there is no CPU or library fallback, and a non-zero status raises
``Fp8Error``.
"""
from __future__ import annotations

import contextlib
import ctypes

from . import _abi
from ._abi import (FP8_PATH_AUTO, FP8_PATH_NATIVE, FP8_PATH_PROMOTE,  # noqa: F401
                   FP8_DEBUG_WAIT_LIMIT_CYCLES, FP8_DEBUG_WITHHOLD_STAGE, FP8_DEBUG_TRACE_BUFFER,
                   FP8_MAX_GROUPS_PER_LAUNCH, FP8_MAX_EXPERTS, FP8_QUANT_POW2, FP8_ACT_NONE,
                   FP8_ACT_RELU, FP8_ACT_GELU, FP8_ACT_GELU_TANH, FP8_ACT_SILU, FP8_TYPE_F32, FP8_TYPE_BF16,
                   FP8_ROUTE_SIGMOID, FP8_ROUTE_ALL, FP8_MAX_TOP, FP8_MOE_MAX_TOKENS,
                   fp8_group_desc)

__all__ = ["fp8_gemm_blockscaled", "fp8_gemm_blockscaled_noalloc", "fp8_gemm_grouped", "group_descs",
           "fp8_gemm_grouped_device", "fp8_grouped_workspace_bytes", "group_table", "fp8_gemm_pertoken",
           "fp8_quantize_blocks", "fp8_gemm_rowcol", "fp8_gemm_blockscaled_residual",
           "fp8_gemm_blockscaled_quant", "fp8_gemm_pertoken_e8m0", "fp8_gemm_block128", "fp8_gemm_block128_fused", "fp8_gemm_experts",
           "fp8_quantize_tokens", "fp8_swiglu_quantize_tokens", "fp8_moe_route", "fp8_moe_route_workspace_bytes",
           "fp8_moe_layer", "fp8_moe_layer_workspace_bytes", "fp8_status_query", "fp8_strerror", "fp8_version", "fp8_debug_set", "fp8_lib_shutdown",
           "Fp8Error", "library"]


class Fp8Error(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        super().__init__(f"{what}: {fp8_strerror(code)} ({code})" if what else fp8_strerror(code))


def library():
    return _abi.load()


_raw_stream = None


def _stream(stream):
    """The stream's handle; None is torch's current stream of the current device
    (through the raw accessor: a Stream object costs 3 us of a call's 6)."""
    global _raw_stream
    if stream is None:
        if _raw_stream is None:
            import torch
            torch.cuda.current_stream()   # initialises CUDA
            _raw_stream = lambda: torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())   # noqa: E731
        return _raw_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _outputs_on(stream, device):
    """The context in which a call's outputs are allocated: on the stream that writes them,
    so that the allocator gives no memory that another stream's queued work still uses."""
    if stream is None or device.type != "cuda":
        return contextlib.nullcontext()
    import torch
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device) if isinstance(stream, int) else stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(rc: int, what: str):
    if rc != 0:
        raise Fp8Error(rc, what)


def fp8_gemm_blockscaled(A, sA, B, sB, C, M=None, N=None, K=None, stream=None, mode=None):
    """C[M,N] (bf16) = block-scaled E4M3 GEMM of A[M,K] and B[N,K] with fp32
    32x32 block scales sA, sB.  Tensors are CUDA tensors (A/B uint8 codes or
    float8_e4m3fn, sA/sB float32, C bfloat16).  ``mode`` None = AUTO."""
    M = A.shape[0] if M is None else M
    K = A.shape[1] if K is None else K
    N = B.shape[0] if N is None else N
    lib = library()
    s = _stream(stream)
    if mode is None:
        rc = lib.fp8_gemm_blockscaled(_ptr(A), _ptr(sA), _ptr(B), _ptr(sB), _ptr(C), M, N, K, s)
    else:
        rc = lib.fp8_gemm_blockscaled_ex(_ptr(A), _ptr(sA), _ptr(B), _ptr(sB), _ptr(C), M, N, K,
                                         int(mode), s)
    _check(rc, "fp8_gemm_blockscaled")
    return C


def fp8_gemm_blockscaled_noalloc(A, sA, B, sB, C, M=None, N=None, K=None, stream=None):
    """Same as fp8_gemm_blockscaled (AUTO path) through the entry point that
    allocates no device memory (its status word is a static array inside the
    library).  For callers that cannot allocate device memory, e.g. a server
    whose caching allocator owns the device.  Make the first call on a device
    outside stream capture: it performs that device's one-time set-up."""
    M = A.shape[0] if M is None else M
    K = A.shape[1] if K is None else K
    N = B.shape[0] if N is None else N
    rc = library().fp8_gemm_blockscaled_noalloc(_ptr(A), _ptr(sA), _ptr(B), _ptr(sB), _ptr(C),
                                                M, N, K, _stream(stream))
    _check(rc, "fp8_gemm_blockscaled_noalloc")
    return C


def fp8_gemm_blockscaled_residual(A, sA, B, sB, R, C, M=None, N=None, K=None, stream=None):
    """C = bf16(block-scaled GEMM + R): the residual R (bf16 [M, N], may be C
    itself) added in fp32 in the epilogue before the one bf16 rounding."""
    M = A.shape[0] if M is None else M
    K = A.shape[1] if K is None else K
    N = B.shape[0] if N is None else N
    _check(library().fp8_gemm_blockscaled_residual(_ptr(A), _ptr(sA), _ptr(B), _ptr(sB), _ptr(R), _ptr(C),
                                                   M, N, K, _stream(stream)), "fp8_gemm_blockscaled_residual")
    return C


def fp8_gemm_blockscaled_quant(A, sA, B, sB, Cq, sC, M=None, N=None, K=None, stream=None):
    """(Cq, sC) = block quantization of the block-scaled GEMM's bf16 output, done
    in its epilogue: Cq E4M3 codes [M, N] (uint8 or float8 storage), sC fp32
    [ceil(M/32), N/32] scales; equal bit for bit to fp8_gemm_blockscaled
    followed by fp8_quantize_blocks."""
    M = A.shape[0] if M is None else M
    K = A.shape[1] if K is None else K
    N = B.shape[0] if N is None else N
    _check(library().fp8_gemm_blockscaled_quant(_ptr(A), _ptr(sA), _ptr(B), _ptr(sB), _ptr(Cq), _ptr(sC),
                                                M, N, K, _stream(stream)), "fp8_gemm_blockscaled_quant")
    return Cq, sC


def fp8_gemm_pertoken_e8m0(A, sA, B, sB, C, M=None, N=None, K=None, stream=None):
    """C = bf16(sum_kb 2^(sA[m][kb]-127) * sB * sum_k A*B): per-token A scales as
    UE8M0 bytes (uint8 [M, K/32]), B block scales fp32 powers of two; the
    native path."""
    M = A.shape[0] if M is None else M
    K = A.shape[1] if K is None else K
    N = B.shape[0] if N is None else N
    _check(library().fp8_gemm_pertoken_e8m0(_ptr(A), _ptr(sA), _ptr(B), _ptr(sB), _ptr(C), M, N, K,
                                            _stream(stream)), "fp8_gemm_pertoken_e8m0")
    return C


def fp8_gemm_rowcol(A, sA, B, sB, C, M=None, N=None, K=None, stream=None):
    """C[M,N] (bf16) = sA[m] * sB[n] * sum_k A[m,k] B[n,k]: per-token (sA, fp32
    [M]) x per-channel (sB, fp32 [N]) scales; per-tensor = constant vectors."""
    M = A.shape[0] if M is None else M
    K = A.shape[1] if K is None else K
    N = B.shape[0] if N is None else N
    _check(library().fp8_gemm_rowcol(_ptr(A), _ptr(sA), _ptr(B), _ptr(sB), _ptr(C), M, N, K,
                                     _stream(stream)), "fp8_gemm_rowcol")
    return C


def fp8_gemm_pertoken(A, sA, B, sB, C, M=None, N=None, K=None, stream=None, mode=None):
    """C[M,N] (bf16) with per-token A scales: sA fp32 [M, K/32] (one per row
    of A per 32-K block), sB fp32 [N/32, K/32] blocks.  mode: None (AUTO) or
    FP8_PATH_* (NATIVE: power-of-two scales on the block-scaled MMA)."""
    M = A.shape[0] if M is None else M
    K = A.shape[1] if K is None else K
    N = B.shape[0] if N is None else N
    if mode is None:
        _check(library().fp8_gemm_pertoken(_ptr(A), _ptr(sA), _ptr(B), _ptr(sB), _ptr(C), M, N, K,
                                           _stream(stream)), "fp8_gemm_pertoken")
    else:
        _check(library().fp8_gemm_pertoken_ex(_ptr(A), _ptr(sA), _ptr(B), _ptr(sB), _ptr(C), M, N, K,
                                              mode, _stream(stream)), "fp8_gemm_pertoken_ex")
    return C


def fp8_quantize_blocks(x, q=None, s=None, stream=None):
    """Block quantization of bf16 activations x [M, K] (CUDA tensor) into E4M3
    codes q [M, K] (uint8) and fp32 scales s [ceil(M/32), K/32]: the A and sA
    operands of fp8_gemm_blockscaled.  Returns (q, s); allocates them when not
    given (on ``stream``)."""
    M, K = x.shape
    if q is None or s is None:
        import torch
        with _outputs_on(stream, x.device):
            if q is None:
                q = torch.empty(M, K, dtype=torch.uint8, device=x.device)
            if s is None:
                s = torch.empty((M + 31) // 32, K // 32, dtype=torch.float32, device=x.device)
    _check(library().fp8_quantize_blocks(_ptr(x), _ptr(q), _ptr(s), M, K, _stream(stream)),
           "fp8_quantize_blocks")
    return q, s


# The 128-granular calls check what the C entry points cannot see (they get addresses and
# sizes): types, layouts, and that every tensor is on the current device.  A call of a few microseconds is bound by this marshalling: the checks are
# written out, without helpers or tuples built per tensor.

class _Calls:
    """The library's functions and torch's types, looked up once (on first use)."""
    loaded = None

    def __init__(self):
        import torch
        self.codes = frozenset((torch.uint8, torch.float8_e4m3fn))
        self.f32, self.bf16, self.i32 = torch.float32, torch.bfloat16, torch.int32
        self.floats = frozenset((torch.float32, torch.bfloat16))
        # the current device, and the current stream of a device
        self.device, self.stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        lib = library()
        self.fused = lib.fp8_gemm_block128_fused
        self.block128, self.experts = lib.fp8_gemm_block128_ex, lib.fp8_gemm_experts_ex
        self.route, self.layer = lib.fp8_moe_route, lib.fp8_moe_layer
        self.quantize, self.swiglu = lib.fp8_quantize_tokens, lib.fp8_swiglu_quantize_tokens
        _Calls.loaded = self


def _refused(what, *tensors):
    """The ValueError for tensors that are not contiguous CUDA tensors of their types on
    the current device (the library launches there)."""
    for name, t, kind in tensors:
        if not (t.dtype in kind if isinstance(kind, frozenset) else t.dtype is kind):
            return ValueError(f"{what}: {name} has type {t.dtype}")
    devices = [t.get_device() for _, t, _ in tensors]
    if min(devices) >= 0:
        where = ", ".join(f"{name} on {d}" for (name, _, _), d in zip(tensors, devices))
        current = _Calls.loaded.device()
        if any(d != current for d in devices):
            return ValueError(f"{what}: tensors must be on the current device {current} ({where})")
    return ValueError(f"{what}: tensors must be contiguous and on the GPU")


def fp8_gemm_block128(A, sA, B, sB, C, stream=None, mode=None):
    """C[M,N] (bf16) = sum over 128-K blocks of sA[m][kb] sB[n/128][kb] A B^T:
    A [M,K] codes with fp32 scales sA [M, ceil(K/128)] (one per token and 128
    values), B [N,K] codes with sB [ceil(N/128), ceil(K/128)] (128 x 128 blocks).
    Codes are uint8 or float8_e4m3fn; every tensor contiguous.  mode: None (AUTO),
    FP8_PATH_PROMOTE (each row's bits independent of M) or FP8_PATH_NATIVE
    (power-of-two scales).  N a multiple of 8, K of 16."""
    M, K = A.shape
    N, kb = B.shape[0], (K + 127) // 128
    if (B.shape != (N, K) or C.shape != (M, N) or sA.shape != (M, kb) or sB.shape != ((N + 127) // 128, kb)):
        raise ValueError("fp8_gemm_block128: shapes of A, sA, B, sB, C do not match")
    d = _Calls.loaded or _Calls()
    dev = A.get_device()   # -1: a host tensor
    if not (A.dtype in d.codes and B.dtype in d.codes and sA.dtype is d.f32 and sB.dtype is d.f32
            and C.dtype is d.bf16 and A.is_contiguous() and sA.is_contiguous() and B.is_contiguous()
            and sB.is_contiguous() and C.is_contiguous()
            and dev >= 0 and sA.get_device() == dev and B.get_device() == dev and sB.get_device() == dev
            and C.get_device() == dev and d.device() == dev):
        raise _refused("fp8_gemm_block128", ("A", A, d.codes), ("sA", sA, d.f32), ("B", B, d.codes),
                       ("sB", sB, d.f32), ("C", C, d.bf16))
    rc = d.block128(A.data_ptr(), sA.data_ptr(), B.data_ptr(), sB.data_ptr(), C.data_ptr(), M, N, K,
                    FP8_PATH_AUTO if mode is None else mode,
                    d.stream(dev) if stream is None else _stream(stream))
    if rc:
        raise Fp8Error(rc, "fp8_gemm_block128")
    return C


def fp8_gemm_block128_fused(A, sA, B, sB, C, bias=None, act=FP8_ACT_NONE, residual=None, stream=None, mode=None):
    """C = bf16(act(product + bias) + residual): fp8_gemm_block128 with the epilogue
    done in fp32 before the one rounding.  bias: None or [N], float32 or bfloat16;
    act: FP8_ACT_NONE, _RELU, _GELU (by the error function), _GELU_TANH or _SILU;
    residual: None or bfloat16 [M,N], which may be C itself.  Other arguments as
    fp8_gemm_block128."""
    M, K = A.shape
    N, kb = B.shape[0], (K + 127) // 128
    if (B.shape != (N, K) or C.shape != (M, N) or sA.shape != (M, kb) or sB.shape != ((N + 127) // 128, kb)
            or (bias is not None and bias.shape != (N,)) or (residual is not None and residual.shape != (M, N))):
        raise ValueError("fp8_gemm_block128_fused: shapes of A, sA, B, sB, C, bias, residual do not match")
    d = _Calls.loaded or _Calls()
    dev = A.get_device()
    if not (A.dtype in d.codes and B.dtype in d.codes and sA.dtype is d.f32 and sB.dtype is d.f32
            and C.dtype is d.bf16 and A.is_contiguous() and sA.is_contiguous() and B.is_contiguous()
            and sB.is_contiguous() and C.is_contiguous()
            and dev >= 0 and sA.get_device() == dev and B.get_device() == dev and sB.get_device() == dev
            and C.get_device() == dev and d.device() == dev
            and (bias is None or (bias.dtype in d.floats and bias.is_contiguous() and bias.get_device() == dev))
            and (residual is None or (residual.dtype is d.bf16 and residual.is_contiguous()
                                      and residual.get_device() == dev))):
        raise _refused("fp8_gemm_block128_fused", ("A", A, d.codes), ("sA", sA, d.f32), ("B", B, d.codes),
                       ("sB", sB, d.f32), ("C", C, d.bf16),
                       *([] if bias is None else [("bias", bias, d.floats)]),
                       *([] if residual is None else [("residual", residual, d.bf16)]))
    rc = d.fused(A.data_ptr(), sA.data_ptr(), B.data_ptr(), sB.data_ptr(),
                 None if bias is None else bias.data_ptr(),
                 FP8_TYPE_BF16 if bias is not None and bias.dtype is d.bf16 else FP8_TYPE_F32, act,
                 None if residual is None else residual.data_ptr(), C.data_ptr(), M, N, K,
                 FP8_PATH_AUTO if mode is None else mode,
                 d.stream(dev) if stream is None else _stream(stream))
    if rc:
        raise Fp8Error(rc, "fp8_gemm_block128_fused")
    return C


def fp8_gemm_experts(A, sA, B, sB, C, offsets, stream=None, mode=None):
    """The product of fp8_gemm_block128 grouped by expert: rows offsets[e] ..
    offsets[e+1]-1 of A [T,K] times B[e] of B [E,N,K] into the same rows of
    C [T,N]; sA [T, ceil(K/128)], sB [E, ceil(N/128), ceil(K/128)], offsets an
    int32 CUDA tensor of E + 1 ascending row numbers, read on the device only.
    Experts without rows cost nothing; rows outside the table are not written."""
    T, K = A.shape
    E, N = B.shape[:2]
    kb = (K + 127) // 128
    if (B.shape != (E, N, K) or C.shape != (T, N) or sA.shape != (T, kb)
            or sB.shape != (E, (N + 127) // 128, kb) or offsets.shape != (E + 1,)):
        raise ValueError("fp8_gemm_experts: shapes of A, sA, B, sB, C, offsets do not match")
    d = _Calls.loaded or _Calls()
    dev = A.get_device()
    if not (A.dtype in d.codes and B.dtype in d.codes and sA.dtype is d.f32 and sB.dtype is d.f32
            and C.dtype is d.bf16 and offsets.dtype is d.i32 and A.is_contiguous() and sA.is_contiguous()
            and B.is_contiguous() and sB.is_contiguous() and C.is_contiguous() and offsets.is_contiguous()
            and dev >= 0 and sA.get_device() == dev and B.get_device() == dev and sB.get_device() == dev
            and C.get_device() == dev and offsets.get_device() == dev and d.device() == dev):
        raise _refused("fp8_gemm_experts", ("A", A, d.codes), ("sA", sA, d.f32), ("B", B, d.codes),
                       ("sB", sB, d.f32), ("C", C, d.bf16), ("offsets", offsets, d.i32))
    rc = d.experts(A.data_ptr(), sA.data_ptr(), B.data_ptr(), sB.data_ptr(), C.data_ptr(), offsets.data_ptr(), T, N, K,
                   E, FP8_PATH_AUTO if mode is None else mode,
                   d.stream(dev) if stream is None else _stream(stream))
    if rc:
        raise Fp8Error(rc, "fp8_gemm_experts")
    return C


def fp8_quantize_tokens(x, q=None, s=None, rows=None, pow2=False, stream=None):
    """bf16 activations x [R, K] (rows may be strided) into E4M3 codes q [M, K]
    and fp32 scales s [M, ceil(K/128)], one per 128 values of a token: the A and
    sA operands of fp8_gemm_block128 and fp8_gemm_experts.  rows: None (M = R)
    or an int32 CUDA tensor [M] of rows of x to take (outside of [0, R): a row of
    zeros).  pow2: scales rounded up to powers of two.  Returns (q, s);
    allocates them when not given (on ``stream``)."""
    R, K = x.shape
    M = R if rows is None else rows.shape[0]
    if q is None or s is None:
        q, s = _token_operands(M, K, q, s, x.device, stream)
    if q.shape != (M, K) or s.shape != (M, (K + 127) // 128):
        raise ValueError("fp8_quantize_tokens: q must be [M, K] and s [M, ceil(K/128)]")
    d = _Calls.loaded or _Calls()
    dev = x.get_device()
    if rows is not None and not (rows.dtype is d.i32 and rows.dim() == 1 and rows.is_contiguous()
                                 and rows.get_device() == dev):
        raise _refused("fp8_quantize_tokens (rows: a vector)", ("rows", rows, d.i32), ("x", x, d.bf16))
    if not (x.dtype is d.bf16 and q.dtype in d.codes and s.dtype is d.f32 and q.is_contiguous()
            and s.is_contiguous() and (x.stride(1) == 1 or K <= 1)
            and dev >= 0 and q.get_device() == dev and s.get_device() == dev and d.device() == dev):
        raise _refused("fp8_quantize_tokens", ("x", x, d.bf16), ("q", q, d.codes), ("s", s, d.f32))
    rc = d.quantize(x.data_ptr(), x.stride(0) if R > 1 else K, R, None if rows is None else rows.data_ptr(),
                    q.data_ptr(), s.data_ptr(), M, K, FP8_QUANT_POW2 if pow2 else 0,
                    d.stream(dev) if stream is None else _stream(stream))
    if rc:
        raise Fp8Error(rc, "fp8_quantize_tokens")
    return q, s


def fp8_swiglu_quantize_tokens(x, q=None, s=None, pow2=False, stream=None):
    """fp8_quantize_tokens of silu(gate) * up, with gate = x[:, :K] and
    up = x[:, K:] of bf16 x [M, 2K] (rows may be strided).  128 values whose
    largest magnitude is below 2^-100 count as zeros (codes 0, scale 1); where the
    product passes the largest fp32 number, the scale is infinite and that value's
    code NaN."""
    M, K2 = x.shape
    K = K2 // 2
    if q is None or s is None:
        q, s = _token_operands(M, K, q, s, x.device, stream)
    if K2 % 2 or q.shape != (M, K) or s.shape != (M, (K + 127) // 128):
        raise ValueError("fp8_swiglu_quantize_tokens: x is [M, 2K], q [M, K] and s [M, ceil(K/128)]")
    d = _Calls.loaded or _Calls()
    dev = x.get_device()
    if not (x.dtype is d.bf16 and q.dtype in d.codes and s.dtype is d.f32 and q.is_contiguous()
            and s.is_contiguous() and (x.stride(1) == 1 or K2 <= 1)
            and dev >= 0 and q.get_device() == dev and s.get_device() == dev and d.device() == dev):
        raise _refused("fp8_swiglu_quantize_tokens", ("x", x, d.bf16), ("q", q, d.codes), ("s", s, d.f32))
    rc = d.swiglu(x.data_ptr(), x.stride(0) if M > 1 else K2, q.data_ptr(), s.data_ptr(), M, K,
                  FP8_QUANT_POW2 if pow2 else 0,
                  d.stream(dev) if stream is None else _stream(stream))
    if rc:
        raise Fp8Error(rc, "fp8_swiglu_quantize_tokens")
    return q, s


def _token_operands(M, K, q, s, device, stream):
    import torch
    with _outputs_on(stream, device):
        q = torch.empty(M, K, dtype=torch.uint8, device=device) if q is None else q
        s = torch.empty(M, (K + 127) // 128, dtype=torch.float32, device=device) if s is None else s
    return q, s


def fp8_moe_route_workspace_bytes(T: int, E: int, top: int) -> int:
    return library().fp8_moe_route_workspace_bytes(int(T), int(E), int(top))


def fp8_moe_route(logits, top, sigmoid=False, renormalize=True, scale=1.0, order=True, out=None, workspace=None,
                  stream=None):
    """The router of a mixture-of-experts layer: the ``top`` experts of each token by
    its logits [T, E] (float32 or bfloat16, rows may be strided).  Returns (weights,
    ids, offsets, rows, places), or (weights, ids) with order=False:

    weights float32 [T, top]: softmax of the logits (sigmoid: their sigmoids) over the
    chosen experts (renormalize=False: over all of them, the sigmoids as they are),
    times scale; ids int32 [T, top]: the experts by descending logit, the lower expert
    first of equal ones.  Logits of -inf or NaN are never chosen: where fewer than top
    are left, ids are -1 and weights 0.  offsets int32 [E + 1], rows int32 [T * top],
    places int32 [T, top]: the pairs (token, expert) in expert order, for
    fp8_quantize_tokens(rows=rows) and fp8_gemm_experts(offsets); places[t, j] is where
    pair (t, j) stands (-1: nowhere), and rows are -1 from offsets[E] on.

    out: the tuple of an earlier call, to be written again; workspace: a uint8 CUDA
    tensor of fp8_moe_route_workspace_bytes(T, E, top) bytes, one for each of the calls
    that may overlap.  Both are allocated when not given (on ``stream``)."""
    T, E = logits.shape
    if out is None or (order and workspace is None):
        out, workspace = _route_outputs(T, E, top, order, out, workspace, logits.device, stream)
    if len(out) != (5 if order else 2):
        raise ValueError("fp8_moe_route: out must be (weights, ids, offsets, rows, places), or (weights, ids) without an order")
    d = _Calls.loaded or _Calls()
    dev = logits.get_device()
    weights, ids = out[0], out[1]
    pairs = (T, top)
    good = (weights.shape == pairs and ids.shape == pairs and logits.dtype in d.floats
            and (logits.stride(1) == 1 or E <= 1) and weights.dtype is d.f32 and ids.dtype is d.i32
            and weights.is_contiguous() and ids.is_contiguous()
            and dev >= 0 and weights.get_device() == dev and ids.get_device() == dev and d.device() == dev)
    at, space, size = (None, None, None), None, 0
    if order:
        offsets, rows, places = out[2], out[3], out[4]
        good = (good and offsets.shape == (E + 1,) and rows.shape == (T * top,) and places.shape == pairs
                and offsets.dtype is d.i32 and rows.dtype is d.i32 and places.dtype is d.i32
                and offsets.is_contiguous() and rows.is_contiguous() and places.is_contiguous()
                and workspace.is_contiguous() and offsets.get_device() == dev and rows.get_device() == dev
                and places.get_device() == dev and workspace.get_device() == dev)
        at = (offsets.data_ptr(), rows.data_ptr(), places.data_ptr())
        space, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if not good:
        shapes = [pairs, pairs, (E + 1,), (T * top,), pairs]
        if any(tuple(t.shape) != shape for t, shape in zip(out, shapes)):
            raise ValueError("fp8_moe_route: out must be weights and ids [T, top], and with an order offsets [E + 1], "
                             "rows [T * top] and places [T, top]")
        raise _refused("fp8_moe_route", ("logits", logits, d.floats), ("weights", weights, d.f32),
                       *[("out", t, d.i32) for t in out[1:]],
                       *([("workspace", workspace, workspace.dtype)] if order else []))
    rc = d.route(logits.data_ptr(), logits.stride(0) if T > 1 else E,
                 FP8_TYPE_BF16 if logits.dtype is d.bf16 else FP8_TYPE_F32, T, E, top,
                 (FP8_ROUTE_SIGMOID if sigmoid else 0) | (0 if renormalize else FP8_ROUTE_ALL), scale,
                 weights.data_ptr(), ids.data_ptr(), at[0], at[1], at[2], space, size,
                 d.stream(dev) if stream is None else _stream(stream))
    if rc:
        raise Fp8Error(rc, "fp8_moe_route")
    return out


def _route_outputs(T, E, top, order, out, workspace, device, stream):
    import torch
    i32 = lambda *n: torch.empty(*n, dtype=torch.int32, device=device)   # noqa: E731
    with _outputs_on(stream, device):
        if out is None:
            out = (torch.empty(T, top, dtype=torch.float32, device=device), i32(T, top))
            if order:
                out += (i32(E + 1), i32(T * top), i32(T, top))
        if order and workspace is None:
            workspace = torch.empty(fp8_moe_route_workspace_bytes(T, E, top), dtype=torch.uint8, device=device)
    return out, workspace


def fp8_moe_layer_workspace_bytes(T: int, top: int, I: int) -> int:   # noqa: E741
    return library().fp8_moe_layer_workspace_bytes(int(T), int(top), int(I))


def fp8_moe_layer(x, weights, ids, gate_up, s_gate_up, down, s_down, out=None, workspace=None, stream=None):
    """A whole mixture-of-experts layer for up to FP8_MOE_MAX_TOKENS tokens:
    out[t] = sum_j weights[t, j] down_e(silu(gate_e x_t) * up_e x_t), e = ids[t, j], as
    bfloat16 [T, H], on unquantized activations x (bfloat16 [T, H]).

    weights float32 and ids int32 [T, top] as fp8_moe_route makes them (an id outside
    [0, E) takes no part); gate_up codes [E, 2I, H] (the gate's rows first) with scales
    s_gate_up [E, ceil(2I/128), ceil(H/128)], down codes [E, H, I] with s_down
    [E, ceil(H/128), ceil(I/128)]; H and I multiples of 16.  workspace: a uint8 CUDA
    tensor of fp8_moe_layer_workspace_bytes(T, top, I) bytes, one for each of the calls
    that may overlap.  out and workspace are allocated when not given (on ``stream``)."""
    T, H = x.shape
    E, I2 = gate_up.shape[:2]
    top, I = weights.shape[-1], I2 // 2   # noqa: E741
    hb = (H + 127) // 128
    if T > FP8_MOE_MAX_TOKENS:
        raise ValueError(f"fp8_moe_layer: {T} tokens; it takes up to {FP8_MOE_MAX_TOKENS} (more: fp8_quantize_tokens, "
                         "fp8_gemm_experts and fp8_swiglu_quantize_tokens)")
    if out is None or workspace is None:
        out, workspace = _layer_outputs(T, top, H, I, out, workspace, x.device, stream)
    if (weights.shape != (T, top) or ids.shape != (T, top) or I2 % 2 or gate_up.shape != (E, I2, H)
            or down.shape != (E, H, I) or s_gate_up.shape != (E, (I2 + 127) // 128, hb)
            or s_down.shape != (E, hb, (I + 127) // 128) or out.shape != (T, H)):
        raise ValueError("fp8_moe_layer: shapes of x, weights, ids, gate_up, s_gate_up, down, s_down, out do not match")
    d = _Calls.loaded or _Calls()
    dev = x.get_device()
    if not (x.dtype is d.bf16 and weights.dtype is d.f32 and ids.dtype is d.i32 and gate_up.dtype in d.codes
            and s_gate_up.dtype is d.f32 and down.dtype in d.codes and s_down.dtype is d.f32 and out.dtype is d.bf16
            and x.is_contiguous() and weights.is_contiguous() and ids.is_contiguous() and gate_up.is_contiguous()
            and s_gate_up.is_contiguous() and down.is_contiguous() and s_down.is_contiguous() and out.is_contiguous()
            and workspace.is_contiguous()
            and dev >= 0 and weights.get_device() == dev and ids.get_device() == dev and gate_up.get_device() == dev
            and s_gate_up.get_device() == dev and down.get_device() == dev and s_down.get_device() == dev
            and out.get_device() == dev and workspace.get_device() == dev and d.device() == dev):
        raise _refused("fp8_moe_layer", ("x", x, d.bf16), ("weights", weights, d.f32), ("ids", ids, d.i32),
                       ("gate_up", gate_up, d.codes), ("s_gate_up", s_gate_up, d.f32), ("down", down, d.codes),
                       ("s_down", s_down, d.f32), ("out", out, d.bf16), ("workspace", workspace, workspace.dtype))
    rc = d.layer(x.data_ptr(), weights.data_ptr(), ids.data_ptr(), gate_up.data_ptr(), s_gate_up.data_ptr(),
                 down.data_ptr(), s_down.data_ptr(), out.data_ptr(), T, top, E, H, I, workspace.data_ptr(),
                 workspace.numel() * workspace.element_size(),
                 d.stream(dev) if stream is None else _stream(stream))
    if rc:
        raise Fp8Error(rc, "fp8_moe_layer")
    return out


def _layer_outputs(T, top, H, I, out, workspace, device, stream):   # noqa: E741
    import torch
    with _outputs_on(stream, device):
        if out is None:
            out = torch.empty(T, H, dtype=torch.bfloat16, device=device)
        if workspace is None:
            workspace = torch.empty(fp8_moe_layer_workspace_bytes(T, top, I), dtype=torch.uint8, device=device)
    return out, workspace


class GroupDescs:
    """The host array of per-group pointer records that fp8_gemm_grouped
    takes, built once (the tensors stay referenced) so that repeated calls on
    the same buffers skip the per-call pointer marshalling."""

    def __init__(self, groups):
        self.groups = list(groups)
        self.G = len(self.groups)
        self.arr = (fp8_group_desc * max(self.G, 1))()
        for g, (a, sa, b, sb, c) in enumerate(self.groups):
            self.arr[g] = fp8_group_desc(*[x if isinstance(x, int) else _ptr(x) for x in (a, sa, b, sb, c)])


def group_descs(groups) -> GroupDescs:
    return GroupDescs(groups)


def fp8_gemm_grouped(groups, Ms, N, K, G=None, stream=None, mode=None):
    """groups: sequence of (A_g, sA_g, B_g, sB_g, C_g) CUDA tensors (or raw
    device pointers), or a GroupDescs built from one; Ms: int32 CUDA tensor of
    G row counts (read on device)."""
    if isinstance(groups, GroupDescs):
        G = groups.G if G is None else G
        arr = groups.arr
    else:
        G = len(groups) if G is None else G
        arr = (fp8_group_desc * max(G, 1))()
        for g, (a, sa, b, sb, c) in enumerate(groups[:G]):
            arr[g] = fp8_group_desc(*[x if isinstance(x, int) else _ptr(x) for x in (a, sa, b, sb, c)])
    lib = library()
    s = _stream(stream)
    ms = Ms if isinstance(Ms, int) else _ptr(Ms)
    if mode is None:
        rc = lib.fp8_gemm_grouped(arr, ms, N, K, G, s)
    else:
        rc = lib.fp8_gemm_grouped_ex(arr, ms, N, K, G, int(mode), s)
    _check(rc, "fp8_gemm_grouped")


def group_table(groups, device):
    """The records of fp8_gemm_grouped_device: an int64 CUDA tensor [G, 5]
    holding each group's (A, sA, B, sB, C) device pointers, in the layout of
    fp8_group_desc.  The tensors must stay alive while launches use it."""
    import torch
    rows = [[x if isinstance(x, int) else _ptr(x) for x in g] for g in groups]
    return torch.tensor(rows, dtype=torch.int64).reshape(len(rows), 5).to(device)


def fp8_grouped_workspace_bytes(G: int) -> int:
    return library().fp8_grouped_workspace_bytes(int(G))


def fp8_gemm_grouped_device(table, Ms, N, K, workspace, G=None, stream=None):
    """Grouped GEMM whose records live in device memory: ``table`` is an
    int64 CUDA tensor [G, 5] of device pointers (see group_table), ``Ms`` an
    int32 CUDA tensor of row counts, ``workspace`` a CUDA tensor of at least
    fp8_grouped_workspace_bytes(G) bytes (128-byte aligned).  Every argument
    stays on the device, so a CUDA graph captured once follows later changes
    of the table and the row counts."""
    G = table.shape[0] if G is None else G
    rc = library().fp8_gemm_grouped_device(_ptr(table), _ptr(Ms), N, K, G, _ptr(workspace),
                                           workspace.numel() * workspace.element_size(), _stream(stream))
    _check(rc, "fp8_gemm_grouped_device")


def fp8_status_query(stream=None) -> int:
    out = ctypes.c_int(0)
    _check(library().fp8_status_query(_stream(stream), ctypes.byref(out)), "fp8_status_query")
    return out.value


def fp8_strerror(code: int) -> str:
    return library().fp8_strerror(int(code)).decode()


def fp8_version() -> int:
    return library().fp8_version()


def fp8_debug_set(key: int, value: int):
    _check(library().fp8_debug_set(int(key), int(value)), "fp8_debug_set")


def fp8_lib_shutdown():
    library().fp8_lib_shutdown()
