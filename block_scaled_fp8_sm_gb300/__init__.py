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
                   FP8_MAX_GROUPS_PER_LAUNCH, FP8_MAX_EXPERTS, FP8_QUANT_POW2, fp8_group_desc)

__all__ = ["fp8_gemm_blockscaled", "fp8_gemm_blockscaled_noalloc", "fp8_gemm_grouped", "group_descs",
           "fp8_gemm_grouped_device", "fp8_grouped_workspace_bytes", "group_table", "fp8_gemm_pertoken",
           "fp8_quantize_blocks", "fp8_gemm_rowcol", "fp8_gemm_blockscaled_residual",
           "fp8_gemm_blockscaled_quant", "fp8_gemm_pertoken_e8m0", "fp8_gemm_block128", "fp8_gemm_experts",
           "fp8_quantize_tokens", "fp8_swiglu_quantize_tokens", "fp8_status_query", "fp8_strerror", "fp8_version", "fp8_debug_set", "fp8_lib_shutdown",
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
        # the current device, and the current stream of a device
        self.device, self.stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        lib = library()
        self.block128, self.experts = lib.fp8_gemm_block128_ex, lib.fp8_gemm_experts_ex
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
