"""B200 (sm_100a) fine-grained block-scaled FP8 GEMM -- Python binding.

A thin ctypes layer over ``libdg.so`` (declared in ``include/dg.h``).  The
functions here only marshal torch tensors into pointers, sizes and the current
CUDA stream; every step of the computation runs in the library's CUDA kernels.
There is no CPU fallback: if the library is missing or the device is not
sm_100, the calls raise.

Entry points (same names as the C ABI):

* ``dg_quantize_1x128(x, pow2=False)`` -> (q, sf)    1 x 128 E4M3 activations
* ``dg_quantize_128x128(w, pow2=False)`` -> (q, sf)  128 x 128 E4M3 weights
* ``dg_quantize_128x1(x, pow2=False)`` -> (q, sf)  1 x 128-along-K groups of an
  operand stored [K, M] (K outermost)
* ``dg_pack_ue8m0(sf, m)`` -> packed int32 UE8M0 scales (4 K groups per word)
* ``dg_pack_ue8m0_128x128(sf, n)`` -> B's 128 x 128 block scales packed per row
* ``dg_fp8_gemm_nt(a, sfa, b, sfb, d, workspace=None)``
* ``dg_fp8_gemm_nt_accumulate(a, sfa, b, sfb, c, d, workspace=None)``  D = C + A B^T
* ``dg_fp8_gemm_nt_noalloc(a, sfa, b, sfb, d)``
* ``dg_fp8_gemm_nt_quantize(a, sfa, b, sfb, pow2=False)`` -> (dq, sfd)  the
  output quantized 1 x 128 in the epilogue (E4M3 codes and MN-major scales)
* ``dg_fp8_gemm_nn / _tn / _tt(a, sfa, b, sfb, d, workspace=None)``  the other
  operand layouts (A stored [K, M] for T, B stored [K, N] for N)
* ``dg_m_grouped_fp8_gemm_nt_contiguous(a, sfa, b, sfb, d, m_indices)``
* ``dg_m_grouped_fp8_gemm_nt_masked(a, sfa, b, sfb, d, masked_m)``
* ``dg_k_grouped_fp8_gemm_nt_contiguous(a, sfa, b, sfb, d, k_sizes, c=None)``
* ``dg_k_grouped_fp8_gemm_tn_contiguous(a, sfa, b, sfb, d, k_sizes, c=None)``
  (a [K, M] and b [K, N])
* ``dg_fp8_gemm_nt_ue8m0(a, sfa, b, sfb, d)``, ``dg_m_grouped_fp8_gemm_nt_masked_ue8m0(
  a, sfa, b, sfb, d, masked_m)``  power-of-two scales as packed UE8M0 words,
  applied by the tensor cores
* ``dg_quantize_mxfp4(x, transpose=False)`` -> (q, sf)  1 x 32 MXFP4 (E2M1 codes,
  UE8M0 scale words) of the rows or the columns of x;
  ``dg_dequantize_mxfp4(q, sf, dtype)`` reads them back
* ``dg_mxfp4_gemm_nt(a, sfa, b, sfb, d)``,
  ``dg_m_grouped_mxfp4_gemm_nt_contiguous(a, sfa, b, sfb, d, m_indices)``,
  ``dg_m_grouped_mxfp4_gemm_nt_masked(a, sfa, b, sfb, d, masked_m)``
* ``dg_moe_route(logits, top_k)`` -> (idx, weights, counts, loss, num_tokens)
  softmax top-k routing with per-expert counts and the balance loss;
  ``dg_moe_route_backward(...)`` -> dlogits
* ``dg_get_device_status()``, helpers ``dg_get_tma_aligned_size``,
  ``dg_get_mk_alignment_for_contiguous_layout``, ``dg_set_num_sms``,
  ``dg_get_num_sms``, ``dg_fp8_gemm_nt_workspace_size``.

``stream`` (a ``torch.cuda.Stream``; the current one if not given) is where a call
runs.  It does not wait for other streams: what its inputs hold must be ready
there.  The MXFP4 and routing calls mark their tensors as used on a stream that
is given, so temporaries may be passed; for the other calls keep the tensors until
the stream is done with them (or call ``record_stream``).

Layouts follow the header: A [M, K] uint8 (E4M3 codes), its scales MN-major
[K/128, ld] (``sf.t()`` of the logical [M, K/128]), B [N, K] uint8 with scales
[ceil(N/128), K/128], D [M, N] bfloat16.
"""

from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdg.so")

DG_OK = 0
DG_DTYPE_F32, DG_DTYPE_BF16 = 0, 1
DG_SCALE_FP32, DG_SCALE_POW2 = 0, 1
DG_ERR_INVALID_ARG, DG_ERR_ALIGNMENT, DG_ERR_UNSUPPORTED_ARCH = -1, -2, -3
DG_ERR_CUDA, DG_ERR_WORKSPACE = -4, -5
DG_ERR_TIMEOUT, DG_ERR_DEVICE_DATA = -6, -7

EXPORTS = [
    "dg_status_string", "dg_get_mk_alignment_for_contiguous_layout",
    "dg_get_tma_aligned_size", "dg_set_num_sms", "dg_get_num_sms",
    "dg_quantize_1x128", "dg_quantize_128x1", "dg_quantize_128x128", "dg_pack_ue8m0",
    "dg_pack_ue8m0_128x128",
    "dg_fp8_gemm_nt", "dg_fp8_gemm_nt_ue8m0", "dg_m_grouped_fp8_gemm_nt_masked_ue8m0",
    "dg_fp8_gemm_nn", "dg_fp8_gemm_tn", "dg_fp8_gemm_tt", "dg_k_grouped_fp8_gemm_tn_contiguous",
    "dg_fp8_gemm_nt_quantize",
    "dg_fp8_gemm_nt_workspace_size", "dg_fp8_gemm_nt_noalloc", "dg_fp8_gemm_nt_accumulate",
    "dg_m_grouped_fp8_gemm_nt_contiguous",
    "dg_m_grouped_fp8_gemm_nt_masked", "dg_k_grouped_fp8_gemm_nt_contiguous",
    "dg_get_device_status",
    "dg_quantize_mxfp4", "dg_dequantize_mxfp4", "dg_mxfp4_gemm_nt",
    "dg_m_grouped_mxfp4_gemm_nt_contiguous", "dg_m_grouped_mxfp4_gemm_nt_masked",
    "dg_moe_route", "dg_moe_route_workspace_size", "dg_moe_route_backward",
]

_lib = None


class DGError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libdg.so (once) and declares the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing; build it with `python -m moe_grouped_gemm_act_b200.build`")
    lib = ctypes.CDLL(path)
    P, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    sig = {
        "dg_status_string": (ctypes.c_char_p, [I]),
        "dg_get_mk_alignment_for_contiguous_layout": (I, []),
        "dg_get_tma_aligned_size": (I64, [I64, I]),
        "dg_set_num_sms": (I, [I]),
        "dg_get_num_sms": (I, []),
        "dg_quantize_1x128": (I, [P, I, I64, I64, I64, I64, P, I64, P, I64, I, P]),
        "dg_quantize_128x128": (I, [P, I64, I64, I64, P, P, I, P]),
        "dg_quantize_128x1": (I, [P, I, I64, I64, I64, P, I64, P, I64, I, P]),
        "dg_pack_ue8m0": (I, [P, I64, I64, I64, I64, P, I64, P]),
        "dg_pack_ue8m0_128x128": (I, [P, I64, I64, I64, P, I64, P]),
        "dg_fp8_gemm_nt_ue8m0": (I, [P, P, I64, P, P, I64, P, I64, I64, I64, P]),
        "dg_m_grouped_fp8_gemm_nt_masked_ue8m0":
            (I, [P, P, I64, P, P, I64, P, P, I, I64, I64, I64, P]),
        "dg_fp8_gemm_nt": (I, [P, P, I64, P, P, P, I64, I64, I64, P, SZ, P]),
        "dg_fp8_gemm_nn": (I, [P, P, I64, P, P, P, I64, I64, I64, P, SZ, P]),
        "dg_fp8_gemm_nt_quantize": (I, [P, P, I64, P, P, P, P, I64, I64, I64, I64, I, P]),
        "dg_fp8_gemm_tn": (I, [P, P, I64, P, P, P, I64, I64, I64, P, SZ, P]),
        "dg_fp8_gemm_tt": (I, [P, P, I64, P, P, P, I64, I64, I64, P, SZ, P]),
        "dg_k_grouped_fp8_gemm_tn_contiguous":
            (I, [P, P, I64, P, P, I64, P, P, P, I, I64, I64, I64, P]),
        "dg_fp8_gemm_nt_workspace_size": (SZ, [I64, I64, I64]),
        "dg_fp8_gemm_nt_noalloc": (I, [P, P, I64, P, P, P, I64, I64, I64, P]),
        "dg_fp8_gemm_nt_accumulate": (I, [P, P, I64, P, P, P, P, I64, I64, I64, P, SZ, P]),
        "dg_m_grouped_fp8_gemm_nt_contiguous":
            (I, [P, P, I64, P, P, P, P, I64, I64, I64, I, P]),
        "dg_m_grouped_fp8_gemm_nt_masked":
            (I, [P, P, I64, P, P, P, P, I, I64, I64, I64, P]),
        "dg_k_grouped_fp8_gemm_nt_contiguous":
            (I, [P, P, I64, P, P, I64, P, P, P, I, I64, I64, I64, P]),
        "dg_get_device_status": (I, [P, ctypes.POINTER(ctypes.c_int)]),
        "dg_quantize_mxfp4": (I, [P, I, I64, I64, I64, I64, I, P, P, P]),
        "dg_dequantize_mxfp4": (I, [P, P, I64, I64, I64, P, I, I64, P]),
        "dg_mxfp4_gemm_nt": (I, [P, P, P, P, P, I64, I64, I64, P]),
        "dg_m_grouped_mxfp4_gemm_nt_contiguous":
            (I, [P, P, P, P, P, P, I64, I64, I64, I, P]),
        "dg_m_grouped_mxfp4_gemm_nt_masked":
            (I, [P, P, P, P, P, P, I, I64, I64, I64, P]),
        "dg_moe_route":
            (I, [P, I, I64, I, I64, I, I, P, P, P, P, P, P, P, SZ, P]),
        "dg_moe_route_workspace_size": (SZ, [I64, I]),
        "dg_moe_route_backward":
            (I, [P, I, I64, I, I64, I, I, P, P, P, P, P, P, P, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().dg_status_string(int(status)).decode()


def _check(rc: int, what: str) -> None:
    if rc != DG_OK:
        raise DGError(rc, what)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _need_cuda(*ts: torch.Tensor) -> None:
    for t in ts:
        if not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors (there is no CPU path)")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def _expect(t: torch.Tensor | None, name: str, dtype: torch.dtype, shape: tuple) -> None:
    """Raises ValueError unless t has this dtype and shape.  A shape entry of
    None accepts any extent; a pair (lo, "ld") accepts any multiple of 4 that
    is at least lo (the leading dimension of an MN-major scale tensor).  The C
    ABI takes raw pointers and cannot check extents, so every tensor is
    checked here before the call."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != len(shape):
        raise ValueError(f"{name} must have {len(shape)} dimensions, got shape {tuple(t.shape)}")
    for i, (got, want) in enumerate(zip(t.shape, shape)):
        if want is None:
            continue
        if isinstance(want, tuple):
            lo = want[0]
            if got < lo or got % 4:
                raise ValueError(f"{name}: dimension {i} is {got}; it must be a multiple of 4 "
                                 f">= {lo} (shape {tuple(t.shape)})")
        elif got != want:
            raise ValueError(f"{name}: dimension {i} is {got}, expected {want} "
                             f"(shape {tuple(t.shape)})")


def _gemm_operands(a, sfa, b, sfb, m, n, k, groups=None, a_batch=None):
    """Checks the FP8 operands and their scales of an NT GEMM: A [.., M, K]
    uint8 with MN-major 1x128 scales [.., K/128, ld >= M], B [.., N, K] uint8
    with 128x128 scales [.., ceil(N/128), K/128]."""
    if k % 128:
        return  # the C ABI rejects it (DG_ERR_INVALID_ARG) before touching memory
    lead_a = () if a_batch is None else (a_batch,)
    lead_b = () if groups is None else (groups,)
    _expect(a, "a", torch.uint8, lead_a + (m, k))
    _expect(sfa, "sfa", torch.float32, lead_a + (k // 128, (m, "ld")))
    _expect(b, "b", torch.uint8, lead_b + (n, k))
    _expect(sfb, "sfb", torch.float32, lead_b + (-(-n // 128), k // 128))


# ------------------------------------------------------------------ helpers
def dg_get_mk_alignment_for_contiguous_layout() -> int:
    return load_library().dg_get_mk_alignment_for_contiguous_layout()


def dg_get_tma_aligned_size(n: int, elem_bytes: int) -> int:
    return load_library().dg_get_tma_aligned_size(n, elem_bytes)


def dg_set_num_sms(n: int) -> None:
    _check(load_library().dg_set_num_sms(n), "dg_set_num_sms")


def dg_get_num_sms() -> int:
    return load_library().dg_get_num_sms()


def dg_fp8_gemm_nt_workspace_size(m: int, n: int, k: int) -> int:
    return load_library().dg_fp8_gemm_nt_workspace_size(m, n, k)


def dg_get_device_status(stream=None) -> int:
    st = ctypes.c_int(0)
    _check(load_library().dg_get_device_status(_stream(stream), ctypes.byref(st)),
           "dg_get_device_status")
    return st.value


# ------------------------------------------------------------------ quantizers
def dg_quantize_1x128(x: torch.Tensor, pow2: bool = False, q=None, sf=None,
                      stream=None):
    """1 x 128 quantization of x [M, K] or [B, M, K] (float32 or bfloat16).

    Returns (q uint8 like x, sf float32 [K/128, ld] or [B, K/128, ld]) with
    ld = dg_get_tma_aligned_size(M, 4); sf[..., g, i] is the scale of row i,
    group g.
    """
    _need_cuda(x)
    batched = x.dim() == 3
    xb = x if batched else x.unsqueeze(0)
    b, m, k = xb.shape
    dtype = {torch.float32: DG_DTYPE_F32, torch.bfloat16: DG_DTYPE_BF16}.get(x.dtype)
    if dtype is None:
        raise ValueError("x must be float32 or bfloat16")
    ld = dg_get_tma_aligned_size(m, 4)
    if q is None:
        q = torch.empty(xb.shape, dtype=torch.uint8, device=x.device)
    if sf is None:
        sf = torch.empty((b, k // 128, ld), dtype=torch.float32, device=x.device)
    _need_cuda(q, sf)
    if k % 128 == 0:  # (otherwise the C ABI rejects the call)
        _expect(q if q.dim() == 3 else q.unsqueeze(0), "q", torch.uint8, (b, m, k))
        _expect(sf if sf.dim() == 3 else sf.unsqueeze(0), "sf", torch.float32,
                (b, k // 128, (m, "ld")))
    rc = load_library().dg_quantize_1x128(
        _ptr(xb), dtype, b, m, k, k, _ptr(q), k, _ptr(sf), sf.shape[-1],
        DG_SCALE_POW2 if pow2 else DG_SCALE_FP32, _stream(stream))
    _check(rc, "dg_quantize_1x128")
    if not batched:
        return q.view(m, k), sf.view(k // 128, sf.shape[-1])
    return q, sf


def dg_quantize_128x1(x: torch.Tensor, pow2: bool = False, q=None, sf=None, stream=None):
    """1 x 128-along-K quantization of an operand stored [K, M] (float32 or
    bfloat16): returns (q uint8 [K, M], sf float32 [K/128, ld]) with ld =
    dg_get_tma_aligned_size(M, 4); sf[g, m] is the scale of column m's K
    group g.  Bit-exact with dg_quantize_1x128 of x.T."""
    _need_cuda(x)
    k, m = x.shape
    dtype = {torch.float32: DG_DTYPE_F32, torch.bfloat16: DG_DTYPE_BF16}.get(x.dtype)
    if dtype is None:
        raise ValueError("x must be float32 or bfloat16")
    if q is None:
        q = torch.empty((k, m), dtype=torch.uint8, device=x.device)
    if sf is None:
        sf = torch.empty((k // 128, dg_get_tma_aligned_size(m, 4)), dtype=torch.float32,
                         device=x.device)
    _need_cuda(q, sf)
    if k % 128 == 0:
        _expect(q, "q", torch.uint8, (k, m))
        _expect(sf, "sf", torch.float32, (k // 128, (m, "ld")))
    rc = load_library().dg_quantize_128x1(
        _ptr(x), dtype, k, m, m, _ptr(q), m, _ptr(sf), sf.shape[-1],
        DG_SCALE_POW2 if pow2 else DG_SCALE_FP32, _stream(stream))
    _check(rc, "dg_quantize_128x1")
    return q, sf


def dg_quantize_128x128(w: torch.Tensor, pow2: bool = False, stream=None):
    """128 x 128 quantization of w [N, K] or [G, N, K] float32.

    Returns (q uint8 like w, sf float32 [ceil(N/128), K/128] or
    [G, ceil(N/128), K/128])."""
    _need_cuda(w)
    if w.dtype != torch.float32:
        raise ValueError("w must be float32")
    grouped = w.dim() == 3
    wb = w if grouped else w.unsqueeze(0)
    g, n, k = wb.shape
    q = torch.empty(wb.shape, dtype=torch.uint8, device=w.device)
    sf = torch.empty((g, -(-n // 128), k // 128), dtype=torch.float32, device=w.device)
    rc = load_library().dg_quantize_128x128(
        _ptr(wb), g, n, k, _ptr(q), _ptr(sf),
        DG_SCALE_POW2 if pow2 else DG_SCALE_FP32, _stream(stream))
    _check(rc, "dg_quantize_128x128")
    if not grouped:
        return q[0], sf[0]
    return q, sf


def dg_pack_ue8m0(sf: torch.Tensor, m: int, packed=None, stream=None) -> torch.Tensor:
    """Packs power-of-two scales sf (float32 [Kg, ld] or [B, Kg, ld], the
    MN-major layout dg_quantize_1x128 returns) of m rows into UE8M0 words:
    int32 [ceil(Kg/4), ld'] (or [B, ceil(Kg/4), ld']), ld' =
    dg_get_tma_aligned_size(m, 4); word (p, i) holds groups 4p .. 4p+3 of row
    i, one byte each, lowest group in the lowest byte.  Scales that are not +0
    or a normal power of two are reported through dg_get_device_status()."""
    _need_cuda(sf)
    if sf.dtype != torch.float32:
        raise ValueError("sf must be float32")
    batched = sf.dim() == 3
    sb = sf if batched else sf.unsqueeze(0)
    b, kg, ld = sb.shape
    words = -(-kg // 4)
    if m > ld:
        raise ValueError(f"m = {m} exceeds the scale rows' leading dimension {ld}")
    if packed is None:
        packed = torch.empty((b, words, dg_get_tma_aligned_size(m, 4)), dtype=torch.int32,
                             device=sf.device)
    _need_cuda(packed)
    _expect(packed if packed.dim() == 3 else packed.unsqueeze(0), "packed", torch.int32,
            (b, words, (m, "ld")))
    rc = load_library().dg_pack_ue8m0(_ptr(sb), b, m, kg, ld, _ptr(packed), packed.shape[-1],
                                      _stream(stream))
    _check(rc, "dg_pack_ue8m0")
    return packed if batched else packed.view(words, packed.shape[-1])


def dg_pack_ue8m0_128x128(sf: torch.Tensor, n: int, packed=None, stream=None) -> torch.Tensor:
    """B's 128 x 128 block scales sf (float32 power-of-two values,
    [ceil(n/128), Kg] or [G, ceil(n/128), Kg], as dg_quantize_128x128(pow2=True)
    returns) written out per row of B in the packed UE8M0 layout: int32
    [ceil(Kg/4), ld] (or [G, ceil(Kg/4), ld]), ld = dg_get_tma_aligned_size(n,
    4); word (p, j) holds groups 4p .. 4p+3 of row j's block."""
    _need_cuda(sf)
    if sf.dtype != torch.float32:
        raise ValueError("sf must be float32")
    grouped = sf.dim() == 3
    sb = sf if grouped else sf.unsqueeze(0)
    g, nb, kg = sb.shape
    if nb != -(-n // 128):
        raise ValueError(f"sf has {nb} row blocks; n = {n} needs {-(-n // 128)}")
    words = -(-kg // 4)
    if packed is None:
        packed = torch.empty((g, words, dg_get_tma_aligned_size(n, 4)), dtype=torch.int32,
                             device=sf.device)
    _need_cuda(packed)
    _expect(packed if packed.dim() == 3 else packed.unsqueeze(0), "packed", torch.int32,
            (g, words, (n, "ld")))
    rc = load_library().dg_pack_ue8m0_128x128(_ptr(sb), g, n, kg, _ptr(packed),
                                              packed.shape[-1], _stream(stream))
    _check(rc, "dg_pack_ue8m0_128x128")
    return packed if grouped else packed.view(words, packed.shape[-1])


# ------------------------------------------------------------------ GEMMs
def dg_fp8_gemm_nt(a, sfa, b, sfb, d, workspace: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """D = A * B^T with 1x128 (sfa, MN-major [K/128, ld]) and 128x128 (sfb)
    scales; d is a preallocated bfloat16 [M, N] tensor, returned."""
    _need_cuda(a, sfa, b, sfb, d)
    m, k = a.shape
    n = b.shape[0]
    _gemm_operands(a, sfa, b, sfb, m, n, k)
    _expect(d, "d", torch.bfloat16, (m, n))
    if workspace is not None:
        _need_cuda(workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load_library().dg_fp8_gemm_nt(
        _ptr(a), _ptr(sfa), sfa.shape[-1], _ptr(b), _ptr(sfb), _ptr(d), m, n, k,
        _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc, "dg_fp8_gemm_nt")
    return d


def _fp8_gemm_layout(name, a_t, b_t, a, sfa, b, sfb, d, workspace, stream):
    """The dense GEMM with A stored [K, M] when a_t, B stored [K, N] when b_t
    (else [M, K] and [N, K]); the scales keep their logical layouts."""
    _need_cuda(a, sfa, b, sfb, d)
    if a_t:
        k, m = a.shape
    else:
        m, k = a.shape
    n = b.shape[1] if b_t else b.shape[0]
    if k % 128 == 0:
        _expect(a, "a", torch.uint8, (k, m) if a_t else (m, k))
        _expect(b, "b", torch.uint8, (k, n) if b_t else (n, k))
        _expect(sfa, "sfa", torch.float32, (k // 128, (m, "ld")))
        _expect(sfb, "sfb", torch.float32, (-(-n // 128), k // 128))
    _expect(d, "d", torch.bfloat16, (m, n))
    if workspace is not None:
        _need_cuda(workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = getattr(load_library(), name)(
        _ptr(a), _ptr(sfa), sfa.shape[-1], _ptr(b), _ptr(sfb), _ptr(d), m, n, k,
        _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc, name)
    return d


def dg_fp8_gemm_nt_quantize(a, sfa, b, sfb, pow2: bool = False, dq=None, sfd=None,
                            stream=None):
    """D = A * B^T quantized 1 x 128 in the GEMM's epilogue: returns (dq uint8
    [M, N] E4M3 codes, sfd float32 [N/128, ld] MN-major scales, ld =
    dg_get_tma_aligned_size(M, 4)) -- bit-identical to dg_quantize_1x128 of
    the BF16 result of the same tile form.  N % 128 == 0."""
    _need_cuda(a, sfa, b, sfb)
    m, k = a.shape
    n = b.shape[0]
    _gemm_operands(a, sfa, b, sfb, m, n, k)
    if n % 128:
        raise ValueError(f"N = {n} must be a multiple of 128")
    if dq is None:
        dq = torch.empty((m, n), dtype=torch.uint8, device=a.device)
    if sfd is None:
        sfd = torch.empty((n // 128, dg_get_tma_aligned_size(m, 4)), dtype=torch.float32,
                          device=a.device)
    _need_cuda(dq, sfd)
    _expect(dq, "dq", torch.uint8, (m, n))
    _expect(sfd, "sfd", torch.float32, (n // 128, (m, "ld")))
    rc = load_library().dg_fp8_gemm_nt_quantize(
        _ptr(a), _ptr(sfa), sfa.shape[-1], _ptr(b), _ptr(sfb), _ptr(dq), _ptr(sfd),
        sfd.shape[-1], m, n, k, DG_SCALE_POW2 if pow2 else DG_SCALE_FP32, _stream(stream))
    _check(rc, "dg_fp8_gemm_nt_quantize")
    return dq, sfd


def dg_fp8_gemm_nn(a, sfa, b, sfb, d, workspace=None, stream=None) -> torch.Tensor:
    """D = A * B^T with A [M, K] and B stored [K, N] (N contiguous, N % 16 == 0)."""
    return _fp8_gemm_layout("dg_fp8_gemm_nn", False, True, a, sfa, b, sfb, d, workspace, stream)


def dg_fp8_gemm_tn(a, sfa, b, sfb, d, workspace=None, stream=None) -> torch.Tensor:
    """D = A * B^T with A stored [K, M] and B stored [K, N] (M, N % 16 == 0)."""
    return _fp8_gemm_layout("dg_fp8_gemm_tn", True, True, a, sfa, b, sfb, d, workspace, stream)


def dg_fp8_gemm_tt(a, sfa, b, sfb, d, workspace=None, stream=None) -> torch.Tensor:
    """D = A * B^T with A stored [K, M] (M % 16 == 0) and B [N, K]."""
    return _fp8_gemm_layout("dg_fp8_gemm_tt", True, False, a, sfa, b, sfb, d, workspace, stream)


def dg_fp8_gemm_nt_accumulate(a, sfa, b, sfb, c, d, workspace: torch.Tensor | None = None,
                              stream=None) -> torch.Tensor:
    """D = C + A * B^T: as dg_fp8_gemm_nt, with c a float32 [M, N] tensor added
    before the BF16 rounding of d; d is returned."""
    _need_cuda(a, sfa, b, sfb, c, d)
    m, k = a.shape
    n = b.shape[0]
    _gemm_operands(a, sfa, b, sfb, m, n, k)
    _expect(c, "c", torch.float32, (m, n))
    _expect(d, "d", torch.bfloat16, (m, n))
    if workspace is not None:
        _need_cuda(workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load_library().dg_fp8_gemm_nt_accumulate(
        _ptr(a), _ptr(sfa), sfa.shape[-1], _ptr(b), _ptr(sfb), _ptr(c), _ptr(d), m, n, k,
        _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc, "dg_fp8_gemm_nt_accumulate")
    return d


def dg_fp8_gemm_nt_noalloc(a, sfa, b, sfb, d, stream=None) -> torch.Tensor:
    """dg_fp8_gemm_nt without a caller-provided workspace, for callers that
    cannot allocate device memory (see include/dg.h): the split-K scratch is
    the library's own fixed 32 MiB per-device array.  Shapes whose preferred
    split needs more raise DGError (DG_ERR_WORKSPACE).  Calls that overlap on
    the GPU share that array and must be ordered."""
    _need_cuda(a, sfa, b, sfb, d)
    m, k = a.shape
    n = b.shape[0]
    _gemm_operands(a, sfa, b, sfb, m, n, k)
    _expect(d, "d", torch.bfloat16, (m, n))
    rc = load_library().dg_fp8_gemm_nt_noalloc(
        _ptr(a), _ptr(sfa), sfa.shape[-1], _ptr(b), _ptr(sfb), _ptr(d), m, n, k,
        _stream(stream))
    _check(rc, "dg_fp8_gemm_nt_noalloc")
    return d


def dg_m_grouped_fp8_gemm_nt_contiguous(a, sfa, b, sfb, d, m_indices,
                                        stream=None) -> torch.Tensor:
    """Contiguous m-grouped GEMM: a [M_total, K], b [G, N, K], m_indices int32
    [M_total] (-1 = padding); padding rows of d are not written."""
    _need_cuda(a, sfa, b, sfb, d, m_indices)
    m_total, k = a.shape
    g, n, _ = b.shape
    _gemm_operands(a, sfa, b, sfb, m_total, n, k, groups=g)
    _expect(d, "d", torch.bfloat16, (m_total, n))
    _expect(m_indices, "m_indices", torch.int32, (m_total,))
    rc = load_library().dg_m_grouped_fp8_gemm_nt_contiguous(
        _ptr(a), _ptr(sfa), sfa.shape[-1], _ptr(b), _ptr(sfb), _ptr(d),
        _ptr(m_indices), m_total, n, k, g, _stream(stream))
    _check(rc, "dg_m_grouped_fp8_gemm_nt_contiguous")
    return d


def dg_m_grouped_fp8_gemm_nt_masked(a, sfa, b, sfb, d, masked_m,
                                    stream=None) -> torch.Tensor:
    """Masked m-grouped GEMM: a [G, M_max, K], sfa [G, K/128, ld], b [G, N, K],
    masked_m int32 [G] on the device; rows >= masked_m[g] of d untouched."""
    _need_cuda(a, sfa, b, sfb, d, masked_m)
    g, m_max, k = a.shape
    n = b.shape[1]
    _gemm_operands(a, sfa, b, sfb, m_max, n, k, groups=g, a_batch=g)
    _expect(d, "d", torch.bfloat16, (g, m_max, n))
    _expect(masked_m, "masked_m", torch.int32, (g,))
    rc = load_library().dg_m_grouped_fp8_gemm_nt_masked(
        _ptr(a), _ptr(sfa), sfa.shape[-1], _ptr(b), _ptr(sfb), _ptr(d),
        _ptr(masked_m), g, m_max, n, k, _stream(stream))
    _check(rc, "dg_m_grouped_fp8_gemm_nt_masked")
    return d


def dg_k_grouped_fp8_gemm_tn_contiguous(a, sfa, b, sfb, d, k_sizes, c=None,
                                        stream=None) -> torch.Tensor:
    """The k-grouped GEMM with both operands stored with the token axis K
    outermost: a [K, M], b [K, N] uint8 (M, N % 16 == 0), scales and the rest
    as in dg_k_grouped_fp8_gemm_nt_contiguous."""
    _need_cuda(a, sfa, b, sfb, d, k_sizes)
    if c is not None:
        _need_cuda(c)
    k, m = a.shape
    n = b.shape[1]
    g = k_sizes.numel()
    if k % 128 == 0:
        _expect(a, "a", torch.uint8, (k, m))
        _expect(sfa, "sfa", torch.float32, (k // 128, (m, "ld")))
        _expect(b, "b", torch.uint8, (k, n))
        _expect(sfb, "sfb", torch.float32, (k // 128, (n, "ld")))
    _expect(d, "d", torch.float32, (g, m, n))
    _expect(k_sizes, "k_sizes", torch.int32, (g,))
    if c is not None:
        _expect(c, "c", torch.float32, (g, m, n))
    rc = load_library().dg_k_grouped_fp8_gemm_tn_contiguous(
        _ptr(a), _ptr(sfa), sfa.shape[-1], _ptr(b), _ptr(sfb), sfb.shape[-1], _ptr(c),
        _ptr(d), _ptr(k_sizes), g, m, n, k, _stream(stream))
    _check(rc, "dg_k_grouped_fp8_gemm_tn_contiguous")
    return d


def dg_k_grouped_fp8_gemm_nt_contiguous(a, sfa, b, sfb, d, k_sizes, c=None,
                                        stream=None) -> torch.Tensor:
    """K-grouped GEMM (MoE weight gradient): a [M, K] and b [N, K] uint8 with
    1x128 scales sfa [K/128, ld_a] and sfb [K/128, ld_b] (both from
    dg_quantize_1x128), k_sizes int32 [G] on the device (multiples of 128
    summing to K), d float32 [G, M, N]; d[g] = c[g] + a_g b_g^T over group
    g's K segment (c float32 [G, M, N] or None).  d is returned."""
    _need_cuda(a, sfa, b, sfb, d, k_sizes)
    if c is not None:
        _need_cuda(c)
    m, k = a.shape
    n = b.shape[0]
    g = k_sizes.numel()
    if k % 128 == 0:  # (otherwise the C ABI rejects the call)
        _expect(a, "a", torch.uint8, (m, k))
        _expect(sfa, "sfa", torch.float32, (k // 128, (m, "ld")))
        _expect(b, "b", torch.uint8, (n, k))
        _expect(sfb, "sfb", torch.float32, (k // 128, (n, "ld")))
    _expect(d, "d", torch.float32, (g, m, n))
    _expect(k_sizes, "k_sizes", torch.int32, (g,))
    if c is not None:
        _expect(c, "c", torch.float32, (g, m, n))
    rc = load_library().dg_k_grouped_fp8_gemm_nt_contiguous(
        _ptr(a), _ptr(sfa), sfa.shape[-1], _ptr(b), _ptr(sfb), sfb.shape[-1], _ptr(c),
        _ptr(d), _ptr(k_sizes), g, m, n, k, _stream(stream))
    _check(rc, "dg_k_grouped_fp8_gemm_nt_contiguous")
    return d


def _ue8m0_scales(sfa, sfb, m, n, k, lead=()):
    """Checks packed UE8M0 scale words: sfa [.., ceil(K/512), ld >= m],
    sfb [.., ceil(K/512), ld >= n], int32."""
    if k % 128:
        return
    words = -(-(k // 128) // 4)
    _expect(sfa, "sfa", torch.int32, lead + (words, (m, "ld")))
    _expect(sfb, "sfb", torch.int32, lead + (words, (n, "ld")))


def dg_fp8_gemm_nt_ue8m0(a, sfa, b, sfb, d, stream=None) -> torch.Tensor:
    """D = A * B^T with power-of-two scales as packed UE8M0 words applied by
    the tensor cores: a [M, K] and b [N, K] uint8, sfa int32 [ceil(K/512),
    ld_a] (dg_pack_ue8m0 of the 1x128 scales), sfb int32 [ceil(K/512), ld_b]
    per row of B (dg_pack_ue8m0_128x128 of the 128x128 block scales); d a
    preallocated bfloat16 [M, N] tensor, returned."""
    _need_cuda(a, sfa, b, sfb, d)
    m, k = a.shape
    n = b.shape[0]
    if k % 128 == 0:
        _expect(a, "a", torch.uint8, (m, k))
        _expect(b, "b", torch.uint8, (n, k))
    _ue8m0_scales(sfa, sfb, m, n, k)
    _expect(d, "d", torch.bfloat16, (m, n))
    rc = load_library().dg_fp8_gemm_nt_ue8m0(
        _ptr(a), _ptr(sfa), sfa.shape[-1], _ptr(b), _ptr(sfb), sfb.shape[-1], _ptr(d), m, n, k,
        _stream(stream))
    _check(rc, "dg_fp8_gemm_nt_ue8m0")
    return d


def dg_m_grouped_fp8_gemm_nt_masked_ue8m0(a, sfa, b, sfb, d, masked_m,
                                          stream=None) -> torch.Tensor:
    """The masked m-grouped GEMM with packed UE8M0 scales: a [G, M_max, K],
    sfa int32 [G, ceil(K/512), ld_a], b [G, N, K], sfb int32 [G, ceil(K/512),
    ld_b] per row of B, masked_m int32 [G] on the device; rows >= masked_m[g]
    of d are untouched."""
    _need_cuda(a, sfa, b, sfb, d, masked_m)
    g, m_max, k = a.shape
    n = b.shape[1]
    if k % 128 == 0:
        _expect(a, "a", torch.uint8, (g, m_max, k))
        _expect(b, "b", torch.uint8, (g, n, k))
    _ue8m0_scales(sfa, sfb, m_max, n, k, lead=(g,))
    _expect(d, "d", torch.bfloat16, (g, m_max, n))
    _expect(masked_m, "masked_m", torch.int32, (g,))
    rc = load_library().dg_m_grouped_fp8_gemm_nt_masked_ue8m0(
        _ptr(a), _ptr(sfa), sfa.shape[-1], _ptr(b), _ptr(sfb), sfb.shape[-1], _ptr(d),
        _ptr(masked_m), g, m_max, n, k, _stream(stream))
    _check(rc, "dg_m_grouped_fp8_gemm_nt_masked_ue8m0")
    return d


# ------------------------------------------------------------------ MXFP4, routing
_DTYPES = {torch.float32: DG_DTYPE_F32, torch.bfloat16: DG_DTYPE_BF16}
_U8, _I32, _F32, _BF16 = torch.uint8, torch.int32, torch.float32, torch.bfloat16


def _on_device(name, fn_args, ts, stream):
    """Calls entry point `name` with fn_args and the stream, on the device that
    the tensors ts share: their own current stream if none is given, whatever
    device is current.  (The raw-stream and current-device
    lookups are the ones under torch.cuda's, without their argument handling,
    which took a third of a small call.)"""
    dev = ts[0].get_device()  # (-1: on the host)
    if dev < 0:
        raise ValueError("all tensors must be CUDA tensors (there is no CPU path)")
    for t in ts:
        if t.get_device() != dev:
            raise ValueError(f"tensors on cuda:{dev} and {t.device}: all must be CUDA tensors on "
                             f"one device")
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
    else:
        raw = stream.cuda_stream
    fn = getattr(_lib or load_library(), name)
    if torch._C._cuda_getDevice() == dev:
        rc = fn(*fn_args, raw)
    else:
        with torch.cuda.device(dev):
            rc = fn(*fn_args, raw)
    if rc != DG_OK:
        raise DGError(rc, name)
    if stream is not None:
        # the caller may drop a tensor while the stream still uses it
        for t in ts:
            t.record_stream(stream)


def _exact(t, name, dtype, shape):
    """_expect for a contiguous tensor of exactly this shape, quick where it holds."""
    if t is None or t.dtype is not dtype or t.shape != shape:
        _expect(t, name, dtype, shape)
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")


def _empty(like, shape, dtype, stream):
    """An uninitialised tensor on like's device for a call on `stream`: it comes
    from that stream's memory pool, so that nothing still running on the current
    stream holds it, and is marked as used on the current stream, where the
    caller gets it."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        t = like.new_empty(shape, dtype=dtype)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _contiguous(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def _rows_2d(x, name):
    """The row stride of a matrix whose rows are contiguous."""
    if x.shape[1] > 1 and x.stride(1) != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    ld = x.stride(0) if x.shape[0] > 1 else x.shape[1]
    if ld < x.shape[1]:
        raise ValueError(f"{name}: rows overlap (row stride {ld} of {x.shape[1]} elements)")
    return ld


def _mx_scales(rows, k):
    """The shape of an operand's MXFP4 scale words."""
    return ((rows + 127) // 128, (k + 127) // 128, 32, 4)


def dg_quantize_mxfp4(x: torch.Tensor, transpose: bool = False, q=None, sf=None, stream=None):
    """MXFP4 quantization (one UE8M0 scale per 32 K elements) of x [M, K] or
    [B, M, K] (float32 or bfloat16), or, with ``transpose``, of the transpose of
    x [K, M].  A 2-D x may have a row stride: with ``transpose`` any, else one of a
    multiple of 16 bytes (and a base on 16 bytes), or DG_ERR_ALIGNMENT is raised.

    Returns (q uint8 [.., M, K/2], sf int32 [.., ceil(M/128), ceil(K/128), 32, 4]),
    the layouts of include/dg.h."""
    if x.dtype not in _DTYPES:
        raise ValueError("x must be float32 or bfloat16")
    if x.dim() not in (2, 3) or (transpose and x.dim() == 3):
        raise ValueError(f"x must be a matrix (or a batch of them, not transposed), got shape "
                         f"{tuple(x.shape)}")
    if x.dim() == 3:
        _contiguous(x)
        lead, (m, k), ld = (x.shape[0],), x.shape[1:], x.shape[2]
    else:
        lead, ld = (), _rows_2d(x, "x")
        m, k = (x.shape[1], x.shape[0]) if transpose else x.shape
    if k <= 0 or k % 32:
        raise ValueError(f"K = {k} must be a positive multiple of 32")
    if lead == (0,):
        raise ValueError("an empty batch")
    if q is None:
        q = _empty(x, lead + (m, k // 2), _U8, stream)
    else:
        _exact(q, "q", _U8, lead + (m, k // 2))
    if sf is None:
        sf = _empty(x, lead + _mx_scales(m, k), _I32, stream)
    else:
        _exact(sf, "sf", _I32, lead + _mx_scales(m, k))
    _on_device("dg_quantize_mxfp4",
               (x.data_ptr(), _DTYPES[x.dtype], lead[0] if lead else 1, m, k, ld, int(transpose),
                q.data_ptr(), sf.data_ptr()), (x, q, sf), stream)
    return q, sf


def dg_dequantize_mxfp4(q: torch.Tensor, sf: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                        out=None, stream=None) -> torch.Tensor:
    """The values of an MXFP4 operand (q [.., M, K/2], sf as dg_quantize_mxfp4
    returns them) in bfloat16 or float32, both exact: [.., M, K]."""
    if out is not None:
        dtype = out.dtype
    if dtype not in _DTYPES:
        raise ValueError("dtype must be float32 or bfloat16")
    if q.dim() not in (2, 3):
        raise ValueError(f"q must be [M, K/2] or [B, M, K/2], got shape {tuple(q.shape)}")
    lead, (m, kh) = tuple(q.shape[:-2]), q.shape[-2:]
    k = 2 * kh
    if k <= 0 or k % 32:
        raise ValueError(f"K = {k} must be a positive multiple of 32")
    if lead == (0,):
        raise ValueError("an empty batch")
    _exact(q, "q", _U8, lead + (m, kh))
    _exact(sf, "sf", _I32, lead + _mx_scales(m, k))
    if out is None:
        out = _empty(q, lead + (m, k), dtype, stream)
    else:
        _exact(out, "out", dtype, lead + (m, k))
    _on_device("dg_dequantize_mxfp4",
               (q.data_ptr(), sf.data_ptr(), lead[0] if lead else 1, m, k, out.data_ptr(),
                _DTYPES[dtype], k), (q, sf, out), stream)
    return out


def _mx_operands(a, sfa, b, sfb, d, m, n, k, lead_a, lead_b):
    """Checks the operands, scales and result of a product; the one expression
    first, since its parts are half of a small call's time one by one."""
    sa, sb = lead_a + _mx_scales(m, k), lead_b + _mx_scales(n, k)
    if (a.dtype is _U8 and b.dtype is _U8 and sfa.dtype is _I32 and sfb.dtype is _I32
            and d.dtype is _BF16 and b.shape == lead_b + (n, k // 2) and sfa.shape == sa
            and sfb.shape == sb and d.shape == lead_a + (m, n)
            and a.shape == lead_a + (m, k // 2) and a.is_contiguous() and b.is_contiguous()
            and sfa.is_contiguous() and sfb.is_contiguous() and d.is_contiguous()):
        return
    _exact(a, "a", _U8, lead_a + (m, k // 2))
    _exact(sfa, "sfa", _I32, sa)
    _exact(b, "b", _U8, lead_b + (n, k // 2))
    _exact(sfb, "sfb", _I32, sb)
    _exact(d, "d", _BF16, lead_a + (m, n))


def dg_mxfp4_gemm_nt(a, sfa, b, sfb, d, stream=None) -> torch.Tensor:
    """D = A * B^T of two MXFP4 operands: a [M, K/2] and b [N, K/2] uint8 with
    their scale words (dg_quantize_mxfp4), N % 8 == 0; d a preallocated bfloat16
    [M, N] tensor, returned."""
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError("a and b must be [M, K/2] and [N, K/2]")
    m, k, n = a.shape[0], 2 * a.shape[1], b.shape[0]
    _mx_operands(a, sfa, b, sfb, d, m, n, k, (), ())
    _on_device("dg_mxfp4_gemm_nt",
               (a.data_ptr(), sfa.data_ptr(), b.data_ptr(), sfb.data_ptr(), d.data_ptr(), m, n, k),
               (a, sfa, b, sfb, d), stream)
    return d


def dg_m_grouped_mxfp4_gemm_nt_contiguous(a, sfa, b, sfb, d, m_indices,
                                          stream=None) -> torch.Tensor:
    """Contiguous m-grouped product of MXFP4 operands: a [M_total, K/2], b [G, N,
    K/2], m_indices int32 [M_total] (-1 = padding); padding rows of d are not
    written."""
    if a.dim() != 2 or b.dim() != 3:
        raise ValueError("a and b must be [M_total, K/2] and [G, N, K/2]")
    m, k = a.shape[0], 2 * a.shape[1]
    g, n = b.shape[:2]
    _mx_operands(a, sfa, b, sfb, d, m, n, k, (), (g,))
    _exact(m_indices, "m_indices", _I32, (m,))
    _on_device("dg_m_grouped_mxfp4_gemm_nt_contiguous",
               (a.data_ptr(), sfa.data_ptr(), b.data_ptr(), sfb.data_ptr(), d.data_ptr(),
                m_indices.data_ptr(), m, n, k, g), (a, sfa, b, sfb, d, m_indices), stream)
    return d


def dg_m_grouped_mxfp4_gemm_nt_masked(a, sfa, b, sfb, d, masked_m, stream=None) -> torch.Tensor:
    """Masked m-grouped product of MXFP4 operands: a [G, M_max, K/2], b [G, N,
    K/2], masked_m int32 [G] on the device (dg_moe_route's counts); rows >=
    masked_m[g] of d are not written."""
    if a.dim() != 3 or b.dim() != 3:
        raise ValueError("a and b must be [G, M_max, K/2] and [G, N, K/2]")
    g, m, k = a.shape[0], a.shape[1], 2 * a.shape[2]
    n = b.shape[1]
    _mx_operands(a, sfa, b, sfb, d, m, n, k, (g,), (g,))
    _exact(masked_m, "masked_m", _I32, (g,))
    _on_device("dg_m_grouped_mxfp4_gemm_nt_masked",
               (a.data_ptr(), sfa.data_ptr(), b.data_ptr(), sfb.data_ptr(), d.data_ptr(),
                masked_m.data_ptr(), g, m, n, k), (a, sfa, b, sfb, d, masked_m), stream)
    return d


def dg_moe_route_workspace_size(t: int, e: int) -> int:
    return load_library().dg_moe_route_workspace_size(t, e)


def _route_logits(logits):
    if logits.dtype not in _DTYPES:
        raise ValueError("logits must be float32 or bfloat16")
    if logits.dim() != 2:
        raise ValueError(f"logits must be [T, E], got shape {tuple(logits.shape)}")
    return logits.shape[0], logits.shape[1], _rows_2d(logits, "logits")


def dg_moe_route(logits: torch.Tensor, top_k: int, normalize: bool = True, token_mask=None,
                 stream=None):
    """Softmax top-k routing of logits [T, E] (float32 or bfloat16, any row
    stride) with the per-expert counts and the balance loss (include/dg.h).
    token_mask: bool or uint8 [T], False for tokens that do not route.

    Returns (idx int32 [T, top_k], weights float32 [T, top_k], counts int32 [E],
    loss float32 [1], num_tokens int32 [1]); -1 / 0 where a token has no choice.
    The five are views of one allocation: each keeps all of it alive (copy a loss that
    is kept for a log).  They carry no autograd graph; the gradient is
    dg_moe_route_backward's."""
    t, e, ld = _route_logits(logits)
    dev = logits.device
    if token_mask is not None:
        if token_mask.dtype not in (torch.bool, torch.uint8):
            raise ValueError("token_mask must be bool or uint8")
        _exact(token_mask, "token_mask", token_mask.dtype, (t,))
    if not 1 <= top_k <= min(e, 32):
        raise ValueError(f"top_k = {top_k} must be in 1 .. min(E, 32), E = {e}")
    if not logits.is_cuda:
        raise ValueError("all tensors must be CUDA tensors (there is no CPU path)")
    # one allocation for the five results (five took half of a small call's time)
    n = t * top_k
    buf = _empty(logits, (2 * n + e + 2,), _I32, stream)
    real = buf.view(_F32)
    idx = buf.as_strided((t, top_k), (top_k, 1), 0)
    weights = real.as_strided((t, top_k), (top_k, 1), n)
    counts = buf.as_strided((e,), (1,), 2 * n)
    num_tokens = buf.as_strided((1,), (1,), 2 * n + e)
    loss = real.as_strided((1,), (1,), 2 * n + e + 1)
    if torch._C._cuda_getDevice() == dev.index:
        nbytes = dg_moe_route_workspace_size(t, e)
    else:
        with torch.cuda.device(dev):
            nbytes = dg_moe_route_workspace_size(t, e)
    ws = _empty(logits, (nbytes,), _U8, stream) if nbytes else None
    at = buf.data_ptr()
    _on_device("dg_moe_route",
               (logits.data_ptr(), _DTYPES[logits.dtype], t, e, ld, top_k, 1 if normalize else 0,
                _ptr(token_mask), at, at + 4 * n, at + 8 * n, at + 4 * (2 * n + e + 1),
                at + 4 * (2 * n + e), _ptr(ws), nbytes),
               (logits,) if token_mask is None else (logits, token_mask), stream)
    return idx, weights, counts, loss, num_tokens


def dg_moe_route_backward(logits, idx, weights, counts, num_tokens, dweights=None, dloss=None,
                          normalize: bool = True, stream=None) -> torch.Tensor:
    """The gradient of dg_moe_route's logits, in their type: from dweights
    (float32 [T, top_k]) and dloss (float32, one element), either None for zero;
    idx, weights, counts and num_tokens as dg_moe_route returned them."""
    t, e, ld = _route_logits(logits)
    if idx.dim() != 2:
        raise ValueError(f"idx must be [T, top_k], got shape {tuple(idx.shape)}")
    k = idx.shape[1]
    ts = [logits, idx, weights, counts, num_tokens]
    _exact(idx, "idx", _I32, (t, k))
    _exact(weights, "weights", _F32, (t, k))
    _exact(counts, "counts", _I32, (e,))
    _exact(num_tokens, "num_tokens", _I32, (1,))
    if dweights is not None:
        _exact(dweights, "dweights", _F32, (t, k))
        ts.append(dweights)
    if dloss is not None:
        if dloss.numel() != 1:
            raise ValueError("dloss must have one element")
        _exact(dloss, "dloss", _F32, dloss.shape)
        ts.append(dloss)
    dlogits = _empty(logits, (t, e), logits.dtype, stream)
    _on_device("dg_moe_route_backward",
               (logits.data_ptr(), _DTYPES[logits.dtype], t, e, ld, k, 1 if normalize else 0,
                idx.data_ptr(), weights.data_ptr(), counts.data_ptr(), num_tokens.data_ptr(),
                _ptr(dweights), _ptr(dloss), dlogits.data_ptr()), ts, stream)
    return dlogits
