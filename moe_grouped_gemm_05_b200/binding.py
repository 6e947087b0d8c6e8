"""Thin ctypes binding of libdg.so (argument marshalling only).

Every step of the GEMM runs in the library's CUDA kernels; this module checks
tensor dtypes/shapes, passes raw device pointers and the current CUDA stream,
and turns negative status codes into exceptions.  Tensors come from PyTorch
(device memory and streams only).  If the library is missing the first call
raises: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdg.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "dg.h")

DG_OK = 0
DG_ERR_NULL = -1
DG_ERR_SHAPE = -2
DG_ERR_ALIGN = -3
DG_ERR_UNSUPPORTED = -4
DG_ERR_CUDA = -5

DG_DEVERR_BAD_SCALE = 0x1
DG_DEVERR_BAD_EXPERT = 0x2
DG_DEVERR_BAD_MASKED_M = 0x4
DG_DEVERR_MIXED_TILE = 0x8
DG_DEVERR_TIMEOUT = 0x10
DG_DEVERR_BAD_LOGIT = 0x20

_SCORES = {"softmax": 0, "sigmoid": 1}

_lib = None


class DGError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"dg status {code}: {msg}")
        self.code = code


def load() -> ctypes.CDLL:
    """Loads libdg.so once (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m moe_grouped_gemm_05_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32p, i = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int
    lib.dg_fp8_gemm_nt.argtypes = [vp, i32p, vp, i32p, vp, i, i, i, vp]
    lib.dg_fp8_gemm_nt_fp32sfa.argtypes = [vp, vp, vp, i32p, vp, i, i, i, vp]
    lib.dg_m_grouped_fp8_gemm_nt_contiguous_fp32sfa.argtypes = [vp, vp, vp, i32p, vp, i32p, i, i, i, i, vp]
    lib.dg_m_grouped_fp8_gemm_nt_masked_fp32sfa.argtypes = [vp, vp, vp, i32p, vp, i32p, i, i, i, i, vp]
    for name in ("dg_fp8_gemm_nn", "dg_fp8_gemm_tn", "dg_fp8_gemm_tt"):
        getattr(lib, name).argtypes = [vp, i32p, vp, i32p, vp, i, i, i, vp]
    lib.dg_m_grouped_fp8_gemm_nt_contiguous.argtypes = [vp, i32p, vp, i32p, vp, i32p, i, i, i, i, vp]
    lib.dg_m_grouped_fp8_gemm_nt_masked.argtypes = [vp, i32p, vp, i32p, vp, i32p, i, i, i, i, vp]
    lib.dg_pack_sf_ue8m0.argtypes = [vp, i32p, i, i, i, vp]
    lib.dg_quantize_fp8_1x128.argtypes = [vp, i, vp, i32p, i, i, i, vp]
    lib.dg_fp8_gemm_nt_ex.argtypes = [vp, i32p, vp, i32p, vp, vp, i, i, i, i, i, vp]
    lib.dg_moe_permute_capacity.argtypes = [i, i, i]
    lib.dg_moe_permute.argtypes = [i32p, i, i, i, vp, i32p, i, vp, i32p, i32p, i32p, i32p, i, vp]
    lib.dg_moe_unpermute_combine.argtypes = [vp, i32p, vp, i, i, i, vp, vp]
    f = ctypes.c_float
    lib.dg_moe_gate.argtypes = [vp, i, vp, i, i, i, i, i, i, i, i, f, vp, vp, vp]
    lib.dg_moe_gate_backward.argtypes = [vp, i, vp, vp, i, i, i, i, i, f, vp, vp]
    lib.dg_int8_gemm_nt.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, vp]
    lib.dg_m_grouped_int8_gemm_nt_contiguous.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, vp]
    lib.dg_m_grouped_int8_gemm_nt_masked.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, vp]
    lib.dg_quantize_int8_per_token.argtypes = [vp, i, vp, vp, i, i, vp]
    lib.dg_moe_quantize_permute_int8.argtypes = [vp, i, i, i, vp, i, i, vp, vp, vp, vp, vp, i, vp]
    lib.dg_packed_sf_words.argtypes = [i, i]
    lib.dg_packed_sf_words.restype = ctypes.c_int64
    lib.dg_get_mk_alignment_for_contiguous_layout.argtypes = []
    lib.dg_get_device_error.argtypes = [vp, ctypes.POINTER(ctypes.c_int)]
    lib.dg_set_num_sms.argtypes = [i]
    lib.dg_set_pdl.argtypes = [i]
    lib.dg_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    lib.dg_set_wait_limit_ns.restype = ctypes.c_uint64
    lib.dg_set_tc_util.argtypes = [i]
    lib.dg_get_num_sms.argtypes = []
    lib.dg_set_config.argtypes = [i, i, i]
    lib.dg_describe_config.argtypes = [i, i, i, i, i, ctypes.c_char_p, i]
    lib.dg_get_last_error.restype = ctypes.c_char_p
    for name in ("dg_fp8_gemm_nt", "dg_m_grouped_fp8_gemm_nt_contiguous", "dg_m_grouped_fp8_gemm_nt_masked",
                 "dg_pack_sf_ue8m0", "dg_get_device_error", "dg_set_config", "dg_describe_config",
                 "dg_quantize_fp8_1x128", "dg_fp8_gemm_nt_ex", "dg_moe_permute_capacity", "dg_moe_permute",
                 "dg_moe_unpermute_combine", "dg_moe_gate", "dg_moe_gate_backward", "dg_int8_gemm_nt",
                 "dg_m_grouped_int8_gemm_nt_contiguous", "dg_m_grouped_int8_gemm_nt_masked",
                 "dg_quantize_int8_per_token", "dg_moe_quantize_permute_int8"):
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def header_functions() -> list[str]:
    """Names of the functions declared in include/dg.h."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(dg_\w+)\s*\(", text)))


def _check(code: int):
    if code != 0:
        raise DGError(code, load().dg_get_last_error().decode())


def _stream() -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t: torch.Tensor) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr())


def _fp8(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise TypeError(f"{name} must be float8_e4m3fn (or its uint8 bytes), got {t.dtype}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    return t


def _i32(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 CUDA tensor")
    return t


def packed_sf_words(mn: int, kb: int) -> tuple[int, int]:
    """(rows, cols) of a packed scale matrix: (ceil(kb/4), align4(mn))."""
    return (kb + 3) // 4, (mn + 3) // 4 * 4


def _packed_numel(t, batch: int, mn: int, kb: int, name: str):
    """Packed scale words may come as [kp, mn4] or [batch, kp, mn4]: what the
    kernels read is batch * kp * mn4 words, so the element count must match."""
    kp, mn4 = packed_sf_words(mn, kb)
    if t.numel() != batch * kp * mn4:
        raise ValueError(f"{name} holds {t.numel()} words; expected {batch} x {kp} x {mn4} "
                         f"(batch x ceil(Kb/4) x align4(MN))")


_INT_MAX = 0x7FFFFFFF


def _c_ints(*sizes):
    """Refuses sizes that are no C ints: ctypes would take them modulo 2^32.

    Called where one of them is negative or beyond 31 bits, which the callers see by themselves in 0.1 us."""
    if max(sizes) > _INT_MAX or min(sizes) < -_INT_MAX - 1:
        raise ValueError(f"sizes {', '.join(str(n) for n in sizes)}: beyond 32 bits")


def _same_device(ref, *tensors):
    """All operands of a call live on one device (None entries are skipped)."""
    dev = ref.get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"operands on different devices: {ref.device} and {t.device}")


def _out(t, dtypes, shape, name: str, device):
    """Checks a caller-provided output tensor."""
    if t.dtype not in dtypes or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {'/'.join(str(d) for d in dtypes)} tensor of shape "
                         f"{tuple(shape)} on {device}")


def pack_sf_ue8m0(sf: torch.Tensor, out=None) -> torch.Tensor:
    """fp32 power-of-two scales [batch?, mn, kb] -> int32 [batch?, ceil(kb/4), align4(mn)] (into `out` if given)."""
    if sf.dtype != torch.float32 or not sf.is_cuda or not sf.is_contiguous():
        raise TypeError("sf must be a contiguous float32 CUDA tensor")
    squeeze = sf.dim() == 2
    s3 = sf.unsqueeze(0) if squeeze else sf
    if s3.dim() != 3:
        raise ValueError("sf must be [mn, kb] or [batch, mn, kb]")
    batch, mn, kb = s3.shape
    if (batch | mn | kb) >> 31:
        _c_ints(batch, mn, kb)
    kp, mn4 = packed_sf_words(mn, kb)
    if out is None:
        out = torch.empty((batch, kp, mn4), dtype=torch.int32, device=sf.device)
    elif (out.dtype != torch.int32 or not out.is_contiguous() or out.numel() != batch * kp * mn4
          or out.device != sf.device):
        raise ValueError("out must be a contiguous int32 tensor of the packed shape on sf's device")
    _check(load().dg_pack_sf_ue8m0(_ptr(s3), _ptr(out), batch, mn, kb, _stream()))
    if out.dim() == 3 and squeeze:
        return out[0]
    return out


def quantize_fp8_1x128(x: torch.Tensor, q=None, sf=None):
    """Per-token 1x128 FP8 quantisation of x[..., M, K] (bf16 or fp32).

    Returns (q float8_e4m3fn [..., M, K], sf int32 [..., ceil(K/512), align4(M)]),
    the `a` / `sfa` operands of the GEMM entry points.
    """
    if x.dtype not in (torch.bfloat16, torch.float32) or not x.is_cuda or not x.is_contiguous():
        raise TypeError("x must be a contiguous bf16 or fp32 CUDA tensor")
    if x.dim() < 2:
        raise ValueError("x must be [..., M, K]")
    *lead, M, K = x.shape
    batch = 1
    for n in lead:
        batch *= n
    if (batch | M | K) >> 31:
        _c_ints(batch, M, K)
    kp, mn4 = packed_sf_words(M, K // 128)
    if q is None:
        q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    if sf is None:
        sf = torch.empty((*lead, kp, mn4), dtype=torch.int32, device=x.device)
    _out(q, (torch.float8_e4m3fn, torch.uint8), x.shape, "q", x.device)
    _out(sf, (torch.int32,), (*lead, kp, mn4), "sf", x.device)
    _check(load().dg_quantize_fp8_1x128(_ptr(x), 0 if x.dtype == torch.bfloat16 else 1, _ptr(q), _ptr(sf), batch,
                                        M, K, _stream()))
    return q, sf


def _sfa_kind(sfa: torch.Tensor, rows_shape: tuple, K: int) -> bool:
    """True when sfa holds fp32 scales [..rows.., K/128] (packed in the kernel), False for packed int32 words."""
    if sfa.dtype == torch.float32:
        if not sfa.is_cuda or not sfa.is_contiguous() or tuple(sfa.shape) != (*rows_shape, K // 128):
            raise ValueError(f"fp32 sfa must be a contiguous CUDA tensor of shape {(*rows_shape, K // 128)}")
        return True
    _i32(sfa, "sfa")
    return False


def fp8_gemm_nt(a, sfa, b, sfb, d=None) -> torch.Tensor:
    """D[M,N] (bf16) = A[M,K] . B[N,K]^T with 1x128 / 128x128 UE8M0 scales.

    sfa: packed int32 words [ceil(Kb/4), align4(M)], or the fp32 power-of-two scales [M, Kb]
    (then the GEMM packs them itself: no separate packing launch).
    """
    _fp8(a, "a"), _fp8(b, "b"), _i32(sfb, "sfb")
    M, K = a.shape
    N, Kb_ = b.shape
    if (M | N | K) >> 31:
        _c_ints(M, N, K)
    if Kb_ != K:
        raise ValueError("a and b disagree on K")
    fp32_sfa = _sfa_kind(sfa, (M,), K)
    if (not fp32_sfa and tuple(sfa.shape) != packed_sf_words(M, K // 128)) or \
            tuple(sfb.shape) != packed_sf_words(-(-N // 128), K // 128):
        raise ValueError("packed scale shapes do not match [ceil(Kb/4), align4(MN)]")
    _same_device(a, sfa, b, sfb, d)
    if d is None:
        d = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    elif d.dtype != torch.bfloat16 or tuple(d.shape) != (M, N) or not d.is_contiguous():
        raise ValueError("d must be a contiguous bf16 [M, N] tensor")
    fn = load().dg_fp8_gemm_nt_fp32sfa if fp32_sfa else load().dg_fp8_gemm_nt
    _check(fn(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(d), M, N, K, _stream()))
    return d


def fp8_gemm(layout: str, a, sfa, b, sfb, d=None) -> torch.Tensor:
    """D[M,N] (bf16) = A . B^T with the operands stored in `layout` ("nt", "nn", "tn" or "tt").

    First letter LHS, second RHS, N = not transposed, T = transposed:
    a is A [M,K] for "n?" and A^T [K,M] for "t?"; b is B [N,K] for "?t" and B^T [K,N] for "?n".
    """
    if layout not in ("nt", "nn", "tn", "tt"):
        raise ValueError(f"unknown layout {layout!r}")
    _fp8(a, "a"), _fp8(b, "b"), _i32(sfa, "sfa"), _i32(sfb, "sfb")
    if not (a.is_contiguous() and b.is_contiguous()):
        raise ValueError("a and b must be contiguous")
    K, M = a.shape if layout[0] == "t" else a.shape[::-1]
    K2, N = b.shape if layout[1] == "n" else b.shape[::-1]
    if (M | N | K) >> 31:
        _c_ints(M, N, K)
    if K2 != K:
        raise ValueError("a and b disagree on K")
    if tuple(sfa.shape) != packed_sf_words(M, K // 128) or tuple(sfb.shape) != packed_sf_words(-(-N // 128), K // 128):
        raise ValueError("packed scale shapes do not match [ceil(Kb/4), align4(MN)]")
    _same_device(a, sfa, b, sfb, d)
    if d is None:
        d = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    elif d.dtype != torch.bfloat16 or tuple(d.shape) != (M, N) or not d.is_contiguous():
        raise ValueError("d must be a contiguous bf16 [M, N] tensor")
    fn = getattr(load(), f"dg_fp8_gemm_{layout}")
    _check(fn(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(d), M, N, K, _stream()))
    return d


def fp8_gemm_nt_ex(a, sfa, b, sfb, c=None, d=None, recipe_b: int = 128, out_dtype=torch.bfloat16) -> torch.Tensor:
    """D = A . B^T (+ C).  recipe_b: rows of B per scale (128 = 128x128 blocks, 1 = per-row "1D1D").

    out_dtype bf16 or float32; c (float32 [M, N]) requires a float32 output.
    """
    _fp8(a, "a"), _fp8(b, "b"), _i32(sfa, "sfa"), _i32(sfb, "sfb")
    M, K = a.shape
    N, Kb_ = b.shape
    if (M | N | K | recipe_b) >> 31:
        _c_ints(M, N, K, recipe_b)
    if Kb_ != K:
        raise ValueError("a and b disagree on K")
    if tuple(sfb.shape) != packed_sf_words(-(-N // recipe_b), K // 128) or tuple(sfa.shape) != packed_sf_words(M, K // 128):
        raise ValueError("packed scale shapes do not match the recipe")
    if c is not None and (c.dtype != torch.float32 or tuple(c.shape) != (M, N) or not c.is_contiguous()):
        raise ValueError("c must be a contiguous float32 [M, N] tensor")
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out_dtype must be bfloat16 or float32")
    _same_device(a, sfa, b, sfb, c, d)
    if d is None:
        d = torch.empty((M, N), dtype=out_dtype, device=a.device)
    else:
        _out(d, (torch.bfloat16, torch.float32), (M, N), "d", a.device)
    _check(load().dg_fp8_gemm_nt_ex(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(c) if c is not None else None,
                                    _ptr(d), M, N, K, recipe_b, 1 if d.dtype == torch.float32 else 0, _stream()))
    return d


def m_grouped_fp8_gemm_nt_contiguous(a, sfa, b, sfb, m_indices, d=None) -> torch.Tensor:
    """Contiguous-layout grouped GEMM: D[m] = A[m] . B[m_indices[m]]^T; -1 rows untouched.

    sfa: packed words or fp32 scales [M_total, Kb] (packed in the kernel)."""
    _fp8(a, "a"), _fp8(b, "b"), _i32(sfb, "sfb"), _i32(m_indices, "m_indices")
    M, K = a.shape
    G, N, Kb_ = b.shape
    if (M | N | K | G) >> 31:
        _c_ints(M, N, K, G)
    if Kb_ != K or m_indices.shape != (M,):
        raise ValueError("shape mismatch")
    fp32_sfa = _sfa_kind(sfa, (M,), K)
    if not fp32_sfa:
        _packed_numel(sfa, 1, M, K // 128, "sfa")
    _packed_numel(sfb, G, -(-N // 128), K // 128, "sfb")
    _same_device(a, sfa, b, sfb, m_indices, d)
    if d is None:
        d = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    elif d.dtype != torch.bfloat16 or tuple(d.shape) != (M, N) or not d.is_contiguous():
        raise ValueError("d must be a contiguous bf16 [M_total, N] tensor")
    fn = load().dg_m_grouped_fp8_gemm_nt_contiguous_fp32sfa if fp32_sfa else load().dg_m_grouped_fp8_gemm_nt_contiguous
    _check(fn(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(d), _ptr(m_indices), M, N, K, G, _stream()))
    return d


def m_grouped_fp8_gemm_nt_masked(a, sfa, b, sfb, masked_m, d=None) -> torch.Tensor:
    """Masked-layout grouped GEMM: rows m < masked_m[g] of expert g; other rows untouched.

    sfa: packed words or fp32 scales [G, M_max, Kb] (packed in the kernel)."""
    _fp8(a, "a"), _fp8(b, "b"), _i32(sfb, "sfb"), _i32(masked_m, "masked_m")
    G, M_max, K = a.shape
    Gb, N, Kb_ = b.shape
    if (G | M_max | N | K) >> 31:
        _c_ints(G, M_max, N, K)
    if Gb != G or Kb_ != K or masked_m.shape != (G,):
        raise ValueError("shape mismatch")
    fp32_sfa = _sfa_kind(sfa, (G, M_max), K)
    if not fp32_sfa:
        _packed_numel(sfa, G, M_max, K // 128, "sfa")
    _packed_numel(sfb, G, -(-N // 128), K // 128, "sfb")
    _same_device(a, sfa, b, sfb, masked_m, d)
    if d is None:
        d = torch.empty((G, M_max, N), dtype=torch.bfloat16, device=a.device)
    elif d.dtype != torch.bfloat16 or tuple(d.shape) != (G, M_max, N) or not d.is_contiguous():
        raise ValueError("d must be a contiguous bf16 [G, M_max, N] tensor")
    fn = load().dg_m_grouped_fp8_gemm_nt_masked_fp32sfa if fp32_sfa else load().dg_m_grouped_fp8_gemm_nt_masked
    _check(fn(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(d), _ptr(masked_m), G, M_max, N, K, _stream()))
    return d


def moe_permute(topk_ids: torch.Tensor, num_experts: int, q: torch.Tensor, sfa: torch.Tensor, out=None):
    """Contiguous-layout permutation of routed tokens.

    Returns a dict with a (float8 [M_cap, K]), sfa (int32 [kp, M_cap]), m_indices, src_of ([M_cap]) and
    row_of ([T, topk]); a / sfa / m_indices are the operands of m_grouped_fp8_gemm_nt_contiguous.
    `out`, if given, is such a dict of preallocated tensors (M_cap = dg_moe_permute_capacity).
    """
    _i32(topk_ids, "topk_ids"), _fp8(q, "q"), _i32(sfa, "sfa")
    T, topk = topk_ids.shape
    if q.dim() != 2 or q.shape[0] != T:
        raise ValueError(f"q must be [T, K] with T = {T} rows, one per token of topk_ids")
    K = q.shape[1]
    if (T | topk | num_experts | K) >> 31:
        _c_ints(T, topk, num_experts, K)
    _packed_numel(sfa, 1, T, K // 128, "sfa")
    _same_device(q, topk_ids, sfa)
    cap = load().dg_moe_permute_capacity(T, topk, num_experts)
    if cap < 0:
        _check(cap)
    kp = (K // 128 + 3) // 4
    dev = q.device
    if out is None:
        out = {
            "a": torch.empty((cap, K), dtype=torch.float8_e4m3fn, device=dev),
            "sfa": torch.empty((kp, cap), dtype=torch.int32, device=dev),
            "m_indices": torch.empty((cap,), dtype=torch.int32, device=dev),
            "src_of": torch.empty((cap,), dtype=torch.int32, device=dev),
            "row_of": torch.empty((T, topk), dtype=torch.int32, device=dev),
        }
    else:
        want = {"a": ((torch.float8_e4m3fn, torch.uint8), (cap, K)), "sfa": ((torch.int32,), (kp, cap)),
                "m_indices": ((torch.int32,), (cap,)), "src_of": ((torch.int32,), (cap,)),
                "row_of": ((torch.int32,), (T, topk))}
        for key, (dtypes, shape) in want.items():
            if key not in out:
                raise ValueError(f"out[{key!r}] is missing")
            _out(out[key], dtypes, shape, f"out[{key!r}]", dev)
    _check(load().dg_moe_permute(_ptr(topk_ids), T, topk, num_experts, _ptr(q), _ptr(sfa), K, _ptr(out["a"]),
                                 _ptr(out["sfa"]), _ptr(out["m_indices"]), _ptr(out["row_of"]), _ptr(out["src_of"]),
                                 cap, _stream()))
    return out


def moe_unpermute_combine(d_perm: torch.Tensor, row_of: torch.Tensor, weights=None, out=None) -> torch.Tensor:
    """out[t] = sum_s weights[t, s] * d_perm[row_of[t, s]] (bf16, FP32 sums)."""
    if d_perm.dtype != torch.bfloat16 or not d_perm.is_contiguous() or not d_perm.is_cuda or d_perm.dim() != 2:
        raise TypeError("d_perm must be a contiguous bf16 [rows, N] CUDA tensor")
    _i32(row_of, "row_of")
    T, topk = row_of.shape
    N = d_perm.shape[1]
    if (T | topk | N) >> 31:
        _c_ints(T, topk, N)
    if weights is not None:
        _out(weights, (torch.float32,), (T, topk), "weights", d_perm.device)
    _same_device(d_perm, row_of)
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=d_perm.device)
    else:
        _out(out, (torch.bfloat16,), (T, N), "out", d_perm.device)
    _check(load().dg_moe_unpermute_combine(_ptr(d_perm), _ptr(row_of), _ptr(weights) if weights is not None else None,
                                           T, topk, N, _ptr(out), _stream()))
    return out


# The current device and the current stream's handle, without the objects that torch.cuda wraps around them
# (1.6 us of an 8 us call).
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _launch_stream(dev: int) -> int:
    """The current stream of device `dev`, which must be the current device: the library launches there."""
    if dev != _current_device():
        raise ValueError(f"operands are on cuda:{dev} but the current device is cuda:{_current_device()}")
    return _current_stream(dev)


def _operand(t, dtypes, shape, name: str, dev: int) -> int:
    """Checks one operand (dtype, shape, contiguity, device number) and returns its address."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)} on cuda:{dev}, got shape "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


_FLOAT_CODES = {torch.bfloat16: 0, torch.float32: 1}
_INT8, _I32T, _F32T, _BF16T = (torch.int8,), (torch.int32,), (torch.float32,), (torch.bfloat16,)
_BF16_F32 = (torch.bfloat16, torch.float32)


def _cuda_matrix(t, dtypes, name: str, dims: int = 2):
    """Checks the leading operand of a call (dtype, rank, a contiguous CUDA tensor); returns its shape and device."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    shape, dev = t.shape, t.get_device()     # -1: the CPU
    if dev < 0 or len(shape) != dims or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor of {dims} dimensions")
    return shape, dev


def moe_gate(logits, topk: int, bias=None, *, score: str = "softmax", n_group: int = 1, topk_group: int = 1,
             group_top: int = 1, renormalize: bool = False, scale: float = 1.0, ids=None, weights=None):
    """Routes tokens to experts: (topk_ids int32 [T, topk], topk_weights float32 [T, topk]) from logits [T, E].

    score: "softmax" or "sigmoid"; bias (float32 [E]) is added to the scores for the choice only.  With
    n_group > 1 only the topk_group best groups stay, by their best expert (group_top=1) or the sum of their
    two best (2).  The weights are scale * score, with renormalize divided by the sum over the chosen ones.
    Experts with logit (or bias) -inf are never chosen; slots left over hold id -1 and weight 0.  The results
    are the topk_ids of the permutations and the weights of moe_unpermute_combine.
    """
    if score not in _SCORES:
        raise ValueError(f"unknown score {score!r}: softmax or sigmoid")
    (T, E), dev = _cuda_matrix(logits, _BF16_F32, "logits")
    if (T | E | topk | n_group | topk_group | group_top) >> 31:
        _c_ints(T, E, topk, n_group, topk_group, group_top)
    if ids is None:
        ids = torch.empty((T, max(0, topk)), dtype=torch.int32, device=logits.device)
    if weights is None:
        weights = torch.empty((T, max(0, topk)), dtype=torch.float32, device=logits.device)
    _check(load().dg_moe_gate(logits.data_ptr(), _FLOAT_CODES[logits.dtype],
                              _operand(bias, _F32T, (E,), "bias", dev) if bias is not None else None, T, E, topk,
                              _SCORES[score], n_group, topk_group, group_top, 1 if renormalize else 0, scale,
                              _operand(ids, _I32T, (T, topk), "ids", dev),
                              _operand(weights, _F32T, (T, topk), "weights", dev), _launch_stream(dev)))
    return ids, weights


def moe_gate_backward(logits, topk_ids, d_weights, *, score: str = "softmax", renormalize: bool = False,
                      scale: float = 1.0, d_logits=None) -> torch.Tensor:
    """Gradient of moe_gate's weights with respect to the logits, with the choice of experts (topk_ids) held.

    d_weights: float32 [T, topk]; score, renormalize and scale as in the forward call.  Returns d_logits in the
    logits' type: zero outside the chosen experts, except for softmax weights that are not renormalised.
    """
    if score not in _SCORES:
        raise ValueError(f"unknown score {score!r}: softmax or sigmoid")
    (T, E), dev = _cuda_matrix(logits, _BF16_F32, "logits")
    topk = topk_ids.shape[-1] if topk_ids.dim() else 0
    if (T | E | topk) >> 31:
        _c_ints(T, E, topk)
    if d_logits is None:
        d_logits = torch.empty_like(logits)
    _check(load().dg_moe_gate_backward(logits.data_ptr(), _FLOAT_CODES[logits.dtype],
                                       _operand(topk_ids, _I32T, (T, topk), "topk_ids", dev),
                                       _operand(d_weights, _F32T, (T, topk), "d_weights", dev), T, E, topk,
                                       _SCORES[score], 1 if renormalize else 0, scale,
                                       _operand(d_logits, (logits.dtype,), (T, E), "d_logits", dev),
                                       _launch_stream(dev)))
    return d_logits


def quantize_int8_per_token(x, q=None, scale=None):
    """Per-token int8 quantisation of x[..., K] (bf16 or fp32): (q int8 [..., K], scale float32 [...]).

    With x [M, K] (or [G, M_max, K]) these are the `a` / `sa` operands of the int8 products.
    """
    shape, dev = _cuda_matrix(x, _BF16_F32, "x", max(1, x.dim()))
    lead, K = shape[:-1], shape[-1]
    M = lead.numel()
    if (M | K) >> 31:
        _c_ints(M, K)
    if q is None:
        q = torch.empty(shape, dtype=torch.int8, device=x.device)
    if scale is None:
        scale = torch.empty(lead, dtype=torch.float32, device=x.device)
    qp, sp = _operand(q, _INT8, shape, "q", dev), _operand(scale, _F32T, lead, "scale", dev)
    _check(load().dg_quantize_int8_per_token(x.data_ptr(), _FLOAT_CODES[x.dtype], qp, sp, M, K,
                                             _launch_stream(dev)))
    return q, scale


def moe_quantize_permute_int8(topk_ids, num_experts: int, x, out=None):
    """Per-token int8 quantisation of routed tokens x [T, K], written into the contiguous expert layout.

    Returns a dict with a (int8 [M_cap, K]), sa (float32 [M_cap]), m_indices, src_of ([M_cap]) and row_of
    ([T, topk]); a / sa / m_indices are the operands of m_grouped_int8_gemm_nt_contiguous.  `out`, if given, is
    such a dict of preallocated tensors (M_cap = dg_moe_permute_capacity).
    """
    (T, K), dev = _cuda_matrix(x, _BF16_F32, "x")
    routed = topk_ids.shape
    if len(routed) != 2 or routed[0] != T:
        raise ValueError(f"topk_ids must be [T, topk] with T = {T} rows, one per token of x")
    topk = routed[1]
    if (T | K | topk | num_experts) >> 31:
        _c_ints(T, K, topk, num_experts)
    lib = load()
    cap = (T * topk + 127 * num_experts + 127) // 128 * 128    # dg_moe_permute_capacity
    if topk <= 0 or num_experts <= 0 or cap > _INT_MAX:
        _check(lib.dg_moe_permute_capacity(T, topk, num_experts))
    if out is None:
        out = {
            "a": torch.empty((cap, K), dtype=torch.int8, device=x.device),
            "sa": torch.empty((cap,), dtype=torch.float32, device=x.device),
            "m_indices": torch.empty((cap,), dtype=torch.int32, device=x.device),
            "src_of": torch.empty((cap,), dtype=torch.int32, device=x.device),
            "row_of": torch.empty((T, topk), dtype=torch.int32, device=x.device),
        }
    try:
        a, sa, m_indices, src_of, row_of = out["a"], out["sa"], out["m_indices"], out["src_of"], out["row_of"]
    except KeyError as key:
        raise ValueError(f"out[{key}] is missing") from None
    rows = (cap,)
    _check(lib.dg_moe_quantize_permute_int8(
        _operand(topk_ids, _I32T, routed, "topk_ids", dev), T, topk, num_experts, x.data_ptr(), _FLOAT_CODES[x.dtype], K,
        _operand(a, _INT8, (cap, K), "out['a']", dev), _operand(sa, _F32T, rows, "out['sa']", dev),
        _operand(m_indices, _I32T, rows, "out['m_indices']", dev),
        _operand(row_of, _I32T, routed, "out['row_of']", dev),
        _operand(src_of, _I32T, rows, "out['src_of']", dev), cap, _launch_stream(dev)))
    return out


def int8_gemm_nt(a, sa, b, sb, d=None, out_dtype=torch.bfloat16) -> torch.Tensor:
    """D[M,N] = sa[m] * sb[n] * (A[M,K] . B[N,K]^T), int8 operands, exact int32 sums.

    sa: float32 [M], one scale per token; sb: float32 [N], one per output channel.  D is bf16, or float32 with
    out_dtype=torch.float32 (or a float32 d).
    """
    (M, K), dev = _cuda_matrix(a, _INT8, "a")
    N = b.shape[0]
    if (M | N | K) >> 31:
        _c_ints(M, N, K)
    if d is None:
        if out_dtype not in _BF16_F32:
            raise ValueError("out_dtype must be bfloat16 or float32")
        d = torch.empty((M, N), dtype=out_dtype, device=a.device)
    _check(load().dg_int8_gemm_nt(a.data_ptr(), _operand(sa, _F32T, (M,), "sa", dev),
                                  _operand(b, _INT8, (N, K), "b", dev), _operand(sb, _F32T, (N,), "sb", dev),
                                  _operand(d, _BF16_F32, (M, N), "d", dev), M, N, K,
                                  1 if d.dtype == torch.float32 else 0, _launch_stream(dev)))
    return d


def m_grouped_int8_gemm_nt_contiguous(a, sa, b, sb, m_indices, d=None) -> torch.Tensor:
    """Contiguous-layout grouped int8 GEMM: D[m] = sa[m] * sb[g] * (A[m] . B[g]^T), g = m_indices[m]; -1 rows
    untouched.  a int8 [M_total, K], sa float32 [M_total], b int8 [G, N, K], sb float32 [G, N], D bf16."""
    (M, K), dev = _cuda_matrix(a, _INT8, "a")
    (G, N, _), _ = _cuda_matrix(b, _INT8, "b", 3)
    if (M | N | K | G) >> 31:
        _c_ints(M, N, K, G)
    if d is None:
        d = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    _check(load().dg_m_grouped_int8_gemm_nt_contiguous(
        a.data_ptr(), _operand(sa, _F32T, (M,), "sa", dev), _operand(b, _INT8, (G, N, K), "b", dev),
        _operand(sb, _F32T, (G, N), "sb", dev), _operand(d, _BF16T, (M, N), "d", dev),
        _operand(m_indices, _I32T, (M,), "m_indices", dev), M, N, K, G, _launch_stream(dev)))
    return d


def m_grouped_int8_gemm_nt_masked(a, sa, b, sb, masked_m, d=None) -> torch.Tensor:
    """Masked-layout grouped int8 GEMM: rows m < masked_m[g] of expert g; other rows untouched.

    a int8 [G, M_max, K], sa float32 [G, M_max], b int8 [G, N, K], sb float32 [G, N], D bf16 [G, M_max, N]."""
    (G, M_max, K), dev = _cuda_matrix(a, _INT8, "a", 3)
    (_, N, _), _ = _cuda_matrix(b, _INT8, "b", 3)
    if (G | M_max | N | K) >> 31:
        _c_ints(G, M_max, N, K)
    if d is None:
        d = torch.empty((G, M_max, N), dtype=torch.bfloat16, device=a.device)
    _check(load().dg_m_grouped_int8_gemm_nt_masked(
        a.data_ptr(), _operand(sa, _F32T, (G, M_max), "sa", dev), _operand(b, _INT8, (G, N, K), "b", dev),
        _operand(sb, _F32T, (G, N), "sb", dev), _operand(d, _BF16T, (G, M_max, N), "d", dev),
        _operand(masked_m, _I32T, (G,), "masked_m", dev), G, M_max, N, K, _launch_stream(dev)))
    return d


def get_device_error() -> int:
    """Returns and clears the device error word (atomically, after the current stream's work)."""
    v = ctypes.c_int(0)
    _check(load().dg_get_device_error(_stream(), ctypes.byref(v)))
    return v.value


def set_wait_limit_ns(ns: int) -> int:
    """Sets the time limit of each pipeline wait in the GEMM kernels; returns the previous one."""
    if ns < 0:
        raise ValueError("the wait limit is a non-negative number of nanoseconds")
    return int(load().dg_set_wait_limit_ns(ns))


def set_num_sms(n: int) -> int:
    _c_ints(n)
    return load().dg_set_num_sms(n)


def set_tc_util(percent: int) -> int:
    """Caps the share of the GPU's SMs (tensor cores) a call may occupy; returns the previous percent."""
    _c_ints(percent)
    prev = load().dg_set_tc_util(percent)
    if prev < 0:
        _check(prev)
    return prev


def set_pdl(enable: bool) -> bool:
    """Programmatic dependent launch on/off for the library's kernels; returns the previous setting."""
    return bool(load().dg_set_pdl(1 if enable else 0))


def set_config(block_n: int, ctas: int = 0, pipes: int = 0) -> None:
    """Forces the N tile width, 1- or 2-CTA tiles and 1 or 2 pipelines per CTA (block_n=0: heuristic)."""
    if (block_n | ctas | pipes) >> 31:
        _c_ints(block_n, ctas, pipes)
    _check(load().dg_set_config(block_n, ctas, pipes))


def describe_config(kind: str, M: int, N: int, K: int, num_groups: int = 1) -> str:
    buf = ctypes.create_string_buffer(64)
    k = {"dense": 0, "contiguous": 1, "masked": 2, "int8_dense": 3, "int8_contiguous": 4, "int8_masked": 5}[kind]
    if (M | N | K | num_groups) >> 31:
        _c_ints(M, N, K, num_groups)
    _check(load().dg_describe_config(k, M, N, K, num_groups, buf, 64))
    return buf.value.decode()


def get_mk_alignment_for_contiguous_layout() -> int:
    return load().dg_get_mk_alignment_for_contiguous_layout()
