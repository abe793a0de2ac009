"""Python binding of libfluxbin.so, the B200 LUT binary GEMV (C ABI in
include/fluxbin.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of the library.  PyTorch supplies device memory and the current
stream.  If the compiled library is missing, importing the binding's
functions raises; there is no CPU fallback.

Names follow the C ABI: fb_pack, fb_pack_bits, fb_unpack, fb_vcm_gather,
fb_lut_build, fb_validate_weights, fb_gemv_workspace_bytes, fb_gemv,
fb_gemv_batched, fb_qk_norm_rope, fb_attn_prompt, fb_attn_tree; ``Weights``
wraps one fb_weights struct and the tensors it points to.
"""

from __future__ import annotations

import ctypes as C
import os
import struct
from typing import Optional, Tuple

import torch

__all__ = [
    "FbError", "Weights", "lib", "library_path", "FB_GEMV_PDL", "FB_GEMV_INDEPENDENT", "FB_GEMV_TEST_WAIT_TIMEOUT",
    "fb_packed_words", "fb_pack", "fb_pack_bits", "fb_unpack", "fb_vcm_gather",
    "fb_lut_build", "fb_validate_weights", "fb_gemv_workspace_bytes", "fb_gemv",
    "fb_gemv_batched", "fb_status_string", "fb_gemv_launch_plan", "fb_gemv_grouped", "fb_device_errors",
    "fb_fit_saliency", "fb_fit_base", "fit", "fb_gemv_group_scales",
    "FB_ROPE_NEIGHBOURS", "rope_frequencies", "fb_qk_norm_rope", "fb_attn_prompt", "fb_attn_tree",
    "fb_attn_tree_workspace_bytes", "fb_attn_errors",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libfluxbin.so")

FB_OK = 0
FB_GEMV_PDL = 1
FB_GEMV_INDEPENDENT = 2
FB_GEMV_TEST_WAIT_TIMEOUT = 0x80000000
FB_ROPE_NEIGHBOURS = 0x10
_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_STATUS = {0: "FB_OK", 1: "FB_ERR_INVALID_VALUE", 2: "FB_ERR_UNSUPPORTED", 3: "FB_ERR_MISALIGNED",
           4: "FB_ERR_WORKSPACE", 5: "FB_ERR_CUDA"}


class FbError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_STATUS.get(status, status)}")


class FbWeightsStruct(C.Structure):
    _fields_ = [
        ("M", C.c_int), ("N", C.c_int), ("K", C.c_int), ("g", C.c_int),
        ("planes", C.c_void_p), ("alpha_r", C.c_void_p), ("alpha_c", C.c_void_p),
        ("nS", C.c_int), ("Ks", C.c_int),
        ("s_idx", C.c_void_p), ("s_planes", C.c_void_p),
        ("s_alpha_r", C.c_void_p), ("s_alpha_c", C.c_void_p),
    ]


class FbHeadsStruct(C.Structure):
    _fields_ = [
        ("q", C.c_void_p), ("k", C.c_void_p), ("v", C.c_void_p), ("t", C.c_int),
        ("T", C.c_int), ("Hq", C.c_int), ("Hkv", C.c_int), ("D", C.c_int),
        ("ldq", C.c_int), ("ldk", C.c_int), ("ldv", C.c_int),
    ]


class FbKvCacheStruct(C.Structure):
    _fields_ = [
        ("k", C.c_void_p), ("v", C.c_void_p), ("t", C.c_int),
        ("pages", C.c_int), ("page_size", C.c_int), ("Hkv", C.c_int), ("D", C.c_int),
    ]


_lib = None


def lib() -> C.CDLL:
    """The loaded C library, with argument types declared."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise RuntimeError(
                f"{library_path} is missing: build it with `python -m lut_binary_gemv_b200.build` "
                "(nvcc, sm_100a). There is no CPU fallback.")
        L = C.CDLL(library_path)
        P, I, S = C.c_void_p, C.c_int, C.c_size_t
        W = C.POINTER(FbWeightsStruct)
        H, KV, F, U = P, P, C.c_float, C.c_uint   # the attention calls' structs, as bytes or by reference
        sig = {
            "fb_packed_words": (S, [I, I, I]),
            "fb_pack": (I, [P, I, I, I, P, P]),
            "fb_pack_bits": (I, [P, I, I, I, P, P]),
            "fb_unpack": (I, [P, I, I, I, P, P]),
            "fb_vcm_gather": (I, [P, I, I, I, I, P, I, I, P, I, P]),
            "fb_lut_build": (I, [P, I, P, I, I, I, P, P]),
            "fb_validate_weights": (I, [W]),
            "fb_gemv_workspace_bytes": (S, [W, I]),
            "fb_gemv": (I, [W, P, I, P, P, S, C.c_uint, P]),
            "fb_gemv_batched": (I, [W, P, I, I, I, P, I, P, S, C.c_uint, P]),
            "fb_gemv_launch_plan": (I, [W, I, C.c_uint, I, P]),
            "fb_gemv_grouped": (I, [P, I, P, I, P, C.c_uint, P]),
            "fb_gemv_group_scales": (I, [W, I, P, I, P, C.c_uint, P]),
            "fb_device_errors": (I, [P, I]),
            "fb_fit_saliency": (I, [P, I, I, I, P, I, I, I, P, P, P]),
            "fb_fit_base": (I, [P, I, I, I, I, P, I, P, P, P]),
            "fb_qk_norm_rope": (I, [H, H, P, P, I, P, P, F, KV, P, U, P]),
            "fb_attn_prompt": (I, [H, P, I, F, P, I, P, U, P]),
            "fb_attn_tree_workspace_bytes": (S, [I, KV, I, I]),
            "fb_attn_errors": (I, [P, I]),
            "fb_attn_tree": (I, [P, I, I, I, KV, P, I, I, P, P, I, I, P, F, P, I, P, P, S, U, P]),
            "fb_status_string": (C.c_char_p, [I]),
            "fb_abi_version": (I, []),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def _check(status: int, what: str):
    if status != FB_OK:
        raise FbError(status, what)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device: torch.device) -> int:
    """The current CUDA stream of `device` as a raw handle (the cheap
    accessor when torch has it: eager calls are bound by host time)."""
    if _raw_stream is not None:
        return _raw_stream(device.index if device.index is not None else torch.cuda.current_device())
    return torch.cuda.current_stream(device).cuda_stream


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def fb_status_string(status: int) -> str:
    return lib().fb_status_string(status).decode()


def fb_packed_words(K: int, M: int, N: int) -> int:
    return lib().fb_packed_words(K, M, N)


def _new_planes(K, M, N, device):
    n = fb_packed_words(K, M, N)
    if n == 0:
        raise FbError(1, "fb_packed_words")
    return torch.empty(n, dtype=torch.int32, device=device)


def fb_pack(signs: torch.Tensor, planes: Optional[torch.Tensor] = None) -> torch.Tensor:
    """signs: int8 [K, M, N] (+1/-1) on the GPU -> packed planes (int32 words)."""
    K, M, N = signs.shape
    signs = signs.contiguous()
    planes = _new_planes(K, M, N, signs.device) if planes is None else planes
    _check(lib().fb_pack(signs.data_ptr(), K, M, N, planes.data_ptr(), _stream(signs.device)), "fb_pack")
    return planes


def fb_pack_bits(bits: torch.Tensor, N: int, planes: Optional[torch.Tensor] = None) -> torch.Tensor:
    """bits: uint8 [K, M, N/8] canonical bit planes on the GPU -> packed planes."""
    K, M, nb = bits.shape
    if nb * 8 != N:
        raise ValueError("bits must have N/8 bytes per row")
    bits = bits.contiguous()
    planes = _new_planes(K, M, N, bits.device) if planes is None else planes
    _check(lib().fb_pack_bits(bits.data_ptr(), K, M, N, planes.data_ptr(), _stream(bits.device)),
           "fb_pack_bits")
    return planes


def fb_unpack(planes: torch.Tensor, K: int, M: int, N: int) -> torch.Tensor:
    signs = torch.empty((K, M, N), dtype=torch.int8, device=planes.device)
    _check(lib().fb_unpack(planes.data_ptr(), K, M, N, signs.data_ptr(), _stream(planes.device)), "fb_unpack")
    return signs


def fb_vcm_gather(src: torch.Tensor, s_idx: torch.Tensor, nS_pad: int) -> torch.Tensor:
    """src: [nvec, n_src] (f32/f16/bf16); s_idx: int32 [nS] -> [nvec, nS_pad]."""
    src2 = src.reshape(-1, src.shape[-1]) if src.dim() != 1 else src.reshape(1, -1)
    nvec, n_src = src2.shape
    if src2.stride(-1) != 1:
        src2 = src2.contiguous()
    nS = s_idx.numel()
    dst = torch.empty((nvec, nS_pad), dtype=src.dtype, device=src.device)
    _check(lib().fb_vcm_gather(src2.data_ptr(), _DTYPES[src.dtype], nvec, n_src, src2.stride(0),
                               _ptr(s_idx) if nS else None, nS, nS_pad, dst.data_ptr(), nS_pad,
                               _stream(src.device)), "fb_vcm_gather")
    return dst if src.dim() != 1 else dst.reshape(-1)


def fb_lut_build(x: torch.Tensor, alpha_c: Optional[torch.Tensor], K: int, g: int) -> torch.Tensor:
    """LUT-BSF tables [K, N/g, 2^g] fp32 for one activation vector x [N]."""
    x = x.contiguous()
    N = x.numel()
    lut = torch.empty((K, N // g, 1 << g), dtype=torch.float32, device=x.device)
    ac = None if alpha_c is None else alpha_c.contiguous()
    _check(lib().fb_lut_build(x.data_ptr(), _DTYPES[x.dtype], _ptr(ac), K, N, g, lut.data_ptr(),
                              _stream(x.device)), "fb_lut_build")
    return lut


class Weights:
    """One fb_weights struct plus the device tensors it points to."""

    def __init__(self, M: int, N: int, K: int, g: int, planes: torch.Tensor, alpha_r: torch.Tensor,
                 alpha_c: Optional[torch.Tensor] = None, nS: int = 0, Ks: int = 0,
                 s_idx: Optional[torch.Tensor] = None, s_planes: Optional[torch.Tensor] = None,
                 s_alpha_r: Optional[torch.Tensor] = None, s_alpha_c: Optional[torch.Tensor] = None):
        self.M, self.N, self.K, self.g, self.nS, self.Ks = M, N, K, g, nS, Ks if nS else 0
        self.planes, self.alpha_r, self.alpha_c = planes, alpha_r, alpha_c
        self.s_idx, self.s_planes, self.s_alpha_r, self.s_alpha_c = s_idx, s_planes, s_alpha_r, s_alpha_c
        self.device = planes.device
        self.struct = FbWeightsStruct(
            M=M, N=N, K=K, g=g, planes=_ptr(planes), alpha_r=_ptr(alpha_r), alpha_c=_ptr(alpha_c),
            nS=nS, Ks=self.Ks, s_idx=_ptr(s_idx) if nS else None, s_planes=_ptr(s_planes) if nS else None,
            s_alpha_r=_ptr(s_alpha_r) if nS else None, s_alpha_c=_ptr(s_alpha_c) if nS else None)

    @property
    def ref(self):
        ref = self.__dict__.get("_ref")
        if ref is None:
            ref = self._ref = C.byref(self.struct)
        return ref

    def with_g(self, g: int) -> "Weights":
        """The same tensors with another LUT group width (the packed layout
        does not depend on g)."""
        return Weights(self.M, self.N, self.K, g, self.planes, self.alpha_r, self.alpha_c, self.nS,
                       self.Ks, self.s_idx, self.s_planes, self.s_alpha_r, self.s_alpha_c)

    @classmethod
    def from_arrays(cls, M, N, K, g, sign_bits, alpha_r, alpha_c=None, s_idx=None, s_sign_bits=None,
                    s_alpha_r=None, s_alpha_c=None, device="cuda") -> "Weights":
        """Upload canonical bit planes and scales (numpy or torch) and pack them on the GPU."""
        dev = torch.device(device)

        def up(a, dtype=None):
            if a is None:
                return None
            t = torch.as_tensor(a)
            if dtype is not None:
                t = t.to(dtype)
            return t.to(dev).contiguous()

        planes = fb_pack_bits(up(sign_bits, torch.uint8), N)
        nS = 0 if s_idx is None else len(s_idx)
        kw = {}
        if nS:
            nS_pad = (nS + 31) // 32 * 32
            kw = dict(nS=nS, Ks=int(s_alpha_r.shape[0]),
                      s_idx=up(torch.as_tensor(s_idx).to(torch.int64).to(torch.int32)),
                      s_planes=fb_pack_bits(up(s_sign_bits, torch.uint8), nS_pad),
                      s_alpha_r=up(s_alpha_r, torch.float32), s_alpha_c=up(s_alpha_c, torch.float32))
        return cls(M, N, K, g, planes, up(alpha_r, torch.float32), up(alpha_c, torch.float32), **kw)

    @classmethod
    def from_problem(cls, p, device="cuda", g: Optional[int] = None) -> "Weights":
        """From a workloads.Problem (its canonical arrays)."""
        return cls.from_arrays(p.M, p.N, p.K, p.g if g is None else g, p.sign_bits, p.alpha_r, p.alpha_c,
                               p.s_idx if p.nS else None, p.s_sign_bits, p.s_alpha_r, p.s_alpha_c,
                               device=device)


def fb_validate_weights(W: Weights) -> int:
    return lib().fb_validate_weights(W.ref)


def fb_gemv_workspace_bytes(W: Weights, batch: int = 1) -> int:
    return lib().fb_gemv_workspace_bytes(W.ref, batch)


def fb_gemv(W: Weights, x: torch.Tensor, y: Optional[torch.Tensor] = None,
            ws: Optional[torch.Tensor] = None, flags: int = 0) -> torch.Tensor:
    """y = W_hat x for one activation vector x [N] (f32/f16/bf16) -> fp32 [M]."""
    if x.stride(-1) != 1:
        x = x.contiguous()
    y = torch.empty(W.M, dtype=torch.float32, device=x.device) if y is None else y
    # the kernels need no workspace (fb_gemv_workspace_bytes is 0): NULL, 0 unless one is given
    wp, wn = (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())
    _check(lib().fb_gemv(W.ref, x.data_ptr(), _DTYPES[x.dtype], y.data_ptr(), wp, wn, flags,
                         _stream(x.device)), "fb_gemv")
    return y


def fb_gemv_batched(W: Weights, X: torch.Tensor, Y: Optional[torch.Tensor] = None,
                    ws: Optional[torch.Tensor] = None, flags: int = 0) -> torch.Tensor:
    """Y[b] = W_hat X[b] for X [B, N] -> fp32 [B, M]."""
    B = X.shape[0]
    if X.stride(-1) != 1:
        X = X.contiguous()
    Y = torch.empty((B, W.M), dtype=torch.float32, device=X.device) if Y is None else Y
    wp, wn = (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())
    _check(lib().fb_gemv_batched(W.ref, X.data_ptr(), _DTYPES[X.dtype], B, X.stride(0), Y.data_ptr(),
                                 Y.stride(0), wp, wn, flags, _stream(X.device)), "fb_gemv_batched")
    return Y


def fb_gemv_launch_plan(W, batch: int = 1, flags: int = 0, sms: int = 148) -> dict:
    """The launch shape fb_gemv would use for W (a Weights or an
    FbWeightsStruct: only its sizes and pointer alignment are read, so no GPU
    is needed)."""
    out = (C.c_int * 6)()
    ref = W.ref if isinstance(W, Weights) else C.byref(W)
    _check(lib().fb_gemv_launch_plan(ref, batch, flags, sms, C.cast(out, C.c_void_p)), "fb_gemv_launch_plan")
    return dict(zip(("C", "cpb", "RB", "warps", "smem", "V"), list(out)))


def fb_device_errors(clear: bool = True) -> int:
    """Error bits raised by GEMV kernels since the last clear (synchronises the device)."""
    flags = C.c_uint(0)
    _check(lib().fb_device_errors(C.cast(C.byref(flags), C.c_void_p), int(clear)), "fb_device_errors")
    return flags.value


def fb_gemv_grouped(Ws, x: torch.Tensor, ys=None, flags: int = 0):
    """One launch for up to 4 matrices of one format that read the same x
    (q/k/v, gate/up): returns [y_m] with y_m = W_hat_m x."""
    n = len(Ws)
    if ys is None:
        ys = [torch.empty(W.M, dtype=torch.float32, device=x.device) for W in Ws]
    wp = (C.POINTER(FbWeightsStruct) * n)(*[C.pointer(W.struct) for W in Ws])
    yp = (C.c_void_p * n)(*[y.data_ptr() for y in ys])
    _check(lib().fb_gemv_grouped(C.cast(wp, C.c_void_p), n, x.data_ptr(), _DTYPES[x.dtype],
                                 C.cast(yp, C.c_void_p), flags, _stream(x.device)), "fb_gemv_grouped")
    return ys


def fb_gemv_group_scales(W: Weights, G: int, x: torch.Tensor, alpha_r_groups: torch.Tensor,
                         y: Optional[torch.Tensor] = None, flags: int = 0) -> torch.Tensor:
    """y = W_hat x with one row scale per group of G input columns:
    alpha_r_groups fp32 [K, N/G, M] (replacing W.alpha_r); W's other tensors
    as for fb_gemv."""
    if x.stride(-1) != 1:
        x = x.contiguous()
    if G <= 0 or W.N % G:
        raise ValueError("G must be a positive divisor of N")
    if (alpha_r_groups.dtype != torch.float32 or not alpha_r_groups.is_contiguous()
            or alpha_r_groups.numel() != W.K * (W.N // G) * W.M):
        raise ValueError("alpha_r_groups: contiguous float32 [K, N/G, M]")
    y = torch.empty(W.M, dtype=torch.float32, device=x.device) if y is None else y
    st = FbWeightsStruct.from_buffer_copy(W.struct)
    st.alpha_r = alpha_r_groups.data_ptr()
    _check(lib().fb_gemv_group_scales(C.byref(st), G, x.data_ptr(), _DTYPES[x.dtype], y.data_ptr(), flags,
                                      _stream(x.device)), "fb_gemv_group_scales")
    return y


def _f32_rows(t: torch.Tensor, what: str) -> torch.Tensor:
    if t.dim() != 2 or t.dtype != torch.float32 or t.stride(1) != 1:
        raise ValueError(f"{what}: a float32 matrix with unit column stride")
    return t


def fb_fit_saliency(W: torch.Tensor, X: torch.Tensor, nS: int) -> Tuple[torch.Tensor, torch.Tensor]:
    """Column scores (diagonal-Hessian proxy) and the nS salient columns.
    W [M, N], X [T, N] fp32 on the GPU -> (score fp32 [N], s_idx int32 [nS],
    ascending)."""
    W, X = _f32_rows(W, "W"), _f32_rows(X, "X")
    M, N = W.shape
    T = X.shape[0]
    if X.shape[1] != N:
        raise ValueError("X must have W's columns")
    score = torch.empty(N, dtype=torch.float32, device=W.device)
    s_idx = torch.empty(max(nS, 0), dtype=torch.int32, device=W.device)
    _check(lib().fb_fit_saliency(W.data_ptr(), M, N, W.stride(0), X.data_ptr(), T, X.stride(0), nS,
                                 score.data_ptr(), s_idx.data_ptr() if nS > 0 else None, _stream(W.device)),
           "fb_fit_saliency")
    return score, s_idx


def fb_fit_base(R: torch.Tensor, sweeps: int, signs: Optional[torch.Tensor] = None,
                alpha_r: Optional[torch.Tensor] = None,
                alpha_c: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """One greedy base on the residual R [M, N] fp32 (updated in place) ->
    (signs int8 [M, N], alpha_r fp32 [M], alpha_c fp32 [N]), written into the
    given outputs when passed (signs: unit column stride; scales contiguous)."""
    R = _f32_rows(R, "R")
    M, N = R.shape
    signs = torch.empty((M, N), dtype=torch.int8, device=R.device) if signs is None else signs
    ar = torch.empty(M, dtype=torch.float32, device=R.device) if alpha_r is None else alpha_r
    ac = torch.empty(N, dtype=torch.float32, device=R.device) if alpha_c is None else alpha_c
    if (signs.shape != (M, N) or signs.dtype != torch.int8 or signs.stride(1) != 1 or ar.shape != (M,)
            or ac.shape != (N,) or not ar.is_contiguous() or not ac.is_contiguous()):
        raise ValueError("fb_fit_base: output shapes")
    _check(lib().fb_fit_base(R.data_ptr(), M, N, R.stride(0), sweeps, signs.data_ptr(), signs.stride(0),
                             ar.data_ptr(), ac.data_ptr(), _stream(R.device)), "fb_fit_base")
    return signs, ar, ac


def fit(W: torch.Tensor, X: torch.Tensor, K: int, Ks: int, nS: int, sweeps: int) -> dict:
    """The whole fit on the GPU: K global bases on R = W, then the salient
    set and Ks bases on the residual's salient columns (gathered by
    fb_vcm_gather, padded to a multiple of 32 with zero columns).  Returns
    signs [K, M, N], alpha_r [K, M], alpha_c [K, N], score [N], s_idx [nS],
    s_signs [Ks, M, nS], s_alpha_r [Ks, M], s_alpha_c [Ks, nS], residual
    [M, N] (after the global bases) and s_residual [M, nS] (after the salient
    ones)."""
    W = _f32_rows(W, "W")
    M, N = W.shape
    dev = W.device
    score, s_idx = fb_fit_saliency(W, X, nS)
    R = W.clone()
    signs = torch.empty((K, M, N), dtype=torch.int8, device=dev)
    ar = torch.empty((K, M), dtype=torch.float32, device=dev)
    ac = torch.empty((K, N), dtype=torch.float32, device=dev)
    for k in range(K):
        fb_fit_base(R, sweeps, signs[k], ar[k], ac[k])
    nS_pad = (nS + 31) // 32 * 32
    # the salient bases run over the padded gather (zero columns past nS);
    # the views below drop the padding
    s_signs = torch.empty((Ks, M, nS_pad), dtype=torch.int8, device=dev)
    s_ar = torch.empty((Ks, M), dtype=torch.float32, device=dev)
    s_ac = torch.empty((Ks, nS_pad), dtype=torch.float32, device=dev)
    RS = None
    if nS > 0 and Ks > 0:
        RS = fb_vcm_gather(R, s_idx, nS_pad)
        for k in range(Ks):
            fb_fit_base(RS, sweeps, s_signs[k], s_ar[k], s_ac[k])
    return {"signs": signs, "alpha_r": ar, "alpha_c": ac, "score": score, "s_idx": s_idx,
            "s_signs": s_signs[:, :, :nS], "s_alpha_r": s_ar, "s_alpha_c": s_ac[:, :nS], "residual": R,
            "s_residual": None if RS is None else RS[:, :nS]}


# ---- attention ---------------------------------------------------------------
#
# Eager calls of small cases are bound by host time, so the checks below read
# each tensor property once and the structs are packed as bytes.

_HEADS = struct.Struct("@PPP8i")      # FbHeadsStruct
_CACHE = struct.Struct("@PP5i4x")     # FbKvCacheStruct
_get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on(device: int, f, *args) -> int:
    """f(*args, stream) on the device the tensors live on, whichever is current."""
    if device != _get_device():
        with torch.cuda.device(device):
            return f(*args, torch.cuda.current_stream(device).cuda_stream)
    return f(*args, torch.cuda.current_stream(device).cuda_stream if _raw_stream is None else _raw_stream(device))


def _pitch(ld: int, what: str) -> int:
    """A pitch as the C ABI takes it: ctypes would cut a longer one off."""
    if ld >= 1 << 31:
        raise ValueError(f"{what}: rows at most 2^31 - 1 elements apart are expected, got {ld}")
    return ld


def _rows(t: torch.Tensor, what: str, device: int, shape, dtype) -> int:
    """The row pitch of [T, H, D] heads on the GPU whose heads are contiguous within a row."""
    if t.dtype == dtype and t.shape == shape and t.get_device() == device >= 0:
        T, H, D = shape
        if t.is_contiguous():
            return H * D
        st = t.stride()
        if (st[2] == 1 or D == 1) and (st[1] == D or H == 1):
            return _pitch(st[0], what) if T > 1 else H * D
        raise ValueError(f"{what}: the heads of a row must be contiguous (only rows may be strided)")
    raise ValueError(f"{what}: a {dtype} tensor {tuple(shape)} on the GPU of the others is expected, "
                     f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _sizes(q: torch.Tensor, k: torch.Tensor):
    """The shape of the queries, of the keys and values, and their type's code."""
    qs, ks = q.shape, k.shape
    t = _DTYPES.get(q.dtype)
    if len(qs) != 3 or len(ks) != 3 or t is None:
        raise ValueError("q, k, v: [T, heads, D] tensors (f32/f16/bf16)")
    return qs, (qs[0], ks[1], qs[2]), t


def _flat(t: torch.Tensor, what: str, dtype, n: int, device: int) -> int:
    """The address of a contiguous tensor of n elements of the given type."""
    if t.dtype != dtype or t.numel() != n or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous {dtype} tensor of {n} elements on the GPU of the others is expected")
    return t.data_ptr()


def _cache_bytes(cache, device: int, dtype):
    """(k_pages, v_pages), each [pages, Hkv, page_size, D] -> the C struct and the shape."""
    k, v = cache
    shape = k.shape
    if (len(shape) != 4 or v.shape != shape or k.dtype != dtype or v.dtype != dtype or k.get_device() != device
            or v.get_device() != device or not k.is_contiguous() or not v.is_contiguous()):
        raise ValueError("cache: two contiguous [pages, Hkv, page_size, D] tensors of the heads' type and device")
    pages, Hkv, page_size, D = shape
    return _CACHE.pack(k.data_ptr(), v.data_ptr(), _DTYPES[dtype], pages, page_size, Hkv, D), shape


def rope_frequencies(rot: int, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """theta^(-2p / rot) for the rot/2 pairs of a rotation: float64, as fb_qk_norm_rope takes them."""
    return float(theta) ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)


def fb_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, pos: Optional[torch.Tensor],
                    inv_freq: Optional[torch.Tensor], q_weight: Optional[torch.Tensor] = None,
                    k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, interleaved: bool = False,
                    cache=None, slots: Optional[torch.Tensor] = None, out_dtype=None,
                    q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                    v_out: Optional[torch.Tensor] = None, flags: int = 0):
    """Norm and rotation of projected heads, and their write into a paged cache, in one pass.

    q [T, Hq, D], k and v [T, Hkv, D] (f32/f16/bf16; rows may be strided, as slices of a fused projection);
    pos int32 [T]; inv_freq float64 [rot/2] (None: no rotation); q_weight, k_weight float32 [D] (None: no norm).
    interleaved: pairs are neighbouring elements, not the halves of the rotated part.  cache = (k_pages, v_pages),
    [pages, Hkv, page_size, D] each, takes the keys and values at slots int32 [T] (slots outside are skipped).
    Returns (q_out, k_out, v_out): q_out is made when not given; k_out and v_out are made only where there is no
    cache.  Their type is out_dtype: by default the cache's, else a given output's, else the heads' (bf16 for
    f32 heads).  The outputs may be the inputs (in place)."""
    qs, ks, t = _sizes(q, k)
    T, Hq, D = qs
    Hkv, dev, dtype = ks[1], q.get_device(), q.dtype
    hin = _HEADS.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), t, T, Hq, Hkv, D, _rows(q, "q", dev, qs, dtype),
                      _rows(k, "k", dev, ks, dtype), _rows(v, "v", dev, ks, dtype))
    dt = out_dtype
    if dt is None:
        given = cache[0] if cache is not None else next((o for o in (q_out, k_out, v_out) if o is not None), None)
        dt = given.dtype if given is not None else dtype if t else torch.bfloat16
    to = _DTYPES.get(dt)
    if to is None:
        raise ValueError("out_dtype: torch.float16 or torch.bfloat16")
    if q_out is None:
        q_out = torch.empty(qs, dtype=dt, device=q.device)
    kv = None
    if cache is None:
        k_out = torch.empty(ks, dtype=dt, device=q.device) if k_out is None else k_out
        v_out = torch.empty(ks, dtype=dt, device=q.device) if v_out is None else v_out
    else:
        kv = _cache_bytes(cache, dev, dt)[0]
    kp = vp = ldk = ldv = 0
    if k_out is not None:
        kp, ldk = k_out.data_ptr(), _rows(k_out, "k_out", dev, ks, dt)
    if v_out is not None:
        vp, ldv = v_out.data_ptr(), _rows(v_out, "v_out", dev, ks, dt)
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    if rot and pos is None:
        raise ValueError("pos: int32 [T] where there is a rotation")
    if (cache is None) != (slots is None):
        raise ValueError("cache and slots go together")
    hout = _HEADS.pack(q_out.data_ptr(), kp, vp, to, T, Hq, Hkv, D, _rows(q_out, "q_out", dev, qs, dt), ldk, ldv)
    _check(_on(dev, lib().fb_qk_norm_rope, hin, hout, None if pos is None else _flat(pos, "pos", torch.int32, T, dev),
               _flat(inv_freq, "inv_freq", torch.float64, rot // 2, dev) if rot else None, rot,
               None if q_weight is None else _flat(q_weight, "q_weight", torch.float32, D, dev),
               None if k_weight is None else _flat(k_weight, "k_weight", torch.float32, D, dev), eps, kv,
               None if slots is None else _flat(slots, "slots", torch.int32, T, dev),
               flags | FB_ROPE_NEIGHBOURS if interleaved else flags), "fb_qk_norm_rope")
    return q_out, k_out, v_out


def fb_attn_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                   scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, flags: int = 0) -> torch.Tensor:
    """Causal attention of packed prompts: q [T, Hq, D], k and v [T, Hkv, D] (f16/bf16, D 64 or 128; rows may be
    strided), sequence s being tokens cu_seqlens[s] .. cu_seqlens[s+1]-1 (int32 [n+1]) -> [T, Hq, D].  scale
    defaults to D^-0.5; lse float32 [T, Hq] takes the logarithms of the softmax's sums.  Rows of no sequence keep
    what `out` holds (unset memory when it is not given)."""
    qs, ks, t = _sizes(q, k)
    T, Hq, D = qs
    dev, dtype = q.get_device(), q.dtype
    h = _HEADS.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), t, T, Hq, ks[1], D, _rows(q, "q", dev, qs, dtype),
                    _rows(k, "k", dev, ks, dtype), _rows(v, "v", dev, ks, dtype))
    if out is None:
        out = torch.empty(qs, dtype=dtype, device=q.device)
    n = cu_seqlens.numel() - 1
    _check(_on(dev, lib().fb_attn_prompt, h, _flat(cu_seqlens, "cu_seqlens", torch.int32, n + 1, dev), n,
               D ** -0.5 if scale is None else scale, out.data_ptr(), _rows(out, "out", dev, qs, dtype),
               None if lse is None else _flat(lse, "lse", torch.float32, T * Hq, dev), flags), "fb_attn_prompt")
    return out


def fb_attn_tree_workspace_bytes(Hq: int, cache, max_draft: int, table_width: int) -> int:
    """Bytes of the workspace that fb_attn_tree needs (0: none) for Hq query heads over the cache."""
    dev = cache[0].get_device()
    return _tree_workspace(dev, Hq, _cache_bytes(cache, dev, cache[0].dtype)[0], max_draft, table_width)


def _tree_workspace(device: int, *args) -> int:
    """The size goes by the SMs of the device that runs the call, whichever is current."""
    if device < 0 or device == _get_device():
        return lib().fb_attn_tree_workspace_bytes(*args)
    with torch.cuda.device(device):
        return lib().fb_attn_tree_workspace_bytes(*args)


def fb_attn_tree(q: torch.Tensor, cache, page_table: torch.Tensor, lens: torch.Tensor,
                 cu_draft: Optional[torch.Tensor] = None, max_draft: int = 1, mask: Optional[torch.Tensor] = None,
                 scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                 flags: int = 0) -> torch.Tensor:
    """Attention of each sequence's newest tokens over the paged cache: q [T, Hq, D] of the cache's type, cache =
    (k_pages, v_pages), page_table int32 [n, width], lens int32 [n] committed keys, cu_draft int32 [n+1] the
    sequences' tokens in q (None: one each, T = n), at most max_draft <= 64 a sequence, whose own keys are in the
    cache at positions lens[s] + j.  mask int64 [T]: bit j of a token's word lets it see drafted token j of its
    sequence (None: a chain, j <= i).  Returns [T, Hq, D]; scale, out and lse as for fb_attn_prompt.  ws (uint8)
    is made when not given."""
    qs, dtype, dev = q.shape, q.dtype, q.get_device()
    if len(qs) != 3 or dtype not in _DTYPES:
        raise ValueError("q: a [T, heads, D] tensor of the cache's type")
    T, Hq, D = qs
    ldq = _rows(q, "q", dev, qs, dtype)
    kv, shape = _cache_bytes(cache, dev, dtype)
    if shape[3] != D:
        raise ValueError("cache: another head width than q's")
    n, ts = lens.numel(), page_table.shape
    if len(ts) != 2 or ts[0] != n or page_table.dtype != torch.int32 or page_table.get_device() != dev:
        raise ValueError("page_table: an int32 [n, width] tensor on q's device")
    width = ld = ts[1]
    if not page_table.is_contiguous():
        ld, unit = page_table.stride()
        if (unit != 1 and width > 1) or (ld < width and n > 1):
            raise ValueError("page_table: unit column stride")
        ld = _pitch(ld, "page_table") if n > 1 else width
    if out is None:
        out = torch.empty(qs, dtype=dtype, device=q.device)
    if ws is None:
        wb = _tree_workspace(dev, Hq, kv, max_draft, width)
        wp = None
        if wb:
            ws = torch.empty(wb, dtype=torch.uint8, device=q.device)
            wp = ws.data_ptr()
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("ws: a contiguous tensor on q's device")
    else:
        wp, wb = ws.data_ptr(), ws.numel() * ws.element_size()
    _check(_on(dev, lib().fb_attn_tree, q.data_ptr(), ldq, T, Hq, kv, page_table.data_ptr(), width, ld,
               _flat(lens, "lens", torch.int32, n, dev),
               None if cu_draft is None else _flat(cu_draft, "cu_draft", torch.int32, n + 1, dev), n, max_draft,
               None if mask is None else _flat(mask, "mask", torch.int64, T, dev),
               D ** -0.5 if scale is None else scale, out.data_ptr(), _rows(out, "out", dev, qs, dtype),
               None if lse is None else _flat(lse, "lse", torch.float32, T * Hq, dev), wp, wb, flags),
           "fb_attn_tree")
    return out


def fb_attn_errors(clear: bool = True) -> int:
    """Error bits raised by attention kernels since the last clear (synchronises the device): 1, a page outside the
    cache or too many drafted tokens; 2, a wait that gave up."""
    flags = C.c_uint(0)
    _check(lib().fb_attn_errors(C.cast(C.byref(flags), C.c_void_p), int(clear)), "fb_attn_errors")
    return flags.value
