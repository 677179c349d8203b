"""Thin Python binding of libtq (argument marshalling only).

Every function takes torch tensors that already live on a CUDA device, checks
their dtype, device, contiguity and shape, and passes raw device pointers and
the current CUDA stream to the C ABI declared in ``include/tq.h``.  All work
runs in libtq's kernels; there is no CPU fallback.  A missing libtq.so, a
tensor on the CPU, or a non-OK status raises.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtq.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "tq.h")

TQ_OK = 0
STATUS_NAMES = {0: "TQ_OK", 1: "TQ_ERR_INVALID_VALUE", 2: "TQ_ERR_UNSUPPORTED",
                3: "TQ_ERR_MISALIGNED", 4: "TQ_ERR_WORKSPACE", 5: "TQ_ERR_LAUNCH"}
QTYPE = {torch.float32: 0, torch.bfloat16: 1}
PATHS = {"auto": 0, "fp32": 1, "bf16_mma": 2}
PATH_NAMES = {v: k for k, v in PATHS.items()}

_lib = None


class TQError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} returned {status_string(status)}")


_P, _I, _L, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
_SIGNATURES = {
    "tq_status_string": ([_I], ctypes.c_char_p),
    "tq_auto_path": ([_I, _I], _I),
    "tq_device_faults": ([ctypes.POINTER(ctypes.c_uint)], _I),
    "tq_check_wait_expiry": ([_P], _I),
    "tq_prepare_queries": ([_P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _P], _I),
    "tq_scores": ([_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P], _I),
    "tq_scores_packed": ([_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P], _I),
    "tq_scores_mse": ([_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P], _I),
    "tq_prepare_queries_hadamard": ([_P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _P], _I),
    "tq_hadamard_rotation": ([_P, _I, _P], _I),
    "tq_decode_workspace_bytes": ([_I, _I, _I, _I], ctypes.c_size_t),
    "tq_decode_mse": ([_P, _P, _P, _P, _I, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, ctypes.c_float,
                       _P, ctypes.c_size_t, _P], _I),
    "tq_decode_prod": ([_P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, ctypes.c_float,
                        _P, ctypes.c_size_t, _P], _I),
    "tq_prepare_queries_split": ([_P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P], _I),
    "tq_scores_split": ([_P, _P, _P, _P, _P, _I, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _P], _I),
    "tq_workspace_bytes": ([_I, _I, _I], _Z),
    "tq_solve": ([_P, _I, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _Z, _I, _P], _I),
    "tq_solve_packed": ([_P, _I, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _Z, _I, _P], _I),
    "tq_pack_indices": ([_P, _P, _L, _I, _I, _P], _I),
    "tq_unpack_indices": ([_P, _P, _L, _I, _I, _P], _I),
    "tq_pack_signs": ([_P, _P, _L, _I, _P], _I),
    "tq_unpack_signs": ([_P, _P, _L, _I, _P], _I),
    "tq_compress_keys": ([_P, _P, _P, _P, _I, _P, _P, _P, _P, _I, _I, _I, _I, _P], _I),
    "tq_compress_keys_packed": ([_P, _P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _P], _I),
    "tq_lloyd_max_codebook": ([_I, _I, _I, _I, _P], _I),
    "tq_haar_rotation": ([_P, _I, _P], _I),
    "tq_append_paged": ([_P, _P, _P, _I, _P, _I, _P, _I, _I, _P, _P, _I, _P], _I),
    "tq_decode_paged_workspace_bytes": ([_I, _I, _I, _I, _I], ctypes.c_size_t),
    "tq_decode_paged": ([_P, _P, _I, _P, _P, _I, _I, _I, ctypes.c_float, _P, _I, _P, _P, _Z, _P], _I),
    "tq_evict_paged_workspace_bytes": ([_I, _I, _I, _I], ctypes.c_size_t),
    "tq_evict_paged": ([_P, _P, _P, _P, _I, _I, _P, _P, _I, _I, _I, _P, _P, _P, _Z, _P], _I),
    "tq_norm_rope": ([_P, _L, _L, _P, _L, _L, _I, _P, _P, _I, ctypes.c_float, _P, _I, _P, _P, _I, _I, _P, _P, _I, _I, _I,
                      _I, _P], _I),
    "tq_append_int8": ([_P, _P, _L, _P, _L, _I, _P, _P, _I, _P, _I, _I, _P], _I),
    "tq_read_int8": ([_P, _P, _P, _I, _P, _P, _I, _P, _I, _I, _P], _I),
    "tq_attend_int8_workspace_bytes": ([_I, _I, _I, _I, _I], ctypes.c_size_t),
    "tq_attend_int8": ([_P, _P, _I, _P, _P, _I, _I, _P, _I, _I, _I, _I, ctypes.c_float, _P, _P, _Z, _P], _I),
    "tq_solve_packed_noalloc": ([_P, _I, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P], _I),
}


def lib() -> ctypes.CDLL:
    """Loads libtq.so once; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with compressed_kv_cache_gb300.build.build()")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = res
        _lib = handle
    return _lib


def declared_functions() -> list[str]:
    """Names of the functions include/tq.h declares."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_]*\s*\*?\s*(tq_[a-z0-9_]+)\s*\(",
                                 text, flags=re.M)))


def status_string(status: int) -> str:
    return lib().tq_status_string(status).decode()


def auto_path(B: int, D: int) -> str:
    return PATH_NAMES[lib().tq_auto_path(B, D)]


def device_faults() -> int:
    """Fault bits the bounded waits of libtq's kernels set on the current device since the
    last call (0 = none; 1 lookup-table scorers, 2 tensor-core scorer, 4 decode, 8
    compressor, 16 check_wait_expiry, 32 a length, slot or page number out of range in a paged
    call, 64 append_paged, 128 attend_int8); reading clears them.  Synchronises with the device."""
    v = ctypes.c_uint(0)
    _check("tq_device_faults", lib().tq_device_faults(ctypes.byref(v)))
    return int(v.value)


def check_wait_expiry() -> None:
    """Runs one warp whose only bounded wait can never complete, on the current stream:
    after about a second it sets fault bit 16 and returns (see device_faults)."""
    _check("tq_check_wait_expiry", lib().tq_check_wait_expiry(_stream()))


def _check(fn: str, status: int) -> None:
    if status != TQ_OK:
        raise TQError(fn, status)


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _dev(t: torch.Tensor, name: str, dtypes) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (libtq has no CPU path)")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _as3(t: torch.Tensor) -> tuple[int, int, int]:
    if t.dim() == 2:
        return 1, t.shape[0], t.shape[1]
    if t.dim() == 3:
        return t.shape[0], t.shape[1], t.shape[2]
    raise ValueError(f"expected a [B,D] or [P,B,D] tensor, got shape {tuple(t.shape)}")


def prepare_queries(Q, Pi, S_mat, out=None):
    """A = Pi q and T = S_mat q.  Q [P,B,D] (or [B,D]) fp32/bf16; Pi, S_mat [H,D,D] (or [D,D])."""
    P, B, D = _as3(Q)
    H = 1 if Pi.dim() == 2 else Pi.shape[0]
    if tuple(Pi.shape[-2:]) != (D, D) or Pi.shape != S_mat.shape:
        raise ValueError("Pi and S_mat must be [H,D,D] or [D,D]")
    A, T = out if out is not None else (torch.empty((P, B, D), device=Q.device, dtype=torch.float32),
                                         torch.empty((P, B, D), device=Q.device, dtype=torch.float32))
    _check("tq_prepare_queries", lib().tq_prepare_queries(
        _dev(Q, "Q", QTYPE), QTYPE[Q.dtype], _dev(Pi, "Pi", (torch.float32,)),
        _dev(S_mat, "S_mat", (torch.float32,)), _dev(A, "A", (torch.float32,)),
        _dev(T, "T", (torch.float32,)), P, H, B, D, _stream()))
    if Q.dim() == 2:
        return A.view(B, D), T.view(B, D)
    return A, T


def prepare_queries_hadamard(Q, signs, S_mat, out=None):
    """A = H diag(s) q (fast Walsh-Hadamard transform) and T = S_mat q.  signs [H,D] (or [D])
    fp32 +-1; S_mat [H,D,D] (or [D,D]); D a power of two."""
    P, B, D = _as3(Q)
    H = 1 if signs.dim() == 1 else signs.shape[0]
    if signs.shape[-1] != D or tuple(S_mat.shape[-2:]) != (D, D):
        raise ValueError("signs must be [H,D] and S_mat [H,D,D]")
    A, T = out if out is not None else (torch.empty((P, B, D), device=Q.device, dtype=torch.float32),
                                         torch.empty((P, B, D), device=Q.device, dtype=torch.float32))
    _check("tq_prepare_queries_hadamard", lib().tq_prepare_queries_hadamard(
        _dev(Q, "Q", QTYPE), QTYPE[Q.dtype], _dev(signs, "signs", (torch.float32,)),
        _dev(S_mat, "S_mat", (torch.float32,)), _dev(A, "A", (torch.float32,)),
        _dev(T, "T", (torch.float32,)), P, H, B, D, _stream()))
    if Q.dim() == 2:
        return A.view(B, D), T.view(B, D)
    return A, T


def hadamard_rotation(signs):
    """Dense Pi = H diag(s) as a float32 [D,D] numpy matrix (host computation in libtq), for
    the compressor and the dense paths."""
    import numpy as np
    s = np.ascontiguousarray(signs, dtype=np.float32)
    D = s.size
    out = np.empty((D, D), dtype=np.float32)
    _check("tq_hadamard_rotation", lib().tq_hadamard_rotation(s.ctypes.data, D, out.ctypes.data))
    return out


def _keys3(t: torch.Tensor, P: int):
    if t.dim() == 2 and P == 1:
        return t.shape[0], t.shape[1]
    if t.dim() == 3 and t.shape[0] == P:
        return t.shape[1], t.shape[2]
    raise ValueError(f"key tensor shape {tuple(t.shape)} does not match P={P}")


def _scores_out(out, P, B, S, like):
    if out is None:
        out = torch.empty((P, B, S), device=like.device, dtype=torch.float32)
    if out.numel() != P * B * S:
        raise ValueError("scores output has the wrong size")
    return out


def scores(A, T, K_idx, signs, gamma, codebook, path="auto", out=None):
    """Scores from an unpacked cache: K_idx uint8 [P,S,D], signs int8 [P,S,D], gamma fp32 [P,S]."""
    P, B, D = _as3(A)
    S, Dk = _keys3(K_idx, P)
    if Dk != D or signs.shape != K_idx.shape or gamma.numel() != P * S:
        raise ValueError("inconsistent key shapes")
    o = _scores_out(out, P, B, S, A)
    _check("tq_scores", lib().tq_scores(
        _dev(A, "A", (torch.float32,)), _dev(T, "T", (torch.float32,)),
        _dev(K_idx, "K_idx", (torch.uint8,)), _dev(signs, "signs", (torch.int8,)),
        _dev(gamma, "gamma", (torch.float32,)), _dev(codebook, "codebook", (torch.float32,)),
        _dev(o, "scores", (torch.float32,)), P, B, S, D, codebook.numel(), PATHS[path], _stream()))
    return o if (out is not None or A.dim() == 3) else o.view(B, S)


def scores_packed(A, T, idx_plane, sign_plane, gamma_f16, codebook, idx_bits, path="auto", out=None):
    """Scores from a bit-packed cache: idx_plane uint8 [P,S,D*bits/8], sign_plane uint8
    [P,S,D/8], gamma_f16 float16 [P,S]."""
    P, B, D = _as3(A)
    S, row = _keys3(idx_plane, P)
    if row * 8 != D * idx_bits or sign_plane.shape[-1] * 8 != D or gamma_f16.numel() != P * S:
        raise ValueError("inconsistent packed key shapes")
    o = _scores_out(out, P, B, S, A)
    _check("tq_scores_packed", lib().tq_scores_packed(
        _dev(A, "A", (torch.float32,)), _dev(T, "T", (torch.float32,)),
        _dev(idx_plane, "idx_plane", (torch.uint8,)), _dev(sign_plane, "sign_plane", (torch.uint8,)),
        _dev(gamma_f16, "gamma_f16", (torch.float16,)), _dev(codebook, "codebook", (torch.float32,)),
        _dev(o, "scores", (torch.float32,)), P, B, S, D, idx_bits, PATHS[path], _stream()))
    return o if (out is not None or A.dim() == 3) else o.view(B, S)


def scores_mse(A, idx_plane, norm_f16, codebook, idx_bits, norm_correction=False, out=None):
    """MSE-only scores: A = Pi q [P,B,D] fp32, idx_plane uint8 [P,S,D*bits/8] (codes of
    the rotated unit keys), norm_f16 float16 [P,S] (key lengths)."""
    P, B, D = _as3(A)
    S, row = _keys3(idx_plane, P)
    if row * 8 != D * idx_bits or norm_f16.numel() != P * S:
        raise ValueError("inconsistent packed key shapes")
    o = _scores_out(out, P, B, S, A)
    _check("tq_scores_mse", lib().tq_scores_mse(
        _dev(A, "A", (torch.float32,)), _dev(idx_plane, "idx_plane", (torch.uint8,)),
        _dev(norm_f16, "norm_f16", (torch.float16,)), _dev(codebook, "codebook", (torch.float32,)),
        _dev(o, "scores", (torch.float32,)), P, B, S, D, idx_bits, 1 if norm_correction else 0,
        _stream()))
    return o if (out is not None or A.dim() == 3) else o.view(B, S)


def decode_mse(A, k_plane, k_norm, k_codebook, k_bits, v_plane, v_norm, v_codebook, v_bits, Pi_v,
               scale=None, workspace=None, out=None):
    """Attention output over MSE-quantized keys and values (rotated-domain decode).
    A = Pi_k q [P,B,128]; planes uint8 [P,S,128*bits/8]; norms float16 [P,S];
    Pi_v [H,128,128] (or [128,128]).  Returns [P,B,128] (or [B,128])."""
    P, B, D = _as3(A)
    S, krow = _keys3(k_plane, P)
    _, vrow = _keys3(v_plane, P)
    H = 1 if Pi_v.dim() == 2 else Pi_v.shape[0]
    if krow * 8 != D * k_bits or vrow * 8 != D * v_bits or k_norm.numel() != P * S or v_norm.numel() != P * S:
        raise ValueError("inconsistent key/value shapes")
    need = int(lib().tq_decode_workspace_bytes(P, B, S, D))
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=A.device, dtype=torch.uint8)
    o = out if out is not None else torch.empty((P, B, D), device=A.device, dtype=torch.float32)
    if scale is None:
        scale = 1.0 / float(D) ** 0.5
    _check("tq_decode_mse", lib().tq_decode_mse(
        _dev(A, "A", (torch.float32,)), _dev(k_plane, "k_plane", (torch.uint8,)),
        _dev(k_norm, "k_norm", (torch.float16,)), _dev(k_codebook, "k_codebook", (torch.float32,)), k_bits,
        _dev(v_plane, "v_plane", (torch.uint8,)), _dev(v_norm, "v_norm", (torch.float16,)),
        _dev(v_codebook, "v_codebook", (torch.float32,)), v_bits, _dev(Pi_v, "Pi_v", (torch.float32,)),
        _dev(o, "out", (torch.float32,)), P, H, B, S, D, float(scale),
        _dev(workspace, "workspace", (torch.uint8,)), workspace.numel(), _stream()))
    return o if (out is not None or A.dim() == 3) else o.view(B, D)


def decode_prod(A, T, k_plane, k_sign_plane, k_gamma, k_codebook, k_bits, v_plane, v_norm, v_codebook,
                v_bits, Pi_v, scale=None, workspace=None, out=None):
    """Attention output over a TurboQuant_prod key cache and MSE-quantized values.
    A, T [P,B,128] from prepare_queries; k_plane uint8 [P,S,128*k_bits/8], k_sign_plane
    uint8 [P,S,16], k_gamma float16 [P,S]; values as for decode_mse.  Returns [P,B,128]
    (or [B,128])."""
    P, B, D = _as3(A)
    if _as3(T) != (P, B, D):
        raise ValueError("A and T must have the same shape")
    S, krow = _keys3(k_plane, P)
    S2, srow = _keys3(k_sign_plane, P)
    _, vrow = _keys3(v_plane, P)
    H = 1 if Pi_v.dim() == 2 else Pi_v.shape[0]
    if (krow * 8 != D * k_bits or srow * 8 != D or S2 != S or vrow * 8 != D * v_bits
            or k_gamma.numel() != P * S or v_norm.numel() != P * S):
        raise ValueError("inconsistent key/value shapes")
    need = int(lib().tq_decode_workspace_bytes(P, B, S, D))
    if workspace is None:
        workspace = torch.empty(max(need, 16), device=A.device, dtype=torch.uint8)
    o = out if out is not None else torch.empty((P, B, D), device=A.device, dtype=torch.float32)
    if scale is None:
        scale = 1.0 / float(D) ** 0.5
    _check("tq_decode_prod", lib().tq_decode_prod(
        _dev(A, "A", (torch.float32,)), _dev(T, "T", (torch.float32,)), _dev(k_plane, "k_plane", (torch.uint8,)),
        _dev(k_sign_plane, "k_sign_plane", (torch.uint8,)), _dev(k_gamma, "k_gamma", (torch.float16,)),
        _dev(k_codebook, "k_codebook", (torch.float32,)), k_bits,
        _dev(v_plane, "v_plane", (torch.uint8,)), _dev(v_norm, "v_norm", (torch.float16,)),
        _dev(v_codebook, "v_codebook", (torch.float32,)), v_bits, _dev(Pi_v, "Pi_v", (torch.float32,)),
        _dev(o, "out", (torch.float32,)), P, H, B, S, D, float(scale),
        _dev(workspace, "workspace", (torch.uint8,)), workspace.numel(), _stream()))
    return o if (out is not None or A.dim() == 3) else o.view(B, D)


def prepare_queries_split(Q, channels, Pi_out, Pi_reg, out=None):
    """A_out = Pi_out q[channels], A_reg = Pi_reg q[other channels] for Q [P,B,D] (or [B,D])
    f32/bf16; channels int32 [n_out] increasing; Pi_out [H,n_out,n_out] (or 2-D), Pi_reg
    [H,n_reg,n_reg].  Returns (A_out, A_reg) fp32."""
    P, B, D = _as3(Q)
    n_out = channels.numel()
    H = 1 if Pi_out.dim() == 2 else Pi_out.shape[0]
    lead = Q.shape[:-1]
    if out is None:
        out = (torch.empty(lead + (n_out,), device=Q.device, dtype=torch.float32),
               torch.empty(lead + (D - n_out,), device=Q.device, dtype=torch.float32))
    A_out, A_reg = out
    _check("tq_prepare_queries_split", lib().tq_prepare_queries_split(
        _dev(Q, "Q", tuple(QTYPE)), QTYPE[Q.dtype], _dev(channels, "channels", (torch.int32,)),
        _dev(Pi_out, "Pi_out", (torch.float32,)), _dev(Pi_reg, "Pi_reg", (torch.float32,)),
        _dev(A_out, "A_out", (torch.float32,)), _dev(A_reg, "A_reg", (torch.float32,)), P, H, B, D, n_out,
        _stream()))
    return A_out, A_reg


def scores_split(A_out, A_reg, out_plane, out_norm, out_codebook, out_bits, reg_plane, reg_norm,
                 reg_codebook, reg_bits, out=None):
    """Scores of the outlier-split cache: [P,B,S] (or [B,S])."""
    P, B, n_out = _as3(A_out)
    _, _, n_reg = _as3(A_reg)
    S, orow = _keys3(out_plane, P)
    S2, rrow = _keys3(reg_plane, P)
    if (S2 != S or orow * 8 != n_out * out_bits or rrow * 8 != n_reg * reg_bits
            or out_norm.numel() != P * S or reg_norm.numel() != P * S):
        raise ValueError("inconsistent split cache shapes")
    o = _scores_out(out, P, B, S, A_out)
    _check("tq_scores_split", lib().tq_scores_split(
        _dev(A_out, "A_out", (torch.float32,)), _dev(A_reg, "A_reg", (torch.float32,)),
        _dev(out_plane, "out_plane", (torch.uint8,)), _dev(out_norm, "out_norm", (torch.float16,)),
        _dev(out_codebook, "out_codebook", (torch.float32,)), out_bits,
        _dev(reg_plane, "reg_plane", (torch.uint8,)), _dev(reg_norm, "reg_norm", (torch.float16,)),
        _dev(reg_codebook, "reg_codebook", (torch.float32,)), reg_bits, _dev(o, "scores", (torch.float32,)),
        P, B, S, n_out, n_reg, _stream()))
    return o if (out is not None or A_out.dim() == 3) else o.view(B, S)


def workspace_bytes(P: int, B: int, D: int) -> int:
    return int(lib().tq_workspace_bytes(P, B, D))


def _workspace(ws, P, B, D, like):
    need = workspace_bytes(P, B, D)
    if ws is None:
        ws = torch.empty(need, device=like.device, dtype=torch.uint8)
    return ws


def solve(Q, K_idx, signs, gamma, Pi, S_mat, codebook, path="auto", workspace=None, out=None):
    """Fused query transform + scoring over an unpacked cache."""
    P, B, D = _as3(Q)
    H = 1 if Pi.dim() == 2 else Pi.shape[0]
    S, Dk = _keys3(K_idx, P)
    if Dk != D:
        raise ValueError("inconsistent key shapes")
    ws = _workspace(workspace, P, B, D, Q)
    o = _scores_out(out, P, B, S, Q)
    _check("tq_solve", lib().tq_solve(
        _dev(Q, "Q", QTYPE), QTYPE[Q.dtype], _dev(K_idx, "K_idx", (torch.uint8,)),
        _dev(signs, "signs", (torch.int8,)), _dev(gamma, "gamma", (torch.float32,)),
        _dev(Pi, "Pi", (torch.float32,)), _dev(S_mat, "S_mat", (torch.float32,)),
        _dev(codebook, "codebook", (torch.float32,)), _dev(o, "scores", (torch.float32,)),
        P, H, B, S, D, codebook.numel(), _dev(ws, "workspace", (torch.uint8,)), ws.numel(),
        PATHS[path], _stream()))
    return o if (out is not None or Q.dim() == 3) else o.view(B, S)


def solve_packed(Q, idx_plane, sign_plane, gamma_f16, Pi, S_mat, codebook, idx_bits, path="auto",
                 workspace=None, out=None):
    """Fused query transform + scoring over a bit-packed cache."""
    P, B, D = _as3(Q)
    H = 1 if Pi.dim() == 2 else Pi.shape[0]
    S, _ = _keys3(idx_plane, P)
    ws = _workspace(workspace, P, B, D, Q)
    o = _scores_out(out, P, B, S, Q)
    _check("tq_solve_packed", lib().tq_solve_packed(
        _dev(Q, "Q", QTYPE), QTYPE[Q.dtype], _dev(idx_plane, "idx_plane", (torch.uint8,)),
        _dev(sign_plane, "sign_plane", (torch.uint8,)), _dev(gamma_f16, "gamma_f16", (torch.float16,)),
        _dev(Pi, "Pi", (torch.float32,)), _dev(S_mat, "S_mat", (torch.float32,)),
        _dev(codebook, "codebook", (torch.float32,)), _dev(o, "scores", (torch.float32,)),
        P, H, B, S, D, idx_bits, _dev(ws, "workspace", (torch.uint8,)), ws.numel(),
        PATHS[path], _stream()))
    return o if (out is not None or Q.dim() == 3) else o.view(B, S)


def pack_indices(K_idx, bits, out=None):
    """uint8 codes [..., D] -> packed plane [..., D*bits/8]."""
    D = K_idx.shape[-1]
    n = K_idx.numel() // D
    o = out if out is not None else torch.empty((*K_idx.shape[:-1], D * bits // 8), device=K_idx.device, dtype=torch.uint8)
    _check("tq_pack_indices", lib().tq_pack_indices(
        _dev(K_idx, "K_idx", (torch.uint8,)), _dev(o, "idx_plane", (torch.uint8,)), n, D, bits, _stream()))
    return o


def unpack_indices(plane, D, bits, out=None):
    n = plane.numel() // (D * bits // 8)
    o = out if out is not None else torch.empty((*plane.shape[:-1], D), device=plane.device, dtype=torch.uint8)
    _check("tq_unpack_indices", lib().tq_unpack_indices(
        _dev(plane, "idx_plane", (torch.uint8,)), _dev(o, "K_idx", (torch.uint8,)), n, D, bits, _stream()))
    return o


def pack_signs(signs, out=None):
    D = signs.shape[-1]
    n = signs.numel() // D
    o = out if out is not None else torch.empty((*signs.shape[:-1], D // 8), device=signs.device, dtype=torch.uint8)
    _check("tq_pack_signs", lib().tq_pack_signs(
        _dev(signs, "signs", (torch.int8,)), _dev(o, "sign_plane", (torch.uint8,)), n, D, _stream()))
    return o


def unpack_signs(plane, D, out=None):
    n = plane.numel() // (D // 8)
    o = out if out is not None else torch.empty((*plane.shape[:-1], D), device=plane.device, dtype=torch.int8)
    _check("tq_unpack_signs", lib().tq_unpack_signs(
        _dev(plane, "sign_plane", (torch.uint8,)), _dev(o, "signs", (torch.int8,)), n, D, _stream()))
    return o


def lloyd_max_codebook(D: int, mse_bits: int, grid_points: int = 400_001, iterations: int = 300):
    """Lloyd-Max codebook (host computation in libtq), float32 numpy array of 2^mse_bits."""
    import numpy as np
    out = np.empty(1 << mse_bits, dtype=np.float32)
    _check("tq_lloyd_max_codebook", lib().tq_lloyd_max_codebook(
        D, mse_bits, grid_points, iterations, out.ctypes.data))
    return out


def haar_rotation(G):
    """Sign-fixed QR rotation of a float64 [D,D] numpy matrix (host computation in libtq)."""
    import numpy as np
    G = np.ascontiguousarray(G, dtype=np.float64)
    D = G.shape[0]
    out = np.empty((D, D), dtype=np.float32)
    _check("tq_haar_rotation", lib().tq_haar_rotation(G.ctypes.data, D, out.ctypes.data))
    return out


def compress_keys(keys, Pi, S_mat, codebook, gamma_dtype=torch.float32):
    """TurboQuant_prod compression on the GPU.  keys fp32 [P,S,D] (or [S,D]); Pi, S_mat
    [H,D,D] (or [D,D]).  Returns (K_idx uint8, signs int8, gamma fp32 or fp16)."""
    P, S, D = _as3(keys)
    H = 1 if Pi.dim() == 2 else Pi.shape[0]
    K_idx = torch.empty(keys.shape, device=keys.device, dtype=torch.uint8)
    signs = torch.empty(keys.shape, device=keys.device, dtype=torch.int8)
    gamma = torch.empty(keys.shape[:-1], device=keys.device, dtype=gamma_dtype)
    g32 = _dev(gamma, "gamma", (torch.float32,)) if gamma_dtype == torch.float32 else None
    g16 = _dev(gamma, "gamma", (torch.float16,)) if gamma_dtype == torch.float16 else None
    _check("tq_compress_keys", lib().tq_compress_keys(
        _dev(keys, "keys", (torch.float32,)), _dev(Pi, "Pi", (torch.float32,)),
        _dev(S_mat, "S_mat", (torch.float32,)), _dev(codebook, "codebook", (torch.float32,)),
        codebook.numel(), _dev(K_idx, "K_idx", (torch.uint8,)), _dev(signs, "signs", (torch.int8,)),
        g32, g16, P, H, S, D, _stream()))
    return K_idx, signs, gamma


def compress_keys_packed(keys, Pi, S_mat, codebook, idx_bits, out=None):
    """TurboQuant_prod compression on the GPU straight into the packed cache.  keys fp32
    [P,S,D] (or [S,D]); Pi, S_mat [H,D,D] (or [D,D]); codebook 2^idx_bits fp32.  Returns
    (idx_plane uint8 [..,S,D*idx_bits/8], sign_plane uint8 [..,S,D/8], gamma fp16 [..,S])."""
    P, S, D = _as3(keys)
    H = 1 if Pi.dim() == 2 else Pi.shape[0]
    lead = keys.shape[:-1]
    if out is None:
        out = (torch.empty(lead + (D * idx_bits // 8,), device=keys.device, dtype=torch.uint8),
               torch.empty(lead + (D // 8,), device=keys.device, dtype=torch.uint8),
               torch.empty(lead, device=keys.device, dtype=torch.float16))
    ip, sp, g = out
    _check("tq_compress_keys_packed", lib().tq_compress_keys_packed(
        _dev(keys, "keys", (torch.float32,)), _dev(Pi, "Pi", (torch.float32,)),
        _dev(S_mat, "S_mat", (torch.float32,)), _dev(codebook, "codebook", (torch.float32,)), idx_bits,
        _dev(ip, "idx_plane", (torch.uint8,)), _dev(sp, "sign_plane", (torch.uint8,)),
        _dev(g, "gamma", (torch.float16,)), P, H, S, D, _stream()))
    return ip, sp, g


class _PagedCacheStruct(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("k_plane", "k_norm", "v_plane", "v_norm", "Pi_k", "Pi_v", "k_codebook",
                                  "v_codebook")] + \
               [(n, _I) for n in ("n_pages", "H", "page_size", "D", "k_bits", "v_bits", "rot_heads")]


class PagedCache:
    """A paged cache of MSE-quantized keys and values: the handle the paged calls take, made
    once per layer.  k_plane uint8 [N,H,page,D*k_bits/8], k_norm float16 [N,H,page], v_plane
    and v_norm likewise; Pi_k, Pi_v fp32 [h,D,D] (or [D,D]), KV head i using rotation i % h;
    k_codebook, v_codebook fp32 of 2^bits ascending centroids.  D is 128, bits 2 to 4, page a
    power of two from 16 to 256.  The tensors stay the caller's (they may be written between
    calls, not resized); all are on one device, and the calls run there.  As everywhere in this
    library arrays begin on a 16-byte boundary, so a slice of lengths, rows or a page table may
    have to be copied first (TQ_ERR_MISALIGNED)."""

    __slots__ = ("k_plane", "k_norm", "v_plane", "v_norm", "Pi_k", "k_codebook", "Pi_v", "v_codebook", "device",
                 "H", "page_size", "D", "k_bits", "v_bits", "_struct", "_ref", "_index")

    def __init__(self, k_plane, k_norm, v_plane, v_norm, Pi_k, k_codebook, Pi_v, v_codebook):
        names = ("k_plane", "k_norm", "v_plane", "v_norm", "Pi_k", "Pi_v", "k_codebook", "v_codebook")
        tensors = (k_plane, k_norm, v_plane, v_norm, Pi_k, Pi_v, k_codebook, v_codebook)
        dtypes = (torch.uint8, torch.float16) * 2 + (torch.float32,) * 4
        ptrs = [_dev(t, n, (d,)) for t, n, d in zip(tensors, names, dtypes)]
        if any(t.device != k_plane.device for t in tensors):
            raise ValueError("the tensors of a cache must be on one device")
        if k_plane.dim() != 4 or v_plane.dim() != 4:
            raise ValueError("k_plane and v_plane must be [pages, H, page, bytes]")
        N, H, page, krow = k_plane.shape
        D = Pi_k.shape[-1]
        if (tuple(v_plane.shape[:3]) != (N, H, page) or tuple(k_norm.shape) != (N, H, page)
                or tuple(v_norm.shape) != (N, H, page)):
            raise ValueError("inconsistent page shapes")
        if Pi_k.dim() not in (2, 3) or tuple(Pi_k.shape[-2:]) != (D, D) or Pi_v.shape != Pi_k.shape:
            raise ValueError("Pi_k and Pi_v must be [h,D,D] or [D,D]")
        kb, vb = krow * 8 // D, v_plane.shape[3] * 8 // D
        if (krow * 8 != D * kb or v_plane.shape[3] * 8 != D * vb or k_codebook.numel() != 1 << kb
                or v_codebook.numel() != 1 << vb):
            raise ValueError("row bytes and codebook sizes do not match")
        self.k_plane, self.k_norm, self.v_plane, self.v_norm = k_plane, k_norm, v_plane, v_norm
        self.Pi_k, self.k_codebook, self.Pi_v, self.v_codebook = Pi_k, k_codebook, Pi_v, v_codebook
        self.device, self.H, self.page_size, self.D, self.k_bits, self.v_bits = k_plane.device, H, page, D, kb, vb
        self._struct = _PagedCacheStruct(*ptrs, N, H, page, D, kb, vb, 1 if Pi_k.dim() == 2 else Pi_k.shape[0])
        self._ref, self._index = ctypes.addressof(self._struct), k_plane.get_device()


def _on(index: int, t: torch.Tensor, name: str, dtype, shape) -> int:
    """Pointer of a tensor of a paged call: its type, device, shape and contiguity are checked."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the cache on cuda:{index}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _paged_call(name: str, index: int, *args) -> None:
    """Calls `name` on device `index` and that device's current stream."""
    fn = getattr(_lib or lib(), name)
    if index == torch.cuda.current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status != TQ_OK:
        raise TQError(name, status)


def _raw_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):         # the same handle, without a Stream object around it
    _raw_stream = torch._C._cuda_getCurrentRawStream       # noqa: F811


def _table(index: int, page_table: torch.Tensor) -> tuple[int, int, int]:
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be a [B, max_pages] tensor")
    B, M = page_table.shape
    return _on(index, page_table, "page_table", torch.int32, (B, M)), B, M


def _workspace_of(index: int, workspace, need: int):
    """The scratch of a paged call, its pointer and size.  The caller holds the tensor until the kernels are launched: memory
    given back before is what the allocator hands out next, to an output of the same call for one."""
    if workspace is None:
        workspace = torch.empty(need, device=torch.device("cuda", index), dtype=torch.uint8)
    n = workspace.numel()
    return workspace, _on(index, workspace, "workspace", torch.uint8, (n,)), n


def append_paged(K, V, rows, cache: PagedCache, page_table, mass=None, positions=None) -> None:
    """Quantises new tokens' keys and values and writes them to their slots.  K, V [n,H,D]
    fp32/bf16; rows int32 [n,3] of (sequence, slot, position), a negative sequence or slot
    skipping the row; page_table int32 [B,max_pages].  mass fp32 and positions int32 [B,H,S]
    (optional) get 0 and the position at the slots written.  No two rows may name one slot."""
    if not isinstance(K, torch.Tensor) or K.dim() != 3 or K.dtype not in QTYPE:
        raise ValueError("K must be a [n, H, D] fp32 or bf16 tensor")
    n, dev, H = K.shape[0], cache._index, cache.H
    shape = (n, H, cache.D)
    tp, B, M = _table(dev, page_table)
    S = 0
    for t in (mass, positions):
        if t is not None:
            S = t.shape[-1] if t.dim() == 3 else 0
            if S < 1:
                raise ValueError("mass and positions must be [B, H, S] tensors with S >= 1")
    _paged_call("tq_append_paged", dev, cache._ref, _on(dev, K, "K", K.dtype, shape), _on(dev, V, "V", K.dtype, shape),
                QTYPE[K.dtype], _on(dev, rows, "rows", torch.int32, (n, 3)), n, tp, B, M,
                None if mass is None else _on(dev, mass, "mass", torch.float32, (B, H, S)),
                None if positions is None else _on(dev, positions, "positions", torch.int32, (B, H, S)), S)


def decode_paged_workspace_bytes(B: int, H: int, G: int, S: int, with_mass: bool) -> int:
    return int(lib().tq_decode_paged_workspace_bytes(B, H, G, S, 1 if with_mass else 0))


def decode_paged(Q, cache: PagedCache, page_table, lengths, mass=None, scale=None, workspace=None, out=None):
    """Attention output of one new token per sequence over the paged cache.  Q [B,H*G,D]
    fp32/bf16 (query head i reads KV head i // G); page_table int32 [B,max_pages], lengths
    int32 [B].  mass fp32 [B,H,S] (optional): the weights each slot received, summed over its
    group's queries, are added to it.  scale defaults to 1/sqrt(D).  Returns Q's shape and
    type; zeros for a sequence of length 0.  Q's type decides the precision: fp32 accuracy for
    fp32, products of fp16 operands for bf16 (the logits keep fp32 accuracy with mass)."""
    if not isinstance(Q, torch.Tensor) or Q.dim() != 3 or Q.dtype not in QTYPE:
        raise ValueError("Q must be a [B, heads, D] fp32 or bf16 tensor")
    dev, H, D = cache._index, cache.H, cache.D
    tp, B, M = _table(dev, page_table)
    heads = Q.shape[1]
    if heads < H or heads % H:
        raise ValueError(f"{heads} query heads over {H} KV heads")
    G = heads // H
    shape, dtype = (B, heads, D), Q.dtype
    qp = _on(dev, Q, "Q", dtype, shape)
    S, mp = 0, None
    if mass is not None:
        S = mass.shape[-1] if mass.dim() == 3 else 0
        if S < 1:
            raise ValueError("mass must be a [B, H, S] tensor with S >= 1")
        mp = _on(dev, mass, "mass", torch.float32, (B, H, S))
    held, wp, wn = _workspace_of(dev, workspace, 0 if workspace is not None else
                                 decode_paged_workspace_bytes(B, H, G, S, mass is not None))
    if out is None:
        out = torch.empty_like(Q)
    _paged_call("tq_decode_paged", dev, cache._ref, qp, QTYPE[dtype], tp, _on(dev, lengths, "lengths", torch.int32, (B,)),
                B, G, M, 1.0 / D ** 0.5 if scale is None else float(scale), mp, S, _on(dev, out, "out", dtype, shape), wp, wn)
    return out


def evict_paged_workspace_bytes(B: int, H: int, S: int, budget: int) -> int:
    return int(lib().tq_evict_paged_workspace_bytes(B, H, S, budget))


def evict_paged(cache: PagedCache, page_table, lengths, seen, mass, positions, budget, recent, workspace=None,
                out=None):
    """Cuts each sequence and KV head to min(length, budget) slots: those whose position is at
    least seen - recent before the others, among either by mass, ties to the lower slot.  Kept rows behind the
    budget move to the slots given up.  lengths, seen int32 [B]; mass fp32, positions int32
    [B,H,S].  Returns (mass, positions) of the slots as they are now (`out`, or new tensors of
    0 and -1 behind the kept slots); `lengths` is the caller's to cut once all layers are done."""
    dev = cache._index
    tp, B, M = _table(dev, page_table)
    if not isinstance(mass, torch.Tensor) or mass.dim() != 3:
        raise ValueError("mass must be a [B, H, S] tensor")
    shape = (B, cache.H, mass.shape[-1])
    S = shape[2]
    mp, pp = _on(dev, mass, "mass", torch.float32, shape), _on(dev, positions, "positions", torch.int32, shape)
    budget, recent = max(-1, min(int(budget), S)), max(-1, min(int(recent), 2 ** 31 - 1))   # both fit an int
    if out is None:
        out = torch.zeros_like(mass), torch.full_like(positions, -1)
    held, wp, wn = _workspace_of(dev, workspace, 0 if workspace is not None else
                                 evict_paged_workspace_bytes(B, cache.H, S, budget))
    _paged_call("tq_evict_paged", dev, cache._ref, tp, _on(dev, lengths, "lengths", torch.int32, (B,)),
                _on(dev, seen, "seen", torch.int32, (B,)), B, M, mp, pp, S, budget, recent,
                _on(dev, out[0], "mass_out", torch.float32, shape),
                _on(dev, out[1], "positions_out", torch.int32, shape), wp, wn)
    return out


def _strided(index: int, t: torch.Tensor, name: str, dtype, shape) -> int:
    """Pointer of a [n, heads, D] tensor whose rows are dense: its type, device and shape are checked."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.stride(2) != 1 and shape[2] > 1:
        raise ValueError(f"{name} must be dense in its last dimension")
    return t.data_ptr()


_INV_TWO_PI = 0x28BE60DB9391054A7F09D5F47D4D377036D8A5664F10E410      # 1 / (2 pi) * 2^192


class Rotary:
    """The rotation of a model's queries and keys: the handle norm_rope takes, made once.  inv_freq:
    radians a position of each pair of coordinates (any sequence of floats, a multiple of 4 of
    them, taken in 64 bits).  axis: which of a token's positions turns each pair (time, height,
    width; default: the only one).  paired: pairs are coordinates (2i, 2i+1) instead of (i, i +
    pairs)."""

    __slots__ = ("turns", "axis", "pairs", "axes", "paired", "_index", "_ptrs")

    def __init__(self, inv_freq, device, axis=None, paired=False):
        import math
        freq = [float(f) for f in inv_freq]
        axes = [0] * len(freq) if axis is None else [int(a) for a in axis]
        if not freq or len(freq) % 4 or len(freq) > 128 or not all(math.isfinite(f) for f in freq):
            raise ValueError("inv_freq must hold a multiple of 4 finite numbers, 128 at most")
        if len(axes) != len(freq) or min(axes) < 0 or max(axes) > 7:
            raise ValueError("axis must name one of up to 8 positions for each frequency")
        ratios = [f.as_integer_ratio() for f in freq]
        bits = [(a * _INV_TWO_PI // b >> 128) & 0xffffffffffffffff for a, b in ratios]      # of 2^64 a turn
        self.turns = torch.tensor([b - (1 << 64) if b >> 63 else b for b in bits], dtype=torch.int64).to(device)
        self.axis = torch.tensor(axes, dtype=torch.uint8).to(device)
        self.pairs, self.axes, self.paired, self._index = len(freq), max(axes) + 1, bool(paired), self.turns.get_device()
        self._ptrs = _dev(self.turns, "turns", (torch.int64,)), _dev(self.axis, "axis", (torch.uint8,))


def norm_rope(q, k, positions, rotary: Rotary, q_weight=None, k_weight=None, eps=1e-6, out=None):
    """Root-mean-square norm of every head of q [n,Hq,D] and k [n,Hk,D] (fp32/bf16, dense in their last
    dimension, as parts of a joint projection are; k may be None), times q_weight and k_weight [D]
    (fp32/bf16; None: no norm), then rotated by positions int32 [n] or [n,axes].  Returns dense (q, k)
    of the same type; `out`: a pair to write to, which may be q and k themselves where these are dense."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3 or q.dtype not in QTYPE:
        raise ValueError("q must be a [n, heads, D] fp32 or bf16 tensor")
    dev, dtype = rotary._index, q.dtype
    n, Hq, D = q.shape
    if not isinstance(positions, torch.Tensor) or positions.dim() not in (1, 2):
        raise ValueError("positions must be a [n] or [n, axes] tensor")
    axes = 1 if positions.dim() == 1 else positions.shape[1]
    if axes < rotary.axes:
        raise ValueError(f"positions have {axes} axes, the rotation takes {rotary.axes}")
    qp, Hk, kp, ks = _strided(dev, q, "q", dtype, (n, Hq, D)), 0, None, (0, 0)
    if k is not None:
        if not isinstance(k, torch.Tensor) or k.dim() != 3:
            raise ValueError("k must be a [n, heads, D] tensor or None")
        Hk = k.shape[1]
        kp, ks = _strided(dev, k, "k", dtype, (n, Hk, D)), k.stride()
    weights, wtype = [], None
    for t, name in ((q_weight, "q_weight"), (k_weight if Hk else None, "k_weight")):
        if t is not None:
            if t.dtype not in QTYPE or wtype not in (None, t.dtype):
                raise TypeError("q_weight and k_weight must be fp32 or bf16, both alike")
            wtype = t.dtype
        weights.append(None if t is None else _on(dev, t, name, t.dtype, (D,)))
    if out is None:
        dense = torch.contiguous_format
        out = torch.empty_like(q, memory_format=dense), None if k is None else torch.empty_like(k, memory_format=dense)
    qs = q.stride()
    _paged_call("tq_norm_rope", dev, qp, qs[0], qs[1], kp, ks[0], ks[1], QTYPE[dtype], weights[0], weights[1], QTYPE.get(wtype, 0),
                eps, _on(dev, positions, "positions", torch.int32, (n,) if positions.dim() == 1 else (n, axes)), axes,
                rotary._ptrs[0], rotary._ptrs[1], rotary.pairs, 1 if rotary.paired else 0,
                _on(dev, out[0], "q_out", dtype, (n, Hq, D)),
                None if k is None else _on(dev, out[1], "k_out", dtype, (n, Hk, D)), n, Hq, Hk, D)
    return out


class _Int8CacheStruct(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("k_codes", "v_codes", "exponents")] + [(n, _I) for n in ("n_pages", "H", "page_size", "D")]


class Int8Cache:
    """A paged cache of keys and values in 8 bits with an exponent for each 16 slots of a head: the handle
    the int8 calls take, made once per layer.  k_codes, v_codes uint8 [N,H,page,D], exponents int8
    [N,H,page/16,2]; D 64 or 128, page a power of two from 16 to 256.  Fresh pages need no
    initial values.  The tensors stay the caller's and every array of a call begins on a 16-byte boundary (slices of starts,
    lengths and positions too), as for PagedCache.

    The calls share a step's form: tokens one behind the other, those of sequence b from starts[b] to
    starts[b+1] (int32 [B+1]), at its slots from lengths[b] (int32 [B], slots in use before the step) on."""

    __slots__ = ("k_codes", "v_codes", "exponents", "device", "H", "page_size", "D", "_struct", "_ref", "_index")

    def __init__(self, k_codes, v_codes, exponents):
        ptrs = [_dev(t, n, (d,)) for t, n, d in ((k_codes, "k_codes", torch.uint8), (v_codes, "v_codes", torch.uint8),
                                                 (exponents, "exponents", torch.int8))]
        if k_codes.device != v_codes.device or k_codes.device != exponents.device:
            raise ValueError("the tensors of a cache must be on one device")
        if k_codes.dim() != 4 or v_codes.shape != k_codes.shape:
            raise ValueError("k_codes and v_codes must be [pages, H, page, D]")
        N, H, page, D = k_codes.shape
        if tuple(exponents.shape) != (N, H, page // 16, 2):
            raise ValueError("exponents must be [pages, H, page / 16, 2]")
        self.k_codes, self.v_codes, self.exponents = k_codes, v_codes, exponents
        self.device, self.H, self.page_size, self.D = k_codes.device, H, page, D
        self._struct = _Int8CacheStruct(*ptrs, N, H, page, D)
        self._ref, self._index = ctypes.addressof(self._struct), k_codes.get_device()


def _step(index: int, starts, lengths, B: int) -> tuple[int, int]:
    return _on(index, starts, "starts", torch.int32, (B + 1,)), _on(index, lengths, "lengths", torch.int32, (B,))


def append_int8(K, V, starts, cache: Int8Cache, page_table, lengths) -> None:
    """Writes a step's keys and values to their slots.  K, V [n,H,D] fp32/bf16, heads dense, tokens at any
    stride (parts of a joint projection); page_table int32 [B,max_pages].  The codes do not depend on
    how a sequence's tokens are cut into steps."""
    if not isinstance(K, torch.Tensor) or K.dim() != 3 or K.dtype not in QTYPE:
        raise ValueError("K must be a [n, H, D] fp32 or bf16 tensor")
    dev, H, D, n = cache._index, cache.H, cache.D, K.shape[0]
    tp, B, M = _table(dev, page_table)
    ptrs = []
    for t, name in ((K, "K"), (V, "V")):
        ptrs += [_strided(dev, t, name, K.dtype, (n, H, D)), t.stride(0)]
        if H > 1 and t.stride(1) != D:
            raise ValueError(f"the heads of {name} must be dense")
    _paged_call("tq_append_int8", dev, cache._ref, *ptrs, QTYPE[K.dtype], *_step(dev, starts, lengths, B), n, tp, B, M)


def read_int8(cache: Int8Cache, page_table, starts, lengths, n: int, dtype=torch.bfloat16, out=None):
    """The values of n slots, keys and values [n,H,D] (exact in fp32 and bf16): those of sequence b from slot
    lengths[b] on in rows starts[b] to starts[b+1].  `out`: a pair to write to, whose other rows stay."""
    if dtype not in QTYPE:
        raise ValueError("dtype must be fp32 or bf16")
    dev, shape = cache._index, (int(n), cache.H, cache.D)
    tp, B, M = _table(dev, page_table)
    if out is None:
        out = torch.empty(shape, device=cache.device, dtype=dtype)
        out = out, torch.empty_like(out)
    _paged_call("tq_read_int8", dev, cache._ref, _on(dev, out[0], "K", dtype, shape), _on(dev, out[1], "V", dtype, shape),
                QTYPE[dtype], *_step(dev, starts, lengths, B), shape[0], tp, B, M)
    return out


def attend_int8_workspace_bytes(n: int, B: int, H: int, G: int, D: int) -> int:
    return int(lib().tq_attend_int8_workspace_bytes(n, B, H, G, D))


def attend_int8(Q, starts, cache: Int8Cache, page_table, lengths, window=None, sinks=0, scale=None, workspace=None, out=None):
    """Attention of a step's tokens over the cache, up to their own slots (append_int8 first).  Q [n,H*G,D]
    fp32/bf16 (query head i reads KV head i // G).  window: how many slots up to its own a token sees
    (None: all), besides the first `sinks` of its sequence.  scale defaults to 1/sqrt(D).  Returns Q's
    shape and type; `out`: a tensor to write to, whose rows behind the last sequence's stay."""
    if not isinstance(Q, torch.Tensor) or Q.dim() != 3 or Q.dtype not in QTYPE:
        raise ValueError("Q must be a [n, heads, D] fp32 or bf16 tensor")
    dev, H, D, dtype = cache._index, cache.H, cache.D, Q.dtype
    tp, B, M = _table(dev, page_table)
    n, heads = Q.shape[0], Q.shape[1]
    if heads < H or heads % H:
        raise ValueError(f"{heads} query heads over {H} KV heads")
    if window is not None and not 0 < window < 2 ** 31 or not 0 <= sinks < 2 ** 31:
        raise ValueError("window must be positive or None, sinks not negative, both below 2^31")
    G, shape = heads // H, (n, heads, D)
    qp = _on(dev, Q, "Q", dtype, shape)
    held, wp, wn = _workspace_of(dev, workspace, 0 if workspace is not None else attend_int8_workspace_bytes(n, B, H, G, D))
    if out is None:
        out = torch.empty_like(Q)
    _paged_call("tq_attend_int8", dev, cache._ref, qp, QTYPE[dtype], *_step(dev, starts, lengths, B), n, G, tp, B, M,
                0 if window is None else window, sinks, 1.0 / D ** 0.5 if scale is None else float(scale),
                _on(dev, out, "out", dtype, shape), wp, wn)
    return out
