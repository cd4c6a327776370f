"""ctypes binding of ``libstce.so`` (argument marshalling only).

Every step of the scoring path runs in the HIP library; this module checks
tensor shapes/dtypes/devices, allocates outputs and workspaces with torch and
passes raw device pointers plus the current HIP stream to the C ABI declared
in ``include/stce.h``.  There is no fallback: without the built library every
entry point raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libstce.so")

STATUS_NONE = (1 << 63) - 1
FIELDS = {1: "temperature", 2: "top_k", 3: "top_p", 4: "min_p", 5: "target"}
FLAG_VALID, FLAG_FILTERED, FLAG_IN_SUPPORT, FLAG_IGNORED, FLAG_LISTED = 1, 2, 4, 8, 32
PROBLEM_IGNORE_INDEX, PROBLEM_PRE_GEMM_TEMPERATURE, PROBLEM_BF16_LANE, PROBLEM_RECOMPUTE_ALL = 1, 2, 4, 8
LANES = {"fp32": 0, "bf16": PROBLEM_BF16_LANE}
# a 32-byte record, then (after all T records) a 64-byte tile list, then a
# support list of NSP (token id, key) pairs
RECORD_BYTES = 32
NTILE = 31
NSP = 128
STATE_BYTES_PER_ROW = RECORD_BYTES + 2 * (1 + NTILE) + 8 * NSP
DT_BF16, DT_F32, DT_FP8, DT_F16 = 1, 2, 3, 4
VALUE_DTYPES = {torch.bfloat16: DT_BF16, torch.float16: DT_F16, torch.float32: DT_F32}
# dtypes a weight of e4m3 codes may come in (the fp8 lane)
FP8_WEIGHT_DTYPES = (torch.uint8, torch.float8_e4m3fn)

SYMBOLS = (
    "stce_state_bytes", "stce_workspace_bytes", "stce_forward", "stce_backward",
    "stce_scaled_logits", "stce_support_from_logits", "stce_support_workspace_bytes",
    "stce_decode_state", "stce_status_string", "stce_last_error", "stce_profile_attach", "stce_schedule",
    "stce_policy_loss", "stce_forward_with_side", "stce_fused_workspace_bytes", "stce_fused_policy_step",
    "stce_recompute_keys", "stce_forward_noalloc", "stce_noalloc_scratch_bytes", "stce_fp8_quantize_rows",
    "stce_token_workspace_bytes", "stce_token_logprobs", "stce_token_logprobs_backward",
    "stce_fp8_quantize_blocks", "stce_fp8_block_matmul_workspace_bytes", "stce_fp8_block_matmul",
)
KERNEL_KINDS = {1: "validate", 2: "projection", 3: "select", 4: "dlogits", 5: "grad_weight",
                6: "grad_hidden", 7: "transpose", 8: "partials", 9: "policy_loss", 10: "dz_keys",
                11: "split_sum", 12: "prescale", 13: "classify", 14: "sparse_grad_weight",
                15: "sparse_grad_hidden", 16: "reproject", 17: "quantize", 18: "tile_lists",
                19: "tile_recompute", 20: "listed_entries", 21: "token_logprobs", 22: "token_merge",
                23: "token_grad", 24: "quantize_blocks", 25: "block_matmul"}
QUANT_TILE, QUANT_TRANSPOSE = 1, 2
FP8_BLOCK = 128
PG_OBJECTIVES = {"cispo": 1, "clip": 2}


class Problem(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int64), ("H", ctypes.c_int64), ("V", ctypes.c_int64),
        ("dtype", ctypes.c_int32), ("flags", ctypes.c_int32),
        ("hidden", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("target", ctypes.c_void_p),
        ("temperature", ctypes.c_void_p), ("top_k", ctypes.c_void_p), ("top_p", ctypes.c_void_p),
        ("min_p", ctypes.c_void_p), ("chunk_rows", ctypes.c_int64), ("vocab_slice", ctypes.c_int64),
        ("ignore_index", ctypes.c_int64), ("pre_gemm_temperature", ctypes.c_float),
        ("weight_scale", ctypes.c_void_p),
    ]


class RowInfo(ctypes.Structure):
    _fields_ = [
        ("key_thr", ctypes.c_uint32), ("id_thr", ctypes.c_int32), ("n", ctypes.c_int32),
        ("flags", ctypes.c_uint32), ("lse_support", ctypes.c_float), ("lse_full", ctypes.c_float),
        ("row_max", ctypes.c_float), ("target_key", ctypes.c_float),
    ]


class Profile(ctypes.Structure):
    _fields_ = [("capacity", ctypes.c_int32), ("count", ctypes.c_int32),
                ("start", ctypes.POINTER(ctypes.c_void_p)), ("stop", ctypes.POINTER(ctypes.c_void_p)),
                ("kind", ctypes.POINTER(ctypes.c_int32))]


class PgParams(ctypes.Structure):
    _fields_ = [
        ("objective", ctypes.c_int32), ("eps_low", ctypes.c_float), ("eps_high", ctypes.c_float),
        ("scale", ctypes.c_float), ("advantages", ctypes.c_void_p), ("old_logprob", ctypes.c_void_p),
        ("state", ctypes.c_void_p),
    ]


class SideOutputs(ctypes.Structure):
    _fields_ = [("lse_full", ctypes.c_void_p), ("entropy_full", ctypes.c_void_p),
                ("entropy_support", ctypes.c_void_p)]


class TokenProblem(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int64), ("V", ctypes.c_int64), ("dtype", ctypes.c_int32), ("flags", ctypes.c_int32),
        ("logits", ctypes.c_void_p), ("ld", ctypes.c_int64), ("temperature", ctypes.c_void_p),
        ("tokens", ctypes.c_void_p), ("K", ctypes.c_int32), ("top_n", ctypes.c_int32),
        ("ignore_index", ctypes.c_int64),
    ]


class TokenOutputs(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("logprob", "lse", "entropy", "top_logprob", "top_id", "stats")]


class BlockMatmul(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("a", ctypes.c_void_p), ("lda", ctypes.c_int64), ("a_scale", ctypes.c_void_p),
        ("a_row_stride", ctypes.c_int64), ("a_block_stride", ctypes.c_int64),
        ("b", ctypes.c_void_p), ("ldb", ctypes.c_int64), ("b_scale", ctypes.c_void_p),
        ("b_row_stride", ctypes.c_int64), ("b_block_stride", ctypes.c_int64),
        ("b_rows", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("out", ctypes.c_void_p),
        ("ldo", ctypes.c_int64), ("accumulate", ctypes.c_int32),
    ]


class StceError(RuntimeError):
    pass


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the HIP library (once) and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise StceError(f"{path} is not built: run sampling_transform_logprob_amd/build.py")
    L = ctypes.CDLL(path)
    P, vp, i64, i32, sz = ctypes.POINTER(Problem), ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    sig = {
        "stce_state_bytes": (sz, [i64]),
        "stce_workspace_bytes": (ctypes.c_int, [P, ctypes.POINTER(sz), ctypes.POINTER(sz)]),
        "stce_forward": (ctypes.c_int, [P, vp, vp, vp, vp, sz, vp]),
        "stce_backward": (ctypes.c_int, [P, vp, vp, vp, vp, i32, vp, vp, sz, vp]),
        "stce_recompute_keys": (ctypes.c_int, [P, vp, vp, vp, vp, sz, vp]),
        "stce_forward_noalloc": (ctypes.c_int, [P, vp, vp, vp, vp]),
        "stce_noalloc_scratch_bytes": (sz, []),
        "stce_fp8_quantize_rows": (ctypes.c_int, [vp, i64, i64, vp, vp, vp]),
        "stce_scaled_logits": (ctypes.c_int, [P, i64, i64, vp, vp, sz, vp]),
        "stce_support_from_logits": (ctypes.c_int, [vp, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]),
        "stce_support_workspace_bytes": (sz, [i64, i64]),
        "stce_decode_state": (ctypes.c_int, [vp, i64, ctypes.POINTER(RowInfo)]),
        "stce_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "stce_last_error": (ctypes.c_char_p, []),
        "stce_profile_attach": (ctypes.c_int, [ctypes.POINTER(Profile)]),
        "stce_schedule": (ctypes.c_int, [P, ctypes.POINTER(i64), ctypes.POINTER(i64)]),
        "stce_policy_loss": (ctypes.c_int, [ctypes.POINTER(PgParams), i64, vp, vp, vp, vp, vp]),
        "stce_forward_with_side": (ctypes.c_int, [P, vp, vp, ctypes.POINTER(SideOutputs), vp, vp, sz, vp]),
        "stce_fused_workspace_bytes": (ctypes.c_int, [P, ctypes.POINTER(sz), ctypes.POINTER(sz)]),
        "stce_fused_policy_step": (ctypes.c_int, [P, ctypes.POINTER(PgParams), vp, vp, vp, vp,
                                                  ctypes.POINTER(SideOutputs), vp, vp, i32, vp, vp, sz, vp]),
        "stce_token_workspace_bytes": (ctypes.c_int, [ctypes.POINTER(TokenProblem), ctypes.POINTER(sz)]),
        "stce_token_logprobs": (ctypes.c_int, [ctypes.POINTER(TokenProblem), ctypes.POINTER(TokenOutputs), vp, vp, sz,
                                               vp]),
        "stce_token_logprobs_backward": (ctypes.c_int, [ctypes.POINTER(TokenProblem), vp, vp, vp, vp, vp, i64, vp]),
        "stce_fp8_quantize_blocks": (ctypes.c_int, [vp, i32, i64, i64, i64, i32, vp, i64, vp, vp]),
        "stce_fp8_block_matmul_workspace_bytes": (ctypes.c_int, [ctypes.POINTER(BlockMatmul), ctypes.POINTER(sz)]),
        "stce_fp8_block_matmul": (ctypes.c_int, [ctypes.POINTER(BlockMatmul), vp, sz, vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype, f.argtypes = res, args
    _lib = L
    return L


def _check(status: int) -> None:
    if status != 0:
        L = load()
        raise StceError(f"{L.stce_status_string(status).decode()}: {L.stce_last_error().decode()}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream() -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _meta(name, t, T, dtype, device):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor or None")
    if t.dim() != 1 or t.shape[0] != T:
        # over-length (or short) per-row metadata is an error, never truncated
        raise ValueError(f"{name} must have shape [{T}], got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t.contiguous()


def make_problem(hidden, weight, target, temperature=None, top_k=None, top_p=None, min_p=None,
                 chunk_rows: int = 0, vocab_slice: int = 0, ignore_index: Optional[int] = None,
                 pre_gemm_temperature: Optional[float] = None, lane: str = "fp32",
                 weight_scale: Optional[torch.Tensor] = None, recompute_all: bool = False):
    """Checked ``stce_problem`` plus the tensors it points into (kept alive).

    ``temperature`` is the per-row tensor applied to the logits after the
    product; ``pre_gemm_temperature`` is instead one scalar applied to the
    hidden states before it (the two do not combine).  ``lane="bf16"`` runs
    the bf16 value program (bf16 keys; the logprob, still an fp32 tensor,
    holds bf16 values, so ``.bfloat16()`` is exact).  A weight of e4m3 codes
    (``torch.uint8`` or ``torch.float8_e4m3fn``) with ``weight_scale`` (fp32
    [V]) and bf16 hidden states selects the fp8 lane."""
    if lane not in LANES:
        raise ValueError(f"lane must be one of {tuple(LANES)}")
    if pre_gemm_temperature is not None and temperature is not None:
        raise ValueError("pass either a per-row temperature tensor or pre_gemm_temperature, not both")
    if hidden.dim() != 2 or weight.dim() != 2 or hidden.shape[1] != weight.shape[1]:
        raise ValueError(f"hidden [T, H] and weight [V, H] expected, got {tuple(hidden.shape)}, {tuple(weight.shape)}")
    if weight.dtype in FP8_WEIGHT_DTYPES:
        if hidden.dtype != torch.bfloat16:
            raise TypeError(f"the fp8 lane takes bf16 hidden states, got {hidden.dtype}")
        if weight_scale is None:
            raise ValueError("an e4m3 weight needs weight_scale (fp32 [V])")
        dt = DT_FP8
        weight = weight.view(torch.uint8)
    else:
        if weight_scale is not None:
            raise ValueError("weight_scale is for an e4m3 weight only")
        if hidden.dtype != weight.dtype:
            raise TypeError(f"hidden ({hidden.dtype}) and weight ({weight.dtype}) must share a dtype")
        dt = {torch.bfloat16: DT_BF16, torch.float32: DT_F32}.get(hidden.dtype)
        if dt is None:
            raise TypeError(
                f"unsupported LM-head dtype {hidden.dtype}: scoring takes bf16 or fp32 hidden/weight, or an "
                "e4m3 weight with per-row scales (the fp8 lane)")
    if hidden.device.type != "cuda" or weight.device != hidden.device:
        raise ValueError("hidden and weight must be on the same GPU")
    T, H = hidden.shape
    V = weight.shape[0]
    dev = hidden.device
    hidden, weight = hidden.contiguous(), weight.contiguous()
    if weight_scale is not None:
        weight_scale = _meta("weight_scale", weight_scale, V, torch.float32, dev)
    target = _meta("target", target, T, torch.int64, dev)
    if target is None:
        raise ValueError("target is required")
    keep = [hidden, weight, target,
            _meta("temperature", temperature, T, torch.float32, dev),
            _meta("top_k", top_k, T, torch.int32, dev),
            _meta("top_p", top_p, T, torch.float32, dev),
            _meta("min_p", min_p, T, torch.float32, dev)]
    flags = (0 if ignore_index is None else PROBLEM_IGNORE_INDEX) | LANES[lane]
    if pre_gemm_temperature is not None:
        flags |= PROBLEM_PRE_GEMM_TEMPERATURE
    if recompute_all:
        flags |= PROBLEM_RECOMPUTE_ALL
    prob = Problem(T, H, V, dt, flags, *[t.data_ptr() if t is not None else None for t in keep], chunk_rows,
                   vocab_slice, 0 if ignore_index is None else int(ignore_index),
                   0.0 if pre_gemm_temperature is None else float(pre_gemm_temperature),
                   None if weight_scale is None else weight_scale.data_ptr())
    keep.append(weight_scale)
    return prob, keep


def workspace_bytes(prob: Problem):
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().stce_workspace_bytes(ctypes.byref(prob), ctypes.byref(f), ctypes.byref(b)))
    return f.value, b.value


def schedule(prob: Problem):
    """(forward rows per chunk, backward vocabulary columns per slice)."""
    c, v = ctypes.c_int64(), ctypes.c_int64()
    _check(load().stce_schedule(ctypes.byref(prob), ctypes.byref(c), ctypes.byref(v)))
    return c.value, v.value


def _raise_rows(status: torch.Tensor, what: str, tensors: dict) -> None:
    v = int(status.item())
    if v == STATUS_NONE:
        return
    row, field = v >> 8, v & 0xFF
    name = FIELDS.get(field, f"field {field}")
    t = tensors.get(name)
    val = "" if t is None else f"={t[row].tolist()!r}"
    raise ValueError(f"{what}: invalid {name}[{row}]{val}")


def forward(hidden, weight, target, temperature=None, top_k=None, top_p=None, min_p=None, *,
            chunk_rows: int = 0, check: bool = True, workspace: Optional[torch.Tensor] = None,
            side: bool = False, ignore_index: Optional[int] = None, pre_gemm_temperature: Optional[float] = None,
            lane: str = "fp32", weight_scale: Optional[torch.Tensor] = None):
    """Selected logprob per row and the per-row state for backward.

    With ``side=True`` also returns a dict of the sweep's side outputs
    (``lse_full``, ``entropy_full``, ``entropy_support``, fp32 [T]).
    """
    prob, keep = make_problem(hidden, weight, target, temperature, top_k, top_p, min_p, chunk_rows,
                              ignore_index=ignore_index, pre_gemm_temperature=pre_gemm_temperature, lane=lane,
                              weight_scale=weight_scale)
    T = prob.T
    fwd_b, _ = workspace_bytes(prob)
    dev = hidden.device
    ws = workspace if workspace is not None else torch.empty(max(fwd_b, 1), dtype=torch.uint8, device=dev)
    logprob = torch.empty(T, dtype=torch.float32, device=dev)
    state = torch.empty(T * STATE_BYTES_PER_ROW, dtype=torch.uint8, device=dev)
    status = torch.empty(1, dtype=torch.int64, device=dev)
    outs = None
    if side:
        outs = {k: torch.empty(T, dtype=torch.float32, device=dev)
                for k in ("lse_full", "entropy_full", "entropy_support")}
        so = SideOutputs(*(outs[k].data_ptr() for k in ("lse_full", "entropy_full", "entropy_support")))
        _check(load().stce_forward_with_side(ctypes.byref(prob), _ptr(logprob), _ptr(state), ctypes.byref(so),
                                             _ptr(status), _ptr(ws), ws.numel(), _stream()))
    else:
        _check(load().stce_forward(ctypes.byref(prob), _ptr(logprob), _ptr(state), _ptr(status), _ptr(ws),
                                   ws.numel(), _stream()))
    if check:
        _raise_rows(status, "stce_forward", dict(temperature=keep[3], top_k=keep[4], top_p=keep[5],
                                                 min_p=keep[6], target=keep[2]))
    return (logprob, state, outs) if side else (logprob, state)


def forward_noalloc(hidden, weight, target, temperature=None, top_k=None, top_p=None, min_p=None, *,
                    chunk_rows: int = 0, check: bool = True, ignore_index: Optional[int] = None,
                    pre_gemm_temperature: Optional[float] = None, lane: str = "fp32",
                    weight_scale: Optional[torch.Tensor] = None):
    """``forward`` through ``stce_forward_noalloc``: the library's static
    scratch instead of a workspace (the outputs are still allocated here)."""
    prob, keep = make_problem(hidden, weight, target, temperature, top_k, top_p, min_p, chunk_rows,
                              ignore_index=ignore_index, pre_gemm_temperature=pre_gemm_temperature, lane=lane,
                              weight_scale=weight_scale)
    T = prob.T
    dev = hidden.device
    logprob = torch.empty(T, dtype=torch.float32, device=dev)
    state = torch.empty(T * STATE_BYTES_PER_ROW, dtype=torch.uint8, device=dev)
    status = torch.empty(1, dtype=torch.int64, device=dev)
    _check(load().stce_forward_noalloc(ctypes.byref(prob), _ptr(logprob), _ptr(state), _ptr(status), _stream()))
    if check:
        _raise_rows(status, "stce_forward_noalloc", dict(temperature=keep[3], top_k=keep[4], top_p=keep[5],
                                                         min_p=keep[6], target=keep[2]))
    return logprob, state


def backward(hidden, weight, target, state, grad_logprob, temperature=None, top_k=None, top_p=None,
             min_p=None, *, need_hidden: bool = True, need_weight: bool = True,
             grad_weight: Optional[torch.Tensor] = None, accumulate_grad_weight: bool = False,
             vocab_slice: int = 0, workspace: Optional[torch.Tensor] = None, ignore_index: Optional[int] = None,
             pre_gemm_temperature: Optional[float] = None, lane: str = "fp32",
             weight_scale: Optional[torch.Tensor] = None, recompute_all: bool = False):
    """(grad_hidden [T, H] in hidden's dtype, grad_weight [V, H] fp32).
    ``recompute_all`` recomputes every row's keys, ignoring the support
    lists the state holds."""
    prob, keep = make_problem(hidden, weight, target, temperature, top_k, top_p, min_p, 0, vocab_slice,
                              ignore_index=ignore_index, pre_gemm_temperature=pre_gemm_temperature, lane=lane,
                              weight_scale=weight_scale, recompute_all=recompute_all)
    T, H, V = prob.T, prob.H, prob.V
    dev = hidden.device
    if grad_logprob.shape != (T,) or grad_logprob.dtype != torch.float32 or grad_logprob.device != dev:
        raise ValueError("grad_logprob must be fp32 [T] on the hidden's device")
    if state.numel() != T * STATE_BYTES_PER_ROW or state.dtype != torch.uint8:
        raise ValueError(f"state must be the uint8 [T*{STATE_BYTES_PER_ROW}] tensor written by forward")
    g = grad_logprob.contiguous()
    _, bwd_b = workspace_bytes(prob)
    ws = workspace if workspace is not None else torch.empty(max(bwd_b, 1), dtype=torch.uint8, device=dev)
    gh = torch.empty(T, H, dtype=hidden.dtype, device=dev) if need_hidden else None
    if need_weight:
        if grad_weight is None:
            grad_weight = torch.empty(V, H, dtype=torch.float32, device=dev)
            accumulate_grad_weight = False
        elif grad_weight.shape != (V, H) or grad_weight.dtype != torch.float32 or not grad_weight.is_contiguous():
            raise ValueError("grad_weight must be a contiguous fp32 [V, H] tensor")
    else:
        grad_weight = None
    _check(load().stce_backward(ctypes.byref(prob), _ptr(g), _ptr(state), _ptr(gh), _ptr(grad_weight),
                                1 if accumulate_grad_weight else 0, None, _ptr(ws), ws.numel(), _stream()))
    return gh, grad_weight


def recompute_keys(hidden, weight, target, state, grad_logprob, temperature=None, top_k=None, top_p=None,
                   min_p=None, *, vocab_slice: int = 0, ignore_index: Optional[int] = None,
                   pre_gemm_temperature: Optional[float] = None, lane: str = "fp32",
                   weight_scale: Optional[torch.Tensor] = None):
    """fp32 keys [T, V] recomputed by the backward's products, exported by
    those launches themselves (parity: they must equal the forward's bit for
    bit).  A row whose keys the backward recomputes on its listed tiles only
    gets those tiles' keys; its other entries stay NaN."""
    prob, keep = make_problem(hidden, weight, target, temperature, top_k, top_p, min_p, 0, vocab_slice,
                              ignore_index=ignore_index, pre_gemm_temperature=pre_gemm_temperature, lane=lane,
                              weight_scale=weight_scale)
    dev = hidden.device
    if state.numel() != prob.T * STATE_BYTES_PER_ROW or state.dtype != torch.uint8:
        raise ValueError(f"state must be the uint8 [T*{STATE_BYTES_PER_ROW}] tensor written by forward")
    _, bwd_b = workspace_bytes(prob)
    ws = torch.empty(max(bwd_b, 1), dtype=torch.uint8, device=dev)
    out = torch.full((prob.T, prob.V), float("nan"), dtype=torch.float32, device=dev)
    g = grad_logprob.contiguous()
    _check(load().stce_recompute_keys(ctypes.byref(prob), _ptr(g), _ptr(state), _ptr(out), _ptr(ws), ws.numel(),
                                      _stream()))
    return out


def scaled_logits(hidden, weight, temperature=None, row0: int = 0, nrows: Optional[int] = None, *,
                  pre_gemm_temperature: Optional[float] = None, lane: str = "fp32",
                  weight_scale: Optional[torch.Tensor] = None):
    """fp32 keys of rows [row0, row0 + nrows) from the forward's kernel:
    s = fl32(h W^T) / T per row, or fl32((h / Ts) W^T) with the scalar
    pre-GEMM temperature Ts; in the bf16 lane the bf16 keys."""
    T = hidden.shape[0]
    nrows = T - row0 if nrows is None else nrows
    target = torch.zeros(T, dtype=torch.int64, device=hidden.device)
    prob, keep = make_problem(hidden, weight, target, temperature, pre_gemm_temperature=pre_gemm_temperature,
                              lane=lane, weight_scale=weight_scale)
    fwd_b, _ = workspace_bytes(prob)
    ws = torch.empty(max(fwd_b, 1), dtype=torch.uint8, device=hidden.device)
    out = torch.empty(nrows, prob.V, dtype=torch.float32, device=hidden.device)
    _check(load().stce_scaled_logits(ctypes.byref(prob), row0, nrows, _ptr(out), _ptr(ws), ws.numel(), _stream()))
    return out


def fp8_quantize_rows(x: torch.Tensor):
    """(codes uint8 [R, H], scales fp32 [R]): the fp8 lane's per-row e4m3
    quantization of bf16 rows ``x`` [R, H] (H a multiple of 16)."""
    if x.dim() != 2 or x.dtype != torch.bfloat16 or x.device.type != "cuda":
        raise ValueError("x must be a bf16 [R, H] tensor on a GPU")
    x = x.contiguous()
    R, H = x.shape
    codes = torch.empty(R, H, dtype=torch.uint8, device=x.device)
    scales = torch.empty(R, dtype=torch.float32, device=x.device)
    _check(load().stce_fp8_quantize_rows(_ptr(x), R, H, _ptr(codes), _ptr(scales), _stream()))
    return codes, scales


def support_from_logits(s, target, top_k=None, top_p=None, min_p=None, *, check: bool = True):
    """Support program + selected logprob on given fp32 keys s [R, V]."""
    if s.dim() != 2 or s.dtype != torch.float32 or s.device.type != "cuda":
        raise ValueError("s must be a fp32 [R, V] GPU tensor")
    s = s.contiguous()
    R, V = s.shape
    dev = s.device
    target = _meta("target", target, R, torch.int64, dev)
    tk = _meta("top_k", top_k, R, torch.int32, dev)
    tp = _meta("top_p", top_p, R, torch.float32, dev)
    mp = _meta("min_p", min_p, R, torch.float32, dev)
    L = load()
    nb = L.stce_support_workspace_bytes(R, V)
    ws = torch.empty(max(nb, 1), dtype=torch.uint8, device=dev)
    logprob = torch.empty(R, dtype=torch.float32, device=dev)
    state = torch.empty(R * STATE_BYTES_PER_ROW, dtype=torch.uint8, device=dev)
    status = torch.empty(1, dtype=torch.int64, device=dev)
    _check(L.stce_support_from_logits(_ptr(s), R, V, _ptr(tk), _ptr(tp), _ptr(mp), _ptr(target), _ptr(logprob),
                                      _ptr(state), _ptr(status), _ptr(ws), ws.numel(), _stream()))
    if check:
        _raise_rows(status, "stce_support_from_logits", dict(top_k=tk, top_p=tp, min_p=mp, target=target))
    return logprob, state


def policy_loss(logprob, advantages, old_logprob, objective: str = "cispo", eps_low: float = 0.2,
                eps_high: float = 0.28, scale: float = 1.0, state: Optional[torch.Tensor] = None):
    """Per-token policy-gradient loss on the selected logprob.

    Returns (loss [T], grad_logprob [T], ratio [T]); grad_logprob is the
    upstream gradient to pass to ``backward`` for d(sum loss)/d(h, W).
    """
    if objective not in PG_OBJECTIVES:
        raise ValueError(f"objective must be one of {tuple(PG_OBJECTIVES)}")
    if logprob.dim() != 1 or logprob.dtype != torch.float32:
        raise ValueError("logprob must be fp32 [T]")
    T = logprob.shape[0]
    dev = logprob.device
    adv = _meta("advantages", advantages, T, torch.float32, dev)
    old = _meta("old_logprob", old_logprob, T, torch.float32, dev)
    if adv is None or old is None:
        raise ValueError("advantages and old_logprob are required")
    lp = logprob.contiguous()
    loss = torch.empty(T, dtype=torch.float32, device=dev)
    grad = torch.empty(T, dtype=torch.float32, device=dev)
    ratio = torch.empty(T, dtype=torch.float32, device=dev)
    pg = PgParams(PG_OBJECTIVES[objective], eps_low, eps_high, scale, adv.data_ptr(), old.data_ptr(),
                  None if state is None else state.data_ptr())
    _check(load().stce_policy_loss(ctypes.byref(pg), T, _ptr(lp), _ptr(loss), _ptr(grad), _ptr(ratio), _stream()))
    return loss, grad, ratio


def policy_loss_step(hidden, weight, target, advantages, old_logprob, temperature=None, top_k=None, top_p=None,
                     min_p=None, *, objective: str = "cispo", eps_low: float = 0.2, eps_high: float = 0.28,
                     scale: float = 1.0, need_hidden: bool = True, need_weight: bool = True,
                     ignore_index: Optional[int] = None, pre_gemm_temperature: Optional[float] = None,
                     lane: str = "fp32"):
    """Fused head + policy-gradient token loss: forward, per-token loss and
    the gradients of ``sum(loss)``.  Returns (loss [T], logprob [T], ratio [T],
    grad_hidden, grad_weight)."""
    logprob, state = forward(hidden, weight, target, temperature, top_k, top_p, min_p, ignore_index=ignore_index,
                             pre_gemm_temperature=pre_gemm_temperature, lane=lane)
    loss, g, ratio = policy_loss(logprob, advantages, old_logprob, objective, eps_low, eps_high, scale, state)
    gh, gw = backward(hidden, weight, target, state, g, temperature, top_k, top_p, min_p,
                      need_hidden=need_hidden, need_weight=need_weight, ignore_index=ignore_index,
                      pre_gemm_temperature=pre_gemm_temperature, lane=lane)
    return loss, logprob, ratio, gh, gw


def fused_workspace_bytes(prob: Problem):
    """(default, minimum) workspace bytes of the fused step; a size between
    them keeps fewer chunks per weight-gradient group."""
    n, m = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().stce_fused_workspace_bytes(ctypes.byref(prob), ctypes.byref(n), ctypes.byref(m)))
    return n.value, m.value


def fused_policy_step(hidden, weight, target, advantages, old_logprob, temperature=None, top_k=None, top_p=None,
                      min_p=None, *, objective: str = "cispo", eps_low: float = 0.2, eps_high: float = 0.28,
                      scale: float = 1.0, need_hidden: bool = True, need_weight: bool = True,
                      grad_weight: Optional[torch.Tensor] = None, accumulate_grad_weight: bool = False,
                      side: bool = False, chunk_rows: int = 0, ignore_index: Optional[int] = None,
                      check: bool = True, workspace: Optional[torch.Tensor] = None,
                      pre_gemm_temperature: Optional[float] = None, lane: str = "fp32",
                      weight_scale: Optional[torch.Tensor] = None, recompute_all: bool = False):
    """The fused head + policy-gradient step (dlogits formed in the forward's
    sweep from the chunk's keys).  Returns a dict with ``loss``, ``logprob``,
    ``ratio`` (fp32 [T]), ``state``, ``grad_hidden`` ([T, H], hidden's dtype,
    or None), ``grad_weight`` (fp32 [V, H] or None) and, with ``side=True``,
    ``lse_full``, ``entropy_full``, ``entropy_support``.  An e4m3 ``weight``
    (uint8 codes) with ``weight_scale`` takes the fp8 lane."""
    if objective not in PG_OBJECTIVES:
        raise ValueError(f"objective must be one of {tuple(PG_OBJECTIVES)}")
    prob, keep = make_problem(hidden, weight, target, temperature, top_k, top_p, min_p, chunk_rows,
                              ignore_index=ignore_index, pre_gemm_temperature=pre_gemm_temperature, lane=lane,
                              weight_scale=weight_scale, recompute_all=recompute_all)
    T, H, V = prob.T, prob.H, prob.V
    dev = hidden.device
    adv = _meta("advantages", advantages, T, torch.float32, dev)
    old = _meta("old_logprob", old_logprob, T, torch.float32, dev)
    if adv is None or old is None:
        raise ValueError("advantages and old_logprob are required")
    keep += [adv, old]
    nb, _ = fused_workspace_bytes(prob)
    ws = workspace if workspace is not None else torch.empty(max(nb, 1), dtype=torch.uint8, device=dev)
    out = {k: torch.empty(T, dtype=torch.float32, device=dev) for k in ("loss", "logprob", "ratio")}
    out["state"] = torch.empty(T * STATE_BYTES_PER_ROW, dtype=torch.uint8, device=dev)
    out["grad_hidden"] = torch.empty(T, H, dtype=hidden.dtype, device=dev) if need_hidden else None
    if need_weight:
        if grad_weight is None:
            grad_weight = torch.empty(V, H, dtype=torch.float32, device=dev)
            accumulate_grad_weight = False
        elif grad_weight.shape != (V, H) or grad_weight.dtype != torch.float32 or not grad_weight.is_contiguous():
            raise ValueError("grad_weight must be a contiguous fp32 [V, H] tensor")
    else:
        grad_weight = None
    out["grad_weight"] = grad_weight
    so = None
    if side:
        for k in ("lse_full", "entropy_full", "entropy_support"):
            out[k] = torch.empty(T, dtype=torch.float32, device=dev)
        so = SideOutputs(*(out[k].data_ptr() for k in ("lse_full", "entropy_full", "entropy_support")))
    pg = PgParams(PG_OBJECTIVES[objective], eps_low, eps_high, scale, adv.data_ptr(), old.data_ptr(), None)
    status = torch.empty(1, dtype=torch.int64, device=dev)
    _check(load().stce_fused_policy_step(ctypes.byref(prob), ctypes.byref(pg), _ptr(out["logprob"]),
                                         _ptr(out["state"]), _ptr(out["loss"]), _ptr(out["ratio"]),
                                         None if so is None else ctypes.byref(so), _ptr(out["grad_hidden"]),
                                         _ptr(grad_weight), 1 if accumulate_grad_weight else 0, _ptr(status),
                                         _ptr(ws), ws.numel(), _stream()))
    if check:
        _raise_rows(status, "stce_fused_policy_step", dict(temperature=keep[3], top_k=keep[4], top_p=keep[5],
                                                            min_p=keep[6], target=keep[2]))
    return out


def decode_state(state: torch.Tensor) -> dict:
    """Per-row state fields as numpy arrays (copies the state to the host),
    with ``ntile`` and ``tiles`` [T, 31] from the rows' tile lists, and
    ``support_ids`` / ``support_keys`` [T, 128] from their support lists."""
    import numpy as np
    host = state.detach().cpu().contiguous()
    n = host.numel() // STATE_BYTES_PER_ROW
    out = (RowInfo * n)()
    _check(load().stce_decode_state(ctypes.c_void_p(host.data_ptr()), n, out))
    arr = np.frombuffer(bytes(out), dtype=np.dtype([
        ("key_thr", "<u4"), ("id_thr", "<i4"), ("n", "<i4"), ("flags", "<u4"),
        ("lse_support", "<f4"), ("lse_full", "<f4"), ("row_max", "<f4"), ("target_key", "<f4")]))
    d = {k: arr[k].copy() for k in arr.dtype.names}
    tb = 2 * (1 + NTILE)
    tl = host[n * RECORD_BYTES:n * (RECORD_BYTES + tb)].numpy().view(np.uint16).reshape(n, 1 + NTILE)
    d["ntile"] = tl[:, 0].astype(np.int64)
    d["tiles"] = tl[:, 1:].astype(np.int64)
    sl = host[n * (RECORD_BYTES + tb):].numpy().view(np.int32).reshape(n, NSP, 2)
    d["support_ids"] = sl[:, :, 0].astype(np.int64)
    d["support_keys"] = sl[:, :, 1].copy().view(np.float32)
    return d


def state_prefix(state: torch.Tensor, rows: int) -> torch.Tensor:
    """The state bytes of the first ``rows`` rows (their records, their tile
    lists, then their support lists), comparable with the state of a call
    over those rows only."""
    T = state.numel() // STATE_BYTES_PER_ROW
    tb, sb = 2 * (1 + NTILE), 8 * NSP
    rec = state[: T * RECORD_BYTES][: rows * RECORD_BYTES]
    til = state[T * RECORD_BYTES: T * (RECORD_BYTES + tb)][: rows * tb]
    sup = state[T * (RECORD_BYTES + tb):][: rows * sb]
    return torch.cat([rec, til, sup])


class ScoreFunction(torch.autograd.Function):
    """Autograd wrapper of the scoring core:

    ``logprob = ScoreFunction.apply(hidden, weight, target, temperature, top_k, top_p, min_p,
    ignore_index, pre_gemm_temperature, lane)`` (arguments after ``target`` optional, as in
    ``forward``).  The backward recomputes through ``backward`` with the
    incoming gradient as ``grad_logprob``; the weight gradient is returned in
    the weight's dtype."""

    @staticmethod
    def forward(ctx, hidden, weight, target, temperature=None, top_k=None, top_p=None, min_p=None,
                ignore_index=None, pre_gemm_temperature=None, lane="fp32"):
        opts = dict(ignore_index=ignore_index, pre_gemm_temperature=pre_gemm_temperature, lane=lane)
        logprob, state = forward(hidden, weight, target, temperature, top_k, top_p, min_p, **opts)
        ctx.save_for_backward(hidden, weight, target, state)
        ctx.meta = (temperature, top_k, top_p, min_p)
        ctx.opts = opts
        return logprob

    @staticmethod
    def backward(ctx, g):
        hidden, weight, target, state = ctx.saved_tensors
        gh, gw = backward(hidden, weight, target, state, g.float().contiguous(), *ctx.meta,
                          need_hidden=ctx.needs_input_grad[0], need_weight=ctx.needs_input_grad[1], **ctx.opts)
        if gw is not None:
            gw = gw.to(weight.dtype)
        return (gh, gw) + (None,) * 8


# ---------------------------------------------------------------------------
# Operators on given arrays: token log probabilities, block-scaled fp8
# quantization and product.  Their arrays may lie on any GPU: the call is made
# on the arrays' device, on its current stream.
# ---------------------------------------------------------------------------
_fast = None


def _load_fast():
    """The marshalling module (see csrc/marshal.cpp) with the library's
    functions bound, or False where it is not built.  It makes the calls below
    with less host time for operands it takes as they stand; everything else,
    and every error, goes through the ctypes calls."""
    global _fast
    L = load()
    try:
        from . import _marshal as m
    except ImportError:
        _fast = False
    else:
        m.bind({n: ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in SYMBOLS[-6:]})
        _fast = m
    return _fast


def _here(x):
    """(module, device index) of the marshalling module where it can take a call
    on x's device: the current one."""
    m = _fast
    if m is None:
        m = _load_fast()
    if m is False or not isinstance(x, torch.Tensor) or not x.is_cuda:
        return None, 0
    i = x.get_device()
    return (m, i) if i == torch._C._cuda_getDevice() else (None, 0)


def _call(fn, dev, *args):
    """fn(*args, stream) on the arrays' device, on its current stream."""
    # (the raw queries: a torch.cuda.Stream object costs as much as a launch)
    i = dev.index
    if i == torch._C._cuda_getDevice():
        _check(fn(*args, torch._C._cuda_getCurrentRawStream(i)))
    else:
        with torch.cuda.device(dev):
            _check(fn(*args, torch._C._cuda_getCurrentRawStream(i)))


def _rows(name, x, dtypes):
    """A 2-d GPU tensor of one of the dtypes with unit-stride rows (a copy
    where the rows are not contiguous), and its row stride."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError(f"{name} must be a 2-d tensor")
    if x.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {tuple(str(d) for d in dtypes)}, got {x.dtype}")
    if not x.is_cuda:
        raise ValueError(f"{name} must be on a GPU, got {x.device}")
    R, C = x.shape
    if x.is_contiguous():
        return x, C
    if (C > 1 and x.stride(1) != 1) or (R > 1 and x.stride(0) < C):
        return x.contiguous(), C
    return x, (x.stride(0) if R > 1 and C else C)


def _tokens(tokens, T, dev):
    """(int64 [T] or [T, K] or None, K)."""
    if tokens is None:
        return None, 0
    if not isinstance(tokens, torch.Tensor) or tokens.dtype != torch.int64:
        raise TypeError("tokens must be an int64 tensor or None")
    if tokens.device != dev:
        raise ValueError(f"tokens is on {tokens.device}, expected {dev}")
    if tokens.dim() not in (1, 2) or tokens.shape[0] != T:
        raise ValueError(f"tokens must have shape [{T}] or [{T}, K], got {tuple(tokens.shape)}")
    return tokens.contiguous(), (1 if tokens.dim() == 1 else tokens.shape[1])


def _token_problem(logits, tokens, temperature, top_n, ignore_index):
    z, ld = _rows("logits", logits, VALUE_DTYPES)
    T, V = z.shape
    dev = z.device
    tok, K = _tokens(tokens, T, dev)
    temp = None if temperature is None else _meta("temperature", temperature, T, torch.float32, dev)
    prob = TokenProblem(T, V, VALUE_DTYPES[z.dtype], 0 if ignore_index is None else PROBLEM_IGNORE_INDEX,
                        z.data_ptr(), ld if ld > V else V, None if temp is None else temp.data_ptr(),
                        None if tok is None else tok.data_ptr(), K, top_n,
                        0 if ignore_index is None else int(ignore_index))
    return prob, (z, tok, temp)


@functools.lru_cache(maxsize=1024)
def _token_workspace(T, V, dtype, top_n):
    """Workspace bytes of ``stce_token_logprobs`` for these sizes."""
    nb = ctypes.c_size_t()
    prob = TokenProblem(T, V, dtype, 0, None, V, None, None, 0, top_n, 0)
    _check(load().stce_token_workspace_bytes(ctypes.byref(prob), ctypes.byref(nb)))
    return nb.value


def _given_workspace(workspace, dev):
    """A caller's workspace (or None) and its bytes."""
    if workspace is None:
        return None, 0
    if workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {dev}")
    return workspace, workspace.numel()


def token_logprobs(logits, tokens=None, temperature=None, *, top_n: int = 0, ignore_index: Optional[int] = None,
                   check: bool = True, workspace: Optional[torch.Tensor] = None):
    """Log probabilities of given tokens under ``logits`` [T, V] (bf16, fp16 or
    fp32; rows may be strided), scaled by a per-row ``temperature`` (fp32 [T]
    or None).  ``tokens`` int64 [T] or [T, K].

    Returns a dict: ``logprob`` (fp32, tokens' shape; absent without tokens),
    ``lse`` and ``entropy`` (fp32 [T]), ``stats`` (fp32 [T, 4], for
    ``token_logprobs_backward``) and, with ``top_n``, the ``top_n`` most likely
    tokens of each row in order, lower id first among equal logits:
    ``top_logprob`` (fp32 [T, top_n]) and ``top_id`` (int64; -1 past a row's
    last token with a logit above -inf).  Masked tokens (-inf) score -inf;
    ``ignore_index`` scores 0.  ``check=False`` skips the report of invalid
    tokens and temperatures, which reads one number back from the GPU."""
    if workspace is None:
        m, i = _here(logits)
        r = m and m.token_logprobs(logits, tokens, temperature, top_n, ignore_index, check, i,
                                   torch._C._cuda_getCurrentRawStream(i))
        if r is not None:
            if r[0]:
                _check(r[0])
            if check:
                _raise_rows(r[2], "stce_token_logprobs", dict(temperature=temperature, target=tokens))
            return r[1]
    prob, keep = _token_problem(logits, tokens, temperature, top_n, ignore_index)
    T, K = prob.T, prob.K
    dev = logits.device
    L = load()
    if workspace is None:
        nb = _token_workspace(T, prob.V, prob.dtype, top_n)
        if nb:
            workspace = torch.empty(nb, dtype=torch.uint8, device=dev)
    workspace, ws_bytes = _given_workspace(workspace, dev)
    # one allocation for the fp32 outputs: a row costs little more than its calls
    buf = torch.empty(T * (6 + K + top_n), dtype=torch.float32, device=dev)
    out = dict(stats=buf.as_strided((T, 4), (4, 1), 0), lse=buf.as_strided((T,), (1,), 4 * T),
               entropy=buf.as_strided((T,), (1,), 5 * T))
    base = buf.data_ptr()
    ptrs = [None, base + 16 * T, base + 20 * T, None, None, base]
    if tokens is not None:
        out["logprob"] = buf.as_strided(tokens.shape, (K, 1)[-tokens.dim():], 6 * T)
        ptrs[0] = base + 24 * T
    if top_n:
        out["top_logprob"] = buf.as_strided((T, top_n), (top_n, 1), (6 + K) * T)
        out["top_id"] = torch.empty((T, top_n), dtype=torch.int64, device=dev)
        ptrs[3], ptrs[4] = base + (24 + 4 * K) * T, out["top_id"].data_ptr()
    status = torch.empty(1, dtype=torch.int64, device=dev) if check else None
    o = TokenOutputs(*ptrs)
    _call(L.stce_token_logprobs, dev, ctypes.byref(prob), ctypes.byref(o), _ptr(status), _ptr(workspace),
          ws_bytes)
    if check:
        _raise_rows(status, "stce_token_logprobs", dict(temperature=keep[2], target=keep[1]))
    return out


def token_logprobs_backward(logits, tokens, stats, grad_logprob=None, grad_entropy=None, grad_lse=None, *,
                            temperature=None, ignore_index: Optional[int] = None,
                            grad_logits: Optional[torch.Tensor] = None):
    """Gradient of ``sum(grad_logprob * logprob) + sum(grad_entropy * entropy)
    + sum(grad_lse * lse)`` with respect to the logits, in their dtype; ``stats``
    is the forward's.  ``grad_logits`` gives the result's place (strided rows
    allowed; not overlapping the logits)."""
    if grad_logits is None:
        m, i = _here(logits)
        r = m and m.token_grad(logits, tokens, stats, grad_logprob, grad_entropy, grad_lse, temperature, ignore_index,
                               i, torch._C._cuda_getCurrentRawStream(i))
        if r is not None:
            if r[0]:
                _check(r[0])
            return r[1]
    prob, keep = _token_problem(logits, tokens, temperature, 0, ignore_index)
    T, V = prob.T, prob.V
    dev = logits.device
    if stats.shape != (T, 4) or stats.dtype != torch.float32 or stats.device != dev or not stats.is_contiguous():
        raise ValueError("stats must be the contiguous fp32 [T, 4] tensor of the forward")
    if grad_logprob is not None:
        if tokens is None or grad_logprob.shape != tokens.shape:
            raise ValueError("grad_logprob must have the tokens' shape")
        if grad_logprob.dtype != torch.float32 or grad_logprob.device != dev:
            raise ValueError("grad_logprob must be fp32 on the logits' device")
        grad_logprob = grad_logprob.contiguous()
    ge = _meta("grad_entropy", grad_entropy, T, torch.float32, dev)
    gl = _meta("grad_lse", grad_lse, T, torch.float32, dev)
    if grad_logits is None:
        grad_logits = torch.empty(T, V, dtype=logits.dtype, device=dev)
    elif (grad_logits.shape != (T, V) or grad_logits.dtype != logits.dtype or grad_logits.device != dev
          or (V > 1 and grad_logits.stride(1) != 1) or (T > 1 and grad_logits.stride(0) < V)):
        raise ValueError("grad_logits must have the logits' shape, dtype and device, with unit-stride rows")
    ldg = max(grad_logits.stride(0), V) if T > 1 else max(V, 1)
    _call(load().stce_token_logprobs_backward, dev, ctypes.byref(prob), _ptr(stats), _ptr(grad_logprob), _ptr(ge),
          _ptr(gl), _ptr(grad_logits), ldg)
    return grad_logits


class TokenLogprobFunction(torch.autograd.Function):
    """Autograd wrapper of ``token_logprobs``:

    ``logprob, lse, entropy, top_logprob, top_id = TokenLogprobFunction.apply(logits, tokens, temperature,
    ignore_index, top_n, check)`` (arguments after ``tokens`` optional; the
    last two outputs None without ``top_n``).  Gradients flow from the first
    three to the logits; the alternatives are values (score them as given
    tokens to differentiate through them)."""

    @staticmethod
    def forward(ctx, logits, tokens, temperature=None, ignore_index=None, top_n=0, check=True):
        out = token_logprobs(logits, tokens, temperature, top_n=top_n, ignore_index=ignore_index, check=check)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(logits, tokens, out["stats"], temperature)
        ctx.ignore_index = ignore_index
        top = (out.get("top_logprob"), out.get("top_id"))
        ctx.mark_non_differentiable(*(t for t in top if t is not None))
        return (out.get("logprob"), out["lse"], out["entropy"]) + top

    @staticmethod
    def backward(ctx, g_logprob, g_lse, g_entropy, *_):
        if g_logprob is None and g_lse is None and g_entropy is None:
            return (None,) * 6
        logits, tokens, stats, temperature = ctx.saved_tensors
        g = token_logprobs_backward(logits, tokens, stats, g_logprob, g_entropy, g_lse, temperature=temperature,
                                    ignore_index=ctx.ignore_index)
        return (g,) + (None,) * 5


def fp8_quantize_blocks(x: torch.Tensor, *, block: str = "row", transpose: bool = False):
    """e4m3 codes and fp32 scales of ``x`` [R, C] (bf16, fp16 or fp32), one
    scale per 128 values: of a row (``block="row"``) or of a 128 x 128 tile
    (``block="tile"``); with ``transpose`` of the transposed matrix.  Returns
    (codes float8_e4m3fn [Q, L rounded up to 16, zeros past L], scales [Q or
    ceil(Q / 128), ceil(L / 128)]) with Q, L = R, C (transposed: C, R): the
    operands of ``fp8_block_matmul``.  (The scales are a view with the block
    index slowest in memory.)"""
    if block not in ("row", "tile"):
        raise ValueError("block must be 'row' or 'tile'")
    m, i = _here(x)
    r = m and m.quantize(x, block == "tile", transpose, i, torch._C._cuda_getCurrentRawStream(i))
    if r is not None:
        if r[0]:
            _check(r[0])
        return r[1], r[2]
    x, ld = _rows("x", x, VALUE_DTYPES)
    R, C = x.shape
    Q, n = (C, R) if transpose else (R, C)
    dev = x.device
    kp = -(-n // 16) * 16
    codes = torch.empty(Q, kp, dtype=torch.float8_e4m3fn, device=dev)
    sr = Q if block == "row" else -(-Q // FP8_BLOCK)
    scales = torch.empty_strided((sr, -(-n // FP8_BLOCK)), (1, sr), dtype=torch.float32, device=dev)
    flags = (QUANT_TILE if block == "tile" else 0) | (QUANT_TRANSPOSE if transpose else 0)
    _call(load().stce_fp8_quantize_blocks, dev, _ptr(x), VALUE_DTYPES[x.dtype], R, C, max(ld, C), flags, _ptr(codes),
          kp, _ptr(scales))
    return codes, scales


def _fp8_operand(name, q, scale, tile_ok):
    q, ld = _rows(name, q, FP8_WEIGHT_DTYPES)
    R, K = q.shape
    kb = -(-K // FP8_BLOCK)
    if K % 16 or ld % 16 or q.data_ptr() % 16:
        raise ValueError(f"{name} must have rows of a multiple of 16 codes, 16-byte aligned (fp8_quantize_blocks pads "
                         f"them so), got {tuple(q.shape)} with row stride {ld}")
    if not isinstance(scale, torch.Tensor) or scale.dtype != torch.float32 or scale.device != q.device:
        raise TypeError(f"{name}_scale must be fp32 on {name}'s device")
    tiles = (-(-R // FP8_BLOCK), kb)
    if tuple(scale.shape) == (R, kb):
        rows = 1
    elif tile_ok and tuple(scale.shape) == tiles:
        rows = FP8_BLOCK
    else:
        want = f"{(R, kb)}" + (f" or {tiles}" if tile_ok else "")
        raise ValueError(f"{name}_scale must have shape {want}, got {tuple(scale.shape)}")
    return q, ld, rows


def fp8_block_matmul(a, a_scale, b, b_scale, out_dtype=torch.bfloat16, *, out: Optional[torch.Tensor] = None,
                     accumulate: bool = False, workspace: Optional[torch.Tensor] = None):
    """``a @ b.T`` of e4m3 codes a [M, K] and b [N, K] (``float8_e4m3fn`` or
    uint8, K a multiple of 16) with a scale per 128 of K: ``a_scale`` [M,
    ceil(K / 128)], ``b_scale`` [N, ceil(K / 128)] or, per 128 x 128 tile,
    [ceil(N / 128), ceil(K / 128)], fp32, any strides.  Returns ``out`` [M, N] in
    ``out_dtype`` (bf16, fp16, fp32), rounded once from fp32 sums; with
    ``accumulate`` the product is added to ``out`` (fp32)."""
    if out is None and not accumulate and workspace is None:
        m, i = _here(a)
        r = m and m.matmul(a, a_scale, b, b_scale, out_dtype, i, torch._C._cuda_getCurrentRawStream(i))
        if r is not None:
            if r[0]:
                _check(r[0])
            return r[1]
    a, lda, _ = _fp8_operand("a", a, a_scale, False)
    b, ldb, b_rows = _fp8_operand("b", b, b_scale, True)
    M, K = a.shape
    N = b.shape[0]
    dev = a.device
    if b.shape[1] != K or b.device != dev:
        raise ValueError(f"a and b must share K and the device, got {tuple(a.shape)}, {tuple(b.shape)}")
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        if out_dtype not in VALUE_DTYPES:
            raise TypeError(f"out_dtype must be bf16, fp16 or fp32, got {out_dtype}")
        out = torch.empty(M, N, dtype=out_dtype, device=dev)
    elif (out.shape != (M, N) or out.dtype not in VALUE_DTYPES or out.device != dev
          or (N > 1 and out.stride(1) != 1) or (M > 1 and out.stride(0) < N)):
        raise ValueError("out must be a bf16, fp16 or fp32 [M, N] tensor on the operands' device with unit-stride rows")
    p = BlockMatmul(M, N, K, a.data_ptr(), lda, a_scale.data_ptr(), a_scale.stride(0),
                    a_scale.stride(1), b.data_ptr(), ldb, b_scale.data_ptr(),
                    b_scale.stride(0), b_scale.stride(1), b_rows, VALUE_DTYPES[out.dtype], out.data_ptr(),
                    max(out.stride(0), N) if M > 1 else N, 1 if accumulate else 0)
    L = load()
    nb = ctypes.c_size_t()
    _check(L.stce_fp8_block_matmul_workspace_bytes(ctypes.byref(p), ctypes.byref(nb)))
    if workspace is None and nb.value:
        workspace = torch.empty(nb.value, dtype=torch.uint8, device=dev)
    workspace, ws_bytes = _given_workspace(workspace, dev)
    _call(L.stce_fp8_block_matmul, dev, ctypes.byref(p), _ptr(workspace), ws_bytes)
    return out


class Fp8BlockLinearFunction(torch.autograd.Function):
    """``Fp8BlockLinearFunction.apply(x, weight)``: the linear layer (or head)
    ``x @ weight.T`` of bf16, fp16 or fp32 x [T, H] and weight [V, H] on e4m3
    operands with block scales (x per row and 128 values, the weight per 128 x
    128 tile), in x's dtype.  The gradients pass the quantizations straight
    through and are such products themselves: the incoming gradient and the
    weight's transpose for dx, both transposed to reduce over the rows for
    dweight, each quantized along its reduction; dweight in the weight's dtype."""

    @staticmethod
    def forward(ctx, x, weight):
        xq, xs = fp8_quantize_blocks(x)
        wq, ws = fp8_quantize_blocks(weight, block="tile")
        ctx.save_for_backward(x, weight)
        return fp8_block_matmul(xq, xs, wq, ws, out_dtype=x.dtype)

    @staticmethod
    def backward(ctx, g):
        x, weight = ctx.saved_tensors
        gx = gw = None
        if ctx.needs_input_grad[0]:
            gq, gs = fp8_quantize_blocks(g)
            wq, ws = fp8_quantize_blocks(weight, block="tile", transpose=True)
            gx = fp8_block_matmul(gq, gs, wq, ws, out_dtype=x.dtype)
        if ctx.needs_input_grad[1]:
            gq, gs = fp8_quantize_blocks(g, transpose=True)
            xq, xs = fp8_quantize_blocks(x, transpose=True)
            gw = fp8_block_matmul(gq, gs, xq, xs, out_dtype=weight.dtype)
        return gx, gw
