"""ctypes binding of libdspark.so (include/dspark.h).  Argument marshalling
only: every step runs in the HIP library.  Tensors are torch tensors on the
GPU; outputs are allocated here with torch and filled by the library on the
current torch stream."""
from __future__ import annotations

import ctypes
import functools
import os
import struct

import torch
from torch.autograd import forward_ad

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None

DTYPE_F32 = 0
DTYPE_BF16 = 1
GREEDY = 0
SAMPLED = 1
MASS = 1 << 24
K_MAX = 1024
STATUS_NAMES = {0: "OK", 1: "ROW_NAN", 2: "ROW_POSINF", 3: "ROW_ZERO_MASS", 4: "DRAW_RANGE",
                5: "ALLOC_INCONSISTENT", 6: "TARGET_INVALID", 7: "DRAFT_INVALID", 8: "BAD_WEIGHT",
                9: "BAD_TOPK", 10: "Q_BAD_LEN", 11: "Q_BAD_ID", 12: "Q_UNSORTED", 13: "Q_NONFINITE",
                14: "Q_NEGATIVE", 15: "Q_NOT_DYADIC", 16: "Q_PADDING", 17: "Q_MASS", 18: "Q_TOKEN",
                19: "BAD_HISTORY", 20: "BAD_PENALTY", 21: "BAD_BIAS", 22: "BAD_MASK",
                23: "BAD_SCORE", 24: "BAD_PARENT", 25: "BAD_LENGTH"}


class DsparkError(RuntimeError):
    pass


class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("n_rows", ctypes.c_int64), ("vocab", ctypes.c_int64), ("row_stride", ctypes.c_int64)]


class Q(ctypes.Structure):
    _fields_ = [("topk", ctypes.c_void_p), ("k_max", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("dense", ctypes.c_void_p), ("sp_ids", ctypes.c_void_p), ("sp_cnt", ctypes.c_void_p),
                ("sp_len", ctypes.c_void_p)]


class QWire(ctypes.Structure):
    _fields_ = [("topk", ctypes.c_void_p), ("k_max", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("dense", ctypes.c_void_p), ("padded", ctypes.c_int64), ("dense_stride", ctypes.c_int64),
                ("sp_ids", ctypes.c_void_p), ("sp_val", ctypes.c_void_p), ("sp_len", ctypes.c_void_p)]


class Shaping(ctypes.Structure):
    _fields_ = [("rows_per_request", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("history", ctypes.c_void_p), ("history_max", ctypes.c_int64), ("history_stride", ctypes.c_int64),
                ("history_len", ctypes.c_void_p), ("prompt_len", ctypes.c_void_p),
                ("draft", ctypes.c_void_p), ("draft_stride", ctypes.c_int64),
                ("repetition", ctypes.c_void_p), ("frequency", ctypes.c_void_p), ("presence", ctypes.c_void_p),
                ("temperature", ctypes.c_void_p),
                ("bias_offset", ctypes.c_void_p), ("bias_ids", ctypes.c_void_p), ("bias_values", ctypes.c_void_p),
                ("bias_total", ctypes.c_int64),
                ("mask", ctypes.c_void_p), ("mask_stride", ctypes.c_int64), ("n_masks", ctypes.c_int64),
                ("mask_row", ctypes.c_void_p)]


class Teacher(ctypes.Structure):
    _fields_ = [("ids", ctypes.c_void_p), ("logits", ctypes.c_void_p), ("len", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("k_max", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class Fp8(ctypes.Structure):
    _fields_ = [("values", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("scale_dtype", ctypes.c_int32),
                ("block_rows", ctypes.c_int32), ("n_rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("row_stride", ctypes.c_int64), ("scale_stride", ctypes.c_int64)]


class State(ctypes.Structure):
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("in_request", ctypes.c_int64), ("in_beam", ctypes.c_int64), ("in_outer", ctypes.c_int64), ("in_row", ctypes.c_int64),
                ("out_request", ctypes.c_int64), ("out_beam", ctypes.c_int64), ("out_outer", ctypes.c_int64), ("out_row", ctypes.c_int64),
                ("outer", ctypes.c_int64), ("rows", ctypes.c_int64), ("row_bytes", ctypes.c_int64)]


BEAM_MAX = 64
BEAM_OUT_MAX = 128
DISTILL_STATS = 5
SCALE_F32 = 0
SCALE_E8M0 = 1

EXPORTS = ["dspark_propose", "dspark_q_alloc", "dspark_sample", "dspark_verify_greedy", "dspark_fused",
           "dspark_q_alloc_weights", "dspark_cr_expf", "dspark_q_encode", "dspark_q_validate", "dspark_margin", "dspark_verify_stochastic", "dspark_verify_ratio", "dspark_sharded_propose", "dspark_sharded_propose_noalloc", "dspark_sharded_q", "dspark_sharded_q_workspace", "dspark_workspace_bytes", "dspark_q_semantic_id",
           "dspark_shape_logits", "dspark_top_logits", "dspark_top_logits_workspace", "dspark_distill",
           "dspark_distill_backward", "dspark_distill_step", "dspark_distill_workspace",
           "dspark_quantize_blocks", "dspark_block_product", "dspark_block_product_workspace",
           "dspark_block_linear", "dspark_block_linear_workspace",
           "dspark_beam_select", "dspark_beam_select_workspace", "dspark_beam_reorder",
           "dspark_status_name", "dspark_last_error", "dspark_abi_version"]


def library_path() -> str:
    return os.environ.get("DSPARK_LIB", os.path.join(_HERE, "libdspark.so"))


def load_library():
    """Loads libdspark.so; raises if it is missing (there is no fallback)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise DsparkError(f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(path)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    RP, QP = ctypes.POINTER(Rows), ctypes.POINTER(Q)
    TP, F32 = ctypes.POINTER(Teacher), ctypes.c_float
    FP = ctypes.POINTER(Fp8)
    sig = {
        "dspark_propose": (ctypes.c_int, [RP, P, P, P, P, SZ, P]),
        "dspark_q_alloc": (ctypes.c_int, [RP, QP, P, P, SZ, P]),
        "dspark_sample": (ctypes.c_int, [QP, I64, I64, P, I64, P, P, P]),
        "dspark_verify_greedy": (ctypes.c_int, [RP, P, P, I64, P, P, P, P, P, P, SZ, P]),
        "dspark_fused": (ctypes.c_int, [RP, RP, I32, QP, P, P, P, P, P, P, P, P, P, P, P, SZ, P]),
        "dspark_q_alloc_weights": (ctypes.c_int, [P, I64, I64, I64, P, P, P, SZ, P]),
        "dspark_cr_expf": (ctypes.c_int, [P, P, I64, P]),
        "dspark_q_encode": (ctypes.c_int, [P, I64, P, P]),
        "dspark_margin": (ctypes.c_int, [RP, P, P]),
        "dspark_sharded_propose": (ctypes.c_int, [RP, I32, P, P, P, P, P, SZ, P]),
        "dspark_sharded_propose_noalloc": (ctypes.c_int, [RP, I32, P, P, P, P, P]),
        "dspark_sharded_q": (ctypes.c_int, [RP, I32, QP, P, P, P, P, P, SZ, P]),
        "dspark_sharded_q_workspace": (SZ, [I64, I32, I32]),
        "dspark_verify_stochastic": (ctypes.c_int, [RP, P, P, I64, P, P, P, P, P, P, P]),
        "dspark_verify_ratio": (ctypes.c_int, [RP, P, P, QP, I64, P, P, P, P, P, P]),
        "dspark_q_validate": (ctypes.c_int, [ctypes.POINTER(QWire), I64, I64, P, P, P, P, P]),
        "dspark_workspace_bytes": (SZ, [I32, I64, I64, I32]),
        "dspark_shape_logits": (ctypes.c_int, [RP, ctypes.POINTER(Shaping), P, I32, I64, P, P]),
        "dspark_top_logits": (ctypes.c_int, [RP, P, I32, F32, P, P, P, P, P, P, SZ, P]),
        "dspark_top_logits_workspace": (SZ, [I64, I64, I32]),
        "dspark_distill": (ctypes.c_int, [RP, TP, F32, P, P, P, P, SZ, P]),
        "dspark_distill_backward": (ctypes.c_int, [RP, TP, F32, P, P, P, P, I64, P]),
        "dspark_distill_step": (ctypes.c_int, [RP, TP, F32, P, P, P, I64, P, P, SZ, P]),
        "dspark_distill_workspace": (SZ, [I64, I64]),
        "dspark_quantize_blocks": (ctypes.c_int, [RP, FP, P]),
        "dspark_block_product": (ctypes.c_int, [FP, FP, P, I32, I64, P, SZ, P]),
        "dspark_block_product_workspace": (SZ, [I64, I64, I64]),
        "dspark_block_linear": (ctypes.c_int, [RP, FP, P, I32, I64, P, SZ, P]),
        "dspark_block_linear_workspace": (SZ, [I64, I64, I64]),
        "dspark_beam_select": (ctypes.c_int, [RP, P, P, I32, I32, I32, P, P, P, P, P, P, P, SZ, P]),
        "dspark_beam_select_workspace": (SZ, [I64, I64, I32]),
        "dspark_beam_reorder": (ctypes.c_int, [P, I32, I64, I32, P, P, P, P]),
        "dspark_q_semantic_id": (ctypes.c_char_p, []),
        "dspark_status_name": (ctypes.c_char_p, [I32]),
        "dspark_last_error": (ctypes.c_char_p, []),
        "dspark_abi_version": (I32, []),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    _LIB = lib
    return lib


def _check(rc: int):
    if rc != 0:
        raise DsparkError(f"libdspark error {rc}: {_LIB.dspark_last_error().decode()}")


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _rows(x: torch.Tensor) -> Rows:
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("logits must be a 2-D [rows, V] tensor with unit column stride")
    if x.dtype == torch.float32:
        dt = DTYPE_F32
    elif x.dtype == torch.bfloat16:
        dt = DTYPE_BF16
    else:
        raise ValueError("logits must be float32 or bfloat16")
    if not x.is_cuda:
        raise ValueError("logits must be on the GPU")
    return Rows(x.data_ptr(), dt, 0, x.shape[0], x.shape[1], x.stride(0))


def _i32(n, dev):
    return torch.empty(n, dtype=torch.int32, device=dev)


def abi_version() -> int:
    return int(load_library().dspark_abi_version())


def q_semantic_id() -> str:
    return load_library().dspark_q_semantic_id().decode()


def status_name(code: int) -> str:
    return load_library().dspark_status_name(int(code)).decode()


def workspace_bytes(op: int, n_rows: int, vocab: int, k_max: int) -> int:
    return int(load_library().dspark_workspace_bytes(op, n_rows, vocab, k_max))


def _make_q(n_rows, V, dev, topk, k_max, want_dense):
    qd = {"topk": topk, "k_max": int(k_max)}
    qd["dense"] = torch.empty((n_rows, V), dtype=torch.int32, device=dev) if want_dense else None
    if topk is not None and k_max > 0:
        qd["sp_ids"] = torch.empty((n_rows, k_max), dtype=torch.int32, device=dev)
        qd["sp_cnt"] = torch.empty((n_rows, k_max), dtype=torch.int32, device=dev)
        qd["sp_len"] = torch.empty(n_rows, dtype=torch.int32, device=dev)
    else:
        qd["sp_ids"] = qd["sp_cnt"] = qd["sp_len"] = None
    return qd


def _qstruct(qd) -> Q:
    return Q(None if qd["topk"] is None else qd["topk"].data_ptr(), qd["k_max"], 0,
             None if qd["dense"] is None else qd["dense"].data_ptr(),
             None if qd["sp_ids"] is None else qd["sp_ids"].data_ptr(),
             None if qd["sp_cnt"] is None else qd["sp_cnt"].data_ptr(),
             None if qd["sp_len"] is None else qd["sp_len"].data_ptr())


def _split_ws(x: torch.Tensor, op: int, split: bool = True):
    """Workspace that lets dense q rows streamed from memory (float32 rows,
    bf16 rows above 131072 ids) be split over several workgroups: (tensor,
    aligned pointer, bytes), or (None, None, 0) when it does not apply."""
    n, V = x.shape
    if not split or (x.dtype == torch.bfloat16 and V <= 131072):
        return None, None, 0
    nbytes = int(load_library().dspark_workspace_bytes(op, n, V, 0))
    if nbytes == 0:
        return None, None, 0
    ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=x.device)
    return ws, ctypes.c_void_p(ws.data_ptr() + (-ws.data_ptr()) % 256), nbytes


def _topk(topk, dev):
    """Per-row k on the device, or None when every row is dense (k = 0 for
    all rows is the same request as no top-k array)."""
    if topk is None:
        return None
    t = torch.as_tensor(topk, dtype=torch.int32)
    if not bool(t.any()):
        return None
    return t.to(dev).contiguous()


def propose(draft: torch.Tensor):
    lib = load_library()
    n, dev = draft.shape[0], draft.device
    am, cf, st = _i32(n, dev), torch.empty(n, dtype=torch.float32, device=dev), _i32(n, dev)
    r = _rows(draft)
    _check(lib.dspark_propose(ctypes.byref(r), _p(am), _p(cf), _p(st), None, 0, _stream()))
    return {"argmax": am, "conf": cf, "status": st}


def q_alloc(draft: torch.Tensor, topk=None, k_max: int = 0, split: bool = True):
    """topk: None (all dense) or per-row k (0 = dense).  split=False keeps
    every streamed dense row on one workgroup (no workspace)."""
    lib = load_library()
    n, V, dev = draft.shape[0], draft.shape[1], draft.device
    tk = _topk(topk, dev)
    want_dense = tk is None or bool((tk == 0).any())
    qd = _make_q(n, V, dev, tk, k_max, want_dense)
    st = _i32(n, dev)
    r, q = _rows(draft), _qstruct(qd)
    ws, wp, wb = _split_ws(draft, 1, split)
    _check(lib.dspark_q_alloc(ctypes.byref(r), ctypes.byref(q), _p(st), wp, wb, _stream()))
    qd["status"] = st
    return qd


def sample(qd, draws: torch.Tensor, row_status: torch.Tensor, vocab: int):
    """draws: uint32-valued int tensor [n_rows, draws_per_row]; row_status is
    updated in place."""
    lib = load_library()
    d = draws.to(torch.int32).contiguous()
    n, dpr = d.shape
    tok = torch.empty((n, dpr), dtype=torch.int32, device=d.device)
    q = _qstruct(qd)
    _check(lib.dspark_sample(ctypes.byref(q), n, vocab, _p(d), dpr, _p(tok), _p(row_status), _stream()))
    return tok


def verify_greedy(target: torch.Tensor, draft_tokens: torch.Tensor, draft_status=None):
    lib = load_library()
    R, dev = draft_tokens.shape[0], target.device
    t = _rows(target)
    out = {k: _i32(R * 6, dev) for k in ("target_argmax", "target_status")}
    out.update({k: _i32(R, dev) for k in ("accept_len", "bonus", "req_status")})
    dt = draft_tokens.to(torch.int32).contiguous()
    ds = None if draft_status is None else draft_status.to(torch.int32).contiguous()
    _check(lib.dspark_verify_greedy(ctypes.byref(t), _p(dt), _p(ds), R, _p(out["target_argmax"]),
                                    _p(out["target_status"]), _p(out["accept_len"]), _p(out["bonus"]),
                                    _p(out["req_status"]), None, 0, _stream()))
    return out


def fused(draft: torch.Tensor, target: torch.Tensor, mode: int, topk=None, k_max: int = 0, draws=None,
          with_q: bool = True, out=None, split: bool = True):
    """The whole step.  draft [5R, V], target [6R, V]; draws [5R] or None.
    `out` may pass preallocated outputs from an earlier call (same shapes)."""
    lib = load_library()
    n, V, dev = draft.shape[0], draft.shape[1], draft.device
    R = n // 5
    if out is None:
        out = {"argmax": _i32(n, dev), "conf": torch.empty(n, dtype=torch.float32, device=dev),
               "status": _i32(n, dev), "sample": _i32(n, dev) if draws is not None else None,
               "target_argmax": _i32(R * 6, dev), "target_status": _i32(R * 6, dev),
               "accept_len": _i32(R, dev), "bonus": _i32(R, dev), "req_status": _i32(R, dev)}
        if with_q:
            tk = _topk(topk, dev)
            want_dense = tk is None or bool((tk == 0).any())
            out["q"] = _make_q(n, V, dev, tk, k_max, want_dense)
        else:
            out["q"] = None
        out["draws"] = None if draws is None else draws.to(torch.int32).contiguous()
        out["_ws"] = _split_ws(draft, 4, split and with_q)
    d, t = _rows(draft), _rows(target)
    q = None if out["q"] is None else ctypes.byref(_qstruct(out["q"]))
    _, wp, wb = out["_ws"]
    _check(lib.dspark_fused(ctypes.byref(d), ctypes.byref(t), mode, q, _p(out["draws"]), _p(out["argmax"]),
                            _p(out["conf"]), _p(out["sample"]), _p(out["status"]), _p(out["target_argmax"]),
                            _p(out["target_status"]), _p(out["accept_len"]), _p(out["bonus"]),
                            _p(out["req_status"]), wp, wb, _stream()))
    return out


def q_alloc_weights(w: torch.Tensor):
    lib = load_library()
    if w.dim() != 2 or w.dtype != torch.float32 or w.stride(1) != 1:
        raise ValueError("w must be a 2-D float32 tensor with unit column stride")
    n_rows, n = w.shape
    counts = torch.empty((n_rows, n), dtype=torch.int32, device=w.device)
    st = _i32(n_rows, w.device)
    _check(lib.dspark_q_alloc_weights(_p(w), n_rows, n, w.stride(0), _p(counts), _p(st), None, 0, _stream()))
    return counts, st


def cr_expf(d: torch.Tensor):
    lib = load_library()
    d = d.contiguous()
    w = torch.empty_like(d)
    _check(lib.dspark_cr_expf(_p(d), _p(w), d.numel(), _stream()))
    return w


def q_encode(counts: torch.Tensor, out: torch.Tensor | None = None):
    """Wire values counts / 2**24 (float32, same shape).  `out` may be the
    counts tensor itself viewed as float32 (in-place encoding)."""
    lib = load_library()
    c = counts.contiguous()
    if out is None:
        out = torch.empty(c.shape, dtype=torch.float32, device=c.device)
    _check(lib.dspark_q_encode(_p(c), c.numel(), _p(out), _stream()))
    return out


def q_validate(vocab: int, topk=None, k_max: int = 0, dense=None, sp_ids=None, sp_val=None, sp_len=None,
               tokens=None, padded=None, want_counts: bool = False):
    """Receiver check of wire q rows.  dense: float32 [n_rows, stride] with
    `padded` (default vocab) values sent per row; sp_*: [n_rows, k_max] and
    [n_rows].  Returns {"status", "dense_counts", "sp_counts"}."""
    lib = load_library()
    ref = dense if dense is not None else sp_len
    n_rows, dev = ref.shape[0], ref.device
    tk = _topk(topk, dev)
    padded = vocab if padded is None else int(padded)
    if dense is not None and (dense.dim() != 2 or dense.stride(1) != 1 or dense.dtype != torch.float32):
        raise ValueError("dense must be a 2-D float32 tensor with unit column stride")
    q = QWire(_p(tk), int(k_max), 0, _p(dense), padded, 0 if dense is None else dense.stride(0),
              _p(sp_ids), _p(sp_val), _p(sp_len))
    st = _i32(n_rows, dev)
    dc = torch.empty((n_rows, vocab), dtype=torch.int32, device=dev) if want_counts and dense is not None else None
    sc = (torch.empty((n_rows, k_max), dtype=torch.int32, device=dev)
          if want_counts and tk is not None and k_max > 0 else None)
    tok = None if tokens is None else tokens.to(torch.int32).contiguous()
    _check(lib.dspark_q_validate(ctypes.byref(q), n_rows, vocab, _p(tok), _p(dc), _p(sc), _p(st), _stream()))
    return {"status": st, "dense_counts": dc, "sp_counts": sc}


def margin(rows: torch.Tensor):
    """top1 - top2 of every row (float32 [n_rows])."""
    lib = load_library()
    r = _rows(rows)
    out = torch.empty(rows.shape[0], dtype=torch.float32, device=rows.device)
    _check(lib.dspark_margin(ctypes.byref(r), _p(out), _stream()))
    return out


def u64_draws(a, dev) -> torch.Tensor:
    """64-bit draws (numpy uint64 or int64 array, or a tensor) as an int64
    device tensor holding the same bits."""
    if isinstance(a, torch.Tensor):
        return a.to(dev, torch.int64).contiguous()
    import numpy as np
    arr = np.ascontiguousarray(a)
    if arr.dtype == np.uint64:
        arr = arr.view(np.int64)
    return torch.from_numpy(arr.astype(np.int64, copy=False)).to(dev)


def verify_stochastic(target: torch.Tensor, draft_tokens: torch.Tensor, target_draws, draft_status=None,
                      out=None):
    """target [6R, V]; draft_tokens [R, 5]; target_draws: 64-bit draws [R, 6]
    (see u64_draws).  `out` may pass the outputs of an earlier call."""
    lib = load_library()
    R, dev = draft_tokens.shape[0], target.device
    if out is None:
        out = {"target_sample": _i32(6 * R, dev), "target_status": _i32(6 * R, dev),
               "accept_len": _i32(R, dev), "bonus": _i32(R, dev), "req_status": _i32(R, dev)}
    t = _rows(target)
    dt = draft_tokens.to(torch.int32).contiguous()
    ds = None if draft_status is None else draft_status.to(torch.int32).contiguous()
    dr = u64_draws(target_draws, dev)
    _check(lib.dspark_verify_stochastic(ctypes.byref(t), _p(dt), _p(ds), R, _p(dr), _p(out["target_sample"]),
                                        _p(out["target_status"]), _p(out["accept_len"]), _p(out["bonus"]),
                                        _p(out["req_status"]), _stream()))
    return out


def verify_ratio(target: torch.Tensor, draft_tokens: torch.Tensor, qd, accept_draws, final_draws,
                 draft_status=None, out=None):
    """Probability-ratio verification.  target [6R, V]; draft_tokens [R, 5];
    qd: the draft rows' q (a dict as q_alloc / fused return it); accept_draws
    64-bit [R, 5]; final_draws 64-bit [R].  Returns accept_len, token,
    req_status (int32 [R])."""
    lib = load_library()
    R, dev = draft_tokens.shape[0], target.device
    if out is None:
        out = {"accept_len": _i32(R, dev), "token": _i32(R, dev), "req_status": _i32(R, dev)}
    t = _rows(target)
    dt = draft_tokens.to(torch.int32).contiguous()
    ds = None if draft_status is None else draft_status.to(torch.int32).contiguous()
    ad, fd = u64_draws(accept_draws, dev), u64_draws(final_draws, dev)
    q = _qstruct(qd)
    _check(lib.dspark_verify_ratio(ctypes.byref(t), _p(dt), _p(ds), ctypes.byref(q), R, _p(ad), _p(fd),
                                   _p(out["accept_len"]), _p(out["token"]), _p(out["req_status"]), _stream()))
    return out


def sharded_propose(rows: torch.Tensor, n_shards: int):
    """Vocabulary-sharded propose emulated on one GPU: argmax, exact-sum S64,
    confidence and status of every row, from n_shards shard workgroups."""
    lib = load_library()
    n, dev = rows.shape[0], rows.device
    out = {"argmax": _i32(n, dev), "s64": torch.empty(n, dtype=torch.float64, device=dev),
           "conf": torch.empty(n, dtype=torch.float32, device=dev), "status": _i32(n, dev)}
    ws = torch.empty(max(1, 48 * n * n_shards), dtype=torch.uint8, device=dev)
    r = _rows(rows)
    _check(lib.dspark_sharded_propose(ctypes.byref(r), int(n_shards), _p(out["argmax"]), _p(out["s64"]),
                                      _p(out["conf"]), _p(out["status"]), _p(ws), ws.numel(), _stream()))
    return out


def sharded_propose_noalloc(rows: torch.Tensor, n_shards: int, out=None):
    """sharded_propose through the allocation-free entry point (the shard
    results stay in the library's device scratch).  `out` may pass the
    outputs of an earlier call."""
    lib = load_library()
    n, dev = rows.shape[0], rows.device
    if out is None:
        out = {"argmax": _i32(n, dev), "s64": torch.empty(n, dtype=torch.float64, device=dev),
               "conf": torch.empty(n, dtype=torch.float32, device=dev), "status": _i32(n, dev)}
    r = _rows(rows)
    _check(lib.dspark_sharded_propose_noalloc(ctypes.byref(r), int(n_shards), _p(out["argmax"]), _p(out["s64"]),
                                              _p(out["conf"]), _p(out["status"]), _stream()))
    return out


def sharded_q(rows: torch.Tensor, n_shards: int, topk=None, k_max: int = 0, draws=None, out=None):
    """The vocabulary-sharded q (dense rows with globally coordinated
    tickets, sparse rows from merged shard top-k) and, with draws, the
    shard-then-token sample; the same outputs as q_alloc plus argmax.  `out`
    may pass the outputs (and workspace) of an earlier call."""
    lib = load_library()
    n, V, dev = rows.shape[0], rows.shape[1], rows.device
    if out is None:
        tk = _topk(topk, dev)
        want_dense = tk is None or bool((tk == 0).any())
        out = _make_q(n, V, dev, tk, k_max, want_dense)
        nbytes = int(lib.dspark_sharded_q_workspace(n, int(n_shards), int(k_max)))
        ws = torch.empty(max(nbytes, 1) + 256, dtype=torch.uint8, device=dev)
        out.update({"status": _i32(n, dev), "argmax": _i32(n, dev),
                    "sample": None if draws is None else _i32(n, dev),
                    "_ws": ws, "_ws_ptr": ws.data_ptr() + (-ws.data_ptr()) % 256, "_ws_bytes": nbytes})
    d = None if draws is None else draws.to(torch.int32).contiguous()
    r, q = _rows(rows), _qstruct(out)
    _check(lib.dspark_sharded_q(ctypes.byref(r), int(n_shards), ctypes.byref(q), _p(d), _p(out["argmax"]),
                                _p(out["sample"]), _p(out["status"]), ctypes.c_void_p(out["_ws_ptr"]),
                                out["_ws_bytes"], _stream()))
    return out


# ---- operators on logit rows: shaping, a teacher's top logits, distillation.
# Their work runs on the rows' device and on that device's current stream.
# Rows that they read or write start 16-byte aligned, as everywhere in the
# library: a contiguous [n, V] tensor has such rows where V is a multiple of 8
# (bf16) or 4 (float32); for other V, rows are the first V columns of a wider
# tensor, and unaligned ones are refused (DsparkError).


def _arg(t, name, dtype, shape, dev):
    """Address of a contiguous argument tensor (None stays None)."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {dev}, "
                         f"not {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _matrix(t, name, dtype, n, dev):
    """(address, columns, row stride) of an [n, columns] argument with unit column stride."""
    if t is None:
        return None, 0, 0
    shape = t.shape
    if t.dtype != dtype or len(shape) != 2 or shape[0] != n or t.device != dev:
        raise ValueError(f"{name} must be a 2-D {dtype} tensor with {n} rows on {dev}")
    cols = shape[1]
    if t.is_contiguous():
        return t.data_ptr(), cols, cols
    if (cols > 1 and t.stride(1) != 1) or (n > 1 and t.stride(0) < cols):
        raise ValueError(f"{name} must have unit column stride and rows that do not overlap")
    return t.data_ptr(), cols, max(t.stride(0), cols)


def _padded(V, dtype):
    """The row stride that keeps rows of V values 16-byte aligned."""
    return -(-V * dtype.itemsize // 16) * 16 // dtype.itemsize


def _empty_rows(n, V, dtype, dev):
    """Rows [n, V] that start 16-byte aligned."""
    wide = _padded(V, dtype)
    rows = torch.empty((n, wide), dtype=dtype, device=dev)
    return rows if wide == V else rows[:, :V]


def _out_rows(out, like, dtype):
    if out is None:
        return _empty_rows(like.shape[0], like.shape[1], dtype, like.device)
    if out.shape != like.shape or out.dtype != dtype or out.device != like.device or out.stride(1) != 1:
        raise ValueError(f"out must be a {dtype} tensor of shape {tuple(like.shape)} with unit column stride on {like.device}")
    return out


def _written(out):
    """Rows of the caller that the library has written count as written in place: torch refuses a backward pass that
    saved them."""
    if out is not None:
        torch.autograd.graph.increment_version(out)


# the current stream's handle, without a torch.cuda.Stream around it where torch offers that (2 us less per call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(dev, f, *args):
    """The library call on dev's current stream, with dev current."""
    if dev.index == torch.cuda.current_device():
        rc = f(*args, _raw_stream(dev.index))
    else:
        with torch.cuda.device(dev):
            rc = f(*args, _raw_stream(dev.index))
    if rc != 0:
        _check(rc)


def shape_logits(rows: torch.Tensor, rows_per_request: int = 1, *, history=None, history_len=None, prompt_len=None,
                 draft=None, repetition=None, frequency=None, presence=None, temperature=None, bias=None, mask=None,
                 mask_row=None, out=None, out_dtype=None):
    """Final logits from raw ones: penalties for repeated tokens, biases,
    temperature and grammar masks (see dspark_shape_logits).  rows [n, V],
    rows_per_request of them for each of the n / rows_per_request requests.
    history int32 [requests, most] with history_len and prompt_len int32
    [requests] (history_len None: every row is full); draft int32 [requests,
    at least rows_per_request - 1]; the penalties and temperature float32
    [requests]; bias (offsets int64 [requests + 1], ids int32, values float32);
    mask int32 (packed bits) [masks, at least (V + 31) // 32] with mask_row
    int32 [n].  out: rows to write, which may be `rows` itself; out_dtype: the
    rows' type (default) or float32.  Returns {"logits", "status"}."""
    lib = load_library()
    r = _rows(rows)
    n, V, dev = rows.shape[0], rows.shape[1], rows.device
    P = int(rows_per_request)
    if P < 1 or n % P:
        raise ValueError("the number of rows must be a multiple of rows_per_request")
    R = n // P
    o = _out_rows(out, rows, out_dtype or (rows.dtype if out is None else out.dtype))
    if o.dtype not in (torch.float32, rows.dtype):
        raise ValueError("out_dtype must be the rows' type or float32")
    h, h_max, h_stride = _matrix(history, "history", torch.int32, R, dev)
    if history is not None and history_len is None:
        history_len = torch.full((R,), h_max, dtype=torch.int32, device=dev)
    if history is not None and h_max == 0:
        h = history_len.data_ptr()  # nothing to read, but the lengths are still checked
    d, d_cols, d_stride = _matrix(draft, "draft", torch.int32, R, dev)
    if draft is not None and d_cols < P - 1:
        raise ValueError("draft must have at least rows_per_request - 1 columns")
    m, m_cols, m_stride = (None, 0, 0) if mask is None else _matrix(mask, "mask", torch.int32, mask.shape[0], dev)
    if mask_row is not None and mask is None:
        raise ValueError("mask_row needs mask")
    if history is None and (history_len is not None or prompt_len is not None):
        raise ValueError("history_len and prompt_len need history")
    if mask is not None and (m_cols < (V + 31) // 32 or mask.shape[0] == 0):
        raise ValueError("mask must have rows of at least (V + 31) // 32 columns")
    offsets, ids, values = bias if bias is not None else (None, None, None)
    if bias is not None and (offsets is None or ids is None or values is None):
        raise ValueError("bias must be (offsets, ids, values)")
    total = 0 if ids is None else ids.numel()
    i32, f32 = torch.int32, torch.float32
    how = Shaping(P, 0, h, h_max, h_stride, _arg(history_len, "history_len", i32, (R,), dev),
                  _arg(prompt_len, "prompt_len", i32, (R,), dev), d, d_stride,
                  _arg(repetition, "repetition", f32, (R,), dev), _arg(frequency, "frequency", f32, (R,), dev),
                  _arg(presence, "presence", f32, (R,), dev), _arg(temperature, "temperature", f32, (R,), dev),
                  _arg(offsets, "bias offsets", torch.int64, (R + 1,), dev), _arg(ids, "bias ids", i32, (total,), dev),
                  _arg(values, "bias values", f32, (total,), dev), total,
                  m, m_stride, 0 if mask is None else mask.shape[0], _arg(mask_row, "mask_row", i32, (n,), dev))
    st = _i32(n, dev)
    _call(dev, lib.dspark_shape_logits, ctypes.byref(r), ctypes.byref(how), o.data_ptr(),
          DTYPE_F32 if o.dtype == torch.float32 else DTYPE_BF16, o.stride(0), st.data_ptr())
    _written(out)
    return {"logits": o, "status": st}


def top_logits(rows: torch.Tensor, k_max: int, topk=None, temperature: float = 1.0):
    """The k_max (or per row topk, int32 [n]) largest finite logits of every
    row by ascending id, and the log-sum-exp of the row over temperature (see
    dspark_top_logits): {"ids", "logits", "len", "lse", "status"}, a teacher
    for distill at that temperature."""
    lib = load_library()
    r = _rows(rows)
    n, V, dev = rows.shape[0], rows.shape[1], rows.device
    k = int(k_max)
    if k < 0 or k > K_MAX:
        raise ValueError("k_max must be in [0, K_MAX]")
    ids, logits = torch.empty((n, k), dtype=torch.int32, device=dev), torch.empty((n, k), dtype=torch.float32, device=dev)
    length, lse, st = _i32(n, dev), torch.empty(n, dtype=torch.float32, device=dev), _i32(n, dev)
    nbytes = lib.dspark_top_logits_workspace(n, V, k)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    _call(dev, lib.dspark_top_logits, ctypes.byref(r), _arg(topk, "topk", torch.int32, (n,), dev), k, float(temperature),
          ids.data_ptr(), logits.data_ptr(), length.data_ptr(), lse.data_ptr(), st.data_ptr(),
          ws.data_ptr() if nbytes else None, nbytes)
    return {"ids": ids, "logits": logits, "len": length, "lse": lse, "status": st}


def _teacher(t, n, dev) -> Teacher:
    ids = t["ids"]
    if ids.dim() != 2 or ids.shape[1] > K_MAX:
        raise ValueError("teacher ids must be [rows, at most K_MAX]")
    k = ids.shape[1]
    return Teacher(_arg(ids, "teacher ids", torch.int32, (n, k), dev),
                   _arg(t["logits"], "teacher logits", torch.float32, (n, k), dev),
                   _arg(t["len"], "teacher len", torch.int32, (n,), dev),
                   _arg(t.get("lse"), "teacher lse", torch.float32, (n,), dev), k, 0)


def _distill_ws(nbytes, dev):
    return (torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None), nbytes


def _distill(student, teacher, temperature):
    """distill's outputs, and its arguments as the library takes them."""
    lib = load_library()
    r = _rows(student)
    n, V, dev = student.shape[0], student.shape[1], student.device
    t = _teacher(teacher, n, dev)
    loss, st = torch.empty(n, dtype=torch.float32, device=dev), _i32(n, dev)
    stats = torch.empty((n, DISTILL_STATS), dtype=torch.float64, device=dev)
    ws, nbytes = _distill_ws(lib.dspark_distill_workspace(n, V), dev)
    _call(dev, lib.dspark_distill, ctypes.byref(r), ctypes.byref(t), float(temperature), loss.data_ptr(),
          stats.data_ptr(), st.data_ptr(), ws.data_ptr() if nbytes else None, nbytes)
    return loss, stats, st, r, t


def distill(student: torch.Tensor, teacher, temperature: float = 1.0):
    """Distillation loss of every student row [n, V] against a teacher's top
    logits (see dspark_distill).  teacher: {"ids", "logits", "len", "lse"} as
    top_logits returns it at the same temperature; without "lse" (or None)
    the teacher is renormalised over its list.  Returns {"loss", "stats",
    "status"}; stats and status go to distill_backward."""
    loss, stats, st, _, _ = _distill(student, teacher, temperature)
    return {"loss": loss, "stats": stats, "status": st}


def distill_backward(student: torch.Tensor, teacher, forward, grad_loss: torch.Tensor, temperature: float = 1.0,
                     out=None):
    """Gradient of sum(grad_loss * loss) with respect to the student rows;
    forward: what distill returned for the same arguments.  out may be the
    student rows themselves (overwritten)."""
    lib = load_library()
    r = _rows(student)
    n, dev = student.shape[0], student.device
    t = _teacher(teacher, n, dev)
    g = _out_rows(out, student, student.dtype)
    _call(dev, lib.dspark_distill_backward, ctypes.byref(r), ctypes.byref(t), float(temperature),
          _arg(forward["stats"], "stats", torch.float64, (n, DISTILL_STATS), dev),
          _arg(forward["status"], "status", torch.int32, (n,), dev),
          _arg(grad_loss, "grad_loss", torch.float32, (n,), dev), g.data_ptr(), g.stride(0))
    _written(out)
    return g


def distill_step(student: torch.Tensor, teacher, weight: torch.Tensor, temperature: float = 1.0, out=None):
    """Loss of every row (unweighted) and the gradient of sum(weight * loss)
    in one call: {"loss", "grad", "status"}.  out as in distill_backward."""
    lib = load_library()
    r = _rows(student)
    n, V, dev = student.shape[0], student.shape[1], student.device
    t = _teacher(teacher, n, dev)
    g = _out_rows(out, student, student.dtype)
    loss, st = torch.empty(n, dtype=torch.float32, device=dev), _i32(n, dev)
    w = _arg(weight, "weight", torch.float32, (n,), dev)
    ws, nbytes = _distill_ws(lib.dspark_distill_workspace(n, V), dev)
    _call(dev, lib.dspark_distill_step, ctypes.byref(r), ctypes.byref(t), float(temperature), w, loss.data_ptr(),
          g.data_ptr(), g.stride(0), st.data_ptr(), ws.data_ptr() if nbytes else None, nbytes)
    _written(out)
    return {"loss": loss, "grad": g, "status": st}


def _places(student, ids, logits, length, lse):
    return (student.data_ptr(), student.stride(), ids.data_ptr(), logits.data_ptr(), length.data_ptr(),
            None if lse is None else lse.data_ptr())


def _distill_grad(ctx, grad_loss):
    # forward has checked the arguments and laid them out: on torch's backward thread Python takes three times as long
    saved = ctx.saved_tensors  # (and torch has checked that nobody wrote to them since)
    r, t, stats, status, shape, V, dev, at = ctx.laid_out
    if _places(*saved) != at:  # a hook on saved tensors gave back others
        student, ids, logits, length, lse = saved
        if student.stride(1) != 1 or (student.data_ptr() | student.stride(0) * student.element_size()) % 16:
            student = _empty_rows(shape[0], V, student.dtype, dev).copy_(student)
        r, t = _rows(student), _teacher({"ids": ids, "logits": logits, "len": length, "lse": lse}, shape[0], dev)
    if grad_loss.dtype is not torch.float32 or not grad_loss.is_contiguous():
        grad_loss = grad_loss.to(torch.float32).contiguous()
    g = torch.empty(shape, dtype=saved[0].dtype, device=dev)
    _call(dev, _LIB.dspark_distill_backward, ctypes.byref(r), ctypes.byref(t), ctx.temperature, stats.data_ptr(),
          status.data_ptr(), grad_loss.data_ptr(), g.data_ptr(), shape[1])
    return g if shape[1] == V else g[:, :V], None, None, None, None, None


class _DistillLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, student, ids, logits, length, lse, temperature):
        loss, stats, st, r, t = _distill(student, {"ids": ids, "logits": logits, "len": length, "lse": lse}, temperature)
        ctx.save_for_backward(student, ids, logits, length, lse)
        n, V = student.shape
        ctx.laid_out = (r, t, stats, st, (n, _padded(V, student.dtype)), V, student.device,
                         _places(student, ids, logits, length, lse))
        ctx.temperature = temperature
        return loss

    @staticmethod
    def backward(ctx, grad_loss):
        if torch.is_grad_enabled():  # a graph of the gradient is asked for: its derivative is refused
            return torch.autograd.function.once_differentiable(_distill_grad)(ctx, grad_loss)
        return _distill_grad(ctx, grad_loss)


def distill_loss(student: torch.Tensor, teacher, temperature: float = 1.0) -> torch.Tensor:
    """distill's loss (float32 [n]) as a differentiable function of the
    student rows, which start 16-byte aligned (other V than multiples of 8 in
    bf16, 4 in float32: the first V columns of a wider tensor).  The teacher is
    constant: its logits must not require a
    gradient.  Rows that the call refuses have loss 0 and gradient 0.  It may be
    captured into a graph with its backward pass, while no eager graph of the
    same leaves is alive."""
    if teacher["logits"].requires_grad or (teacher.get("lse") is not None and teacher["lse"].requires_grad):
        raise ValueError("the teacher is constant: detach its logits and lse")
    return _DistillLoss.apply(student, teacher["ids"], teacher["logits"], teacher["len"], teacher.get("lse"),
                              float(temperature))


# ---- the vocabulary head in 8-bit floating point: quantisation in blocks of
# 128, the product that makes logit rows, and its gradient.  A quantised
# matrix is {"values": float8_e4m3fn [rows, cols], "scales"}: cols a multiple
# of 16, the last ones zeros where the matrix is narrower; scales float32 or
# float8_e8m0fnu, one for each 128 columns of a row (hidden states, gradients)
# or of 128 rows (weights).


def _fp8(q, name, block_rows, dev) -> Fp8:
    values, scales = q["values"], q["scales"]
    if values.dtype != torch.float8_e4m3fn or values.dim() != 2 or values.device != dev:
        raise ValueError(f"{name} values must be a 2-D float8_e4m3fn tensor on {dev}")
    n, cols = values.shape
    blocks = (-(-n // block_rows), -(-cols // 128))
    if scales.dtype not in (torch.float32, torch.float8_e8m0fnu) or scales.shape != blocks or scales.device != dev:
        raise ValueError(f"{name} scales must be a float32 or float8_e8m0fnu tensor of shape {blocks} on {dev}")
    if cols % 16 or cols == 0:
        raise ValueError(f"{name} must have a multiple of 16 columns (fill up with zeros)")
    if values.stride(1) != 1 or (n > 1 and values.stride(0) < cols):
        raise ValueError(f"{name} values must have unit column stride and rows that do not overlap")
    if (blocks[1] > 1 and scales.stride(1) != 1) or (blocks[0] > 1 and scales.stride(0) < blocks[1]):
        raise ValueError(f"{name} scales must have unit column stride and rows that do not overlap")
    return Fp8(values.data_ptr(), scales.data_ptr(), SCALE_F32 if scales.dtype == torch.float32 else SCALE_E8M0,
               block_rows, n, cols, values.stride(0) if n > 1 else cols, scales.stride(0) if blocks[0] > 1 else blocks[1])


def quantize_blocks(x: torch.Tensor, block_rows: int = 1, scale_dtype=torch.float32):
    """Rows x [n, width] in e4m3 with a scale for each 128 columns of
    block_rows (1 or 128) rows (see dspark_quantize_blocks): {"values"
    float8_e4m3fn [n, width rounded up to a multiple of 16], "scales"}.
    scale_dtype: float32, or float8_e8m0fnu for powers of two.  No gradient
    flows through it."""
    lib = load_library()
    r = _rows(x)
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    if scale_dtype not in (torch.float32, torch.float8_e8m0fnu):
        raise ValueError("scale_dtype must be float32 or float8_e8m0fnu")
    n, width = x.shape
    dev, cols, blocks = x.device, -(-width // 16) * 16, -(-width // 128)
    values = torch.empty((n, cols), dtype=torch.float8_e4m3fn, device=dev)
    scales = torch.empty((-(-n // block_rows), blocks), dtype=scale_dtype, device=dev)
    f = Fp8(values.data_ptr(), scales.data_ptr(), SCALE_F32 if scale_dtype is torch.float32 else SCALE_E8M0, block_rows, n, cols, cols, blocks)
    _call(dev, lib.dspark_quantize_blocks, ctypes.byref(r), ctypes.byref(f))
    return {"values": values, "scales": scales}


def transpose_blocks(w, cols: int):
    """The transpose of a quantised weight matrix whose first `cols` columns
    are its own (the rest fill up): what head_logits needs for the gradient.
    It is laid out once, with torch."""
    values, scales = w["values"], w["scales"]
    n = values.shape[0]
    if not 0 < cols <= values.shape[1]:
        raise ValueError("cols must be in [1, the matrix's columns]")
    t = torch.zeros((cols, -(-n // 16) * 16), dtype=torch.uint8, device=values.device)
    t[:, :n] = values.view(torch.uint8)[:, :cols].t()
    return {"values": t.view(torch.float8_e4m3fn), "scales": scales[:, :-(-cols // 128)].t().contiguous()}


def _product_out(n, V, out, out_dtype, dev):
    if out is None:
        out = _empty_rows(n, V, out_dtype, dev)
    elif out.shape != (n, V) or out.dtype != out_dtype or out.device != dev or out.stride(1) != 1 or (n > 1 and out.stride(0) < V):
        raise ValueError(f"out must be a {out_dtype} tensor of shape {(n, V)} with unit column stride on {dev}")
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("out_dtype must be float32 or bfloat16")
    return out, DTYPE_F32 if out_dtype == torch.float32 else DTYPE_BF16, out.stride(0) if n > 1 else max(out.stride(0), V)


@functools.lru_cache(maxsize=1024)
def _head_workspace(call, n, V, cols):
    return getattr(load_library(), f"dspark_{call}_workspace")(n, V, cols)


def block_product(x, w, out_dtype=torch.bfloat16, out=None) -> torch.Tensor:
    """Logit rows [n, V] of quantised rows x (a scale for each row's blocks)
    and a quantised matrix w of V rows (a scale for blocks of 128 rows), both
    with scales of one type (see dspark_block_product).  out: rows to write.
    No gradient flows through it."""
    lib = load_library()
    dev = x["values"].device
    fx, fw = _fp8(x, "x", 1, dev), _fp8(w, "w", 128, dev)
    o, dt, stride = _product_out(fx.n_rows, fw.n_rows, out, out_dtype, dev)
    nbytes = _head_workspace("block_product", fx.n_rows, fw.n_rows, fx.cols)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    _call(dev, lib.dspark_block_product, ctypes.byref(fx), ctypes.byref(fw), o.data_ptr(), dt, stride,
          ws.data_ptr() if nbytes else None, nbytes)
    _written(out)
    return o


def block_linear(x: torch.Tensor, w, out_dtype=None, out=None) -> torch.Tensor:
    """The same from rows x [n, width] in float32 or bf16, quantised on the
    way (see dspark_block_linear); out_dtype: x's type by default.  No gradient
    flows through it, whatever x requires: head_logits is the differentiable
    form."""
    lib = load_library()
    r = _rows(x)
    n, dev = x.shape[0], x.device
    fw = _fp8(w, "w", 128, dev)
    o, dt, stride = _product_out(n, fw.n_rows, out, out_dtype or (x.dtype if out is None else out.dtype), dev)
    nbytes = _head_workspace("block_linear", n, fw.n_rows, x.shape[1])
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    _call(dev, lib.dspark_block_linear, ctypes.byref(r), ctypes.byref(fw), o.data_ptr(), dt, stride,
          ws.data_ptr() if nbytes else None, nbytes)
    _written(out)
    return o


def _aligned_rows(x):
    """x itself, or a copy whose rows start 16-byte aligned."""
    if x.stride(1) == 1 and x.stride(0) >= x.shape[1] and (x.data_ptr() | x.stride(0) * x.element_size()) % 16 == 0:
        return x
    return _empty_rows(x.shape[0], x.shape[1], x.dtype, x.device).copy_(x)


def _head_grad(ctx, grad):
    values, scales = ctx.saved_tensors
    return block_linear(_aligned_rows(grad), {"values": values, "scales": scales}, ctx.dtype), None, None


class _HeadLogits(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, head, out_dtype):
        t = head["transposed"]
        ctx.save_for_backward(t["values"], t["scales"])
        ctx.dtype = x.dtype
        return block_linear(x, head["weight"], out_dtype)

    @staticmethod
    def backward(ctx, grad):
        if torch.is_grad_enabled():  # a graph of the gradient is asked for: its derivative is refused
            return torch.autograd.function.once_differentiable(_head_grad)(ctx, grad)
        return _head_grad(ctx, grad)


def _no_tangents(x, w, t):
    if forward_ad.unpack_dual(x).tangent is not None:
        raise NotImplementedError("head_logits has no forward-mode derivative")
    if any(forward_ad.unpack_dual(q[k]).tangent is not None for q in (w, t) if q is not None for k in ("values", "scales")):
        raise ValueError("the head is constant: detach it")


def head_logits(x: torch.Tensor, head, out_dtype=None) -> torch.Tensor:
    """Logits [n, V] of hidden states x [n, width] (float32 or bf16, rows
    16-byte aligned) and a head {"weight": a quantised matrix [V, width],
    "transposed": transpose_blocks(weight, width)}, a differentiable function
    of x: the logits' gradient is quantised in blocks of 128 tokens, as x is in
    blocks of 128 channels, and multiplied with the transposed head.  (An entry
    below a 460,000th of its block's largest, a label's, say, becomes zero: see
    dspark_block_linear.)  The head is constant; without a gradient "transposed"
    is not needed.  There is no forward-mode derivative, nor a second one.  It
    may be captured into a graph with its backward pass, while no eager graph of
    the same leaves is alive."""
    w, t, grad = head["weight"], head.get("transposed"), torch.is_grad_enabled()
    if getattr(forward_ad, "_current_level", 0) >= 0:  # (without a dual level there is none: not looked for, 3 us less)
        _no_tangents(x, w, t)
    if grad and (w["values"].requires_grad or w["scales"].requires_grad or
                 (t is not None and (t["values"].requires_grad or t["scales"].requires_grad))):
        raise ValueError("the head is constant: detach it")
    if x.requires_grad and grad:
        if t is None:
            raise ValueError('the gradient needs head["transposed"] (see transpose_blocks)')
        if x.dim() != 2 or t["values"].shape[0] != x.shape[1]:
            raise ValueError('head["transposed"] must have a row for each channel of x')
        if t["values"].shape[1] != -(-head["weight"]["values"].shape[0] // 16) * 16:
            raise ValueError('head["transposed"] must have a column for each token, filled up to a multiple of 16')
        return _HeadLogits.apply(x, head, out_dtype)
    return block_linear(x, head["weight"], out_dtype)


# ---- beam search on logit rows.


def beam_select(rows: torch.Tensor, scores: torch.Tensor, n_out: int | None = None, *, finished=None, end_token: int = -1):
    """The n_out (default: twice the beams, or as many as a call may select) best
    continuations of each request's beams (see dspark_beam_select).  rows
    [requests * beams, V]; scores float32 [requests, beams], -inf for an empty
    slot; finished int32 [requests, beams], nonzero for an ended beam, which
    continues with end_token at its score.  Returns {"parent", "token",
    "score", "finished"} ([requests, n_out]), "len" and "status" ([requests])."""
    lib = load_library()
    r = _rows(rows)
    n, V, dev = rows.shape[0], rows.shape[1], rows.device
    if scores.dim() != 2 or scores.numel() != n:
        raise ValueError("scores must be [requests, beams] with a row of logits for each")
    R, beams = scores.shape
    k = min(2 * beams, BEAM_OUT_MAX, 4096 // max(beams, 1)) if n_out is None else int(n_out)
    i32 = torch.int32
    s, f = _arg(scores, "scores", torch.float32, (R, beams), dev), _arg(finished, "finished", i32, (R, beams), dev)
    # (few allocations: each costs the host as much as a tenth of a small call)
    parent, token, ended = torch.empty((3, R, max(k, 0)), dtype=i32, device=dev).unbind()
    score = torch.empty((R, max(k, 0)), dtype=torch.float32, device=dev)
    length, st = torch.empty((2, R), dtype=i32, device=dev).unbind()
    nbytes = lib.dspark_beam_select_workspace(n, V, k)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    _call(dev, lib.dspark_beam_select, ctypes.byref(r), s, f, beams, k, int(end_token), parent.data_ptr(), token.data_ptr(),
          score.data_ptr(), ended.data_ptr(), length.data_ptr(), st.data_ptr(), ws.data_ptr() if nbytes else None, nbytes)
    return {"parent": parent, "token": token, "score": score, "finished": ended, "len": length, "status": st}


@functools.lru_cache(maxsize=1024)
def _layout(size, stride, es, axis):
    """(strides of requests, beams, outer, positions in bytes), (outer, positions, bytes of a position) of a state."""
    inner, reach = 1, 1
    for d in range(len(size) - 1, min(axis, len(size) - 1), -1):
        if size[d] > 1 and stride[d] != reach:
            raise ValueError("a state's dimensions after its positions must be contiguous")
        inner, reach = inner * size[d], reach * size[d]
    if len(size) <= axis:  # no positions: everything after the beams is one row
        for d in range(len(size) - 1, 1, -1):
            if size[d] > 1 and stride[d] != inner:
                raise ValueError("a state without positions must be contiguous after its beams")
            inner *= size[d]
        return (stride[0] * es, stride[1] * es, 0, 0), (1, 0, inner * es)
    outer, step = 1, 0
    for d in range(axis - 1, 1, -1):  # the dimensions between beams and positions, as one
        if size[d] == 1:
            continue
        if outer > 1 and stride[d] != step * outer:
            raise ValueError("a state's dimensions between its beams and positions must lie evenly")
        if outer == 1:
            step = stride[d]
        outer *= size[d]
    return (stride[0] * es, stride[1] * es, step * es, stride[axis] * es), (outer, size[axis], inner * es)


def beam_reorder(states, parent: torch.Tensor, length=None, *, axis: int = 2, out=None):
    """Gives every slot the state of its parent (see dspark_beam_reorder).
    states: a sequence of tensors [requests, beams, ...] (every layer's caches,
    say), reordered in place, or into `out`, tensors of the same shapes and
    types; parent int32 [requests, beams].  length int32 [requests]: only the
    first length[r] positions, which dimension `axis` counts; states of fewer
    dimensions are taken whole.  A tensor that is written shares no element with
    any other of them (views beside each other in one tensor are fine, two
    sets of caches exchanged within one call are not).  Returns {"states",
    "status"}."""
    lib = load_library()
    states = list(states)
    if not states:
        raise ValueError("no states")
    into = states if out is None else list(out)
    if parent.dim() != 2:
        raise ValueError("parent must be [requests, beams]")
    R, beams = parent.shape
    dev = parent.device
    if not parent.is_cuda:
        raise ValueError("parent must be on the GPU")
    if axis < 2:
        raise ValueError("axis counts from the dimensions after requests and beams: 2 or more")
    if len(into) != len(states):
        raise ValueError("out must be as many tensors as states")
    laid, fewest = [], None  # State records, field by field; the positions of those that hold nothing
    for x, y in zip(states, into):
        size = x.shape
        if len(size) < 2 or size[0] != R or size[1] != beams or x.device != dev:
            raise ValueError(f"a state must be a tensor [{R}, {beams}, ...] on {dev}")
        es = x.element_size()
        strides, counts = _layout(size, x.stride(), es, axis)
        if y is x:
            to = strides
        else:
            if y.shape != size or y.dtype != x.dtype or y.device != dev:
                raise ValueError("out must be tensors of the states' shapes, types and device")
            to = _layout(size, y.stride(), es, axis)[0]
        if x.numel():
            laid += (x.data_ptr(), y.data_ptr(), *strides, *to, *counts)
        elif len(size) > axis:
            fewest = size[axis] if fewest is None else min(fewest, size[axis])
    st = _i32(R, dev)
    if not (R and beams):
        return {"states": into, "status": st.zero_()}
    if fewest is not None and length is not None:  # (the library does not see those states: their limit is put into the lengths)
        length = torch.where(length <= fewest, length, -1)
    if not laid:  # parents and lengths are still checked, with a byte for each beam in the states' place
        nothing = torch.empty((R, beams), dtype=torch.uint8, device=dev)
        strides, counts = _layout(nothing.shape, nothing.stride(), 1, axis)
        laid += (nothing.data_ptr(), nothing.data_ptr(), *strides, *strides, *counts)
    _call(dev, lib.dspark_beam_reorder, struct.pack(f"{len(laid)}q", *laid), len(laid) // 13, R, beams,
          _arg(parent, "parent", torch.int32, (R, beams), dev), _arg(length, "length", torch.int32, (R,), dev), st.data_ptr())
    torch.autograd.graph.increment_version(into)  # (as _written does)
    return {"states": into, "status": st}
