"""GB300-native batched beam-search step, KV-cache reorder and blockwise verify.

A thin ctypes binding over ``libvbs.so`` (declared in ``include/vbs.h``): every
function here only marshals torch tensors into pointers, sizes and the current
CUDA stream; all of the work runs in the library's CUDA kernels.  There is no
fallback: if the library is missing, every call raises.
"""

from __future__ import annotations

import ctypes
import os

import torch

__all__ = ["BeamSearch", "PagedKV", "PagedKV8", "CrossAttention", "kv_reorder", "bpd_propose", "bpd_verify", "VbsError", "lib",
           "LP_GNMT", "LP_POWER", "ES_FALSE", "ES_TRUE", "ES_NEVER", "F32", "BF16", "BPD_EXACT", "BPD_TOPK",
           "BPD_DISTANCE", "gather_shard_partials"]

F32, BF16 = 0, 1
I8, E4M3 = 0, 1
LP_GNMT, LP_POWER = 0, 1
BPD_EXACT, BPD_TOPK, BPD_DISTANCE = 0, 1, 2
ES_FALSE, ES_TRUE, ES_NEVER = 0, 1, 2
OK, EINVAL, ECUDA, ENOMEM, ESTATE, EALIGN, ETIMEOUT, EINPUT, ESCRATCH, EBOUNDS = 0, -1, -2, -3, -4, -5, -6, -7, -8, -9

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libvbs.so")
CHECKED_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libvbs_checked.so")

_c_int, _c_i64, _c_f, _vp = ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p
_pp = ctypes.POINTER(ctypes.c_void_p)

# name -> (restype, argtypes); mirrors include/vbs.h
SIGNATURES = {
    "vbs_strerror": (ctypes.c_char_p, [_c_int]),
    "vbs_version": (_c_int, []),
    "bs_init": (_c_int, [_pp, _c_int, _c_int, _c_int, _c_int, ctypes.c_double, _c_int, _c_int, _c_int, _c_int, _c_int,
                         _c_int, _vp]),
    "bs_reset": (_c_int, [_vp, _vp, _vp]),
    "bs_step": (_c_int, [_vp, _vp, _c_i64, _vp, _vp, _vp, _vp, _vp]),
    "bs_finalize": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp]),
    "bs_finalize_n": (_c_int, [_vp, _vp, _vp, _c_int, _vp, _vp, _vp]),
    "bs_finished": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "bs_seqs": (_c_int, [_vp, _pp]),
    "bs_steps": (_c_int, [_vp, ctypes.POINTER(_c_int)]),
    "bs_status": (_c_int, [_vp]),
    "bs_destroy": (_c_int, [_vp]),
    "bs_expand_static": (_c_int, [_vp, _c_i64, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp, _vp]),
    "kv_reorder": (_c_int, [_vp, _vp, _vp, _vp, _c_int, _c_int, _vp]),
    "vbs_stateless_status": (_c_int, [_vp]),
    "kv_paged_init": (_c_int, [_pp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _vp, _vp]),
    "kv_paged_prefill": (_c_int, [_vp, _c_int]),
    "kv_paged_build": (_c_int, [_vp, _vp, _c_i64, _vp, _vp, _vp, _vp]),
    "kv_paged_slots": (_c_int, [_vp, _c_int, _vp, _vp, _c_i64, _vp, _vp, _vp, _vp]),
    "kv8_init": (_c_int, [_pp, _vp, _c_int, _vp, _c_int, _c_int]),
    "kv8_append": (_c_int, [_vp, _c_int, _vp, _vp, _c_i64, _c_i64, _c_i64, _c_i64, _c_int, _c_i64, _vp]),
    "kv8_read": (_c_int, [_vp, _c_int, _c_i64, _vp, _vp, _vp]),
    "kv8_plan": (_c_int, [_vp, _vp, _c_int]),
    "kv8_attention": (_c_int, [_vp, _c_int, _vp, _c_i64, _c_i64, _c_i64, _c_f, _vp, _c_i64, _c_i64, _c_i64]),
    "kv8_destroy": (_c_int, [_vp]),
    "xattn_init": (_c_int, [_pp, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _vp]),
    "xattn_run": (_c_int, [_vp, _vp, _c_i64, _c_i64, _c_i64, _c_int, _vp, _c_i64, _c_i64, _c_i64, _vp, _c_i64, _c_i64,
                           _c_i64, _c_int, _vp, _c_f, _vp, _c_i64, _c_i64, _c_i64]),
    "xattn_kernel": (_c_int, [_vp, ctypes.POINTER(_c_int)]),
    "xattn_status": (_c_int, [_vp]),
    "xattn_destroy": (_c_int, [_vp]),
    "kv_paged_state": (_c_int, [_vp, _pp, _pp, _pp, _pp, _pp]),
    "kv_paged_prepare": (_c_int, [_vp, _c_int]),
    "kv_paged_reorder": (_c_int, [_vp, _vp, _c_int]),
    "bs_step_two_pass": (_c_int, [_vp, _vp, _c_i64, _vp, _vp, _vp, _vp, _vp]),
    "bs_shard_partial_bytes": (_c_int, [_vp, _vp]),
    "bs_step_shard": (_c_int, [_vp, _vp, _c_i64, _c_int, _c_int, _vp, _vp]),
    "bs_step_merge_shards": (_c_int, [_vp, _c_int, _vp, _vp, _vp, _vp, _vp, _vp]),
    "bs_step_paged": (_c_int, [_vp, _vp, _c_i64, _vp, _vp, _vp, _vp, _vp, _vp, _c_int]),
    "kv_paged_copy": (_c_int, [_vp]),
    "kv_paged_table": (_c_int, [_vp, _pp, ctypes.POINTER(_c_int)]),
    "kv_paged_counts": (_c_int, [_vp, _vp, _vp]),
    "kv_paged_copy_table": (_c_int, [_vp, _vp]),
    "kv_paged_save": (_c_int, [_vp]),
    "kv_paged_cow_slots": (_c_int, [_vp, ctypes.POINTER(_c_i64)]),
    "kv_paged_restore": (_c_int, [_vp]),
    "kv_paged_status": (_c_int, [_vp]),
    "kv_paged_destroy": (_c_int, [_vp]),
    "bpd_propose": (_c_int, [_vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp]),
    "bpd_verify": (_c_int, [_vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp]),
    "bpd_verify_approx": (_c_int, [_vp, _vp, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _vp, _vp,
                                   _vp]),
    "vbs_peak_copy": (_c_int, [_vp, _vp, _c_i64, _c_int, _vp]),
    "vbs_peak_read": (_c_int, [_vp, _c_i64, _c_int, _c_int, _vp, _vp]),
    "vbs_checked_record": (_c_int, [ctypes.POINTER(_c_int), ctypes.POINTER(_c_int), ctypes.POINTER(_c_i64)]),
}

_LIB = None


class VbsError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        msg = lib().vbs_strerror(status).decode() if _LIB is not None else str(status)
        super().__init__(f"{what}: {msg} ({status})" if what else f"{msg} ({status})")
        self.status = status


def lib():
    """Load libvbs.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m verify_bs_step_gb300._build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _LIB = L
    return _LIB


def load_checked():
    """The checked build (libvbs_checked.so: device bounds checks on), loaded with the same
    signatures; swap it in with `use_library(...)`."""
    if not os.path.exists(CHECKED_LIB_PATH):
        raise RuntimeError(f"{CHECKED_LIB_PATH} is missing: build it with `python -m verify_bs_step_gb300._build`")
    L = ctypes.CDLL(CHECKED_LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args
    return L


def use_library(L):
    """Make every call of this module go to library L (returns the one it replaces)."""
    global _LIB
    old, _LIB = _LIB, L
    return old


def checked_record():
    """(checked build?, site, index) of the first failed device bounds check since the last call."""
    c, site, idx = _c_int(), _c_int(), _c_i64()
    _check(lib().vbs_checked_record(ctypes.byref(c), ctypes.byref(site), ctypes.byref(idx)), "vbs_checked_record")
    return bool(c.value), site.value, idx.value


def _check(st: int, what: str):
    if st != OK:
        raise VbsError(st, what)


def _dev_ptr(t: torch.Tensor, name: str, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return _vp(t.data_ptr())


def _stream(device=None):
    return _vp(torch.cuda.current_stream(device).cuda_stream)


def _dtype_code(dt) -> int:
    if dt == torch.bfloat16:
        return BF16
    if dt == torch.float32:
        return F32
    raise ValueError(f"logits dtype must be bfloat16 or float32, got {dt}")


class _Context:
    """A context of the library, destroyed when its last holder lets go of it."""

    def __init__(self, ptr: _vp, destroy):
        self.ptr, self.destroy = ptr, destroy

    def __del__(self):
        try:
            self.destroy(self.ptr)
        except Exception:
            pass


class _DeviceArray:
    """Device memory of a context as an array that torch.as_tensor() takes without a copy; the tensor
    holds it, and it holds the context."""

    def __init__(self, context: _Context, ptr: int, shape, typestr: str):
        self.context = context
        self.__cuda_array_interface__ = {"data": (ptr, False), "shape": tuple(shape), "typestr": typestr,
                                         "strides": None, "version": 2}


def _raw_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# the same without making a Stream object, where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)


class _StreamOrder:
    """Orders a call on a context's stream after the work of the stream that is current when the call is
    made, and what follows it there after the call, where the two differ."""

    def __init__(self, device):
        self.device = torch.device(device)
        self.stream = torch.cuda.current_stream(self.device)
        self.index = self.stream.device.index
        self.raw = self.stream.cuda_stream

    def run(self, fn, name: str, tensors, *args):
        if _raw_stream(self.index) == self.raw:
            st = fn(*args)
            if st == OK:
                return
        else:
            cur = torch.cuda.current_stream(self.device)
            self.stream.wait_stream(cur)
            st = fn(*args)
            cur.wait_stream(self.stream)
            for t in tensors:                       # not to be reused before the context's stream is done
                t.record_stream(self.stream)
        _check(st, name)


def _cuda(t: torch.Tensor, name: str, dtype) -> int:
    if not t.is_cuda or t.dtype != dtype:
        raise ValueError(f"{name} must be a {dtype} CUDA tensor")
    return t.data_ptr()


class BeamSearch:
    """Batched beam search over `batch` sentences x W beams (libvbs bs_*).

    Holds the decode's device buffers (scores [R] fp32, seqs [R, max_len+1]
    int32, beam_idx [R], tokens [R], an all-done flag) so steps allocate nothing.
    All work goes on the stream that is current at construction.
    """

    def __init__(self, batch: int, W: int, V: int, *, eos: int = -1, alpha: float = 1.0,
                 early_stopping: int = ES_FALSE, lp_kind: int = LP_GNMT, max_len: int = 64, bos: int = 0,
                 pad: int = -1, dtype=torch.bfloat16, device="cuda"):
        self.batch, self.W, self.V, self.max_len = batch, W, V, max_len
        self.R = batch * W
        self.device = torch.device(device)
        self.dtype = dtype
        self._stream_obj = torch.cuda.current_stream(self.device)
        self.stream = _vp(self._stream_obj.cuda_stream)
        ctx = _vp()
        _check(lib().bs_init(ctypes.byref(ctx), batch, W, V, eos, alpha, early_stopping, lp_kind, max_len, bos,
                             pad, _dtype_code(dtype), self.stream), "bs_init")
        self.ctx = ctx
        dev = self.device
        self.scores = torch.empty(self.R, dtype=torch.float32, device=dev)
        self.seqs = torch.empty(self.R, max_len + 1, dtype=torch.int32, device=dev)
        self.beam_idx = torch.empty(self.R, dtype=torch.int32, device=dev)
        self.tokens = torch.empty(self.R, dtype=torch.int32, device=dev)
        self.all_done = torch.zeros(1, dtype=torch.int32, device=dev)
        self.reset()

    def reset(self):
        _check(lib().bs_reset(self.ctx, _vp(self.scores.data_ptr()), _vp(self.seqs.data_ptr())), "bs_reset")

    def step(self, logits: torch.Tensor):
        """One step on logits [R, V] (unit stride along V); returns (beam_idx, tokens, scores) views."""
        if logits.dim() != 2 or logits.shape[0] != self.R or logits.shape[1] != self.V or logits.stride(1) != 1:
            raise ValueError(f"logits must be [{self.R}, {self.V}] with unit stride along V")
        if logits.dtype != self.dtype:
            raise ValueError(f"logits must be {self.dtype}")
        _check(lib().bs_step(self.ctx, _dev_ptr(logits, "logits"), logits.stride(0), _vp(self.scores.data_ptr()),
                             _vp(self.seqs.data_ptr()), _vp(self.beam_idx.data_ptr()),
                             _vp(self.tokens.data_ptr()), _vp(self.all_done.data_ptr())), "bs_step")
        return self.beam_idx, self.tokens, self.scores

    def step_two_pass(self, logits: torch.Tensor):
        """step() through the two-pass coarse-selection ablation (reads the logits twice)."""
        if logits.dim() != 2 or logits.shape[0] != self.R or logits.shape[1] != self.V or logits.stride(1) != 1:
            raise ValueError(f"logits must be [{self.R}, {self.V}] with unit stride along V")
        if logits.dtype != self.dtype:
            raise ValueError(f"logits must be {self.dtype}")
        _check(lib().bs_step_two_pass(self.ctx, _dev_ptr(logits, "logits"), logits.stride(0),
                                      _vp(self.scores.data_ptr()), _vp(self.seqs.data_ptr()),
                                      _vp(self.beam_idx.data_ptr()), _vp(self.tokens.data_ptr()),
                                      _vp(self.all_done.data_ptr())), "bs_step_two_pass")
        return self.beam_idx, self.tokens, self.scores

    def shard_partial(self, logits_shard: torch.Tensor, v0: int) -> torch.Tensor:
        """The partial of vocabulary columns [v0, v0 + Vs) of this step's logits (a [R, Vs] view,
        unit stride along V): a uint8 device tensor of bs_shard_partial_bytes()."""
        if logits_shard.dim() != 2 or logits_shard.shape[0] != self.R or logits_shard.stride(1) != 1:
            raise ValueError(f"logits_shard must be [{self.R}, Vs] with unit stride along V")
        if logits_shard.dtype != self.dtype:
            raise ValueError(f"logits must be {self.dtype}")
        n = ctypes.c_int64()
        _check(lib().bs_shard_partial_bytes(self.ctx, ctypes.byref(n)), "bs_shard_partial_bytes")
        out = torch.empty(n.value, dtype=torch.uint8, device=self.device)
        _check(lib().bs_step_shard(self.ctx, _dev_ptr(logits_shard, "logits"), logits_shard.stride(0), v0,
                                   logits_shard.shape[1], _vp(self.scores.data_ptr()), _vp(out.data_ptr())),
               "bs_step_shard")
        return out

    def merge_shards(self, partials: torch.Tensor):
        """Finish the step from the shards' partials ([n_shards, bytes] uint8, contiguous, device);
        returns (beam_idx, tokens, scores) views like step()."""
        if partials.dim() != 2 or not partials.is_contiguous() or partials.dtype != torch.uint8:
            raise ValueError("partials must be a contiguous [n_shards, bytes] uint8 tensor")
        _check(lib().bs_step_merge_shards(self.ctx, partials.shape[0], _dev_ptr(partials, "partials"),
                                          _vp(self.scores.data_ptr()), _vp(self.seqs.data_ptr()),
                                          _vp(self.beam_idx.data_ptr()), _vp(self.tokens.data_ptr()),
                                          _vp(self.all_done.data_ptr())), "bs_step_merge_shards")
        return self.beam_idx, self.tokens, self.scores

    def step_paged(self, logits: torch.Tensor, kv: "PagedKV", t_valid: int):
        """step() plus the table remap of kv.reorder(beam_idx, t_valid); the copy-on-write
        runs at kv.copy().  Returns (beam_idx, tokens, scores) views."""
        if logits.dim() != 2 or logits.shape[0] != self.R or logits.shape[1] != self.V or logits.stride(1) != 1:
            raise ValueError(f"logits must be [{self.R}, {self.V}] with unit stride along V")
        if logits.dtype != self.dtype:
            raise ValueError(f"logits must be {self.dtype}")
        _check(lib().bs_step_paged(self.ctx, _dev_ptr(logits, "logits"), logits.stride(0),
                                   _vp(self.scores.data_ptr()), _vp(self.seqs.data_ptr()),
                                   _vp(self.beam_idx.data_ptr()), _vp(self.tokens.data_ptr()),
                                   _vp(self.all_done.data_ptr()), kv.ctx, t_valid), "bs_step_paged")
        return self.beam_idx, self.tokens, self.scores

    def finalize(self, n_return: int = 1):
        """(out_seqs [batch * n, max_len+1] int32, out_len [batch * n] int32, out_score [batch * n] fp32):
        the best n_return hypotheses of each sentence, best first (sentence b's j-th in row b * n + j)."""
        rows = self.batch * n_return
        out = torch.empty(rows, self.max_len + 1, dtype=torch.int32, device=self.device)
        out_len = torch.empty(rows, dtype=torch.int32, device=self.device)
        out_score = torch.empty(rows, dtype=torch.float32, device=self.device)
        if n_return == 1:
            _check(lib().bs_finalize(self.ctx, _vp(self.scores.data_ptr()), _vp(self.seqs.data_ptr()),
                                     _vp(out.data_ptr()), _vp(out_len.data_ptr()), _vp(out_score.data_ptr())),
                   "bs_finalize")
        else:
            _check(lib().bs_finalize_n(self.ctx, _vp(self.scores.data_ptr()), _vp(self.seqs.data_ptr()), n_return,
                                       _vp(out.data_ptr()), _vp(out_len.data_ptr()), _vp(out_score.data_ptr())),
                   "bs_finalize_n")
        return out, out_len, out_score

    def finished(self):
        """The finished sets: dict of count [B], ns [R] fp64, len [R], serial [R], tokens [R, max_len+1], done [B]."""
        d = self.device
        f = {"count": torch.empty(self.batch, dtype=torch.int32, device=d),
             "ns": torch.empty(self.R, dtype=torch.float64, device=d),
             "len": torch.empty(self.R, dtype=torch.int32, device=d),
             "serial": torch.empty(self.R, dtype=torch.int32, device=d),
             "tokens": torch.empty(self.R, self.max_len + 1, dtype=torch.int32, device=d),
             "done": torch.empty(self.batch, dtype=torch.int32, device=d)}
        _check(lib().bs_finished(self.ctx, *[_vp(f[k].data_ptr()) for k in
                                             ("count", "ns", "len", "serial", "tokens", "done")]), "bs_finished")
        return f

    def steps(self) -> int:
        n = _c_int()
        _check(lib().bs_steps(self.ctx, ctypes.byref(n)), "bs_steps")
        return n.value

    def status(self) -> int:
        """Synchronise and return the device status word (0 = OK)."""
        return lib().bs_status(self.ctx)

    def close(self):
        if getattr(self, "ctx", None) is not None and self.ctx.value:
            lib().bs_destroy(self.ctx)
            self.ctx = _vp()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def bs_expand_static(logits: torch.Tensor, scores_in: torch.Tensor, W: int, scores_out: torch.Tensor | None = None,
                     beam_idx: torch.Tensor | None = None, tokens: torch.Tensor | None = None):
    """One beam expansion (no end-of-sequence token) through the allocation-free entry point.

    logits: CUDA [batch*W, V] (row stride may exceed V), float32 or bfloat16; scores_in: float32
    [batch*W].  Returns (beam_idx, tokens, scores_out).  The library itself allocates nothing;
    the output tensors this wrapper creates when none are given are torch's.
    """
    if logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be [rows, V] with unit column stride")
    R, V = logits.shape
    if W < 1 or R % W:
        raise ValueError("rows must be a multiple of W")
    dev = logits.device
    if scores_out is None:
        scores_out = torch.empty(R, dtype=torch.float32, device=dev)
    if beam_idx is None:
        beam_idx = torch.empty(R, dtype=torch.int32, device=dev)
    if tokens is None:
        tokens = torch.empty(R, dtype=torch.int32, device=dev)
    # the kernels read and write R contiguous entries of each on the logits' device
    for name, t in (("scores_in", scores_in), ("scores_out", scores_out), ("beam_idx", beam_idx),
                    ("tokens", tokens)):
        if t.numel() != R or not t.is_contiguous() or t.device != dev:
            raise ValueError(f"{name} must be a contiguous tensor of {R} entries on {dev}")
    _check(lib().bs_expand_static(_dev_ptr(logits, "logits"), logits.stride(0), R // W, W, V,
                                  _dtype_code(logits.dtype), _dev_ptr(scores_in, "scores_in", torch.float32),
                                  _dev_ptr(scores_out, "scores_out", torch.float32),
                                  _dev_ptr(beam_idx, "beam_idx", torch.int32),
                                  _dev_ptr(tokens, "tokens", torch.int32), _stream(dev)),
           "bs_expand_static")
    return beam_idx, tokens, scores_out


def peak_copy(src: torch.Tensor, dst: torch.Tensor, grid: int):
    """Copy src's bytes into dst with the library's vector-copy kernel (`grid` CTAs)."""
    if not (src.is_contiguous() and dst.is_contiguous()) or src.nbytes != dst.nbytes:
        raise ValueError("src and dst must be contiguous and of equal size")
    _check(lib().vbs_peak_copy(_dev_ptr(src, "src"), _dev_ptr(dst, "dst"), src.nbytes, grid, _stream(src.device)),
           "vbs_peak_copy")


def peak_read(src: torch.Tensor, grid: int, mode: int, sink: torch.Tensor):
    """Read src's bytes with the library's read-only streaming kernel (mode 0: vector loads,
    mode 1: bulk-copy ring); sink is an int32 tensor of at least `grid` entries."""
    if not src.is_contiguous() or sink.numel() < grid or sink.dtype != torch.int32:
        raise ValueError("src must be contiguous; sink int32 with >= grid entries")
    _check(lib().vbs_peak_read(_dev_ptr(src, "src"), src.nbytes, grid, mode, _dev_ptr(sink, "sink"),
                               _stream(src.device)), "vbs_peak_read")


class _KvDesc(ctypes.Structure):
    _fields_ = [("layers", _c_int), ("heads", _c_int), ("head_dim", _c_int), ("t_max", _c_int),
                ("elem_bytes", _c_int)]


def kv_reorder(src: torch.Tensor, dst: torch.Tensor, beam_idx: torch.Tensor, t_valid: int):
    """dst[:, :, r, :, :t_valid] = src[:, :, beam_idx[r], :, :t_valid] for beam_idx[r] >= 0.

    src, dst: contiguous [L, 2, rows, H, T_max, D] CUDA tensors; beam_idx: int32 [rows].
    """
    if src.shape != dst.shape or src.dim() != 6 or src.shape[1] != 2:
        raise ValueError("src and dst must be [L, 2, rows, H, T_max, D]")
    if not (src.is_contiguous() and dst.is_contiguous()):
        raise ValueError("src and dst must be contiguous")
    L, _, rows, H, T, D = src.shape
    desc = _KvDesc(L, H, D, T, src.element_size())
    _check(lib().kv_reorder(ctypes.byref(desc), _dev_ptr(src, "src"), _dev_ptr(dst, "dst"),
                            _dev_ptr(beam_idx, "beam_idx", torch.int32), rows, t_valid, _stream(src.device)),
           "kv_reorder")


class PagedKV:
    """Paged KV cache with copy-on-write (libvbs kv_paged_*).

    The pool is a [batch * blocks_per_sentence, L, 2, H, block, D] tensor; the
    library owns the block table, the reference counts and the free stacks.
    """

    def __init__(self, batch: int, W: int, L: int, H: int, D: int, *, blocks_per_sentence: int,
                 max_blocks: int, block: int = 16, dtype=torch.bfloat16, device="cuda", pool=None):
        self.batch, self.W, self.R = batch, W, batch * W
        self.L, self.H, self.D, self.block = L, H, D, block
        self.S, self.max_blocks = blocks_per_sentence, max_blocks
        self.device = torch.device(device)
        if pool is None:
            pool = torch.zeros(batch * blocks_per_sentence, L, 2, H, block, D, dtype=dtype, device=self.device)
        self.pool = pool
        self._order = _StreamOrder(self.device)
        self.stream = _vp(self._order.raw)
        desc = _KvDesc(L, H, D, max_blocks * block, pool.element_size())
        ctx = _vp()
        _check(lib().kv_paged_init(ctypes.byref(ctx), ctypes.byref(desc), batch, W, blocks_per_sentence, block,
                                   max_blocks, _dev_ptr(pool, "pool"), self.stream), "kv_paged_init")
        self.ctx = ctx
        self._context = _Context(ctx, lib().kv_paged_destroy)
        ptr = [_vp() for _ in range(5)]
        _check(lib().kv_paged_state(self.ctx, *[ctypes.byref(p) for p in ptr]), "kv_paged_state")
        shapes = ((self.R, max_blocks), (self.R,), (batch * self.S,), (batch * self.S,), (batch,))
        self._views = tuple(torch.as_tensor(_DeviceArray(self._context, p.value, s, "<i4"), device=self.device)
                            for p, s in zip(ptr, shapes))

    def prefill(self, P: int):
        _check(lib().kv_paged_prefill(self.ctx, P), "kv_paged_prefill")

    def build(self, lens: torch.Tensor, cap: int | None = None):
        """prefill() for prompts of different lengths, laid out on the GPU with no host round trip.

        lens: int32 [batch] on the device.  Afterwards prepare(t), reorder(.., t) and
        BeamSearch.step_paged(.., t) count positions after each sentence's own prompt.  With cap (room
        for that many tokens): returns the prompts' slot map (slots int64 [cap], pos int32 [cap],
        row int32 [cap], cu int32 [batch + 1]); unused entries are -1."""
        if lens.shape != (self.batch,) or not lens.is_contiguous():
            raise ValueError(f"lens must be a contiguous int32 [{self.batch}] tensor")
        lp = _cuda(lens, "lens", torch.int32)
        if cap is None:
            self._order.run(lib().kv_paged_build, "kv_paged_build", (lens,), self.ctx, lp, 0, None, None, None, None)
            return None
        out, args = self._slot_outputs(self.batch, cap)
        self._order.run(lib().kv_paged_build, "kv_paged_build", (lens,) + out, self.ctx, lp, *args)
        return out

    def slot_map(self, start: torch.Tensor, count: torch.Tensor, cap: int):
        """The slot map of positions [start[i], start[i] + count[i]) of every row (tensors of R entries) or
        of every sentence's first row (batch entries), int32 on the device, as build() returns it."""
        n = start.numel()
        if n not in (self.batch, self.R) or start.shape != (n,) or count.shape != (n,):
            raise ValueError(f"start and count must have {self.R} (or {self.batch}) entries each")
        if not (start.is_contiguous() and count.is_contiguous()):
            raise ValueError("start and count must be contiguous")
        sp, cp = _cuda(start, "start", torch.int32), _cuda(count, "count", torch.int32)
        out, args = self._slot_outputs(n, cap)
        self._order.run(lib().kv_paged_slots, "kv_paged_slots", (start, count) + out, self.ctx, n, sp, cp, *args)
        return out

    def _slot_outputs(self, n: int, cap: int):
        if cap < 0:
            raise ValueError("cap must not be negative")
        dev = self.device                           # (four allocations cost less than one and its views)
        slots = torch.empty(cap, dtype=torch.int64, device=dev)
        pos = torch.empty(cap, dtype=torch.int32, device=dev)
        row = torch.empty(cap, dtype=torch.int32, device=dev)
        cu = torch.empty(n + 1, dtype=torch.int32, device=dev)
        return (slots, pos, row, cu), (cap, slots.data_ptr(), pos.data_ptr(), row.data_ptr(), cu.data_ptr())

    def views(self):
        """The allocator's state as int32 tensors on the library's own memory (no copy; they keep it
        allocated and are not to be written): table [R, max_blocks], blocks per row [R], reference counts, free stacks
        [batch * blocks_per_sentence] and their heights [batch]."""
        return self._views

    def prepare(self, t_write: int):
        _check(lib().kv_paged_prepare(self.ctx, t_write), "kv_paged_prepare")

    def reorder(self, beam_idx: torch.Tensor, t_valid: int):
        _check(lib().kv_paged_reorder(self.ctx, _dev_ptr(beam_idx, "beam_idx", torch.int32), t_valid),
               "kv_paged_reorder")

    def copy(self):
        """Run the copy-on-write tasks that BeamSearch.step_paged recorded."""
        _check(lib().kv_paged_copy(self.ctx), "kv_paged_copy")

    def save(self):
        """Snapshot the allocator state on the device (no host round trip)."""
        _check(lib().kv_paged_save(self.ctx), "kv_paged_save")

    def restore(self):
        """Return the allocator to the last snapshot (no host round trip)."""
        _check(lib().kv_paged_restore(self.ctx), "kv_paged_restore")

    def table(self) -> torch.Tensor:
        """A copy of the block table [R, max_blocks] (int32, on the device)."""
        out = torch.empty(self.R, self.max_blocks, dtype=torch.int32, device=self.device)
        _check(lib().kv_paged_copy_table(self.ctx, _vp(out.data_ptr())), "kv_paged_copy_table")
        return out

    def counts(self):
        """(refcnt [batch * blocks_per_sentence], nblk [R]) as int32 device tensors."""
        rc = torch.empty(self.batch * self.S, dtype=torch.int32, device=self.device)
        nb = torch.empty(self.R, dtype=torch.int32, device=self.device)
        _check(lib().kv_paged_counts(self.ctx, _vp(rc.data_ptr()), _vp(nb.data_ptr())), "kv_paged_counts")
        return rc, nb

    def cow_slots(self) -> int:
        """Filled slots copied by copy-on-write since init (synchronises)."""
        n = _c_i64()
        _check(lib().kv_paged_cow_slots(self.ctx, ctypes.byref(n)), "kv_paged_cow_slots")
        return n.value

    def status(self) -> int:
        return lib().kv_paged_status(self.ctx)

    def close(self):
        # the library's memory goes with the last of this object and the views() still held
        self._views = self._context = None
        self.ctx = _vp()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class PagedKV8(PagedKV):
    """A PagedKV held in 8 bits (torch.int8 or torch.float8_e4m3fn), with one power-of-two scale per
    (block, layer, k/v, head) in `scales` [batch * blocks_per_sentence, L, 2, H] (fp32), and the
    attention that reads it.

    `heads` is the number of query heads (a multiple of H), `max_q` the most query tokens per row of one
    attend() call (up to 32).  D is a multiple of 16 up to 256.
    """

    def __init__(self, batch: int, W: int, L: int, H: int, D: int, *, heads: int, blocks_per_sentence: int,
                 max_blocks: int, block: int = 16, max_q: int = 1, dtype=torch.float8_e4m3fn, device="cuda",
                 pool=None, scales=None):
        self.ctx8 = _vp()
        if dtype not in (torch.int8, torch.float8_e4m3fn):
            raise ValueError(f"dtype must be int8 or float8_e4m3fn, got {dtype}")
        NB = batch * blocks_per_sentence
        if pool is not None and (pool.dtype != dtype or not pool.is_contiguous()
                                 or pool.shape != (NB, L, 2, H, block, D)):
            raise ValueError(f"pool must be a contiguous {dtype} [{NB}, {L}, 2, {H}, {block}, {D}] tensor")
        super().__init__(batch, W, L, H, D, blocks_per_sentence=blocks_per_sentence, max_blocks=max_blocks,
                         block=block, dtype=dtype, device=device, pool=pool)
        if scales is None:
            scales = torch.zeros(NB, L, 2, H, dtype=torch.float32, device=self.device)
        if scales.shape != (NB, L, 2, H) or not scales.is_contiguous():
            raise ValueError(f"scales must be a contiguous float32 [{NB}, {L}, 2, {H}] tensor")
        self.scales, self.heads, self.max_q = scales, heads, max_q
        self._q_shape = None                        # of the planned step
        _check(lib().kv8_init(ctypes.byref(self.ctx8), self.ctx, I8 if dtype == torch.int8 else E4M3,
                              _dev_ptr(scales, "scales", torch.float32), heads, max_q), "kv8_init")

    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor):
        """Write k, v [N, H, D] (bfloat16 or float32, unit stride along D) at slots (int64 [N], -1: skipped).

        Tokens of one block stand next to each other in ascending order (skipped ones may part them), as build()
        and slot_map() list them; a run that starts a block sets its scales, one that continues it can only raise them."""
        N = slots.numel()
        shape, ks, vs = (N, self.H, self.D), k.stride(), v.stride()
        if k.shape != shape or v.shape != shape or ks[2] != 1 or vs[2] != 1:
            raise ValueError(f"k and v must be [{N}, {self.H}, {self.D}] with unit stride along D")
        if k.dtype != v.dtype:
            raise ValueError("k and v must have one dtype")
        if slots.dim() != 1 or not slots.is_contiguous():
            raise ValueError("slots must be a contiguous int64 [N] tensor")
        dt = k.dtype
        code = _dtype_code(dt)
        self._order.run(lib().kv8_append, "kv8_append", (k, v, slots), self.ctx8, layer, _cuda(k, "k", dt),
                        _cuda(v, "v", dt), ks[0], ks[1], vs[0], vs[1], code, N, _cuda(slots, "slots", torch.int64))

    def read(self, layer: int, slots: torch.Tensor):
        """(k, v) bfloat16 [N, H, D]: the values that slots (int64 [N]) hold, exactly; zeros for -1."""
        if slots.dim() != 1 or not slots.is_contiguous():
            raise ValueError("slots must be a contiguous int64 [N] tensor")
        n = slots.shape[0]
        k = torch.empty(n, self.H, self.D, dtype=torch.bfloat16, device=self.device)
        v = torch.empty(n, self.H, self.D, dtype=torch.bfloat16, device=self.device)
        self._order.run(lib().kv8_read, "kv8_read", (slots, k, v), self.ctx8, layer, n,
                        _cuda(slots, "slots", torch.int64), k.data_ptr(), v.data_ptr())
        return k, v

    def plan(self, ctx_len: torch.Tensor, n_q: int = 1):
        """Prepare a step's attention: ctx_len (int32 [R] on the device) is each row's number of cached
        positions, its n_q new tokens among them.  Call it whenever the tables or lengths have changed:
        after build(), prefill(), prepare(), reorder(), restore() or a beam step, attend() refuses to go on with the
        plan before."""
        if ctx_len.shape != (self.R,) or not ctx_len.is_contiguous():
            raise ValueError(f"ctx_len must be a contiguous int32 [{self.R}] tensor")
        self._order.run(lib().kv8_plan, "kv8_plan", (ctx_len,), self.ctx8, _cuda(ctx_len, "ctx_len", torch.int32), n_q)
        self._q_shape = (self.R, n_q, self.heads, self.D)

    def attend(self, layer: int, q: torch.Tensor, scale: float | None = None, out: torch.Tensor | None = None):
        """softmax(scale q k^T) v of q [R, n_q, heads, D] (bfloat16, unit stride along D) over each row's
        cached positions up to the token's own (plan() has set n_q); scale defaults to D ** -0.5."""
        shape = self._q_shape or (self.R, q.shape[1] if q.dim() > 1 else 0, self.heads, self.D)
        qs = _rows4(q, "q", shape)
        out, os_ = _output(out, shape, self.device)
        self._order.run(lib().kv8_attention, "kv8_attention", (q, out), self.ctx8, layer, q.data_ptr(), qs[0], qs[1], qs[2],
                        self.D ** -0.5 if scale is None else scale, out.data_ptr(), os_[0], os_[1], os_[2])
        return out

    def close(self):
        if getattr(self, "ctx8", None) is not None and self.ctx8.value:
            lib().kv8_destroy(self.ctx8)
            self.ctx8 = _vp()
        super().close()


def _rows4(t: torch.Tensor, name: str, shape):
    """The strides of a bfloat16 tensor of this shape."""
    st = t.stride()
    if t.shape != shape or st[3] != 1:
        raise ValueError(f"{name} must be {list(shape)} with unit stride along the last axis, got {list(t.shape)}")
    if not t.is_cuda or t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be a bfloat16 CUDA tensor")
    return st


def _output(out, shape, device):
    """The caller's output or a new one, and its strides."""
    if out is not None:
        return out, _rows4(out, "out", shape)
    row = shape[2] * shape[3]
    return torch.empty(shape, dtype=torch.bfloat16, device=device), (shape[1] * row, row, shape[3])


class CrossAttention:
    """Attention of decoder rows to their sentence's encoder states (libvbs xattn_*).

    `batch` sentences of W rows each read one set of keys and values; `heads` query heads share
    `kv_heads`.  Work goes on the stream that is current at construction.
    """

    def __init__(self, batch: int, W: int, heads: int, D: int, *, kv_heads: int | None = None, max_q: int = 1,
                 max_len: int = 1024, device="cuda"):
        self.ctx = _vp()
        self.batch, self.W, self.R, self.heads, self.D = batch, W, batch * W, heads, D
        self.kv_heads = heads if kv_heads is None else kv_heads
        self.max_q, self.max_len = max_q, max_len
        self.device = torch.device(device)
        self._order = _StreamOrder(self.device)
        _check(lib().xattn_init(ctypes.byref(self.ctx), batch, W, heads, self.kv_heads, D, max_q, max_len,
                                _vp(self._order.raw)), "xattn_init")

    def attend(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, enc_len: torch.Tensor,
               scale: float | None = None, out: torch.Tensor | None = None):
        """softmax(scale q k^T) v: q [R, n_q, heads, D], k and v [batch, S, kv_heads, D] (bfloat16, unit stride
        along D), over positions below enc_len (int32 [batch]) of the row's sentence; zeros where that is 0.
        scale defaults to D ** -0.5."""
        n_q = q.shape[1] if q.dim() == 4 else 0
        S = k.shape[1] if k.dim() == 4 else 0
        shape, kv_shape = (self.R, n_q, self.heads, self.D), (self.batch, S, self.kv_heads, self.D)
        qs, ks, vs = _rows4(q, "q", shape), _rows4(k, "k", kv_shape), _rows4(v, "v", kv_shape)
        if enc_len.shape != (self.batch,) or not enc_len.is_contiguous():
            raise ValueError(f"enc_len must be a contiguous int32 [{self.batch}] tensor")
        lp = _cuda(enc_len, "enc_len", torch.int32)
        out, os_ = _output(out, shape, self.device)
        self._order.run(lib().xattn_run, "xattn_run", (q, k, v, enc_len, out), self.ctx, q.data_ptr(), qs[0], qs[1], qs[2],
                        n_q, k.data_ptr(), ks[0], ks[1], ks[2], v.data_ptr(), vs[0], vs[1], vs[2], S, lp,
                        self.D ** -0.5 if scale is None else scale, out.data_ptr(), os_[0], os_[1], os_[2])
        return out

    @property
    def tiles(self):
        """Whether the last attend() took the tcgen05 tiles (many rows) or, False, the split kernel; None before it."""
        n = _c_int()
        _check(lib().xattn_kernel(self.ctx, ctypes.byref(n)), "xattn_kernel")
        return None if n.value < 0 else bool(n.value)

    def status(self) -> int:
        """Synchronise and return the device status word (0 = OK)."""
        return lib().xattn_status(self.ctx)

    def close(self):
        if getattr(self, "ctx", None) is not None and self.ctx.value:
            lib().xattn_destroy(self.ctx)
            self.ctx = _vp()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def bpd_propose(logits: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """Predict: argmax over V of logits [B, k, V] (dense) -> int32 [B, k]."""
    if logits.dim() != 3 or not logits.is_contiguous():
        raise ValueError("logits must be a contiguous [B, k, V] tensor")
    B, k, V = logits.shape
    if out is None:
        out = torch.empty(B, k, dtype=torch.int32, device=logits.device)
    _check(lib().bpd_propose(_dev_ptr(logits, "logits"), B, k, V, _dtype_code(logits.dtype),
                             _dev_ptr(out, "out", torch.int32), _stream(logits.device)), "bpd_propose")
    return out


def bpd_verify(logits: torch.Tensor, proposals: torch.Tensor, eos: int = -1, khat: torch.Tensor | None = None,
               next_out: torch.Tensor | None = None, criterion: int = 0, param: int = 0, min_accept: int = 1):
    """Verify + accept on combined logits [B, k, k, V] -> (khat int32 [B], next proposals int32 [B, k]).

    criterion BPD_EXACT (default), BPD_TOPK (param = top-k size) or BPD_DISTANCE (param =
    largest token distance), and min_accept (the minimum accepted block): the relaxed
    verify of bpd_verify_approx."""
    if logits.dim() != 4 or logits.shape[1] != logits.shape[2] or not logits.is_contiguous():
        raise ValueError("logits must be a contiguous [B, k, k, V] tensor")
    B, k, _, V = logits.shape
    if proposals.shape != (B, k) or not proposals.is_contiguous():
        raise ValueError("proposals must be a contiguous [B, k] int32 tensor")
    if khat is None:
        khat = torch.empty(B, dtype=torch.int32, device=logits.device)
    if next_out is None:
        next_out = torch.empty(B, k, dtype=torch.int32, device=logits.device)
    if criterion == BPD_EXACT and min_accept == 1:
        _check(lib().bpd_verify(_dev_ptr(logits, "logits"), _dev_ptr(proposals, "proposals", torch.int32), B, k, V,
                                _dtype_code(logits.dtype), eos, _dev_ptr(khat, "khat", torch.int32),
                                _dev_ptr(next_out, "next", torch.int32), _stream(logits.device)), "bpd_verify")
    else:
        _check(lib().bpd_verify_approx(_dev_ptr(logits, "logits"), _dev_ptr(proposals, "proposals", torch.int32), B,
                                       k, V, _dtype_code(logits.dtype), eos, criterion, param, min_accept,
                                       _dev_ptr(khat, "khat", torch.int32), _dev_ptr(next_out, "next", torch.int32),
                                       _stream(logits.device)), "bpd_verify_approx")
    return khat, next_out


def gather_shard_partials(partial: torch.Tensor, group=None) -> torch.Tensor:
    """All-gather one shard partial per rank (torch.distributed, rank order): [world, bytes].

    Each rank of a vocabulary-parallel LM head holds the columns of one shard; after
    BeamSearch.shard_partial this exchange gives every rank the partials that
    BeamSearch.merge_shards takes.
    """
    import torch.distributed as dist
    world = dist.get_world_size(group)
    out = torch.empty(world, partial.numel(), dtype=partial.dtype, device=partial.device)
    dist.all_gather(list(out.unbind(0)), partial.contiguous(), group=group)
    return out
