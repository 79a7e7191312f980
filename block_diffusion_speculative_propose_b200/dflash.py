"""Thin Python binding over the C ABI in include/dflash.h (libdflash.so).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Torch tensors supply device memory and streams; outputs that the
caller does not pass are allocated here with ``torch.empty``.  If the shared
library is missing this module raises — there is no fallback.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from typing import Dict, List, Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdflash.so")

STATUS = {
    0: "DFLASH_OK",
    -1: "DFLASH_ERR_INVALID_ARG",
    -2: "DFLASH_ERR_CUDA",
    -3: "DFLASH_ERR_WORKSPACE",
    -4: "DFLASH_ERR_UNSUPPORTED_SHAPE",
    -5: "DFLASH_ERR_DEVICE_BOUNDS",
    -6: "DFLASH_ERR_UNIMPLEMENTED",
    -7: "DFLASH_ERR_DEVICE_TIMEOUT",
    -8: "DFLASH_ERR_RANGE",
    -9: "DFLASH_ERR_EXCHANGE",
}
DEVERR_TIMEOUT, DEVERR_SLOT, DEVERR_TABLE, DEVERR_TOKEN, DEVERR_POSITION = 1, 2, 4, 8, 16
KERNEL_KINDS = 17


class DFlashError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


class _Config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int), ("n_layers", ctypes.c_int),
                ("n_q_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("intermediate", ctypes.c_int),
                ("vocab", ctypes.c_int), ("n_target_layers", ctypes.c_int),
                ("target_layer_ids", ctypes.POINTER(ctypes.c_int)),
                ("block_size", ctypes.c_int), ("mask_token_id", ctypes.c_int),
                ("page_size", ctypes.c_int), ("rms_eps", ctypes.c_float),
                ("rope_theta", ctypes.c_float), ("max_position", ctypes.c_int)]


_PP = ctypes.POINTER(ctypes.c_void_p)
# dflash_allreduce_fn: int (*)(float* data, size_t count, void* stream, void* user)
ALLREDUCE_FN = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p,
                                ctypes.c_void_p)


class _Weights(ctypes.Structure):
    _fields_ = [("fc_w", ctypes.c_void_p), ("hidden_norm_w", ctypes.c_void_p),
                ("embed", ctypes.c_void_p), ("lm_head", ctypes.c_void_p),
                ("final_norm_w", ctypes.c_void_p)] + [
        (n, _PP) for n in ("in_norm_w", "post_norm_w", "wq", "wk", "wv", "wo", "q_norm_w",
                           "k_norm_w", "w_gate", "w_up", "w_down")]


class _StepIO(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("n", ctypes.c_int),
                ("prev_drafts", ctypes.c_void_p), ("target_logits", ctypes.c_void_p),
                ("target_positions", ctypes.c_void_p), ("last_token_indices", ctypes.c_void_p),
                ("num_draft", ctypes.c_void_p), ("prev_sampled", ctypes.c_void_p),
                ("prev_width", ctypes.c_int), ("prev_num_draft", ctypes.c_void_p),
                ("aux", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("max_pages_per_seq", ctypes.c_int), ("k_cache", _PP), ("v_cache", _PP),
                ("num_pages", ctypes.c_int), ("out_tokens", ctypes.c_void_p),
                ("num_accepted", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("slot_mapping", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("bonus", ctypes.c_void_p), ("draft_tokens", ctypes.c_void_p),
                ("block_tokens", ctypes.c_void_p), ("device_error", ctypes.c_void_p)]


class _TargetConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("hidden", "n_layers", "n_q_heads", "n_kv_heads",
                                            "head_dim", "intermediate", "vocab")] + \
               [("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_float),
                ("max_len", ctypes.c_int), ("n_capture", ctypes.c_int),
                ("capture_layers", ctypes.POINTER(ctypes.c_int))]


_TARGET_SINGLE = ("embed", "final_norm_w", "lm_head")
_TARGET_LAYER = ("in_norm_w", "post_norm_w", "wq", "wk", "wv", "wo", "q_norm_w", "k_norm_w",
                 "w_gate", "w_up", "w_down")


class _TargetWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in _TARGET_SINGLE] + \
               [(n, _PP) for n in _TARGET_LAYER]


class _AttnPlan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("tcgen05", "keys_per_tile", "ring_depth",
                                            "ctas_per_sm", "chunk_keys", "max_splits",
                                            "cluster", "persistent", "transposed_pv")]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libdflash.so (built in-tree by ``build.py``); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "block_diffusion_speculative_propose_b200/build.py")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    i64 = ctypes.c_int64
    sig = {
        "dflash_create": ([ctypes.POINTER(_Config), ctypes.POINTER(_Weights), i32,
                           ctypes.POINTER(vp)], i32),
        "dflash_create_vocab_shard": ([ctypes.POINTER(_Config), ctypes.POINTER(_Weights), i32,
                                       i32, i32, ctypes.POINTER(vp)], i32),
        "dflash_destroy": ([vp], None),
        "dflash_inject_workspace_bytes": ([vp, i32], sz),
        "dflash_propose_workspace_bytes": ([vp, i32, i32], sz),
        "dflash_propose_final_rows_offset": ([vp, i32, i32], sz),
        "dflash_set_wait_limit": ([i32, ctypes.c_longlong], i32),
        "dflash_plan_gemm_info": ([i32] * 6 + [ctypes.POINTER(_GemmPlan)], i32),
        "dflash_create_tp_shard": ([ctypes.POINTER(_Config), ctypes.POINTER(_Weights), i32, i32,
                                    i32, i32, i32, ctypes.POINTER(vp)], i32),
        "dflash_propose_tp": ([vp, vp, vp, vp, i32, i32, _PP, _PP, i32, vp, vp, vp, sz, vp,
                               ALLREDUCE_FN, vp], i32),
        "dflash_aux_capture_layers": ([ctypes.POINTER(ctypes.c_int), i32, i32,
                                       ctypes.POINTER(ctypes.c_int)], i32),
        "dflash_target_create": ([ctypes.POINTER(_TargetConfig), ctypes.POINTER(_TargetWeights),
                                  i32, ctypes.POINTER(vp)], i32),
        "dflash_target_destroy": ([vp], None),
        "dflash_target_workspace_bytes": ([vp, i32], sz),
        "dflash_target_forward": ([vp, vp, i32, i32, vp, vp, vp, sz, vp], i32),
        "dflash_target_check_device_errors": ([vp, ctypes.POINTER(ctypes.c_uint)], i32),
        "dflash_selftest_wait_timeout": ([vp, vp], i32),
        "dflash_verify_workspace_bytes": ([i32, i32, i32], sz),
        "dflash_linear_workspace_bytes": ([vp, i32, i32, i32], sz),
        "dflash_attention_workspace_bytes": ([vp, i32, i32], sz),
        "dflash_paged_slots": ([vp, vp, i32, vp, i32, i32, vp, vp], i32),
        "dflash_prepare_proposal_inputs": ([vp, i32, vp, i32, vp, i32, vp, vp, i32, vp, vp,
                                            i32, i32, i32, vp, vp, vp, vp, vp, vp], i32),
        "dflash_inject_context": ([vp, vp, vp, vp, i32, _PP, _PP, i32, vp, sz, vp], i32),
        "dflash_propose": ([vp, vp, vp, vp, i32, i32, _PP, _PP, i32, vp, vp, vp, vp, sz, vp],
                           i32),
        "dflash_propose_keys": ([vp, vp, vp, vp, i32, i32, _PP, _PP, i32, vp, vp, vp, sz, vp],
                                i32),
        "dflash_finalize_draft_keys": ([vp, vp, i32, i32, i32, vp, vp, vp, vp], i32),
        "dflash_verify_greedy": ([vp, vp, i32, i32, i32, vp, vp, vp, vp, sz, vp], i32),
        "dflash_verify_greedy_noalloc": ([vp, vp, i32, i32, i32, vp, vp, vp, vp], i32),
        "dflash_sample_tokens": ([vp, i64, i32, i32] + [vp] * 9, i32),
        "dflash_verify_sampled_workspace_bytes": ([i32, i32], sz),
        "dflash_verify_sampled": ([vp, vp, i64, i32, i32, i32] + [vp] * 11 + [sz, vp], i32),
        "dflash_spec_step_workspace_bytes": ([vp, i32, i32, i32], sz),
        "dflash_spec_step": ([vp, ctypes.POINTER(_StepIO), vp, sz, vp], i32),
        "dflash_step_graph_create": ([vp, ctypes.POINTER(_StepIO), vp, sz, ctypes.POINTER(vp)],
                                     i32),
        "dflash_step_graph_launch": ([vp, vp], i32),
        "dflash_step_graph_destroy": ([vp], None),
        "dflash_linear": ([vp, vp, vp, i32, i32, i32, vp, vp, sz, vp], i32),
        "dflash_linear_ex": ([vp, vp, vp, i32, i32, i32, vp, i32, i32, vp, sz, vp], i32),
        "dflash_append_kv": ([vp, vp, i64, vp, i64, vp, vp, i64, vp, vp, vp, vp, i32, vp, vp, i32,
                              vp], i32),
        "dflash_block_attention": ([vp, vp, vp, vp, i32, i32, vp, vp, i32, vp, vp, sz, vp],
                                   i32),
        "dflash_prefix_attention_workspace_bytes": ([vp, i32, i32, i32, i32], sz),
        "dflash_prefix_attention": ([vp, vp, i32, i32, vp, vp, i32, i32, i32, vp, vp, i32, vp, vp,
                                     sz, vp], i32),
        "dflash_plan_attention_info": ([i32] * 10 + [ctypes.POINTER(_AttnPlan)], i32),
        "dflash_check_device_errors": ([vp, ctypes.POINTER(ctypes.c_uint)], i32),
        "dflash_launch_count": ([vp], ctypes.c_ulonglong),
        "dflash_kernel_name": ([i32], ctypes.c_char_p),
        "dflash_profile_enable": ([vp, i32], i32),
        "dflash_profile_read": ([vp, i32, ctypes.POINTER(ctypes.c_int),
                                 ctypes.POINTER(ctypes.c_double)], i32),
        "dflash_profile_disable": ([vp], i32),
        "dflash_status_string": ([i32], ctypes.c_char_p),
        "dflash_version": ([], ctypes.c_char_p),
    }
    for name, (args, res) in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    _lib = L
    return L


def _check(status: int, where: str) -> None:
    if status != 0:
        raise DFlashError(status, where)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _want(t: torch.Tensor, dtype: torch.dtype, name: str) -> None:
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")


def _rows(t: torch.Tensor, shape, name: str, dev: int):
    """(pointer, row stride in elements) of a tensor [n, *shape] on CUDA device
    ``dev`` whose rows are packed inside and any distance apart."""
    if dev < 0 or t.get_device() != dev:
        raise ValueError(f"{name}: expected a CUDA tensor on the call's device, got {t.device}")
    size, step = t.shape, t.stride()
    if size[1:] != shape:
        raise ValueError(f"{name}: expected rows of {tuple(shape)}, got {tuple(size[1:])}")
    row = 1
    for i in range(len(size) - 1, 0, -1):
        if size[i] > 1 and step[i] != row:
            raise ValueError(f"{name}: rows must be packed inside")
        row *= size[i]
    return t.data_ptr(), (step[0] if size[0] > 1 else row)


def _is(t: torch.Tensor, dtype: torch.dtype, shape, name: str, dev: int) -> int:
    """The pointer of a packed tensor of this type and shape on CUDA device ``dev``."""
    if t.dtype is not dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected {list(shape)}, got {list(t.shape)}")
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor on the call's CUDA device, "
                         f"got {t.device}")
    return t.data_ptr()


def _bytes(t: torch.Tensor, name: str, dev: int):
    """(pointer, bytes) of a packed buffer of any type on CUDA device ``dev``."""
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor on the call's CUDA device, "
                         f"got {t.device}")
    return t.data_ptr(), t.numel() * t.element_size()


def _word(t: Optional[torch.Tensor], name: str, dev: int) -> Optional[int]:
    """The pointer of a 32-bit word (or more) on CUDA device ``dev``, or None."""
    if t is None:
        return None
    ptr, n = _bytes(t, name, dev)
    if n < 4 or t.element_size() < 4:
        raise ValueError(f"{name}: expected a word of 32 bits, got {t.numel()} of {t.dtype}")
    return ptr


def _stream(stream, dev: Optional[int] = None) -> int:
    """A stream's raw handle; None: the current stream, of device ``dev`` if given."""
    if stream is None:
        # the raw handle of torch.cuda.current_stream(), without the object around it
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()
                                                  if dev is None else dev)
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _on_stream(stream, device: torch.device):
    """Context in which a call's stream is the current one: scratch allocated there is
    that stream's own, and belongs to the graph if the stream is being captured."""
    if stream is None:
        if device.index is None or device.index == torch.cuda.current_device():
            return contextlib.nullcontext()
        stream = torch.cuda.current_stream(device)
    return torch.cuda.stream(_stream_object(stream, device))


def _stream_object(stream, device: torch.device) -> torch.cuda.Stream:
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return (torch.cuda.ExternalStream(int(stream), device=device) if int(stream)
            else torch.cuda.default_stream(device))


def _ptr_array(ts: Sequence[torch.Tensor]):
    arr = (ctypes.c_void_p * len(ts))(*[_ptr(t) for t in ts])
    return ctypes.cast(arr, _PP), arr


class Workspace:
    """Device scratch owned by the caller (a uint8 tensor), grown on demand.  A buffer
    belongs to the stream that it was allocated for, so one that is replaced is reused
    only behind that stream's work; one that another stream, or a capture, has taken
    too is kept as long as the workspace."""

    def __init__(self, device):
        self.device = torch.device(device)
        self.buf = torch.empty(0, dtype=torch.uint8, device=self.device)
        self._owner, self._shared = None, False
        self._kept: List[torch.Tensor] = []

    def get(self, nbytes: int, stream=None) -> torch.Tensor:
        """At least ``nbytes`` of scratch for work on ``stream`` (None: the current one)."""
        with _on_stream(stream, self.device):
            raw = _stream(None, self.device.index)
            if self.buf.numel() < nbytes:
                if self._shared:
                    self._kept.append(self.buf)
                self.buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.device)
                self._owner, self._shared = raw, False
            if raw != self._owner or torch.cuda.is_current_stream_capturing():
                self._shared = True
        return self.buf


class DFlash:
    """A library handle: packed draft weights + RoPE table on one device.

    ``cfg`` uses the field names of ``dflash_config``; ``weights`` the names of
    ``dflash_weights`` (bf16 CUDA tensors; per-layer entries are lists).  The
    handle keeps references to every tensor whose pointer the library keeps.
    ``vocab_shard=(start, count)`` builds one rank's shard of the tensor-parallel
    LM head (dflash_create_vocab_shard): ``weights["lm_head"]`` is then that
    shard's [count, H] rows, and the handle proposes through propose_keys."""

    def __init__(self, cfg: Dict, weights: Dict, device: int = 0, max_position: int = 0,
                 vocab_shard: Optional[Sequence[int]] = None, tp: Optional[Sequence[int]] = None):
        L = lib()
        self.cfg = dict(cfg)
        self.device = torch.device("cuda", device)
        n_layers = cfg["n_layers"]
        self._keep: List = []
        tl = cfg.get("target_layer_ids")
        tl_arr = None
        if tl is not None:
            tl_arr = (ctypes.c_int * len(tl))(*tl)
            self._keep.append(tl_arr)
        maxpos = max_position or cfg.get("max_position", 65536)
        self.max_position = maxpos
        c = _Config(cfg["hidden"], n_layers, cfg["n_q_heads"], cfg["n_kv_heads"],
                    cfg["head_dim"], cfg["intermediate"], cfg["vocab"],
                    cfg["n_target_layers"],
                    ctypes.cast(tl_arr, ctypes.POINTER(ctypes.c_int)) if tl_arr else None,
                    cfg["block_size"], cfg["mask_token_id"], cfg.get("page_size", 16),
                    cfg.get("rms_eps", 1e-6), cfg.get("rope_theta", 1e6), maxpos)
        w = _Weights()
        for k in ("fc_w", "hidden_norm_w", "embed", "lm_head", "final_norm_w"):
            t = weights[k]
            _want(t, torch.bfloat16, k)
            self._keep.append(t)
            setattr(w, k, _ptr(t))
        for k in ("in_norm_w", "post_norm_w", "wq", "wk", "wv", "wo", "q_norm_w", "k_norm_w",
                  "w_gate", "w_up", "w_down"):
            ts = list(weights[k])
            if len(ts) != n_layers:
                raise ValueError(f"{k}: expected {n_layers} layers")
            for t in ts:
                _want(t, torch.bfloat16, k)
            self._keep.extend(ts)
            pp, arr = _ptr_array(ts)
            self._keep.append(arr)
            setattr(w, k, pp)
        h = ctypes.c_void_p()
        self.tp = (0, 1) if tp is None else (int(tp[0]), int(tp[1]))
        if tp is not None:
            # one tensor-parallel rank: `weights` is the whole model (every rank
            # passes the same); the library copies out this rank's slices
            self.vocab_shard = ((0, cfg["vocab"]) if vocab_shard is None else
                                (int(vocab_shard[0]), int(vocab_shard[1])))
            _check(L.dflash_create_tp_shard(ctypes.byref(c), ctypes.byref(w), device,
                                            self.tp[0], self.tp[1], self.vocab_shard[0],
                                            self.vocab_shard[1], ctypes.byref(h)),
                   "dflash_create_tp_shard")
        elif vocab_shard is None:
            self.vocab_shard = (0, cfg["vocab"])
            _check(L.dflash_create(ctypes.byref(c), ctypes.byref(w), device, ctypes.byref(h)),
                   "dflash_create")
        else:
            self.vocab_shard = (int(vocab_shard[0]), int(vocab_shard[1]))
            _check(L.dflash_create_vocab_shard(ctypes.byref(c), ctypes.byref(w), device,
                                               self.vocab_shard[0], self.vocab_shard[1],
                                               ctypes.byref(h)), "dflash_create_vocab_shard")
        self.h = h
        self.ws = Workspace(self.device)
        # this handle's own query heads, kv heads, head size, page size and device
        self._heads = (cfg["n_q_heads"] // self.tp[1], cfg["n_kv_heads"] // self.tp[1],
                       cfg["head_dim"], cfg.get("page_size", 16), device)
        self._prefix_bytes: Dict = {}

    def close(self) -> None:
        if getattr(self, "h", None):
            torch.cuda.synchronize(self.device)
            lib().dflash_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ---------------------------------------------------------------- sizes
    def inject_workspace_bytes(self, n: int) -> int:
        return lib().dflash_inject_workspace_bytes(self.h, n)

    def propose_workspace_bytes(self, B: int, max_pages_per_seq: int) -> int:
        return lib().dflash_propose_workspace_bytes(self.h, B, max_pages_per_seq)

    def propose_final_rows(self, workspace: torch.Tensor, B: int,
                           max_pages_per_seq: int) -> torch.Tensor:
        """View of the [B*K, hidden] fp16 rows that the last proposal with this
        workspace handed to the LM head (diagnostics)."""
        off = int(lib().dflash_propose_final_rows_offset(self.h, B, max_pages_per_seq))
        K, H = self.cfg["block_size"] - 1, self.cfg["hidden"]
        n = B * K * H * 2
        if off < 0 or off + n > workspace.numel():
            raise DFlashError(-1, "dflash_propose_final_rows_offset")
        return workspace[off:off + n].view(torch.float16).view(B * K, H)

    # ---------------------------------------------------------------- calls
    def inject_context(self, aux, positions, slot_mapping, k_cache, v_cache,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> None:
        n = int(aux.shape[0])
        _want(aux, torch.bfloat16, "aux")
        _want(positions, torch.int64, "positions")
        _want(slot_mapping, torch.int64, "slot_mapping")
        need = self.inject_workspace_bytes(n) if n else 0
        ws = workspace if workspace is not None else self.ws.get(need, stream)
        kp, ka = _ptr_array(k_cache)
        vp, va = _ptr_array(v_cache)
        _check(lib().dflash_inject_context(self.h, _ptr(aux), _ptr(positions),
                                           _ptr(slot_mapping), n, kp, vp,
                                           int(k_cache[0].shape[0]), _ptr(ws), ws.numel(),
                                           _stream(stream)),
               "dflash_inject_context")

    def propose(self, bonus_tokens, seq_lens, block_table, k_cache, v_cache,
                draft_tokens=None, block_tokens=None, logits_out=None,
                workspace: Optional[torch.Tensor] = None, stream=None):
        B = int(bonus_tokens.shape[0])
        bs = self.cfg["block_size"]
        _want(bonus_tokens, torch.int32, "bonus_tokens")
        _want(seq_lens, torch.int32, "seq_lens")
        _want(block_table, torch.int32, "block_table")
        W = int(block_table.shape[1])
        if draft_tokens is None:
            draft_tokens = torch.empty(B, bs - 1, dtype=torch.int32, device=self.device)
        need = self.propose_workspace_bytes(B, W) if B else 0
        ws = workspace if workspace is not None else self.ws.get(need, stream)
        kp, ka = _ptr_array(k_cache)
        vp, va = _ptr_array(v_cache)
        _check(lib().dflash_propose(self.h, _ptr(bonus_tokens), _ptr(seq_lens),
                                    _ptr(block_table), B, W, kp, vp, int(k_cache[0].shape[0]),
                                    _ptr(draft_tokens), _ptr(block_tokens), _ptr(logits_out),
                                    _ptr(ws), ws.numel(), _stream(stream)),
               "dflash_propose")
        return draft_tokens

    def spec_step_workspace_bytes(self, B: int, n: int, max_pages_per_seq: int) -> int:
        return lib().dflash_spec_step_workspace_bytes(self.h, B, n, max_pages_per_seq)

    def _step_io(self, prev_drafts, target_logits, target_positions, last_token_indices,
                 num_draft, aux, block_table, k_cache, v_cache, prev_sampled, prev_num_draft,
                 out, device_error):
        """Marshal the buffers of one speculative step into dflash_step_io;
        returns (io, outputs, objects to keep alive)."""
        B, n = int(last_token_indices.shape[0]), int(target_positions.shape[0])
        bs = self.cfg["block_size"]
        _want(prev_drafts, torch.int32, "prev_drafts")
        _want(target_logits, torch.float32, "target_logits")
        _want(target_positions, torch.int64, "target_positions")
        _want(last_token_indices, torch.int32, "last_token_indices")
        _want(num_draft, torch.int32, "num_draft")
        _want(aux, torch.bfloat16, "aux")
        _want(block_table, torch.int32, "block_table")
        if prev_sampled is not None:
            _want(prev_sampled, torch.int32, "prev_sampled")
        if prev_num_draft is not None:
            _want(prev_num_draft, torch.int32, "prev_num_draft")
        dev = self.device
        o = dict(out or {})
        shapes = {"out_tokens": ((B, bs), torch.int32), "num_accepted": ((B,), torch.int32),
                  "positions": ((n,), torch.int64), "slot_mapping": ((n,), torch.int64),
                  "seq_lens": ((B,), torch.int32), "bonus": ((B,), torch.int32),
                  "draft_tokens": ((B, bs - 1), torch.int32),
                  "block_tokens": ((B, bs), torch.int32)}
        for k, (shape, dt) in shapes.items():
            if k not in o:
                o[k] = torch.empty(shape, dtype=dt, device=dev)
            _want(o[k], dt, k)
        kp, ka = _ptr_array(k_cache)
        vp, va = _ptr_array(v_cache)
        io = _StepIO(B, n, _ptr(prev_drafts), _ptr(target_logits), _ptr(target_positions),
                     _ptr(last_token_indices), _ptr(num_draft), _ptr(prev_sampled),
                     int(prev_sampled.shape[1]) if prev_sampled is not None else 0,
                     _ptr(prev_num_draft), _ptr(aux), _ptr(block_table),
                     int(block_table.shape[1]), kp, vp, int(k_cache[0].shape[0]),
                     _ptr(o["out_tokens"]), _ptr(o["num_accepted"]), _ptr(o["positions"]),
                     _ptr(o["slot_mapping"]), _ptr(o["seq_lens"]), _ptr(o["bonus"]),
                     _ptr(o["draft_tokens"]), _ptr(o["block_tokens"]), _ptr(device_error))
        keep = [prev_drafts, target_logits, target_positions, last_token_indices, num_draft,
                aux, block_table, list(k_cache), list(v_cache), prev_sampled, prev_num_draft,
                device_error, ka, va]
        return io, o, keep

    def spec_step(self, prev_drafts, target_logits, target_positions, last_token_indices,
                  num_draft, aux, block_table, k_cache, v_cache, prev_sampled=None,
                  prev_num_draft=None, out=None, device_error=None, workspace=None,
                  stream=None) -> Dict[str, torch.Tensor]:
        """One whole speculative step (dflash_spec_step): verify -> prepare ->
        inject -> propose on the device.  Returns the outputs by name
        (out_tokens, num_accepted, positions, slot_mapping, seq_lens, bonus,
        draft_tokens, block_tokens); tensors given in ``out`` are written in place."""
        io, o, keep = self._step_io(prev_drafts, target_logits, target_positions,
                                    last_token_indices, num_draft, aux, block_table, k_cache,
                                    v_cache, prev_sampled, prev_num_draft, out, device_error)
        need = self.spec_step_workspace_bytes(io.B, io.n, io.max_pages_per_seq) if io.B else 0
        ws = workspace if workspace is not None else self.ws.get(need, stream)
        _check(lib().dflash_spec_step(self.h, ctypes.byref(io), _ptr(ws), ws.numel(),
                                      _stream(stream)), "dflash_spec_step")
        return o

    def step_graph(self, prev_drafts, target_logits, target_positions, last_token_indices,
                   num_draft, aux, block_table, k_cache, v_cache, prev_sampled=None,
                   prev_num_draft=None, out=None, device_error=None,
                   workspace=None) -> "StepGraph":
        """The same step captured once into a library-owned CUDA graph
        (dflash_step_graph_create) over these buffers; see StepGraph."""
        io, o, keep = self._step_io(prev_drafts, target_logits, target_positions,
                                    last_token_indices, num_draft, aux, block_table, k_cache,
                                    v_cache, prev_sampled, prev_num_draft, out, device_error)
        need = self.spec_step_workspace_bytes(io.B, io.n, io.max_pages_per_seq) if io.B else 0
        ws = workspace if workspace is not None else torch.empty(
            max(need, 256), dtype=torch.uint8, device=self.device)
        g = ctypes.c_void_p()
        _check(lib().dflash_step_graph_create(self.h, ctypes.byref(io), _ptr(ws), ws.numel(),
                                              ctypes.byref(g)), "dflash_step_graph_create")
        return StepGraph(self, g, o, keep + [ws, io])

    def propose_keys(self, bonus_tokens, seq_lens, block_table, k_cache, v_cache,
                     draft_keys=None, logits_out=None, workspace: Optional[torch.Tensor] = None,
                     stream=None):
        """dflash_propose_keys: this handle's vocabulary shard's greedy-pick keys,
        [B, K] int64, ready for an all-reduce MAX across the shards."""
        B = int(bonus_tokens.shape[0])
        bs = self.cfg["block_size"]
        _want(bonus_tokens, torch.int32, "bonus_tokens")
        _want(seq_lens, torch.int32, "seq_lens")
        _want(block_table, torch.int32, "block_table")
        W = int(block_table.shape[1])
        if draft_keys is None:
            draft_keys = torch.empty(B, bs - 1, dtype=torch.int64, device=self.device)
        _want(draft_keys, torch.int64, "draft_keys")
        need = self.propose_workspace_bytes(B, W) if B else 0
        ws = workspace if workspace is not None else self.ws.get(need, stream)
        kp, ka = _ptr_array(k_cache)
        vp, va = _ptr_array(v_cache)
        _check(lib().dflash_propose_keys(self.h, _ptr(bonus_tokens), _ptr(seq_lens),
                                         _ptr(block_table), B, W, kp, vp,
                                         int(k_cache[0].shape[0]), _ptr(draft_keys),
                                         _ptr(logits_out), _ptr(ws), ws.numel(),
                                         _stream(stream)), "dflash_propose_keys")
        return draft_keys

    def propose_tp(self, bonus_tokens, seq_lens, block_table, k_cache, v_cache, exchange,
                   draft_keys=None, logits_out=None, workspace: Optional[torch.Tensor] = None,
                   stream=None):
        """dflash_propose_tp on a tensor-parallel shard: `exchange(data_ptr,
        count, stream_ptr) -> int` must sum the `count` fp32 values at the
        device pointer over every rank, in place, ordered on that stream (0 on
        success).  Returns this rank's vocabulary shard's keys [B, K] int64."""
        B = int(bonus_tokens.shape[0])
        bs = self.cfg["block_size"]
        _want(bonus_tokens, torch.int32, "bonus_tokens")
        _want(seq_lens, torch.int32, "seq_lens")
        _want(block_table, torch.int32, "block_table")
        W = int(block_table.shape[1])
        if draft_keys is None:
            draft_keys = torch.empty(B, bs - 1, dtype=torch.int64, device=self.device)
        need = self.propose_workspace_bytes(B, W) if B else 0
        ws = workspace if workspace is not None else self.ws.get(need, stream)
        kp, ka = _ptr_array(k_cache)
        vp, va = _ptr_array(v_cache)

        def hook(data, count, st, user):
            try:
                return int(exchange(int(data), int(count), st))
            except Exception:
                return 1
        cb = ALLREDUCE_FN(hook)
        _check(lib().dflash_propose_tp(self.h, _ptr(bonus_tokens), _ptr(seq_lens),
                                       _ptr(block_table), B, W, kp, vp,
                                       int(k_cache[0].shape[0]), _ptr(draft_keys),
                                       _ptr(logits_out), _ptr(ws), ws.numel(), _stream(stream),
                                       cb, None), "dflash_propose_tp")
        return draft_keys

    def linear(self, A, W, out=None, block_n: int = 0, splits: int = 0, workspace=None,
               stream=None):
        M, K = A.shape
        N = W.shape[0]
        _want(A, torch.bfloat16, "A")
        _want(W, torch.bfloat16, "W")
        if out is None:
            out = torch.empty(M, N, dtype=torch.float32, device=self.device)
        need = lib().dflash_linear_workspace_bytes(self.h, M, N, K) if M else 0
        if splits > 1:
            bn = block_n or 256
            tiles = -(-M // 128) * -(-N // bn)
            need = max(need, 2 * (tiles * splits + 1) * min(M, 128) * bn * 4)
        ws = workspace if workspace is not None else self.ws.get(need, stream)
        _check(lib().dflash_linear_ex(self.h, _ptr(A), _ptr(W), M, N, K, _ptr(out), block_n,
                                      splits, _ptr(ws), ws.numel(), _stream(stream)),
               "dflash_linear")
        return out

    def append_kv(self, k, v, positions, slot_mapping, k_cache, v_cache, k_norm=None, q=None,
                  q_norm=None, q_out=None, stream=None) -> Optional[torch.Tensor]:
        """Keys and values [n, Hkv, d] (and queries [n, Hq, d]) of one layer that
        the caller projected: optional RMSNorm per head, rotation, and the paged
        scatter (dflash_append_kv).  The rows may be slices of one fused
        projection.  Returns the rotated queries, packed, if q is given."""
        n = k.shape[0]
        hq, hkv, d, page, dev = self._heads
        bf = torch.bfloat16
        for t in (k, v, q):
            if t is not None and (t.dtype is not bf or t.shape[0] != n):
                raise ValueError(f"k, v, q: expected {n} rows of bfloat16")
        pool = (k_cache.shape[0], hkv, page, d)
        kp, ks = _rows(k, (hkv, d), "k", dev)
        vp, vs = _rows(v, (hkv, d), "v", dev)
        qp, qs, op = None, 0, None
        if q is not None:
            qp, qs = _rows(q, (hq, d), "q", dev)
            if q_out is None:
                q_out = torch.empty(n, hq, d, dtype=bf, device=self.device)
        if q_out is not None:
            op = _is(q_out, bf, (n, hq, d), "q_out", dev)
        _check(lib().dflash_append_kv(
            self.h, kp, ks, vp, vs,
            None if k_norm is None else _is(k_norm, bf, (d,), "k_norm", dev), qp, qs,
            None if q_norm is None else _is(q_norm, bf, (d,), "q_norm", dev), op,
            _is(positions, torch.int64, (n,), "positions", dev),
            _is(slot_mapping, torch.int64, (n,), "slot_mapping", dev), n,
            _is(k_cache, bf, pool, "k_cache", dev),
            _is(v_cache, bf, pool, "v_cache", dev), pool[0],
            _stream(stream, dev)), "dflash_append_kv")
        return q_out

    def block_attention(self, q, seq_lens, block_table, k_cache, v_cache, o=None,
                        workspace=None, stream=None):
        B = int(seq_lens.shape[0])
        W = int(block_table.shape[1])
        if o is None:
            o = torch.empty(q.shape[0], q.shape[1] * q.shape[2], dtype=torch.float16,
                            device=self.device)
        need = lib().dflash_attention_workspace_bytes(self.h, B, W) if B else 0
        ws = workspace if workspace is not None else self.ws.get(need, stream)
        _check(lib().dflash_block_attention(self.h, _ptr(q), _ptr(seq_lens), _ptr(block_table),
                                            B, W, _ptr(k_cache), _ptr(v_cache),
                                            int(k_cache.shape[0]), _ptr(o), _ptr(ws),
                                            ws.numel(), _stream(stream)),
               "dflash_block_attention")
        return o

    def prefix_attention_workspace_bytes(self, B: int, q_len: int, max_pages_per_seq: int,
                                         prefix_pages: int) -> int:
        return lib().dflash_prefix_attention_workspace_bytes(self.h, B, q_len, max_pages_per_seq,
                                                             prefix_pages)

    def prefix_attention(self, q, seq_lens, block_table, prefix_pages: int, k_cache, v_cache,
                         causal: bool = False, o=None, workspace=None, stream=None):
        """Attention of q [B*q_len, Hq, d] over a batch whose first
        ``prefix_pages`` pages (block_table's row 0) are the same for every
        request (dflash_prefix_attention).  Returns o [B*q_len, Hq*d] fp16."""
        B, W, n = seq_lens.shape[0], block_table.shape[1], q.shape[0]
        hq, hkv, d, page, dev = self._heads
        if n % B if B else n:
            raise ValueError(f"q: expected [{B} * q_len, {hq}, {d}]")
        q_len = n // B if B else 1
        if o is None:
            o = torch.empty(n, hq * d, dtype=torch.float16, device=self.device)
        elif o.numel() != n * hq * d:
            raise ValueError(f"o: expected [{n}, {hq * d}]")
        ws = workspace
        if ws is None:
            key = (B, q_len, W, prefix_pages)
            need = self._prefix_bytes.get(key)
            if need is None:
                need = self.prefix_attention_workspace_bytes(*key)
                self._prefix_bytes[key] = need
            # a captured call has scratch of its graph's own: another graph's may run
            # while the handle's is in use
            with _on_stream(stream, self.device):
                ws = (torch.empty(need, dtype=torch.uint8, device=self.device)
                      if torch.cuda.is_current_stream_capturing() else self.ws.get(need))
        bf, pool = torch.bfloat16, (k_cache.shape[0], hkv, page, d)
        _check(lib().dflash_prefix_attention(
            self.h, _is(q, bf, (n, hq, d), "q", dev), q_len, int(causal),
            _is(seq_lens, torch.int32, (B,), "seq_lens", dev),
            _is(block_table, torch.int32, (B, W), "block_table", dev), B, W, prefix_pages,
            _is(k_cache, bf, pool, "k_cache", dev),
            _is(v_cache, bf, pool, "v_cache", dev), pool[0],
            _is(o, torch.float16, o.shape, "o", dev), *_bytes(ws, "workspace", dev),
            _stream(stream, dev)),
            "dflash_prefix_attention")
        return o

    # ---------------------------------------------------------- diagnostics
    def launch_count(self) -> int:
        return int(lib().dflash_launch_count(self.h))

    def profile_enable(self, max_launches: int) -> None:
        _check(lib().dflash_profile_enable(self.h, max_launches), "dflash_profile_enable")

    def profile_disable(self) -> None:
        _check(lib().dflash_profile_disable(self.h), "dflash_profile_disable")

    def profile_read(self) -> Dict[str, tuple]:
        """{kernel family: (launches, total ms)} since the last read."""
        n = KERNEL_KINDS
        cnt = (ctypes.c_int * n)()
        tot = (ctypes.c_double * n)()
        _check(lib().dflash_profile_read(self.h, n, cnt, tot), "dflash_profile_read")
        return {lib().dflash_kernel_name(k).decode(): (cnt[k], tot[k])
                for k in range(n) if cnt[k]}

    def check_device_errors(self) -> int:
        bits = ctypes.c_uint(0)
        lib().dflash_check_device_errors(self.h, ctypes.byref(bits))
        return int(bits.value)

    def check_device_status(self):
        """(status, bits) of dflash_check_device_errors."""
        bits = ctypes.c_uint(0)
        s = int(lib().dflash_check_device_errors(self.h, ctypes.byref(bits)))
        return s, int(bits.value)

    def selftest_wait_timeout(self, stream=None) -> None:
        """Enqueue a kernel whose one bounded wait runs out (diagnostics)."""
        _check(lib().dflash_selftest_wait_timeout(self.h, _stream(stream)),
               "dflash_selftest_wait_timeout")


def aux_capture_layers(target_layer_ids: Sequence[int], target_n_layers: int) -> List[int]:
    """Capture layers (pre-layer states) for a draft checkpoint's
    target_layer_ids (states after layer i): each id plus one."""
    n = len(target_layer_ids)
    ids = (ctypes.c_int * max(n, 1))(*target_layer_ids)
    out = (ctypes.c_int * max(n, 1))()
    _check(lib().dflash_aux_capture_layers(ids, n, int(target_n_layers), out),
           "dflash_aux_capture_layers")
    return [int(out[i]) for i in range(n)]


class TargetModel:
    """The library's small causal target model (dflash_target_*): fp32
    weights (CUDA tensors, names of ``dflash_target_weights``), one sequence.
    ``forward(tokens, start_pos)`` returns (logits [n, V] fp32, aux
    [n, n_capture * H] bf16)."""

    def __init__(self, cfg: Dict, weights: Dict, capture_layers: Sequence[int],
                 max_len: int, device: int = 0):
        L = lib()
        self.cfg = dict(cfg)
        self.device = torch.device("cuda", device)
        self.n_capture = len(capture_layers)
        self._keep: List = []
        cap = (ctypes.c_int * max(self.n_capture, 1))(*capture_layers)
        self._keep.append(cap)
        c = _TargetConfig(cfg["hidden"], cfg["n_layers"], cfg["n_q_heads"], cfg["n_kv_heads"],
                          cfg["head_dim"], cfg["intermediate"], cfg["vocab"],
                          cfg.get("rms_eps", 1e-6), cfg.get("rope_theta", 1e6), int(max_len),
                          self.n_capture, ctypes.cast(cap, ctypes.POINTER(ctypes.c_int)))
        w = _TargetWeights()
        for k in _TARGET_SINGLE:
            t = weights[k]
            _want(t, torch.float32, k)
            self._keep.append(t)
            setattr(w, k, _ptr(t))
        for k in _TARGET_LAYER:
            ts = list(weights[k])
            if len(ts) != cfg["n_layers"]:
                raise ValueError(f"{k}: expected {cfg['n_layers']} layers")
            for t in ts:
                _want(t, torch.float32, k)
            self._keep.extend(ts)
            pp, arr = _ptr_array(ts)
            self._keep.append(arr)
            setattr(w, k, pp)
        h = ctypes.c_void_p()
        _check(L.dflash_target_create(ctypes.byref(c), ctypes.byref(w), device, ctypes.byref(h)),
               "dflash_target_create")
        self.h = h
        self.ws = Workspace(self.device)

    def close(self) -> None:
        if getattr(self, "h", None):
            torch.cuda.synchronize(self.device)
            lib().dflash_target_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def forward(self, tokens: torch.Tensor, start_pos: int, logits=None, aux=None, stream=None):
        _want(tokens, torch.int32, "tokens")
        n = int(tokens.numel())
        H, V = self.cfg["hidden"], self.cfg["vocab"]
        if logits is None:
            logits = torch.empty(n, V, dtype=torch.float32, device=self.device)
        if aux is None and self.n_capture:
            aux = torch.empty(n, self.n_capture * H, dtype=torch.bfloat16, device=self.device)
        ws = self.ws.get(lib().dflash_target_workspace_bytes(self.h, max(n, 1)), stream)
        _check(lib().dflash_target_forward(self.h, _ptr(tokens), n, int(start_pos), _ptr(logits),
                                           _ptr(aux), _ptr(ws), ws.numel(), _stream(stream)),
               "dflash_target_forward")
        return logits, aux

    def check_device_errors(self) -> int:
        bits = ctypes.c_uint(0)
        lib().dflash_target_check_device_errors(self.h, ctypes.byref(bits))
        return int(bits.value)


def set_wait_limit(device: int, cycles: int) -> None:
    """Cycles after which every bounded wait of the library's kernels on
    `device` gives up (diagnostics; default 4e9)."""
    _check(lib().dflash_set_wait_limit(int(device), int(cycles)), "dflash_set_wait_limit")


class StepGraph:
    """A speculative step captured into a CUDA graph owned by the library.
    ``launch()`` replays it on a stream; ``out`` holds its output tensors.  The
    graph keeps the pointers of the buffers it was built on (held here): write
    new inputs into those tensors between launches."""

    def __init__(self, owner: DFlash, g, out: Dict[str, torch.Tensor], keep: List):
        self._owner = owner     # the handle must outlive the graph
        self.g = g
        self.out = out
        self._keep = keep

    def launch(self, stream=None) -> None:
        _check(lib().dflash_step_graph_launch(self.g, _stream(stream)),
               "dflash_step_graph_launch")

    def close(self) -> None:
        if getattr(self, "g", None):
            torch.cuda.synchronize(self._owner.device)
            lib().dflash_step_graph_destroy(self.g)
            self.g = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def finalize_draft_keys(draft_keys, bonus_tokens, block_size: int, vocab: int,
                        draft_tokens=None, block_tokens=None, device_error=None, stream=None):
    """dflash_finalize_draft_keys: drafts [B, K] (and block tokens [B, bs])
    from the keys exchanged across vocabulary shards."""
    B = int(bonus_tokens.shape[0])
    _want(draft_keys, torch.int64, "draft_keys")
    _want(bonus_tokens, torch.int32, "bonus_tokens")
    dev = draft_keys.device
    if draft_tokens is None:
        draft_tokens = torch.empty(B, block_size - 1, dtype=torch.int32, device=dev)
    if block_tokens is None:
        block_tokens = torch.empty(B, block_size, dtype=torch.int32, device=dev)
    _check(lib().dflash_finalize_draft_keys(_ptr(draft_keys), _ptr(bonus_tokens), B, block_size,
                                            vocab, _ptr(draft_tokens), _ptr(block_tokens),
                                            _ptr(device_error), _stream(stream)),
           "dflash_finalize_draft_keys")
    return draft_tokens, block_tokens


def attention_plan(B: int, n_kv_heads: int, max_pages_per_seq: int, block_size: int,
                   q_per_kv: int, head_dim: int = 128, page_size: int = 16, num_sms: int = 148,
                   forced_ring: int = 0, cluster: bool = False,
                   persistent: bool = False, tile32: bool = False) -> Dict[str, int]:
    """dflash_plan_attention_info: the attention launch plan for this geometry
    (host only)."""
    out = _AttnPlan()
    flags = (1 if cluster else 0) | (2 if persistent else 0) | (4 if tile32 else 0)
    _check(lib().dflash_plan_attention_info(B, n_kv_heads, max_pages_per_seq, page_size,
                                            block_size, q_per_kv, head_dim, num_sms,
                                            forced_ring, flags, ctypes.byref(out)),
           "dflash_plan_attention_info")
    return {n: getattr(out, n) for n, _ in _AttnPlan._fields_}


class _GemmPlan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("pair", "tile_m", "tile_n", "k_splits", "stream_k",
                                            "staged", "tiles", "grid")]


def gemm_plan(M: int, N: int, K: int, group: int = 32, num_sms: int = 148,
              pair_split_cap: int = 37) -> Dict[str, int]:
    """dflash_plan_gemm_info: the GEMM launch plan for this shape (host only)."""
    out = _GemmPlan()
    _check(lib().dflash_plan_gemm_info(M, N, K, group, num_sms, pair_split_cap,
                                       ctypes.byref(out)), "dflash_plan_gemm_info")
    return {n: getattr(out, n) for n, _ in _GemmPlan._fields_}


def verify_workspace_bytes(B: int, K: int, V: int) -> int:
    return lib().dflash_verify_workspace_bytes(B, K, V)


def verify_greedy(drafts, target_logits, out_tokens=None, num_accepted=None, bonus=None,
                  workspace=None, stream=None):
    """Greedy acceptance (dflash_verify_greedy); returns (out_tokens, n, bonus)."""
    B, K1, V = target_logits.shape
    K = K1 - 1
    dev = target_logits.device
    _want(drafts, torch.int32, "drafts")
    _want(target_logits, torch.float32, "target_logits")
    if out_tokens is None:
        out_tokens = torch.empty(B, K + 1, dtype=torch.int32, device=dev)
    if num_accepted is None:
        num_accepted = torch.empty(B, dtype=torch.int32, device=dev)
    if bonus is None:
        bonus = torch.empty(B, dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = torch.empty(max(verify_workspace_bytes(B, K, V), 256), dtype=torch.uint8,
                                device=dev)
    _check(lib().dflash_verify_greedy(_ptr(drafts), _ptr(target_logits), B, K, V,
                                      _ptr(out_tokens), _ptr(num_accepted), _ptr(bonus),
                                      _ptr(workspace), workspace.numel(), _stream(stream)),
           "dflash_verify_greedy")
    return out_tokens, num_accepted, bonus


def verify_greedy_noalloc(drafts, target_logits, out_tokens=None, num_accepted=None,
                          bonus=None, stream=None):
    """Greedy acceptance without a workspace (dflash_verify_greedy_noalloc), for
    callers that cannot allocate device scratch; returns (out_tokens, n, bonus).
    The library's fixed scratch is shared by all calls: keep calls on one stream."""
    B, K1, V = target_logits.shape
    K = K1 - 1
    dev = target_logits.device
    _want(drafts, torch.int32, "drafts")
    _want(target_logits, torch.float32, "target_logits")
    if out_tokens is None:
        out_tokens = torch.empty(B, K + 1, dtype=torch.int32, device=dev)
    if num_accepted is None:
        num_accepted = torch.empty(B, dtype=torch.int32, device=dev)
    if bonus is None:
        bonus = torch.empty(B, dtype=torch.int32, device=dev)
    _check(lib().dflash_verify_greedy_noalloc(_ptr(drafts), _ptr(target_logits), B, K, V,
                                              _ptr(out_tokens), _ptr(num_accepted), _ptr(bonus),
                                              _stream(stream)),
           "dflash_verify_greedy_noalloc")
    return out_tokens, num_accepted, bonus


def _settings(n: int, temperature, top_k, top_p, min_p, dev: int):
    """Pointers of the per-row sampling settings, each checked for type and length."""
    f, shape = torch.float32, (n,)
    return (None if temperature is None else _is(temperature, f, shape, "temperature", dev),
            None if top_k is None else _is(top_k, torch.int32, shape, "top_k", dev),
            None if top_p is None else _is(top_p, f, shape, "top_p", dev),
            None if min_p is None else _is(min_p, f, shape, "min_p", dev))


def sample_tokens(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, tokens=None,
                  probs=None, return_probs: bool = False, device_error=None, stream=None):
    """One token per row of ``logits`` [rows, V] fp32 (rows any distance apart)
    from the uniform numbers ``u`` [rows] (dflash_sample_tokens); the settings
    are per-row tensors or None.  Returns the tokens [rows] int32, with
    ``return_probs`` (or ``probs``) the pair (tokens, probabilities)."""
    _want(logits, torch.float32, "logits")
    (rows, V), dev = logits.shape, logits.get_device()
    ptr, ld = _rows(logits, (V,), "logits", dev)
    if tokens is None:
        tokens = torch.empty(rows, dtype=torch.int32, device=logits.device)
    if probs is None and return_probs:
        probs = torch.empty(rows, dtype=torch.float32, device=logits.device)
    _check(lib().dflash_sample_tokens(
        ptr, ld, rows, V, *_settings(rows, temperature, top_k, top_p, min_p, dev),
        _is(u, torch.float32, (rows,), "u", dev),
        _is(tokens, torch.int32, (rows,), "tokens", dev),
        None if probs is None else _is(probs, torch.float32, (rows,), "probs", dev),
        _word(device_error, "device_error", dev), _stream(stream, dev)), "dflash_sample_tokens")
    return tokens if probs is None else (tokens, probs)


@functools.lru_cache(maxsize=None)
def verify_sampled_workspace_bytes(B: int, K: int) -> int:
    return lib().dflash_verify_sampled_workspace_bytes(B, K)


def verify_sampled(drafts, target_logits, u_accept, u_sample, temperature=None, top_k=None,
                   top_p=None, min_p=None, out_tokens=None, num_accepted=None, bonus=None,
                   device_error=None, workspace=None, stream=None):
    """Acceptance of greedy drafts [B, K] against a sampling target
    (dflash_verify_sampled): ``u_accept`` [B, K] and ``u_sample`` [B] are uniform
    numbers, the settings [B] tensors or None.  Returns (out_tokens, n, bonus),
    as verify_greedy."""
    _want(target_logits, torch.float32, "target_logits")
    B, K1, V = target_logits.shape
    K, dev, i32 = K1 - 1, target_logits.get_device(), torch.int32
    step = target_logits.stride()
    if not target_logits.is_cuda or (V > 1 and step[2] != 1) or (
            B > 1 and K1 > 1 and step[0] != K1 * step[1]):
        raise ValueError("target_logits: expected CUDA rows, packed inside, equally far apart")
    ld = step[1] if K1 > 1 else step[0] if B > 1 else V
    device = target_logits.device
    if out_tokens is None:
        out_tokens = torch.empty(B, K1, dtype=i32, device=device)
    if num_accepted is None:
        num_accepted = torch.empty(B, dtype=i32, device=device)
    if bonus is None:
        bonus = torch.empty(B, dtype=i32, device=device)
    if workspace is None:
        with _on_stream(stream, device):      # reused only behind that stream's work
            workspace = torch.empty(max(verify_sampled_workspace_bytes(B, K), 256),
                                    dtype=torch.uint8, device=device)
    _check(lib().dflash_verify_sampled(
        _is(drafts, i32, (B, K), "drafts", dev), target_logits.data_ptr(), ld, B, K, V,
        *_settings(B, temperature, top_k, top_p, min_p, dev),
        _is(u_accept, torch.float32, (B, K), "u_accept", dev),
        _is(u_sample, torch.float32, (B,), "u_sample", dev),
        _is(out_tokens, i32, (B, K1), "out_tokens", dev),
        _is(num_accepted, i32, (B,), "num_accepted", dev), _is(bonus, i32, (B,), "bonus", dev),
        _word(device_error, "device_error", dev), *_bytes(workspace, "workspace", dev),
        _stream(stream, dev)), "dflash_verify_sampled")
    return out_tokens, num_accepted, bonus


def paged_slots(positions, req_ids, block_table, page_size: int = 16, slots=None,
                stream=None):
    """_paged_slots on the device (dflash_paged_slots)."""
    n = int(positions.shape[0])
    _want(positions, torch.int64, "positions")
    _want(req_ids, torch.int64, "req_ids")
    _want(block_table, torch.int32, "block_table")
    if slots is None:
        slots = torch.empty(n, dtype=torch.int64, device=positions.device)
    _check(lib().dflash_paged_slots(_ptr(positions), _ptr(req_ids), n, _ptr(block_table),
                                    int(block_table.shape[1]), page_size, _ptr(slots),
                                    _stream(stream)), "dflash_paged_slots")
    return slots


def prepare_proposal_inputs(target_positions, last_token_indices, cur_sampled, cur_num_draft,
                            block_table, page_size: int, vocab: int, prev_sampled=None,
                            prev_num_draft=None, device_error=None, stream=None):
    """Proposal inputs with the async rejection correction on the device
    (dflash_prepare_proposal_inputs).  Returns (positions, slot_mapping,
    seq_lens, bonus) ready for DFlash.inject_context / DFlash.propose."""
    n, B = int(target_positions.shape[0]), int(last_token_indices.shape[0])
    _want(target_positions, torch.int64, "target_positions")
    _want(last_token_indices, torch.int32, "last_token_indices")
    _want(cur_sampled, torch.int32, "cur_sampled")
    _want(cur_num_draft, torch.int32, "cur_num_draft")
    _want(block_table, torch.int32, "block_table")
    if prev_sampled is not None:
        _want(prev_sampled, torch.int32, "prev_sampled")
        _want(prev_num_draft, torch.int32, "prev_num_draft")
    dev = target_positions.device
    positions = torch.empty(n, dtype=torch.int64, device=dev)
    slots = torch.empty(n, dtype=torch.int64, device=dev)
    seq_lens = torch.empty(B, dtype=torch.int32, device=dev)
    bonus = torch.empty(B, dtype=torch.int32, device=dev)
    pw = int(prev_sampled.shape[1]) if prev_sampled is not None else 0
    _check(lib().dflash_prepare_proposal_inputs(
        _ptr(target_positions), n, _ptr(last_token_indices), B, _ptr(cur_sampled),
        int(cur_sampled.shape[1]), _ptr(cur_num_draft), _ptr(prev_sampled), pw,
        _ptr(prev_num_draft), _ptr(block_table), int(block_table.shape[1]), page_size, vocab,
        _ptr(positions), _ptr(slots), _ptr(seq_lens), _ptr(bonus), _ptr(device_error),
        _stream(stream)), "dflash_prepare_proposal_inputs")
    return positions, slots, seq_lens, bonus


def status_string(s: int) -> str:
    return lib().dflash_status_string(s).decode()


def version() -> str:
    return lib().dflash_version().decode()
