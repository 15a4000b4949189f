"""logit_masking_amd -- Python binding of libcg.so, the MI355X constrained-decoding
hot path (grammar -> pushdown automaton tables, token bitmask, masked
sampling, state advance).  Argument marshalling only: every step runs in the
library's HIP kernels.  Device buffers are torch tensors; torch supplies
memory and the current HIP stream, nothing else.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libcg.so")

CG_OK, CG_E_ARG, CG_E_PARSE, CG_E_UNSUPPORTED, CG_E_LIMIT, CG_E_VOCAB, CG_E_DEVICE, CG_E_EVAL, CG_E_INVALID = \
    0, -1, -2, -3, -4, -5, -6, -7, -8
ROW_OK, ROW_DONE, ROW_CAPPED, ROW_REJECTED, ROW_NOOP, ROW_INJECT = 0, 1, 2, 3, 4, 5
FLAG_DONE, FLAG_CAPPED = 1, 2
HOST_ONLY = 1
STATE_BYTES = 24
DTYPE_F32, DTYPE_BF16 = 0, 1
MAX_ROW_VOCAB, MAX_TOP = 4194304, 1024  # CG_MAX_ROW_VOCAB, CG_MAX_TOP
FILL_NOALLOC_SCRATCH_BYTES = 16 << 20  # CG_FILL_NOALLOC_SCRATCH_BYTES

# Symbols the C ABI (include/cg.h) exports.
EXPORTS = ["cg_compile_grammar", "cg_free_grammar", "cg_grammar_info", "cg_init_state", "cg_fill_workspace_bytes",
           "cg_fill_bitmask", "cg_sample_advance", "cg_sample_advance_fill",
           "cg_sample_advance_plan", "cg_fill_walk", "cg_force_bytes", "cg_eval_calc", "cg_draft_workspace_bytes",
           "cg_fill_draft", "cg_contract_model_spec", "cg_contract_reverse", "cg_cache_stats", "cg_cache_clear",
           "cg_eval_strop", "cg_fill_bitmask_noalloc",
           "cg_sample_workspace_bytes", "cg_apply_mask_sample", "cg_advance", "cg_try_input", "cg_last_error",
           "cg_filter_workspace_bytes", "cg_filter_sample", "cg_top_workspace_bytes", "cg_top_logits",
           "cg_distill_topk", "cg_distill_topk_grad"]


class CgError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"[{code}] {msg}")
        self.code = code


class Options(ctypes.Structure):
    _fields_ = [("gen_cap", ctypes.c_uint32), ("flags", ctypes.c_uint32)]


class Info(ctypes.Structure):
    _fields_ = [("vocab_size", ctypes.c_int32), ("words_per_row", ctypes.c_int32),
                ("max_token_len", ctypes.c_int32), ("n_states", ctypes.c_int32),
                ("table_entries", ctypes.c_int32), ("table_bytes", ctypes.c_int32),
                ("compile_ms", ctypes.c_double), ("state_masks", ctypes.c_int32), ("pad", ctypes.c_int32),
                ("total_ms", ctypes.c_double), ("max_bytes", ctypes.c_int64)]


_lib = None


def lib():
    """Load libcg.so; fails loudly when it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with logit_masking_amd/build.py")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        L.cg_compile_grammar.argtypes = [ctypes.c_char_p, sz, vp, vp, i32, ctypes.POINTER(Options),
                                         ctypes.POINTER(vp)]
        L.cg_free_grammar.argtypes = [vp]
        L.cg_free_grammar.restype = None
        L.cg_grammar_info.argtypes = [vp, ctypes.POINTER(Info)]
        L.cg_init_state.argtypes = [vp, vp, i32, vp]
        L.cg_fill_workspace_bytes.argtypes = [vp, i32]
        L.cg_fill_workspace_bytes.restype = sz
        L.cg_fill_bitmask.argtypes = [vp, vp, i32, vp, i32, vp, vp]
        L.cg_fill_bitmask_noalloc.argtypes = [vp, vp, i32, vp, i32, vp]
        L.cg_sample_workspace_bytes.argtypes = [i32, i32]
        L.cg_sample_workspace_bytes.restype = sz
        L.cg_apply_mask_sample.argtypes = [vp, i32, i32, i32, i64, vp, i32, vp, vp, vp, vp, vp, vp, vp]
        L.cg_advance.argtypes = [vp, vp, i32, vp, vp, vp, vp]
        L.cg_force_bytes.argtypes = [vp, vp, i32, vp, sz, vp, vp, vp]
        L.cg_contract_model_spec.argtypes = [ctypes.c_char_p, sz, vp, sz, ctypes.POINTER(sz),
                                             ctypes.POINTER(ctypes.c_int32)]
        L.cg_contract_reverse.argtypes = [ctypes.c_char_p, sz, vp, sz, vp, sz, ctypes.POINTER(sz)]
        L.cg_draft_workspace_bytes.argtypes = [vp, i32, i32]
        L.cg_eval_strop.argtypes = [vp, sz, vp, sz, ctypes.POINTER(sz)]
        L.cg_eval_strop.restype = ctypes.c_int
        L.cg_cache_stats.argtypes = [ctypes.POINTER(i32), ctypes.POINTER(i64), ctypes.POINTER(i64)]
        L.cg_cache_stats.restype = ctypes.c_int
        L.cg_cache_clear.argtypes = []
        L.cg_cache_clear.restype = ctypes.c_int
        L.cg_draft_workspace_bytes.restype = sz
        L.cg_fill_draft.argtypes = [vp, vp, vp, i32, vp, i32, vp, vp, i32, vp, vp, vp]
        L.cg_eval_calc.argtypes = [vp, sz, ctypes.POINTER(ctypes.c_int64)]
        L.cg_sample_advance.argtypes = [vp, vp, i32, i32, i64, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.cg_sample_advance_fill.argtypes = [vp, vp, i32, i32, i64, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.cg_sample_advance_plan.argtypes = [vp, vp, i32, i32, i64, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.cg_fill_walk.argtypes = [vp, vp, i32, vp, i32, vp, vp]
        L.cg_try_input.argtypes = [vp, vp, sz, ctypes.POINTER(sz), ctypes.POINTER(ctypes.c_int)]
        L.cg_last_error.restype = ctypes.c_char_p
        for name in ("cg_compile_grammar", "cg_grammar_info", "cg_init_state", "cg_fill_bitmask",
                     "cg_fill_bitmask_noalloc", "cg_sample_advance",
                     "cg_sample_advance_fill", "cg_sample_advance_plan", "cg_fill_walk",
                     "cg_force_bytes", "cg_eval_calc", "cg_fill_draft", "cg_contract_model_spec",
                     "cg_contract_reverse",
                     "cg_apply_mask_sample", "cg_advance", "cg_try_input"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(rc):
    if rc != CG_OK:
        raise CgError(rc, lib().cg_last_error().decode(errors="replace"))


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(getattr(stream, "cuda_stream", stream) or 0)


def _dev(t, dtype, name, ndim=None):
    import torch
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")
    return t


def _states(t, name="states"):
    """Rows of cg_state: a contiguous [B, 24] uint8 device tensor."""
    import torch
    _dev(t, torch.uint8, name, 2)
    if t.shape[1] != STATE_BYTES:
        raise ValueError(f"{name} must be [B, {STATE_BYTES}] (cg_state rows)")
    return t


class Grammar:
    """A compiled grammar (cg_compile_grammar) bound to a vocabulary."""

    def __init__(self, spec_json: bytes, blob: bytes, offsets, gen_cap: int = 2048, host_only: bool = False):
        import numpy as np
        L = lib()
        if isinstance(spec_json, str):
            spec_json = spec_json.encode()
        off = np.ascontiguousarray(np.asarray(offsets, dtype=np.uint32))
        bl = np.frombuffer(blob if blob else b"\0", dtype=np.uint8)
        self._keep = (off, bl)
        h = ctypes.c_void_p()
        opts = Options(gen_cap, HOST_ONLY if host_only else 0)
        _check(L.cg_compile_grammar(spec_json, len(spec_json), bl.ctypes.data, off.ctypes.data, len(off) - 1,
                                    ctypes.byref(opts), ctypes.byref(h)))
        self._h = h
        self.V = len(off) - 1
        self.W = (self.V + 63) // 64
        self.gen_cap = gen_cap

    def __del__(self):
        h = getattr(self, "_h", None)
        if h and _lib is not None:
            _lib.cg_free_grammar(h)
            self._h = None

    def info(self) -> dict:
        i = Info()
        _check(lib().cg_grammar_info(self._h, ctypes.byref(i)))
        return {k: getattr(i, k) for k, _ in Info._fields_}

    def try_input(self, data: bytes):
        """(refused_at, complete) of the host walker over the packed table."""
        buf = ctypes.create_string_buffer(data, len(data)) if data else None
        ra, cp = ctypes.c_size_t(), ctypes.c_int()
        _check(lib().cg_try_input(self._h, buf, len(data), ctypes.byref(ra), ctypes.byref(cp)))
        return ra.value, bool(cp.value)

    # ---- device calls (async on the current stream) --------------------
    def new_states(self, B: int, device="cuda"):
        import torch
        return torch.empty((B, STATE_BYTES), dtype=torch.uint8, device=device)

    def init_state(self, states, stream=None):
        import torch
        _states(states)
        _check(lib().cg_init_state(self._h, _ptr(states), states.shape[0], _stream(stream)))

    def fill_workspace_bytes(self, B: int) -> int:
        return int(lib().cg_fill_workspace_bytes(self._h, B))

    def new_fill_workspace(self, B: int, device="cuda"):
        """Device buffer for fill_bitmask over B rows (no initialisation needed)."""
        import torch
        return torch.empty(max(2, (self.fill_workspace_bytes(B) + 15) // 16 * 2), dtype=torch.int64, device=device)

    def fill_bitmask(self, states, mask, workspace=None, stream=None):
        """workspace: from new_fill_workspace(B); None allocates one for this call."""
        import torch
        _states(states)
        _dev(mask, torch.int64, "mask", 2)
        if mask.shape[0] < states.shape[0]:
            raise ValueError("mask has fewer rows than states")
        B = states.shape[0]
        if workspace is None:
            workspace = self.new_fill_workspace(B, states.device)
        if workspace.numel() * workspace.element_size() < self.fill_workspace_bytes(B):
            raise ValueError("fill workspace too small")
        _check(lib().cg_fill_bitmask(self._h, _ptr(states), B, _ptr(mask), mask.shape[1], _ptr(workspace),
                                     _stream(stream)))

    def fill_bitmask_noalloc(self, states, mask, stream=None):
        """cg_fill_bitmask_noalloc: fill_bitmask with the library's own
        per-device scratch (no workspace; calls on one device must not
        overlap)."""
        import torch
        _states(states)
        _dev(mask, torch.int64, "mask", 2)
        if mask.shape[0] < states.shape[0]:
            raise ValueError("mask has fewer rows than states")
        _check(lib().cg_fill_bitmask_noalloc(self._h, _ptr(states), states.shape[0], _ptr(mask), mask.shape[1],
                                             _stream(stream)))

    def sample_advance(self, logits, mask, temperature, seed, steps, workspace, out_ids, out_logprob, states,
                       status, stream=None):
        """cg_sample_advance: apply_mask_sample + advance in one launch (same
        tensors and meanings as those two calls; steps is read, then bumped)."""
        import torch
        if logits.dtype == torch.float32:
            dt = DTYPE_F32
        elif logits.dtype == torch.bfloat16:
            dt = DTYPE_BF16
        else:
            raise ValueError("logits must be float32 or bfloat16")
        if not logits.is_cuda or logits.dim() != 2 or logits.stride(1) != 1 or logits.shape[1] < self.V:
            raise ValueError("logits must be a 2-D device tensor [B, >= vocab] with unit column stride")
        B = logits.shape[0]
        _dev(mask, torch.int64, "mask", 2)
        _dev(temperature, torch.float32, "temperature", 1)
        _dev(seed, torch.int64, "seed", 1)
        _states(states)
        for t, n in ((steps, "steps"), (out_ids, "out_ids"), (status, "status")):
            _dev(t, torch.int32, n, 1)
        _dev(out_logprob, torch.float32, "out_logprob", 1)
        if workspace.numel() * workspace.element_size() < sample_workspace_bytes(B, self.V):
            raise ValueError("workspace too small")
        for t, n in ((mask, "mask"), (temperature, "temperature"), (seed, "seed"), (steps, "steps"),
                     (out_ids, "out_ids"), (out_logprob, "out_logprob"), (states, "states"), (status, "status")):
            if t.shape[0] < B:
                raise ValueError(f"{n} has fewer rows than logits")
        _check(lib().cg_sample_advance(self._h, _ptr(logits), dt, B, logits.stride(0), _ptr(mask), mask.shape[1],
                                       _ptr(temperature), _ptr(seed), _ptr(steps), _ptr(workspace), _ptr(out_ids),
                                       _ptr(out_logprob), _ptr(states), _ptr(status), _stream(stream)))

    def sample_advance_fill(self, logits, mask, temperature, seed, steps, workspace, out_ids, out_logprob, states,
                            status, fill_workspace=None, stream=None, split=False):
        """cg_sample_advance_fill: sample_advance, then the next step's mask
        written over `mask` (fill_workspace: from new_fill_workspace(B); None
        allocates one for this call).  split=True makes the first of its two
        launches only (cg_sample_advance_plan); fill_walk completes the mask."""
        import torch
        if logits.dtype == torch.float32:
            dt = DTYPE_F32
        elif logits.dtype == torch.bfloat16:
            dt = DTYPE_BF16
        else:
            raise ValueError("logits must be float32 or bfloat16")
        if not logits.is_cuda or logits.dim() != 2 or logits.stride(1) != 1 or logits.shape[1] < self.V:
            raise ValueError("logits must be a 2-D device tensor [B, >= vocab] with unit column stride")
        B = logits.shape[0]
        _dev(mask, torch.int64, "mask", 2)
        _dev(temperature, torch.float32, "temperature", 1)
        _dev(seed, torch.int64, "seed", 1)
        _states(states)
        for t, n in ((steps, "steps"), (out_ids, "out_ids"), (status, "status")):
            _dev(t, torch.int32, n, 1)
        _dev(out_logprob, torch.float32, "out_logprob", 1)
        if workspace.numel() * workspace.element_size() < sample_workspace_bytes(B, self.V):
            raise ValueError("workspace too small")
        for t, n in ((mask, "mask"), (temperature, "temperature"), (seed, "seed"), (steps, "steps"),
                     (out_ids, "out_ids"), (out_logprob, "out_logprob"), (states, "states"), (status, "status")):
            if t.shape[0] < B:
                raise ValueError(f"{n} has fewer rows than logits")
        if fill_workspace is None:
            fill_workspace = self.new_fill_workspace(B)
        elif fill_workspace.numel() * fill_workspace.element_size() < self.fill_workspace_bytes(B):
            raise ValueError("fill workspace too small")
        fn = lib().cg_sample_advance_plan if split else lib().cg_sample_advance_fill
        _check(fn(self._h, _ptr(logits), dt, B, logits.stride(0), _ptr(mask), mask.shape[1], _ptr(temperature),
                  _ptr(seed), _ptr(steps), _ptr(workspace), _ptr(out_ids), _ptr(out_logprob), _ptr(states),
                  _ptr(status), _ptr(fill_workspace), _stream(stream)))

    def fill_walk(self, states, mask, workspace, stream=None):
        """cg_fill_walk: the second launch of sample_advance_fill (after
        split=True, with the same mask and fill workspace)."""
        import torch
        _states(states)
        _dev(mask, torch.int64, "mask", 2)
        B = states.shape[0]
        if mask.shape[0] < B:
            raise ValueError("mask has fewer rows than states")
        _dev(workspace, None, "workspace")
        if workspace.numel() * workspace.element_size() < self.fill_workspace_bytes(B):
            raise ValueError("fill workspace too small")
        _check(lib().cg_fill_walk(self._h, _ptr(states), B, _ptr(mask), mask.shape[1], _ptr(workspace),
                                  _stream(stream)))

    def advance(self, states, ids, steps, status, stream=None):
        import torch
        _states(states)
        for t, n in ((ids, "ids"), (steps, "steps"), (status, "status")):
            _dev(t, torch.int32, n, 1)
            if t.shape[0] < states.shape[0]:
                raise ValueError(f"{n} has fewer rows than states")
        _check(lib().cg_advance(self._h, _ptr(states), states.shape[0], _ptr(ids), _ptr(steps), _ptr(status),
                                _stream(stream)))

    def draft_workspace_bytes(self, B: int, k: int) -> int:
        return int(lib().cg_draft_workspace_bytes(self._h, B, k))

    def fill_draft(self, states, steps, draft, path_states, masks, accept_len, workspace=None, stream=None):
        """cg_fill_draft: draft [B, k] int32 (-1 pads); path_states [B, k+1, 24]
        uint8; masks [B, k+1, W] int64; accept_len [B] int32; steps [B] int32
        or None."""
        import torch
        _states(states)
        B = states.shape[0]
        _dev(draft, torch.int32, "draft", 2)
        k = draft.shape[1]
        if draft.shape[0] < B:
            raise ValueError("draft has fewer rows than states")
        _dev(path_states, torch.uint8, "path_states", 3)
        if path_states.shape[2] != STATE_BYTES:
            raise ValueError(f"path_states must be [B, k+1, {STATE_BYTES}]")
        _dev(masks, torch.int64, "masks", 3)
        _dev(accept_len, torch.int32, "accept_len", 1)
        if steps is not None:
            _dev(steps, torch.int32, "steps", 1)
        if path_states.shape[0] < B or path_states.shape[1] != k + 1 or masks.shape[0] < B or masks.shape[1] != k + 1:
            raise ValueError("path_states / masks must be [B, k+1, ...]")
        if workspace is None:
            n = self.draft_workspace_bytes(B, k)
            workspace = torch.empty(max(2, (n + 15) // 16 * 2), dtype=torch.int64, device=states.device)
        if workspace.numel() * workspace.element_size() < self.draft_workspace_bytes(B, k):
            raise ValueError("draft workspace too small")
        _check(lib().cg_fill_draft(self._h, _ptr(states), _ptr(steps), B, _ptr(draft), k, _ptr(path_states),
                                   _ptr(masks), masks.shape[2], _ptr(accept_len), _ptr(workspace), _stream(stream)))

    def force_bytes(self, states, data, offsets, status, stream=None):
        """cg_force_bytes: row r walks data[offsets[r]:offsets[r+1]] (uint8 /
        int32 device tensors, offsets has B+1 entries)."""
        import torch
        _states(states)
        B = states.shape[0]
        _dev(data, torch.uint8, "data", 1)
        _dev(offsets, torch.int32, "offsets", 1)
        if offsets.shape[0] < B + 1:
            raise ValueError("offsets needs B+1 entries")
        _dev(status, torch.int32, "status", 1)
        if status.shape[0] < B:
            raise ValueError("status has fewer rows than states")
        _check(lib().cg_force_bytes(self._h, _ptr(states), B, _ptr(data), data.numel(), _ptr(offsets),
                                    _ptr(status), _stream(stream)))


def eval_calc(span: bytes):
    """cg_eval_calc: (CG_OK, value) or (error code, message)."""
    if isinstance(span, str):
        span = span.encode()
    buf = ctypes.create_string_buffer(span, len(span)) if span else None
    v = ctypes.c_int64()
    rc = lib().cg_eval_calc(buf, len(span), ctypes.byref(v))
    if rc != CG_OK:
        return rc, lib().cg_last_error().decode(errors="replace")
    return CG_OK, v.value


def eval_strop(span: bytes):
    """cg_eval_strop: (CG_OK, result bytes) or (error code, message)."""
    if isinstance(span, str):
        span = span.encode()
    buf = ctypes.create_string_buffer(span, len(span)) if span else None
    rc, out = _sized_call(lambda b, c, n: lib().cg_eval_strop(buf, len(span), b, c, n))
    if rc != CG_OK:
        return rc, lib().cg_last_error().decode(errors="replace")
    return CG_OK, out


def cache_stats():
    """(entries, hits, misses) of the library's grammar cache."""
    e, h, m = ctypes.c_int32(), ctypes.c_int64(), ctypes.c_int64()
    _check(lib().cg_cache_stats(ctypes.byref(e), ctypes.byref(h), ctypes.byref(m)))
    return e.value, h.value, m.value


def cache_clear():
    _check(lib().cg_cache_clear())


def _sized_call(fn, *args):
    """Call an output-buffer function, growing the buffer once if needed."""
    cap = 1 << 16
    for _ in range(2):
        buf = ctypes.create_string_buffer(cap)
        n = ctypes.c_size_t()
        rc = fn(*args, buf, cap, ctypes.byref(n))
        if rc != CG_E_LIMIT:
            return rc, buf.raw[:n.value]
        cap = n.value + 1
    return rc, b""


def contract_model_spec(ext_spec):
    """cg_contract_model_spec: (model-facing spec bytes, replaced fields)."""
    if isinstance(ext_spec, str):
        ext_spec = ext_spec.encode()
    nf = ctypes.c_int32()
    rc, out = _sized_call(lambda b, c, n: lib().cg_contract_model_spec(ext_spec, len(ext_spec), b, c, n,
                                                                       ctypes.byref(nf)))
    _check(rc)
    return out, nf.value


def contract_reverse(ext_spec, text: bytes):
    """cg_contract_reverse: (rc, output bytes, message); rc is CG_OK or
    CG_E_INVALID (other codes raise)."""
    if isinstance(ext_spec, str):
        ext_spec = ext_spec.encode()
    tb = ctypes.create_string_buffer(text, len(text)) if text else None
    rc, out = _sized_call(lambda b, c, n: lib().cg_contract_reverse(ext_spec, len(ext_spec), tb, len(text), b, c, n))
    if rc not in (CG_OK, CG_E_INVALID):
        _check(rc)
    msg = "" if rc == CG_OK else lib().cg_last_error().decode(errors="replace")
    return rc, out, msg


def sample_workspace_bytes(B: int, V: int) -> int:
    return int(lib().cg_sample_workspace_bytes(B, V))


def new_workspace(B: int, V: int, device="cuda"):
    """A workspace for apply_mask_sample (possibly empty)."""
    import torch
    n = sample_workspace_bytes(B, V)
    return torch.zeros(max(1, (n + 15) // 16 * 2), dtype=torch.float64, device=device)


def apply_mask_sample(logits, mask, temperature, seed, step, workspace, out_ids, out_logprob, vocab=None,
                      stream=None):
    """cg_apply_mask_sample on torch tensors: logits [B, stride] float32 or
    bfloat16, mask [B, W] int64, temperature [B] float32, seed [B] int64
    (the u64 bits), step [B] int32, outputs ids [B] int32, logprob [B] float32."""
    import torch
    if logits.dtype == torch.float32:
        dt = DTYPE_F32
    elif logits.dtype == torch.bfloat16:
        dt = DTYPE_BF16
    else:
        raise ValueError("logits must be float32 or bfloat16")
    if not logits.is_cuda or logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be a 2-D device tensor with unit column stride")
    B = logits.shape[0]
    V = logits.shape[1] if vocab is None else vocab
    _dev(mask, torch.int64, "mask", 2)
    _dev(temperature, torch.float32, "temperature", 1)
    _dev(seed, torch.int64, "seed", 1)
    _dev(step, torch.int32, "step", 1)
    _dev(out_ids, torch.int32, "out_ids", 1)
    _dev(out_logprob, torch.float32, "out_logprob", 1)
    if workspace.numel() * workspace.element_size() < sample_workspace_bytes(B, V):
        raise ValueError("workspace too small")
    for t, n in ((mask, "mask"), (temperature, "temperature"), (seed, "seed"), (step, "step"),
                 (out_ids, "out_ids"), (out_logprob, "out_logprob")):
        if t.shape[0] < B:
            raise ValueError(f"{n} has fewer rows than logits")
    _check(lib().cg_apply_mask_sample(_ptr(logits), dt, B, V, logits.stride(0), _ptr(mask), mask.shape[1],
                                      _ptr(temperature), _ptr(seed), _ptr(step), _ptr(workspace), _ptr(out_ids),
                                      _ptr(out_logprob), _stream(stream)))


# ---- row operators: filtered sampling, top logits, distillation ---------------
# Every tensor of a call lives on the logits' device; the call runs on that
# device's current stream (or `stream`), whatever device is current.

_row_fns = None


def _row_lib():
    """The row operators' functions with their prototypes, set once."""
    global _row_fns
    if _row_fns is None:
        L = lib()
        vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        rows = [vp, i32, i32, i32, i64, vp, i32]
        for name, args, res in (
                ("cg_filter_workspace_bytes", [i32, i32], sz),
                ("cg_filter_sample", rows + [vp] * 9, ctypes.c_int),
                ("cg_top_workspace_bytes", [i32, i32, i32], sz),
                ("cg_top_logits", rows + [i32] + [vp] * 5, ctypes.c_int),
                ("cg_distill_topk", rows + [vp, vp, i32, f32, vp, vp, vp, vp, i64, vp], ctypes.c_int),
                ("cg_distill_topk_grad", rows + [vp, vp, i32, f32, vp, vp, vp, i64, vp], ctypes.c_int)):
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, res
        _row_fns = L
    return _row_fns


def _rows(logits, mask, vocab):
    """(dtype code, rows, vocab, row stride, mask address, words) of the logits and mask of a row operator."""
    import torch
    dtype = logits.dtype
    if dtype is torch.bfloat16:
        dt = DTYPE_BF16
    elif dtype is torch.float32:
        dt = DTYPE_F32
    else:
        raise ValueError("logits must be float32 or bfloat16")
    if not logits.is_cuda or logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be a 2-D device tensor with unit column stride")
    B, cols = logits.shape
    V = cols if vocab is None else vocab
    if not 1 <= V <= cols:
        raise ValueError("vocab out of range of the logits' columns")
    if V > MAX_ROW_VOCAB:
        raise ValueError(f"vocab above {MAX_ROW_VOCAB}")
    stride = logits.stride(0)
    if stride < V:
        if B > 1:
            raise ValueError("logits' rows overlap")
        stride = V  # a row of its own may have any stride
    if mask is None:
        return dt, B, V, stride, None, 0
    _row_arg(mask, torch.int64, "mask", logits.get_device(), B, None)
    if mask.shape[1] < (V + 63) // 64:
        raise ValueError("mask has fewer than ceil(vocab / 64) words per row")
    return dt, B, V, stride, mask.data_ptr(), mask.shape[1]


def _row_arg(t, dtype, name, device, rows, cols=0):
    """The address of a contiguous tensor on device number `device` with at
    least `rows` rows: 1-D for cols = 0, else 2-D with `cols` columns (None:
    any number)."""
    shape = t.shape
    if (t.dtype is dtype and t.get_device() == device and t.is_contiguous() and shape[0] >= rows and
            (len(shape) == 1 if cols == 0 else len(shape) == 2 and (cols is None or shape[1] == cols))):
        return t.data_ptr()
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on the logits' device")
    if t.dim() != (1 if cols == 0 else 2) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with {1 if cols == 0 else 2} dims")
    if shape[0] < rows:
        raise ValueError(f"{name} has fewer rows than logits")
    raise ValueError(f"{name} must have {cols} columns")


def _workspace_arg(t, need, logits):
    if t is None:
        if need:
            raise ValueError("a workspace is needed")
        return None
    if t.get_device() != logits.get_device() or not t.is_contiguous():
        raise ValueError("workspace must be contiguous on the logits' device")
    if t.numel() * t.element_size() < need:
        raise ValueError("workspace too small")
    return t.data_ptr()


def _row_call(fn, device, stream, *args):
    """fn(*args, stream) on device number `device`."""
    import torch
    if stream is None:
        # the handle alone (without the Stream object around it: 1 us of a call's 10)
        raw = torch._C._cuda_getCurrentRawStream(device) or None
    else:
        raw = getattr(stream, "cuda_stream", stream) or None
    if device == torch.cuda.current_device():
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, raw)
    if rc != CG_OK:
        _check(rc)


def filter_workspace_bytes(B: int, V: int) -> int:
    return int(_row_lib().cg_filter_workspace_bytes(B, V))


def new_filter_workspace(B: int, V: int, device="cuda"):
    """A workspace for filter_sample (possibly empty)."""
    import torch
    return torch.empty((filter_workspace_bytes(B, V) + 15) // 16 * 2, dtype=torch.int64, device=device)


def filter_sample(logits, mask, temperature, top_k, top_p, min_p, uniform, workspace, out_ids, out_logprob, vocab=None,
                  stream=None):
    """cg_filter_sample on torch tensors: logits [B, >= vocab] float32 or
    bfloat16, mask [B, W] int64 or None, temperature [B] float32, top_k [B]
    int32, top_p and min_p [B] float32 (each of the three may be None: no such
    filter), uniform [B] float32 in [0, 1); workspace from
    new_filter_workspace(B, vocab) or None; outputs ids [B] int32, logprob [B]
    float32."""
    import torch
    L = _row_lib()
    dt, B, V, stride, m, words = _rows(logits, mask, vocab)
    f32, i32, dev = torch.float32, torch.int32, logits.get_device()
    _row_call(L.cg_filter_sample, dev, stream, logits.data_ptr(), dt, B, V, stride, m, words,
              _row_arg(temperature, f32, "temperature", dev, B),
              None if top_k is None else _row_arg(top_k, i32, "top_k", dev, B),
              None if top_p is None else _row_arg(top_p, f32, "top_p", dev, B),
              None if min_p is None else _row_arg(min_p, f32, "min_p", dev, B),
              _row_arg(uniform, f32, "uniform", dev, B),
              _workspace_arg(workspace, L.cg_filter_workspace_bytes(B, V), logits),
              _row_arg(out_ids, i32, "out_ids", dev, B), _row_arg(out_logprob, f32, "out_logprob", dev, B))


def top_workspace_bytes(B: int, V: int, k: int) -> int:
    return int(_row_lib().cg_top_workspace_bytes(B, V, k))


def new_top_workspace(B: int, V: int, k: int, device="cuda"):
    """A workspace for top_logits (possibly empty)."""
    import torch
    return torch.empty((top_workspace_bytes(B, V, k) + 15) // 16 * 2, dtype=torch.int64, device=device)


def top_logits(logits, mask, workspace, out_ids, out_logits, out_lse, vocab=None, stream=None):
    """cg_top_logits on torch tensors: logits and mask as for filter_sample,
    workspace from new_top_workspace(B, vocab, k) or None; outputs ids [B, k]
    int32, logits [B, k] float32 (k <= MAX_TOP is their column count), lse [B]
    float32."""
    import torch
    L = _row_lib()
    dt, B, V, stride, m, words = _rows(logits, mask, vocab)
    if out_ids.dim() != 2:
        raise ValueError("out_ids must be [B, k]")
    k, dev = out_ids.shape[1], logits.get_device()
    _row_call(L.cg_top_logits, dev, stream, logits.data_ptr(), dt, B, V, stride, m, words, k,
              _workspace_arg(workspace, L.cg_top_workspace_bytes(B, V, k), logits),
              _row_arg(out_ids, torch.int32, "out_ids", dev, B, k),
              _row_arg(out_logits, torch.float32, "out_logits", dev, B, k),
              _row_arg(out_lse, torch.float32, "out_lse", dev, B))


def _distill_args(logits, mask, teacher_ids, teacher_logits, temperature, vocab):
    import torch
    dt, B, V, stride, m, words = _rows(logits, mask, vocab)
    if teacher_ids.dim() != 2:
        raise ValueError("teacher_ids must be [rows, k]")
    k, dev = teacher_ids.shape[1], logits.get_device()
    return dev, B, (logits.data_ptr(), dt, B, V, stride, m, words,
                       _row_arg(teacher_ids, torch.int32, "teacher_ids", dev, B, k),
                       _row_arg(teacher_logits, torch.float32, "teacher_logits", dev, B, k), k, temperature)


def _grad_arg(grad, logits, args):
    """(address, row stride) of a gradient: the logits themselves, or rows apart from them."""
    b, dt, B, V, x_stride = args[:5]
    if grad.dtype is not logits.dtype or grad.get_device() != logits.get_device():
        raise ValueError("out_grad must have the logits' dtype and device")
    shape, strides = grad.shape, grad.stride()
    if len(shape) != 2 or strides[1] != 1 or shape[0] < B or shape[1] < V:
        raise ValueError("out_grad must be [rows, >= vocab] with unit column stride")
    a, stride = grad.data_ptr(), strides[0]
    if stride < V:
        if B > 1:
            raise ValueError("out_grad's rows overlap")
        stride = V
    if a != b or stride != x_stride:
        size = 2 if dt == DTYPE_BF16 else 4
        if B and a < b + ((B - 1) * x_stride + V) * size and b < a + ((B - 1) * stride + V) * size:
            # they may still lie between the logits' rows
            if x_stride != stride or not V <= (a - b) // size % stride <= stride - V:
                raise ValueError("out_grad overlaps the logits (it may only be the same rows)")
    return a, stride


def distill_topk(logits, mask, teacher_ids, teacher_logits, temperature, out_loss, out_lse=None, weight=None,
                 out_grad=None, vocab=None, stream=None):
    """cg_distill_topk on torch tensors: student logits [rows, >= vocab]
    float32 or bfloat16, mask [rows, W] int64 or None, teacher_ids [rows, k]
    int32, teacher_logits [rows, k] float32 (what top_logits writes),
    temperature a number; outputs loss [rows] float32, lse [rows] float32 or
    None and, given weight [rows] float32, the gradient of sum(weight * loss)
    in out_grad [rows, >= vocab] of the logits' dtype (it may be `logits`)."""
    import torch
    L = _row_lib()
    dev, B, args = _distill_args(logits, mask, teacher_ids, teacher_logits, temperature, vocab)
    f32 = torch.float32
    if (weight is None) != (out_grad is None):
        raise ValueError("weight and out_grad go together")
    g, gs = (None, 0) if out_grad is None else _grad_arg(out_grad, logits, args)
    _row_call(L.cg_distill_topk, dev, stream, *args, _row_arg(out_loss, f32, "out_loss", dev, B),
              None if out_lse is None else _row_arg(out_lse, f32, "out_lse", dev, B),
              None if weight is None else _row_arg(weight, f32, "weight", dev, B), g, gs)


def distill_topk_grad(logits, mask, teacher_ids, teacher_logits, temperature, lse, weight, out_grad, vocab=None,
                      stream=None):
    """cg_distill_topk_grad: distill_topk's gradient alone, from the lse it wrote."""
    import torch
    L = _row_lib()
    dev, B, args = _distill_args(logits, mask, teacher_ids, teacher_logits, temperature, vocab)
    g, gs = _grad_arg(out_grad, logits, args)
    _row_call(L.cg_distill_topk_grad, dev, stream, *args, _row_arg(lse, torch.float32, "lse", dev, B),
              _row_arg(weight, torch.float32, "weight", dev, B), g, gs)


_distill_fn = None


def _distill_function():
    """The autograd function behind distill_topk_loss (torch is imported only when a call needs it)."""
    global _distill_fn
    if _distill_fn is None:
        import torch

        class DistillTopK(torch.autograd.Function):
            @staticmethod
            def forward(ctx, logits, mask, teacher_ids, teacher_logits, temperature, vocab):
                rows = logits.shape[0]
                loss = torch.empty(rows, dtype=torch.float32, device=logits.device)
                lse = torch.empty_like(loss)
                distill_topk(logits, mask, teacher_ids, teacher_logits, temperature, loss, lse, vocab=vocab)
                ctx.save_for_backward(logits, mask, teacher_ids, teacher_logits, lse)
                ctx.temperature, ctx.vocab = temperature, vocab
                return loss

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, weight):
                logits, mask, teacher_ids, teacher_logits, lse = ctx.saved_tensors
                whole = ctx.vocab is None or ctx.vocab == logits.shape[1]
                grad = (torch.empty if whole else torch.zeros)(logits.shape, dtype=logits.dtype, device=logits.device)
                distill_topk_grad(logits, mask, teacher_ids, teacher_logits, ctx.temperature, lse,
                                  weight.float().contiguous(), grad, vocab=ctx.vocab)
                return grad, None, None, None, None, None

        _distill_fn = DistillTopK
    return _distill_fn


def distill_topk_loss(logits, teacher_ids, teacher_logits, mask=None, temperature=1.0, vocab=None):
    """The per-position losses of cg_distill_topk, differentiable by the
    logits: logits [..., >= vocab], teacher_ids and teacher_logits [..., k],
    mask [..., W] or None; float32 losses of the leading shape."""
    lead = logits.shape[:-1]
    for t, n in ((teacher_ids, "teacher_ids"), (teacher_logits, "teacher_logits"), (mask, "mask")):
        if t is not None and t.shape[:-1] != lead:
            raise ValueError(f"{n} must have the logits' leading shape")
    x = logits.reshape(-1, logits.shape[-1])
    if x.stride(-1) != 1:
        x = x.contiguous()
    ids = teacher_ids.reshape(-1, teacher_ids.shape[-1]).contiguous()
    top = teacher_logits.reshape(-1, teacher_logits.shape[-1]).contiguous()
    if mask is not None:
        mask = mask.reshape(-1, mask.shape[-1]).contiguous()
    return _distill_function().apply(x, mask, ids, top, temperature, vocab).reshape(lead)
