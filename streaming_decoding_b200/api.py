"""Python binding of libwedlm: the C-ABI calls under the same names, with
argument marshalling only.  Every step of the decode path runs in the CUDA
library; this module never computes any part of it.

Host arrays are numpy; device buffers are torch CUDA tensors (PyTorch supplies
device memory and streams)."""
from __future__ import annotations

import ctypes
import math

import numpy as np

from . import _lib
from ._lib import ModelCfg, SeqStats, StepParams, WedlmError

C = _lib.header_constants()
DTYPE = {"f32": C["WEDLM_DTYPE_F32"], "bf16": C["WEDLM_DTYPE_BF16"]}


def _ptr(a) -> int:
    if a is None:
        return 0
    if isinstance(a, np.ndarray):
        return a.ctypes.data
    return int(a.data_ptr())  # torch tensor


def _check(st: int, where: str, ctx=None):
    if st != 0:
        detail = _lib.load().wedlm_last_error(ctx).decode() if ctx else ""
        raise WedlmError(st, where, detail)


def step_params(lam: float, tau: float, tau_none: bool = False, logit_scale: float = 1.0, blockwise: bool = False,
                temperature: float = 0.0, seed: int = 0) -> StepParams:
    return StepParams(float(lam), float(tau), 1 if tau_none else 0, float(logit_scale), 1 if blockwise else 0,
                      float(temperature), int(seed))


class Engine:
    """One libwedlm context (one model, a batch of sequence slots)."""

    def __init__(self, dims: dict, max_batch: int, max_window: int, max_ctx: int, dtype: str | None = None,
                 num_pages: int = 0, prefill_chunk: int = 0, stream=None):
        self.lib = _lib.load()
        self.dims = dict(dims)
        dtype = dtype or dims.get("dtype", "f32")
        self.dtype = dtype
        cfg = ModelCfg(dims["L"], dims["d"], dims["hq"], dims["hkv"], dims["hd"], dims["F"], dims["V"],
                       dims["mask_id"], float(dims["theta"]), float(dims["eps"]), DTYPE[dtype], max_batch,
                       max_window, max_ctx, num_pages, prefill_chunk)
        self.max_batch, self.max_window, self.max_ctx = max_batch, max_window, max_ctx
        self.stream = stream
        h = ctypes.c_void_p()
        _check(self.lib.wedlm_create(ctypes.byref(cfg), ctypes.c_void_p(_stream_handle(stream)), ctypes.byref(h)),
               "wedlm_create")
        self.ctx = h

    # -- lifetime ---------------------------------------------------------
    def close(self):
        if getattr(self, "ctx", None):
            self.lib.wedlm_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()

    # -- weights ------------------------------------------------------------
    def load_weights(self, kind: int, layer: int, src):
        """src: numpy array (host) or torch CUDA tensor (device); float32 or bf16 (uint16 bits / torch.bfloat16)."""
        if isinstance(src, np.ndarray):
            src = np.ascontiguousarray(src)
            dt = C["WEDLM_DTYPE_BF16"] if src.dtype == np.uint16 else C["WEDLM_DTYPE_F32"]
            if src.dtype not in (np.uint16, np.float32):
                raise TypeError(src.dtype)
            mem = C["WEDLM_MEM_HOST"]
        else:
            import torch
            dt = C["WEDLM_DTYPE_BF16"] if src.dtype in (torch.bfloat16, torch.int16) else C["WEDLM_DTYPE_F32"]
            mem = C["WEDLM_MEM_DEVICE"] if src.is_cuda else C["WEDLM_MEM_HOST"]
            src = src.contiguous()
        _check(self.lib.wedlm_load_weights(self.ctx, kind, layer, _ptr(src), dt, mem), "wedlm_load_weights",
               self.ctx)

    def load_model(self, weight_iter):
        for kind, layer, arr in weight_iter:
            self.load_weights(kind, layer, arr)

    # -- sequences -----------------------------------------------------------
    def prefill(self, slot: int, prompt, max_new_tokens: int, window: int):
        p = np.ascontiguousarray(np.asarray(prompt, dtype=np.int32))
        _check(self.lib.wedlm_prefill(self.ctx, slot, p.ctypes.data if len(p) else None, len(p), max_new_tokens,
                                      window), "wedlm_prefill", self.ctx)

    def kv_reset(self, slot: int = -1):
        _check(self.lib.wedlm_kv_reset(self.ctx, slot), "wedlm_kv_reset", self.ctx)

    def stream_step(self, params: StepParams):
        """One decode step: returns (committed tokens per slot, counts, active)."""
        committed = np.zeros((self.max_batch, self.max_window), np.int32)
        counts = np.zeros(self.max_batch, np.int32)
        active = np.zeros(1, np.int32)
        _check(self.lib.wedlm_stream_step(self.ctx, ctypes.byref(params), committed.ctypes.data, counts.ctypes.data,
                                          active.ctypes.data), "wedlm_stream_step", self.ctx)
        return [committed[b, :counts[b]].tolist() for b in range(self.max_batch)], counts, int(active[0])

    def stream_step_into(self, params: StepParams, committed: np.ndarray, counts: np.ndarray, active: np.ndarray):
        """Same as stream_step with caller-provided (e.g. pinned) host buffers."""
        _check(self.lib.wedlm_stream_step(self.ctx, ctypes.byref(params), _ptr(committed), _ptr(counts),
                                          _ptr(active)), "wedlm_stream_step", self.ctx)

    def stream_step_async(self, params: StepParams, n_steps: int = 1):
        _check(self.lib.wedlm_stream_step_async(self.ctx, ctypes.byref(params), n_steps), "wedlm_stream_step_async",
               self.ctx)

    def read_generated(self, slot: int) -> list:
        buf = np.zeros(self.max_ctx, np.int32)
        n = ctypes.c_int32()
        _check(self.lib.wedlm_read_generated(self.ctx, slot, buf.ctypes.data, len(buf), ctypes.byref(n)),
               "wedlm_read_generated", self.ctx)
        return buf[:n.value].tolist()

    def stats(self, slot: int) -> dict:
        s = SeqStats()
        _check(self.lib.wedlm_get_stats(self.ctx, slot, ctypes.byref(s)), "wedlm_get_stats", self.ctx)
        return {f: getattr(s, f) for f, _ in SeqStats._fields_}

    def kernel_launches(self) -> int:
        n = ctypes.c_int64()
        _check(self.lib.wedlm_kernel_launches(self.ctx, ctypes.byref(n)), "wedlm_kernel_launches")
        return n.value

    def autotune(self, enable: bool = True):
        _check(self.lib.wedlm_autotune(self.ctx, 1 if enable else 0), "wedlm_autotune", self.ctx)

    def keep_logits(self, enable: bool = True):
        """Test hook: True writes logits every step (two-pass LM head + entropy)."""
        _check(self.lib.wedlm_debug_keep_logits(self.ctx, 1 if enable else 0), "wedlm_debug_keep_logits", self.ctx)

    def force_fused_entropy(self, enable: bool = True):
        """Test hook: greedy bf16 steps always take the fused LM-head entropy epilogue."""
        _check(self.lib.wedlm_debug_keep_logits(self.ctx, 2 if enable else 0), "wedlm_debug_keep_logits", self.ctx)

    def debug_capture(self, enable: bool = True):
        """Keep the residual stream at every layer boundary of each decode step (test hook)."""
        _check(self.lib.wedlm_debug_capture(self.ctx, 1 if enable else 0), "wedlm_debug_capture", self.ctx)

    def debug_residual(self, layer: int, rows: int) -> np.ndarray:
        """x entering `layer` (layer = L: after the last layer), [rows][d] fp32, of the last step."""
        out = np.empty((rows, self.dims["d"]), np.float32)
        _check(self.lib.wedlm_debug_residual(self.ctx, layer, out.ctypes.data, rows), "wedlm_debug_residual",
               self.ctx)
        return out

    def gemm_plan(self, kind: str, rows: int):
        """(tile_w, tile_n, k_splits, us) recorded for a projection kind ('gemm_qkv', ...) at `rows`, or None."""
        tw, tn, ks, us = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32(), ctypes.c_float()
        st = self.lib.wedlm_gemm_plan(self.ctx, C["WEDLM_PROF_" + kind.upper()], rows, ctypes.byref(tw),
                                      ctypes.byref(tn), ctypes.byref(ks), ctypes.byref(us))
        return (tw.value, tn.value, ks.value, round(us.value, 2)) if st == 0 else None

    def gemm_schedule(self, kind: str, rows: int):
        """Names of the schedule features of the recorded plan (CTA pairs, hybrid or
        cluster K split, ...), or None."""
        sc = ctypes.c_int32()
        st = self.lib.wedlm_gemm_schedule(self.ctx, C["WEDLM_PROF_" + kind.upper()], rows, ctypes.byref(sc))
        if st != 0:
            return None
        names = {1: "cta_pair", 2: "hybrid_split", 4: "cluster_split", 8: "co_resident_fixup",
                 16: "two_weight_subtiles", 32: "bk32"}
        return [n for bit, n in names.items() if sc.value & bit]

    def profile_enable(self, on: bool = True):
        _check(self.lib.wedlm_profile_enable(self.ctx, 1 if on else 0), "wedlm_profile_enable", self.ctx)

    def profile_read(self) -> dict:
        """{kind: (total ms, launches)} for kinds WEDLM_PROF_* since profile_enable."""
        nk = C["WEDLM_PROF_KINDS"]
        ms = np.zeros(nk, np.float64)
        n = np.zeros(nk, np.int64)
        _check(self.lib.wedlm_profile_read(self.ctx, ms.ctypes.data, n.ctypes.data), "wedlm_profile_read", self.ctx)
        names = {v: k[len("WEDLM_PROF_"):].lower() for k, v in C.items()
                 if k.startswith("WEDLM_PROF_") and k != "WEDLM_PROF_KINDS"}
        return {names[i]: (float(ms[i]), int(n[i])) for i in range(nk)}

    # -- test hooks ---------------------------------------------------------
    def debug_read(self, item: str, shape, dtype):
        out = np.zeros(shape, dtype)
        _check(self.lib.wedlm_debug_read(self.ctx, C["WEDLM_DBG_" + item], out.ctypes.data, out.nbytes),
               "wedlm_debug_read", self.ctx)
        return out

    def last_rows(self):
        v = self.debug_read("ROWSTRIDE", 2, np.int32)
        return int(v[0]), int(v[1])

    def debug_kv(self, slot: int, layer: int, pos0: int, n: int):
        hkv, hd = self.dims["hkv"], self.dims["hd"]
        k = np.zeros((n, hkv, hd), np.float32)
        v = np.zeros((n, hkv, hd), np.float32)
        _check(self.lib.wedlm_debug_kv(self.ctx, slot, layer, pos0, n, k.ctypes.data, v.ctypes.data),
               "wedlm_debug_kv", self.ctx)
        return k, v

    def get_window(self, slot: int):
        f = np.zeros(self.max_window, np.uint8)
        t = np.zeros(self.max_window, np.int32)
        n = ctypes.c_int32()
        _check(self.lib.wedlm_debug_get_window(self.ctx, slot, f.ctypes.data, t.ctypes.data, self.max_window,
                                               ctypes.byref(n)), "wedlm_debug_get_window", self.ctx)
        return f[:n.value].copy(), t[:n.value].copy()

    def set_window(self, slot: int, filled, tokens):
        f = np.ascontiguousarray(np.asarray(filled, np.uint8))
        t = np.ascontiguousarray(np.asarray(tokens, np.int32))
        _check(self.lib.wedlm_debug_set_window(self.ctx, slot, f.ctypes.data, t.ctypes.data, len(f)),
               "wedlm_debug_set_window", self.ctx)

    SCHEDULE_BITS = {"cta_pair": 1, "hybrid_split": 2, "cluster_split": 4, "co_resident_fixup": 8,
                     "two_weight_subtiles": 16, "bk32": 32, "fused_entropy": 64}

    def set_plan(self, kind: str, rows: int, tile_n: int, k_splits: int = 1, schedule=()):
        """Test hook: pin the GEMM launch shape of a projection kind at `rows` (see
        wedlm_debug_set_plan); `schedule` is a list of names.  Returns False if the
        shape cannot be built as asked."""
        bits = 0
        for name in schedule:
            bits |= self.SCHEDULE_BITS[name]
        st = self.lib.wedlm_debug_set_plan(self.ctx, C["WEDLM_PROF_" + kind.upper()], rows, tile_n, k_splits, bits)
        if st == C["WEDLM_ERR_INVALID_ARG"]:
            return False
        _check(st, "wedlm_debug_set_plan", self.ctx)
        return True

    def read_weight(self, kind: int, layer: int, nbytes: int) -> np.ndarray:
        """Test hook: the first `nbytes` of a weight tensor's device storage (uint8)."""
        out = np.empty(nbytes, np.uint8)
        _check(self.lib.wedlm_debug_read_weight(self.ctx, kind, layer, out.ctypes.data, nbytes),
               "wedlm_debug_read_weight", self.ctx)
        return out

    def set_page(self, slot: int, index: int, page: int) -> int:
        """Overwrite one device page-table entry, unchecked (fault-injection hook); returns the old entry."""
        old = ctypes.c_int32()
        _check(self.lib.wedlm_debug_set_page(self.ctx, slot, index, page, ctypes.byref(old)),
               "wedlm_debug_set_page", self.ctx)
        return int(old.value)


def _stream_handle(stream) -> int:
    if stream is None:
        return 0
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


# -- stand-alone stage launches (device buffers are torch CUDA tensors) -----
def reorder_window(filled, n, S, stride: int, stream=None):
    import torch
    n_seq = filled.shape[0]
    dev = filled.device
    perm = torch.empty((n_seq, stride), dtype=torch.int32, device=dev)
    pos = torch.empty_like(perm)
    k = torch.empty(n_seq, dtype=torch.int32, device=dev)
    nf = torch.empty_like(k)
    _check(_lib.load().wedlm_reorder_window(_ptr(filled), _ptr(n), _ptr(S), n_seq, stride, _ptr(perm), _ptr(pos),
                                            _ptr(k), _ptr(nf), _stream_handle(stream)), "wedlm_reorder_window")
    return perm, pos, k, nf


def entropy_select(logits, vocab: int, mask_id: int, filled, n, stride: int, params: StepParams, stream=None):
    import torch
    n_seq = filled.shape[0]
    dev = logits.device
    ht = torch.empty((n_seq, stride), dtype=torch.float32, device=dev)
    am = torch.empty((n_seq, stride), dtype=torch.int32, device=dev)
    fill = torch.empty((n_seq, stride), dtype=torch.uint8, device=dev)
    _check(_lib.load().wedlm_entropy_select(_ptr(logits), vocab, mask_id, _ptr(filled), _ptr(n), n_seq, stride,
                                            ctypes.byref(params), _ptr(ht), _ptr(am), _ptr(fill),
                                            _stream_handle(stream)), "wedlm_entropy_select")
    return ht, am, fill


def entropy_select_noalloc(logits, vocab: int, mask_id: int, filled, n, stride: int, params: StepParams,
                           stream=None):
    """entropy_select without any device allocation (scratch in a fixed library array)."""
    import torch
    n_seq = filled.shape[0]
    dev = logits.device
    ht = torch.empty((n_seq, stride), dtype=torch.float32, device=dev)
    am = torch.empty((n_seq, stride), dtype=torch.int32, device=dev)
    fill = torch.empty((n_seq, stride), dtype=torch.uint8, device=dev)
    _check(_lib.load().wedlm_entropy_select_noalloc(_ptr(logits), vocab, mask_id, _ptr(filled), _ptr(n), n_seq,
                                                    stride, ctypes.byref(params), _ptr(ht), _ptr(am), _ptr(fill),
                                                    _stream_handle(stream)), "wedlm_entropy_select_noalloc")
    return ht, am, fill


def entropy_select_async(logits, vocab: int, mask_id: int, filled, n, stride: int, params: StepParams,
                         workspace=None, out=None, stream=None):
    """Asynchronous entropy selection on caller scratch (wedlm_entropy_select_async).
    Returns (htilde, argmax, fill, workspace); the first int32 of the workspace is
    the call's device error word (read it after synchronising)."""
    import torch
    n_seq = filled.shape[0]
    dev = logits.device
    lib = _lib.load()
    if workspace is None:
        nb = ctypes.c_int64()
        _check(lib.wedlm_entropy_select_workspace_bytes(n_seq, stride, ctypes.byref(nb)),
               "wedlm_entropy_select_workspace_bytes")
        workspace = torch.zeros(int(nb.value), dtype=torch.uint8, device=dev)
    if out is None:
        out = (torch.empty((n_seq, stride), dtype=torch.float32, device=dev),
               torch.empty((n_seq, stride), dtype=torch.int32, device=dev),
               torch.empty((n_seq, stride), dtype=torch.uint8, device=dev))
    ht, am, fill = out
    _check(lib.wedlm_entropy_select_async(_ptr(logits), vocab, mask_id, _ptr(filled), _ptr(n), n_seq, stride,
                                          ctypes.byref(params), _ptr(ht), _ptr(am), _ptr(fill), _ptr(workspace),
                                          workspace.numel(), _stream_handle(stream)), "wedlm_entropy_select_async")
    return ht, am, fill, workspace


def attention_workspace(n_seq: int, stride: int, n_heads: int, n_kv_heads: int, max_ctx: int, device="cuda"):
    """A zeroed workspace for attention_bf16 (uint8 CUDA tensor)."""
    import torch
    nb = ctypes.c_int64()
    _check(_lib.load().wedlm_attention_workspace_bytes(n_seq, stride, n_heads, n_kv_heads, max_ctx, ctypes.byref(nb)),
           "wedlm_attention_workspace_bytes")
    return torch.zeros(int(nb.value), dtype=torch.uint8, device=device)


def attention_bf16(q, kv_pool, page_table, S, n, stride: int, n_heads: int, n_kv_heads: int, max_ctx: int,
                   workspace, out=None, stream=None):
    """Asynchronous reordered-causal paged attention (wedlm_attention_bf16).
    q [n_seq*stride, n_heads, 128] bf16; kv_pool [pages, 2, n_kv_heads, 16, 128]
    bf16; page_table [n_seq, pages_per_seq] int32; S, n [n_seq] int32; workspace
    from attention_workspace().  Returns `out`; read attention_error(workspace)
    after synchronising."""
    import torch
    n_seq = page_table.shape[0]
    if out is None:
        out = torch.empty_like(q)
    _check(_lib.load().wedlm_attention_bf16(_ptr(q), _ptr(kv_pool), kv_pool.shape[0], n_heads, n_kv_heads,
                                            _ptr(page_table), page_table.shape[1], _ptr(S), _ptr(n), n_seq, stride,
                                            max_ctx, _ptr(out), _ptr(workspace), workspace.numel(),
                                            _stream_handle(stream)), "wedlm_attention_bf16")
    return out


def attention_error(workspace) -> int:
    """The device error word of an attention workspace (synchronise first)."""
    return int(workspace[:4].view(dtype=__import__("torch").int32)[0].item())


# -- 4-bit KV cache and page operations --------------------------------------
# These take torch CUDA tensors of one device (which need not be the current
# one) and raise ValueError where a tensor's type, shape, device or layout is
# not the documented one.  stream: a torch.cuda.Stream or a cudaStream_t handle;
# None is torch's current stream of the tensors' device.  Results a call
# allocates belong to that stream.
# A decode step makes one such call per layer, so the checks are kept to a
# microsecond or two.
def _want(cond, what):
    if not cond:
        raise ValueError(what)


def _on(t, index, dtype, shape, name):
    """A contiguous tensor of the given dtype and shape on CUDA device `index`."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name}: wants a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")


def _index(t, name):
    """The index of a tensor's CUDA device."""
    index = t.get_device()
    _want(index >= 0, f"{name}: wants a CUDA tensor")
    return index


def _launch(name, index, stream, *args):
    """Call the library with device `index` current, the stream as last argument."""
    import torch
    fn = getattr(_lib.load(), name)
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream_handle(stream)
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            st = fn(*args, handle)
    if st != 0:
        _check(st, name)


def _empty_on(stream, index, shape, dtype):
    """A new tensor of the launch's stream (of the current one for a plain handle)."""
    import torch
    if stream is None or isinstance(stream, int):
        return torch.empty(shape, dtype=dtype, device=index)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=index)


def kv4_pool(num_pages: int, n_kv_heads: int, n_layers: int | None = None, device="cuda"):
    """A zeroed pool of 4-bit pages: uint8 [n_layers,] num_pages, n_kv_heads, 2, WEDLM_KV4_HALF_PAGE."""
    import torch
    shape = (num_pages, n_kv_heads, 2, C["WEDLM_KV4_HALF_PAGE"])
    return torch.zeros(shape if n_layers is None else (n_layers, *shape), dtype=torch.uint8, device=device)


def _kv4_args(kv4_pool, page_table, S, n, index):
    import torch
    half, int32 = C["WEDLM_KV4_HALF_PAGE"], torch.int32
    pool, table = kv4_pool.shape, page_table.shape
    if len(pool) != 4 or pool[2] != 2 or pool[3] != half:
        raise ValueError(f"kv4_pool: wants [pages, kv heads, 2, {half}]")
    if len(table) != 2:
        raise ValueError("page_table: wants [n_seq, pages_per_seq]")
    n_seq, width = table
    per_seq = (n_seq,)
    # (one test of all that `_on` tests, then the argument that fails)
    if (kv4_pool.dtype is not torch.uint8 or page_table.dtype is not int32 or S.dtype is not int32 or n.dtype is not int32
            or S.shape != per_seq or n.shape != per_seq or kv4_pool.get_device() != index
            or page_table.get_device() != index or S.get_device() != index or n.get_device() != index
            or not (kv4_pool.is_contiguous() and page_table.is_contiguous() and S.is_contiguous() and n.is_contiguous())):
        _on(kv4_pool, index, torch.uint8, pool, "kv4_pool")
        _on(page_table, index, int32, table, "page_table")
        _on(S, index, int32, per_seq, "S")
        _on(n, index, int32, per_seq, "n")
    return n_seq, width, pool[0], pool[1]


def _rows_arg(t, rows, hkv, index, dtype, name):
    """Rows [rows, hkv, 128] whose heads lie side by side; any row stride the library takes."""
    st = t.stride()
    if (t.shape != (rows, hkv, 128) or t.get_device() != index or t.dtype != dtype or st[2] != 1
            or (hkv > 1 and st[1] != 128)):
        raise ValueError(f"{name}: wants {dtype} [{rows}, {hkv}, 128] on cuda:{index} with the heads of a row side by "
                         f"side, got {t.dtype} {tuple(t.shape)} strides {st} on {t.device}")
    return st[0] if rows > 1 else hkv * 128


def _rows_dtype(dtype):
    import torch
    if dtype is torch.float32:
        return C["WEDLM_DTYPE_F32"]
    if dtype is torch.bfloat16:
        return C["WEDLM_DTYPE_BF16"]
    raise ValueError(f"rows are float32 or bfloat16, got {dtype}")


def _error_word(t, index):
    import torch
    dtype = t.dtype
    if (t.get_device() != index or not t.is_contiguous() or
            t.numel() < (1 if dtype is torch.int32 else 4 if dtype is torch.uint8 else math.inf)):
        raise ValueError("error: wants an int32 tensor or a workspace on the same device")


def kv4_append(k, v, kv4_pool, page_table, S, n, stride: int, error, k_scale: float = 1.0, v_scale: float = 1.0,
               stream=None):
    """Write K/V rows into a 4-bit cache (wedlm_kv4_append).  k, v
    [n_seq*stride, n_kv_heads, 128] float32 or bfloat16 (views with a row stride
    are taken as they are); kv4_pool from kv4_pool(); page_table [n_seq,
    pages_per_seq], S, n [n_seq] int32; error: an int32 tensor, or the workspace
    of attention_kv4, whose first word records errors (attention_error)."""
    index = _index(k, "k")
    n_seq, width, pages, hkv = _kv4_args(kv4_pool, page_table, S, n, index)
    dtype = k.dtype
    ks = _rows_arg(k, n_seq * stride, hkv, index, dtype, "k")
    vs = _rows_arg(v, n_seq * stride, hkv, index, dtype, "v")
    _error_word(error, index)
    _launch("wedlm_kv4_append", index, stream, k.data_ptr(), v.data_ptr(), _rows_dtype(dtype), ks, vs,
            kv4_pool.data_ptr(), pages, hkv, page_table.data_ptr(), width, S.data_ptr(), n.data_ptr(),
            n_seq, stride, k_scale, v_scale, error.data_ptr())


def kv4_read(kv4_pool, page_table, S, n, stride: int, error, dtype=None, k_scale: float = 1.0, v_scale: float = 1.0,
             out=None, stream=None):
    """Rows of a 4-bit cache, widened (wedlm_kv4_read): (k, v), each
    [n_seq*stride, n_kv_heads, 128] in dtype (bfloat16 unless given), or written
    into out = (k, v).  Rows r >= n[b] are left as they are."""
    index = _index(kv4_pool, "kv4_pool")
    n_seq, width, pages, hkv = _kv4_args(kv4_pool, page_table, S, n, index)
    if out is None:
        import torch
        out = tuple(_empty_on(stream, index, (n_seq * stride, hkv, 128), dtype or torch.bfloat16) for _ in range(2))
    k, v = out
    _want(dtype is None or k.dtype == dtype, "out and dtype disagree")
    dtype = k.dtype
    ks = _rows_arg(k, n_seq * stride, hkv, index, dtype, "k")
    vs = _rows_arg(v, n_seq * stride, hkv, index, dtype, "v")
    _error_word(error, index)
    _launch("wedlm_kv4_read", index, stream, kv4_pool.data_ptr(), pages, hkv, page_table.data_ptr(),
            width, S.data_ptr(), n.data_ptr(), n_seq, stride, k_scale, v_scale, k.data_ptr(),
            v.data_ptr(), _rows_dtype(dtype), ks, vs, error.data_ptr())
    return k, v


def attention_kv4_workspace(n_seq: int, stride: int, n_heads: int, n_kv_heads: int, max_ctx: int, device="cuda"):
    """A zeroed workspace for attention_kv4 (uint8 CUDA tensor)."""
    import torch
    nb = ctypes.c_int64()
    with torch.cuda.device(torch.device(device)):
        _check(_lib.load().wedlm_attention_kv4_workspace_bytes(n_seq, stride, n_heads, n_kv_heads, max_ctx,
                                                               ctypes.byref(nb)), "wedlm_attention_kv4_workspace_bytes")
        return torch.zeros(int(nb.value), dtype=torch.uint8, device=device)


def attention_kv4(q, kv4_pool, page_table, S, n, stride: int, n_heads: int, n_kv_heads: int, max_ctx: int, workspace,
                  k_scale: float = 1.0, v_scale: float = 1.0, out=None, stream=None):
    """attention_bf16 over a 4-bit cache (wedlm_attention_kv4).  q and out
    [n_seq*stride, n_heads, 128] bfloat16; the cache arguments as in kv4_append;
    workspace from attention_kv4_workspace() with these sizes or others that
    need as much.  Returns `out`; read attention_error(workspace) after
    synchronising."""
    import torch
    index = _index(q, "q")
    n_seq, width, pages, hkv = _kv4_args(kv4_pool, page_table, S, n, index)
    _want(hkv == n_kv_heads, "kv4_pool has another number of KV heads")
    shape = (n_seq * stride, n_heads, 128)
    _on(q, index, torch.bfloat16, shape, "q")
    if out is None:
        out = _empty_on(stream, index, shape, torch.bfloat16)
    else:
        _on(out, index, torch.bfloat16, shape, "out")
    _on(workspace, index, torch.uint8, workspace.shape, "workspace")
    _launch("wedlm_attention_kv4", index, stream, q.data_ptr(), kv4_pool.data_ptr(), pages, n_heads, hkv,
            page_table.data_ptr(), width, S.data_ptr(), n.data_ptr(), n_seq, stride, max_ctx, k_scale,
            v_scale, out.data_ptr(), workspace.data_ptr(), workspace.numel())
    return out


class KVPages:
    """Pages of a cache kept on the device, and the operations on them
    (wedlm_kv_pages_*): all asynchronous, without a host round trip.

    pool [n_layers, num_pages, ...] of any type, each page contiguous and pages
    side by side (layers may lie further apart); page_table [n_seq,
    pages_per_seq] (-1 behind a sequence's pages), S [n_seq] (committed tokens)
    and refs [num_pages] (sequences holding a page; 0 = free), int32.  The
    tensors are used in place and stay the caller's.  Lists are int32 tensors."""

    def __init__(self, pool, page_table, S, refs, workspace=None):
        import torch
        self.index = index = _index(pool, "pool")
        _want(pool.dim() >= 3 and pool.numel() > 0 and pool[0].is_contiguous(),
              "pool: wants [n_layers, num_pages, ...] with contiguous layers")
        layers, pages = pool.shape[:2]
        _want(page_table.dim() == 2, "page_table: wants [n_seq, pages_per_seq]")
        n_seq = page_table.shape[0]
        _on(page_table, index, torch.int32, page_table.shape, "page_table")
        _on(S, index, torch.int32, (n_seq,), "S")
        _on(refs, index, torch.int32, (pages,), "refs")
        nb = ctypes.c_int64()
        _check(_lib.load().wedlm_kv_pages_workspace_bytes(pages, n_seq, ctypes.byref(nb)),
               "wedlm_kv_pages_workspace_bytes")
        if workspace is None:
            workspace = torch.zeros(int(nb.value), dtype=torch.uint8, device=index)
            # (operations may come on any stream, and a caller does not see this memory: it is zero from here on)
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream(index).synchronize()
        _on(workspace, index, torch.uint8, workspace.shape, "workspace")
        self.pool, self.page_table, self.S, self.refs, self.workspace = pool, page_table, S, refs, workspace
        size = pool.element_size()
        stride = pool.stride(0) if layers > 1 else pool[0].numel()
        self._desc = _lib.KVPagesDesc(_ptr(pool), stride * size, pool[0, 0].numel() * size, _ptr(page_table), _ptr(S),
                                      _ptr(refs), layers, pages, n_seq, page_table.shape[1])
        self._by = ctypes.byref(self._desc)
        self._ws = (workspace.data_ptr(), workspace.numel())

    def _list(self, t, name, n=None):
        import torch
        _on(t, self.index, torch.int32, (t.numel() if n is None else n,), name)
        return t.numel()

    def _call(self, name, stream, *args):
        _launch(name, self.index, stream, self._by, *args, *self._ws)

    def copy(self, src, dst, stream=None):
        """Page dst[i] := page src[i] in every layer."""
        n = self._list(src, "src")
        self._list(dst, "dst", n)
        self._call("wedlm_kv_pages_copy", stream, src.data_ptr(), dst.data_ptr(), n)

    def reserve(self, seqs, tokens, stream=None):
        """Free pages for seqs[i] until it has room for tokens[i] tokens."""
        n = self._list(seqs, "seqs")
        self._list(tokens, "tokens", n)
        self._call("wedlm_kv_pages_reserve", stream, seqs.data_ptr(), tokens.data_ptr(), n)

    def fork(self, parents, children, stream=None):
        """children[i], a sequence without pages, becomes a copy of parents[i] that shares its full pages."""
        n = self._list(parents, "parents")
        self._list(children, "children", n)
        self._call("wedlm_kv_pages_fork", stream, parents.data_ptr(), children.data_ptr(), n)

    def free(self, seqs, stream=None):
        """Drop the sequences: their pages lose a reference, rows become -1 and S 0."""
        n = self._list(seqs, "seqs")
        self._call("wedlm_kv_pages_free", stream, seqs.data_ptr(), n)

    def compact(self, map=None, stream=None):
        """Move the u pages in use to ids 0 .. u - 1; map [num_pages] int32 receives the new ids."""
        if map is not None:
            self._list(map, "map", self.refs.numel())
        self._call("wedlm_kv_pages_compact", stream, _ptr(map))

    def error(self) -> int:
        """The device error word (synchronise first)."""
        return attention_error(self.workspace)


def linear_bf16(X, W, stream=None, tile_n: int = 0, k_splits: int = 0, cta_pair: bool = False,
                hybrid: bool = False, cluster_k: bool = False):
    """Y = X W^T (fp32) on the tcgen05 GEMM; X [M][K], W [N][K] torch.bfloat16 CUDA tensors.
    tile_n / k_splits pin the launch shape (0 = automatic); cta_pair runs CTA-pair
    tiles of 256 weight rows (tile_n 128 or 256); hybrid splits K only for the
    tiles of the last partial round of the persistent grid; cluster_k makes the
    k_splits (2..4) slices of a tile one thread-block cluster reduced through
    distributed shared memory."""
    import torch
    M, K = X.shape
    N = W.shape[0]
    Y = torch.empty((M, N), dtype=torch.float32, device=X.device)
    X, W = X.contiguous(), W.contiguous()
    lib = _lib.load()
    if cta_pair or hybrid or cluster_k:
        sched = (1 if cta_pair else 0) | (2 if hybrid else 0) | (4 if cluster_k else 0)
        _check(lib.wedlm_linear_bf16_sched(_ptr(X), _ptr(W), _ptr(Y), M, N, K, tile_n, k_splits, sched,
                                           _stream_handle(stream)), "wedlm_linear_bf16_sched")
    else:
        _check(lib.wedlm_linear_bf16_plan(_ptr(X), _ptr(W), _ptr(Y), M, N, K, tile_n, k_splits,
                                          _stream_handle(stream)), "wedlm_linear_bf16_plan")
    return Y
