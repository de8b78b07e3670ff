"""Thin ctypes binding of libdinfer.so (include/dinfer.h, include/dinfer_ops.h).

Argument marshalling only: every step of the decoder runs in the CUDA
library.  torch tensors provide device memory and streams.  Loading fails
loudly when the library is missing or no GPU is visible -- there is no CPU
path.
"""
from __future__ import annotations

import ctypes
import os
from typing import List, Optional, Sequence

import torch

from . import inputs as _inputs

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdinfer.so")

OK, EINVAL, ENOMEM, ECUDA, EDEVICE, ESTATE = 0, -1, -2, -3, -4, -5
FP32, BF16 = 0, 1


class ModelDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_layers", "d_model", "n_heads", "head_dim", "ffn", "vocab",
                                              "mask_id", "n_experts", "top_k", "expert_ffn")] + \
               [("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_float), ("logit_scale", ctypes.c_float),
                ("dtype", ctypes.c_int32), ("max_batch", ctypes.c_int32), ("max_seq", ctypes.c_int32)]


class Stats(ctypes.Structure):
    _fields_ = [("n_blocks", ctypes.c_int32), ("iterations", ctypes.c_int32), ("refreshes", ctypes.c_int32),
                ("ms_device", ctypes.c_float), ("iters_per_block", ctypes.POINTER(ctypes.c_int32))]


class DinferError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"dinfer status {status}: {msg}")
        self.status = status


class KvCache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v")] + \
               [(n, ctypes.c_int64) for n in ("layer_stride", "page_stride", "token_stride", "head_stride")] + \
               [(n, ctypes.c_void_p) for n in ("table", "lens", "refs", "state")] + \
               [(n, ctypes.c_int32) for n in ("n_layers", "num_pages", "page_size", "kv_heads", "head_dim", "dtype",
                                              "max_seqs", "max_pages")]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libdinfer.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m block_denoising_gb300.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    L.dinfer_num_weights.argtypes = [ctypes.POINTER(ModelDesc)]
    L.dinfer_num_weights.restype = i32
    L.dinfer_create.argtypes = [ctypes.POINTER(ModelDesc), ctypes.POINTER(vp), vp, ctypes.POINTER(vp)]
    L.dinfer_create.restype = i32
    L.dinfer_destroy.argtypes = [vp]
    L.dinfer_destroy.restype = None
    L.dinfer_last_error.argtypes = [vp]
    L.dinfer_last_error.restype = ctypes.c_char_p
    L.dinfer_prefill_cache.argtypes = [vp, vp, vp, i32, i32, i32, i32, f32, i32, vp]
    L.dinfer_prefill_cache.restype = i32
    L.dinfer_block_step.argtypes = [vp, vp, vp, f32, vp]
    L.dinfer_block_step.restype = i32
    L.dinfer_generate.argtypes = [vp, vp, i32, i32, i32, i32, f32, vp, ctypes.POINTER(Stats)]
    L.dinfer_generate.restype = i32
    L.dinfer_set_debug_outputs.argtypes = [vp, vp, vp, vp]
    L.dinfer_set_debug_outputs.restype = i32
    L.dinfer_set_eos.argtypes = [vp, i32]
    L.dinfer_set_eos.restype = i32
    L.dinfer_set_cache_mode.argtypes = [vp, i32, i32]
    L.dinfer_set_cache_mode.restype = i32
    L.dinfer_set_debug_hidden.argtypes = [vp, vp, vp]
    L.dinfer_set_debug_hidden.restype = i32
    L.dinfer_sync.argtypes = [vp]
    L.dinfer_sync.restype = i32
    L.dinfer_moe_experts_touched.argtypes = [vp, ctypes.POINTER(ctypes.c_int64)]
    L.dinfer_moe_experts_touched.restype = i32
    L.dinfer_op_workspace_bytes.argtypes = []
    L.dinfer_op_workspace_bytes.restype = sz
    L.dinfer_op_gemm_bf16.argtypes = [vp, vp, vp, i32, i32, i32, vp, sz, vp]
    L.dinfer_op_gemm_bf16.restype = i32
    L.dinfer_op_lmhead_bf16.argtypes = [vp, vp, i32, i32, i32, i32, f32, vp, vp, vp, vp, sz, vp]
    L.dinfer_op_lmhead_bf16.restype = i32
    L.dinfer_op_attention_bf16.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp, sz, vp]
    L.dinfer_op_attention_bf16.restype = i32
    L.dinfer_op_moe_ffn_bf16.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp]
    L.dinfer_op_moe_ffn_bf16.restype = i32
    i64 = ctypes.c_int64
    L.dinfer_kv_state_ints.argtypes = [i32, i32]
    L.dinfer_kv_state_ints.restype = sz
    L.dinfer_kv_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), vp]
    L.dinfer_kv_status.restype = i32
    L.dinfer_kv_set.argtypes = [vp, vp, vp, vp, vp]
    L.dinfer_kv_set.restype = i32
    L.dinfer_kv_extend.argtypes = [vp, vp, vp, i32, vp]
    L.dinfer_kv_extend.restype = i32
    L.dinfer_kv_append.argtypes = [vp, i32, vp, vp, i32, vp, vp, i64, i64, i32, vp]
    L.dinfer_kv_append.restype = i32
    L.dinfer_kv_fork.argtypes = [vp, vp, vp, i32, i32, vp]
    L.dinfer_kv_fork.restype = i32
    L.dinfer_kv_free.argtypes = [vp, vp, i32, vp]
    L.dinfer_kv_free.restype = i32
    L.dinfer_kv_compact.argtypes = [vp, vp, vp]
    L.dinfer_kv_compact.restype = i32
    L.dinfer_kv_attention.argtypes = [vp, i32, vp, i32, vp, vp, i64, i64, i32, i32, i32, f32, vp, sz, vp]
    L.dinfer_kv_attention.restype = i32
    L.dinfer_op_window_attention.argtypes = [vp, vp, vp, vp, i32, i32, vp, vp, i32, i32, i32, i32, i32, i64, i64, i64,
                                             i64, i32, i32, i32, f32, vp, sz, vp]
    L.dinfer_op_window_attention.restype = i32
    _lib = L
    return L


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(st: int, ctx=None):
    if st != OK:
        msg = lib().dinfer_last_error(ctx).decode(errors="replace")
        raise DinferError(st, msg)


def desc_from_config(cfg: _inputs.ModelConfig, max_batch: int, max_seq: int) -> ModelDesc:
    return ModelDesc(cfg.n_layers, cfg.d_model, cfg.n_heads, cfg.head_dim, cfg.ffn, cfg.vocab, cfg.mask_id,
                     cfg.n_experts, cfg.top_k, cfg.expert_ffn, cfg.rms_eps, cfg.rope_theta, cfg.logit_scale,
                     FP32 if cfg.dtype == "fp32" else BF16, max_batch, max_seq)


class Decoder:
    """A dinfer context over caller-owned device weights (kept alive here)."""

    def __init__(self, cfg: _inputs.ModelConfig, weights: Sequence[torch.Tensor], max_batch: int, max_seq: int,
                 stream: Optional[torch.cuda.Stream] = None):
        L = lib()
        self.cfg = cfg
        self.desc = desc_from_config(cfg, max_batch, max_seq)
        n = L.dinfer_num_weights(ctypes.byref(self.desc))
        if n != len(weights):
            raise ValueError(f"model takes {n} weights, got {len(weights)}")
        self.weights: List[torch.Tensor] = [w.contiguous() for w in weights]
        arr = (ctypes.c_void_p * n)(*[w.data_ptr() for w in self.weights])
        # calls are ordered on this stream (default: torch's current stream)
        self.stream = stream if stream is not None else torch.cuda.current_stream()
        h = ctypes.c_void_p()
        st = L.dinfer_create(ctypes.byref(self.desc), arr, ctypes.c_void_p(self.stream.cuda_stream), ctypes.byref(h))
        _check(st, None)
        self.h = h

    def close(self):
        if getattr(self, "h", None):
            lib().dinfer_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def prefill_cache(self, ids: torch.Tensor, mask: torch.Tensor, block_start: int, block_len: int,
                      threshold: float, commit: bool = True, committed: Optional[torch.Tensor] = None):
        b, L = ids.shape
        _check(lib().dinfer_prefill_cache(self.h, _ptr(ids), _ptr(mask), b, L, block_start, block_len,
                                          float(threshold), int(commit), _ptr(committed)), self.h)

    def block_step(self, ids: torch.Tensor, mask: torch.Tensor, threshold: float,
                   committed: Optional[torch.Tensor] = None):
        _check(lib().dinfer_block_step(self.h, _ptr(ids), _ptr(mask), float(threshold), _ptr(committed)), self.h)

    def generate(self, prompt: torch.Tensor, gen_length: int, block_length: int, threshold: float,
                 out: Optional[torch.Tensor] = None):
        """prompt [b, P] int32 (host or device) -> (out [b, P+G] int32, stats dict)."""
        b, P = prompt.shape
        if out is None:
            out = torch.empty((b, P + gen_length), dtype=torch.int32, device=prompt.device)
        nblk = gen_length // block_length if block_length > 0 else 0
        ipb = (ctypes.c_int32 * max(1, nblk))()
        stats = Stats(0, 0, 0, 0.0, ctypes.cast(ipb, ctypes.POINTER(ctypes.c_int32)))
        _check(lib().dinfer_generate(self.h, _ptr(prompt), b, P, gen_length, block_length, float(threshold),
                                     _ptr(out), ctypes.byref(stats)), self.h)
        return out, {"n_blocks": stats.n_blocks, "iterations": stats.iterations, "refreshes": stats.refreshes,
                     "ms_device": stats.ms_device, "iters_per_block": list(ipb)[:nblk]}

    def set_debug_outputs(self, logits=None, tok=None, conf=None):
        _check(lib().dinfer_set_debug_outputs(self.h, _ptr(logits), _ptr(tok), _ptr(conf)), self.h)

    def set_eos(self, eos_id: int = -1):
        """End-of-sequence id of generate (-1: none)."""
        _check(lib().dinfer_set_eos(self.h, int(eos_id)), self.h)

    CACHE_MODES = {"dual": 0, "none": 1, "prefix": 2, "vicinity": 3}

    def set_cache_mode(self, mode: str, window: int = 0):
        """KV-cache policy of the cached iterations: "dual", "none", "prefix" or "vicinity" (window w)."""
        _check(lib().dinfer_set_cache_mode(self.h, self.CACHE_MODES[mode], int(window)), self.h)

    def set_debug_hidden(self, hidden=None, final_in=None):
        """Per-layer residual stream [n_layers, rows, d] fp32 and LM-head input [rows, d] of the block rows."""
        _check(lib().dinfer_set_debug_hidden(self.h, _ptr(hidden), _ptr(final_in)), self.h)

    def sync(self):
        _check(lib().dinfer_sync(self.h), self.h)

    def moe_experts_touched(self):
        """(MoE layer forward, expert) pairs that received rows since the
        previous call (the count restarts); 0 for dense models."""
        n = ctypes.c_int64(0)
        _check(lib().dinfer_moe_experts_touched(self.h, ctypes.byref(n)), self.h)
        return int(n.value)


# ---------------------------------------------------------------------------
# kernel-level entry points
# ---------------------------------------------------------------------------
class OpWorkspace:
    def __init__(self, device="cuda"):
        n = lib().dinfer_op_workspace_bytes()
        self.buf = torch.zeros(n, dtype=torch.uint8, device=device)
        self.nbytes = n

    def check(self):
        """Raise if a kernel run on this workspace reported a device-side error
        (the status word of the device state at the head of the workspace)."""
        st = int(self.buf[:32].view(torch.int32)[6].item())
        if st:
            raise DinferError(EDEVICE, f"device status 0x{st:x}")


def _stream_ptr():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def op_gemm_bf16(X: torch.Tensor, W: torch.Tensor, ws: OpWorkspace, Y: Optional[torch.Tensor] = None):
    M, K = X.shape
    N = W.shape[0]
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=X.device)
    _check(lib().dinfer_op_gemm_bf16(_ptr(X), _ptr(W), _ptr(Y), M, N, K, _ptr(ws.buf), ws.nbytes, _stream_ptr()))
    return Y


def op_lmhead_bf16(X: torch.Tensor, W: torch.Tensor, mask_id: int, scale: float, ws: OpWorkspace,
                   want_logits: bool = False):
    M, K = X.shape
    V = W.shape[0]
    tok = torch.empty(M, dtype=torch.int32, device=X.device)
    conf = torch.empty(M, dtype=torch.float32, device=X.device)
    logits = torch.empty((M, V), dtype=torch.float32, device=X.device) if want_logits else None
    _check(lib().dinfer_op_lmhead_bf16(_ptr(X), _ptr(W), M, V, K, mask_id, float(scale), _ptr(tok), _ptr(conf),
                                       _ptr(logits), _ptr(ws.buf), ws.nbytes, _stream_ptr()))
    return tok, conf, logits


def op_attention_bf16(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, rows_per_seq: int, ws: OpWorkspace,
                      out: Optional[torch.Tensor] = None):
    b, L, d = k.shape
    heads = d // 128
    if out is None:
        out = torch.empty_like(q)
    _check(lib().dinfer_op_attention_bf16(_ptr(q), _ptr(k), _ptr(v), _ptr(out), b, rows_per_seq, L, heads,
                                          _ptr(ws.buf), ws.nbytes, _stream_ptr()))
    return out


def op_moe_ffn_bf16(X: torch.Tensor, router: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor, top_k: int,
                    ws: OpWorkspace):
    """Routed expert FFN output [M, d] fp32 and the routing (ids [M, k], weights [M, k])."""
    M, d = X.shape
    E, two_fe, _ = w13.shape
    out = torch.empty((M, d), dtype=torch.float32, device=X.device)
    ids = torch.empty((M, top_k), dtype=torch.int32, device=X.device)
    w = torch.empty((M, top_k), dtype=torch.float32, device=X.device)
    _check(lib().dinfer_op_moe_ffn_bf16(_ptr(X), _ptr(router), _ptr(w13), _ptr(w2), M, d, E, top_k, two_fe // 2,
                                        _ptr(out), _ptr(ids), _ptr(w), _ptr(ws.buf), ws.nbytes, _stream_ptr()))
    return out, ids, w


# ---------------------------------------------------------------------------
# paged KV cache and windowed prompt attention (include/dinfer_kv.h)
# ---------------------------------------------------------------------------
_DTYPES = {torch.float32: FP32, torch.bfloat16: BF16}
KV_BAD_SEQ, KV_NO_PAGES, KV_BAD_PAGE, KV_SHARED, KV_FULL = 1, 2, 4, 8, 16


def _require(ok, what: str):
    if not ok:
        raise ValueError(what)


def _rows_of(t: torch.Tensor, name: str, heads: Optional[int], head_dim: int, dtype, gpu: int):
    """Checks [rows, heads, head_dim] with packed head rows; returns rows, heads and the row stride."""
    shape, s = t.shape, t.stride()
    if (len(shape) == 3 and shape[2] == head_dim and (heads is None or shape[1] == heads) and t.dtype is dtype
            and t.get_device() == gpu and s[2] == 1 and (s[1] == head_dim or shape[1] == 1)):
        return shape[0], shape[1], s[0]
    raise ValueError(f"{name}: [rows, {'heads' if heads is None else heads}, {head_dim}] {dtype} on cuda:{gpu} with "
                     f"the heads of a row packed expected, got {list(shape)} {t.dtype} on {t.device} with strides {s}")


def _ints(t: Optional[torch.Tensor], name: str, gpu: int, n: Optional[int] = None):
    """Address of a contiguous int32 vector on the GPU (None: NULL)."""
    if t is None:
        return None
    shape = t.shape
    if (t.dtype is torch.int32 and len(shape) == 1 and t.get_device() == gpu and t.is_contiguous()
            and (n is None or shape[0] == n)):
        return t.data_ptr()
    raise ValueError(f"{name}: a contiguous int32 vector {'' if n is None else f'of {n} '}on cuda:{gpu} expected, got "
                     f"{list(t.shape)} {t.dtype} on {t.device}")


def _i32(x: int) -> int:
    """x, or int32's end next to it: ctypes would take the lower 32 bits of a larger one (a window of 2^32 as 0)."""
    return x if -0x80000000 <= x <= 0x7fffffff else 0x7fffffff if x > 0 else -0x80000000


def _run_on(gpu: int, fn, *args):
    """One library call on torch's current stream of the operands' GPU, which becomes the current one for it."""
    if gpu == torch._C._cuda_getDevice():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(gpu))
    else:
        with torch.cuda.device(gpu):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(gpu))
    if st != OK:
        _check(st)


class PagedKV:
    """A paged KV cache over caller-owned tensors (dinfer_kv.h): k, v viewed as
    [layers, pages, page_size, kv_heads, head_dim] in any non-overlapping order
    with packed head rows; table [max_seqs, max_pages], lens [max_seqs] and refs
    [pages] int32.  All calls run on torch's current stream of the tensors'
    device."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor):
        _require(k.dim() == 5 and k.shape == v.shape and k.stride() == v.stride() and k.dtype == v.dtype
                 and k.device == v.device, "k, v: two [layers, pages, page_size, kv_heads, head_dim] views alike expected")
        _require(k.dtype in _DTYPES and k.is_cuda, "k, v: float32 or bfloat16 on a GPU expected")
        _require(k.stride(4) == 1, "k, v: the elements of a head must be packed")
        dev = k.device
        _require(table.dim() == 2 and table.dtype == torch.int32 and table.device == dev and table.is_contiguous(),
                 f"table: contiguous int32 [max_seqs, max_pages] on {dev} expected")
        self.max_seqs, self.max_pages = table.shape
        layers, pages, page, heads, hd = k.shape
        gpu = k.get_device()
        lens_p, refs_p = _ints(lens, "lens", gpu, self.max_seqs), _ints(refs, "refs", gpu, pages)
        L = lib()
        self.k, self.v, self.table, self.lens, self.refs = k, v, table, lens, refs
        self.device, self.gpu, self.dtype, self.kv_heads, self.head_dim = dev, gpu, k.dtype, heads, hd
        self.state = torch.zeros(L.dinfer_kv_state_ints(pages, self.max_seqs), dtype=torch.int32, device=dev)
        st = k.stride()
        self.desc = KvCache(k.data_ptr(), v.data_ptr(), st[0], st[1], st[2], st[3], table.data_ptr(), lens_p, refs_p,
                            self.state.data_ptr(), layers, pages, page, heads, hd, _DTYPES[k.dtype], self.max_seqs,
                            self.max_pages)
        self._desc = ctypes.addressof(self.desc)

    @classmethod
    def empty(cls, layers: int, pages: int, page_size: int, kv_heads: int, head_dim: int, max_seqs: int,
              max_pages: int, dtype=torch.bfloat16, device="cuda"):
        """A new cache without sequences."""
        k, v = (torch.empty((layers, pages, page_size, kv_heads, head_dim), dtype=dtype, device=device) for _ in range(2))
        return cls(k, v, torch.full((max_seqs, max_pages), -1, dtype=torch.int32, device=device),
                   torch.zeros(max_seqs, dtype=torch.int32, device=device),
                   torch.zeros(pages, dtype=torch.int32, device=device))

    def set_tables(self, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor):
        """Takes over another set of tables of the same sizes (a snapshot, a scheduler's own plan)."""
        _require(table.shape == self.table.shape and lens.shape == self.lens.shape and refs.shape == self.refs.shape,
                 "table, lens, refs: the cache's sizes expected")
        at = [t if t.dtype is torch.int32 and t.get_device() == self.gpu and t.is_contiguous()
              else t.to(self.device, torch.int32).contiguous() for t in (table, lens, refs)]
        _run_on(self.gpu, lib().dinfer_kv_set, self._desc, at[0].data_ptr(), at[1].data_ptr(), at[2].data_ptr())

    def extend(self, add: Optional[torch.Tensor] = None, seqs: Optional[torch.Tensor] = None):
        """Sequences seqs (default: the first ones, one per entry of add; all) grow by add tokens (default: one each)."""
        n = seqs.shape[0] if seqs is not None else add.shape[0] if add is not None else self.max_seqs
        _require(seqs is not None or n <= self.max_seqs, "add: more entries than sequences")
        gpu = self.gpu
        _run_on(gpu, lib().dinfer_kv_extend, self._desc, _ints(seqs, "seqs", gpu), _ints(add, "add", gpu, n), n)

    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor, rows: Optional[torch.Tensor] = None,
               seqs: Optional[torch.Tensor] = None):
        """Stores the last rows of each sequence: k, v [rows, kv_heads, head_dim]; rows [n + 1] the entries'
        first rows (default: one row per sequence)."""
        gpu = self.gpu
        total, _, ks = _rows_of(k, "k", self.kv_heads, self.head_dim, self.dtype, gpu)
        also, _, vs = _rows_of(v, "v", self.kv_heads, self.head_dim, self.dtype, gpu)
        _require(total == also, "k, v: as many rows expected")
        n = rows.shape[0] - 1 if rows is not None else total
        _require(seqs is not None or n <= self.max_seqs, "more entries than sequences")
        _run_on(gpu, lib().dinfer_kv_append, self._desc, _i32(layer), _ints(seqs, "seqs", gpu, n), _ints(rows, "rows", gpu), n,
                k.data_ptr(), v.data_ptr(), ks, vs, total)

    def fork(self, src: torch.Tensor, dst: torch.Tensor, share: bool = True):
        """Sequences dst (not in use) become copies of src, sharing the full pages or copying all of them."""
        n = src.shape[0]
        gpu = self.gpu
        _run_on(gpu, lib().dinfer_kv_fork, self._desc, _ints(src, "src", gpu), _ints(dst, "dst", gpu, n), n, int(share))

    def free(self, seqs: torch.Tensor):
        _run_on(self.gpu, lib().dinfer_kv_free, self._desc, _ints(seqs, "seqs", self.gpu), seqs.shape[0])

    def compact(self, live: Optional[torch.Tensor] = None):
        """Packs the pages in use to the front; live (optional, int32 [1]) receives how many there are."""
        _run_on(self.gpu, lib().dinfer_kv_compact, self._desc, _ints(live, "live", self.gpu, 1))

    def attention(self, layer: int, q: torch.Tensor, ws: OpWorkspace, window: int = -1, sinks: int = 0,
                  scale: Optional[float] = None, seqs: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
        """Attention of each sequence's last token: q [n, heads, head_dim] -> [n, heads, head_dim] (out may be q)."""
        hd, dtype, gpu = self.head_dim, self.dtype, self.gpu
        n, heads, qs = _rows_of(q, "q", None, hd, dtype, gpu)
        _require(seqs is not None or n <= self.max_seqs, "q: more rows than sequences")
        _require(ws.buf.get_device() == gpu, "ws: a workspace on the cache's device expected")
        if out is None:
            out, os_ = torch.empty_like(q, memory_format=torch.contiguous_format), heads * hd
        else:
            also, _, os_ = _rows_of(out, "out", heads, hd, dtype, gpu)
            _require(also == n, "out: as many rows as q expected")
        _run_on(gpu, lib().dinfer_kv_attention, self._desc, _i32(layer), _ints(seqs, "seqs", gpu, n), n, q.data_ptr(),
                out.data_ptr(), qs, os_, heads, _i32(window), _i32(sinks), hd ** -0.5 if scale is None else scale,
                ws.buf.data_ptr(), ws.nbytes)
        return out

    def check(self):
        """Raise if an entry of an earlier call was skipped (DinferError names why); clears the status."""
        _run_on(self.gpu, lib().dinfer_kv_status, self._desc, None)


def op_window_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, ws: OpWorkspace,
                        cu_q: Optional[torch.Tensor] = None, cu_k: Optional[torch.Tensor] = None, left: int = -1,
                        right: int = -1, sinks: int = 0, scale: Optional[float] = None,
                        out: Optional[torch.Tensor] = None):
    """Attention with a sliding window and sinks: q [rows, heads, head_dim], k, v [keys, kv_heads, head_dim];
    cu_q, cu_k [batch + 1] the sequences' first rows and keys (default: one sequence of all); out must not overlap
    q, k or v."""
    dtype, gpu = q.dtype, q.get_device()
    _require(dtype in _DTYPES and q.is_cuda and q.dim() == 3, "q: float32 or bfloat16 [rows, heads, head_dim] on a GPU expected")
    hd = q.shape[2]
    rows, heads, qs = _rows_of(q, "q", None, hd, dtype, gpu)
    keys, kv_heads, ks = _rows_of(k, "k", None, hd, dtype, gpu)
    also, _, vs = _rows_of(v, "v", kv_heads, hd, dtype, gpu)
    _require(keys == also, "k, v: as many keys expected")
    batch = 1 if cu_q is None else cu_q.shape[0] - 1
    cq, ck = _ints(cu_q, "cu_q", gpu), _ints(cu_k, "cu_k", gpu, None if cu_q is None else batch + 1)
    _require(ws.buf.get_device() == gpu, "ws: a workspace on the operands' device expected")
    if out is None:
        out, os_ = torch.empty_like(q, memory_format=torch.contiguous_format), heads * hd
    else:
        also, _, os_ = _rows_of(out, "out", heads, hd, dtype, gpu)
        _require(also == rows, "out: as many rows as q expected")
    _run_on(gpu, lib().dinfer_op_window_attention, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), _DTYPES[dtype],
            batch, cq, ck, rows, keys, heads, kv_heads, hd, qs, ks, vs, os_, _i32(left), _i32(right), _i32(sinks),
            hd ** -0.5 if scale is None else scale, ws.buf.data_ptr(), ws.nbytes)
    return out
