"""Thin Python binding of libdspark (include/dspark.h) over ctypes.

Argument marshalling only: every step of the draft-and-verify path runs in the
library's CUDA kernels. torch provides device memory and the stream. There is
no fallback: if the library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes as C
import os
from typing import Dict, Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libdspark.so")

MAX_LAYERS = 16
GREEDY, PROBABILISTIC, BLOCK = 0, 1, 2
FMT_BF16, FMT_FP8, FMT_NVFP4, FMT_MXFP4 = 0, 1, 2, 3

STATUS = {0: "OK", 1: "ERR_NULL", 2: "ERR_ALIGN", 3: "ERR_SHAPE", 4: "ERR_UNSUPPORTED", 5: "ERR_CUDA",
          6: "ERR_WORKSPACE", 16: "ERR_TIMEOUT", 17: "ERR_BAD_INPUT", 18: "ERR_OOB"}
EXPORTS = ("dspark_create", "dspark_destroy", "dspark_workspace_bytes", "dspark_fuse_ctx", "dspark_draft_block",
           "dspark_markov_rollout", "dspark_confidence", "dspark_verify", "dspark_check", "dspark_status_str",
           "dspark_fuse_ctx_noalloc", "dspark_kv_append", "dspark_qcache_plan", "dspark_qcache_append",
           "dspark_qcache_attend", "dspark_qcache_workspace_bytes", "dspark_qcache_check")


class Geom(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("hidden", "n_aux", "n_layers", "n_heads", "q_lora", "kv_lora", "d_nope",
                                       "d_rope", "d_v", "inter", "vocab", "rank", "block")] + [
        ("rope_theta", C.c_float), ("eps", C.c_float), ("yarn_factor", C.c_float), ("yarn_orig_ctx", C.c_int),
        ("yarn_alpha", C.c_float), ("yarn_beta", C.c_float), ("page_size", C.c_int), ("weight_format", C.c_int)]


class Mat(C.Structure):
    _fields_ = [("data", C.c_void_p), ("scale", C.c_void_p), ("global_scale", C.c_float)]


class LayerWeights(C.Structure):
    _fields_ = [("attn_norm", C.c_void_p), ("w_qkv_a", C.c_void_p), ("q_a_norm", C.c_void_p),
                ("kv_a_norm", C.c_void_p), ("w_q_b", Mat), ("w_kv_b", C.c_void_p), ("w_o", Mat),
                ("mlp_norm", C.c_void_p), ("w_gate", Mat), ("w_up", Mat), ("w_down", Mat)]


class Weights(C.Structure):
    _fields_ = [("w_fc", Mat), ("layers", LayerWeights * MAX_LAYERS), ("final_norm", C.c_void_p),
                ("w_lm", C.c_void_p), ("markov_w1", C.c_void_p), ("markov_w2", C.c_void_p),
                ("w_conf", C.c_void_p), ("b_conf", C.c_float)]


class KV(C.Structure):
    _fields_ = [("pools", C.c_void_p * MAX_LAYERS), ("n_pages", C.c_int), ("page_table", C.c_void_p),
                ("max_pages", C.c_int), ("ctx_len", C.c_void_p), ("max_ctx", C.c_int)]


class Sample(C.Structure):
    _fields_ = [("draft_mode", C.c_int), ("verify_mode", C.c_int), ("temperature", C.c_float),
                ("top_p", C.c_float), ("seed", C.c_uint64), ("step", C.c_uint32)]


class QCacheStruct(C.Structure):
    _fields_ = [("kv_lora", C.c_int), ("d_rope", C.c_int), ("page_size", C.c_int), ("n_layers", C.c_int),
                ("codes", C.c_void_p * MAX_LAYERS), ("scales", C.c_void_p * MAX_LAYERS), ("n_pages", C.c_int),
                ("page_table", C.c_void_p), ("max_pages", C.c_int)]


class QPlanArgs(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("length", "want", "ring", "ring_state", "length_out", "ring_state_out",
                                          "cu_new", "slots", "positions", "seg_row")]


class QAttnArgs(C.Structure):
    _fields_ = [("q", C.c_void_p), ("q_stride", C.c_int64), ("cu_q", C.c_void_p), ("length", C.c_void_p),
                ("n_heads", C.c_int), ("total_q", C.c_int), ("causal", C.c_int), ("scale", C.c_float),
                ("o", C.c_void_p), ("o_stride", C.c_int64), ("lse", C.c_void_p)]


class DSparkError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {STATUS.get(status, status)} ({status})")
        self.status = status


_lib = None


def lib():
    """Load libdspark.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libdspark.so is not built ({LIB_PATH}); run __graft_entry__.build()")
        L = C.CDLL(LIB_PATH)
        vp, i, sz = C.c_void_p, C.c_int, C.c_size_t
        L.dspark_create.argtypes = [C.POINTER(Geom), C.POINTER(Weights), C.POINTER(vp)]
        L.dspark_destroy.argtypes = [vp]
        L.dspark_destroy.restype = None
        L.dspark_workspace_bytes.argtypes = [vp, i, i]
        L.dspark_workspace_bytes.restype = sz
        L.dspark_fuse_ctx.argtypes = [vp, vp, vp, i, vp, sz, vp]
        L.dspark_draft_block.argtypes = [vp, vp, C.POINTER(KV), vp, vp, i, vp, sz, vp]
        L.dspark_markov_rollout.argtypes = [vp, vp, vp, C.POINTER(Sample), vp, vp, i, vp, sz, vp]
        L.dspark_confidence.argtypes = [vp, vp, vp, i, vp]
        L.dspark_verify.argtypes = [vp, vp, vp, vp, C.POINTER(Sample), vp, vp, i, vp, sz, vp]
        L.dspark_check.argtypes = [vp, vp, vp]
        L.dspark_fuse_ctx_noalloc.argtypes = [vp, vp, vp, i, vp]
        L.dspark_kv_append.argtypes = [vp, vp, i, vp, C.POINTER(KV), i, vp, sz, vp]
        L.dspark_qcache_plan.argtypes = [C.POINTER(QCacheStruct), C.POINTER(QPlanArgs), i, i, i, vp, sz, vp]
        L.dspark_qcache_append.argtypes = [C.POINTER(QCacheStruct), vp, i, C.c_int64, C.c_int64, vp, i, vp, i, vp, sz, vp]
        L.dspark_qcache_attend.argtypes = [C.POINTER(QCacheStruct), i, C.POINTER(QAttnArgs), i, vp, sz, vp]
        L.dspark_qcache_workspace_bytes.argtypes = [C.POINTER(QCacheStruct), i]
        L.dspark_qcache_workspace_bytes.restype = sz
        L.dspark_qcache_check.argtypes = [vp, vp]
        L.dspark_status_str.argtypes = [i]
        L.dspark_status_str.restype = C.c_char_p
        for f in EXPORTS:
            if f not in ("dspark_destroy", "dspark_workspace_bytes", "dspark_status_str", "dspark_qcache_workspace_bytes"):
                getattr(L, f).restype = i
        _lib = L
    return _lib


def geom_struct(G, weight_format: int = FMT_BF16) -> Geom:
    return Geom(hidden=G.hidden, n_aux=G.n_aux, n_layers=G.n_layers, n_heads=G.n_heads, q_lora=G.q_lora,
                kv_lora=G.kv_lora, d_nope=G.d_nope, d_rope=G.d_rope, d_v=G.d_v, inter=G.inter, vocab=G.vocab,
                rank=G.rank, block=G.block, rope_theta=G.rope_theta, eps=G.eps, yarn_factor=G.yarn_factor,
                yarn_orig_ctx=G.yarn_orig_ctx, yarn_alpha=G.yarn_alpha, yarn_beta=G.yarn_beta,
                page_size=G.page_size, weight_format=weight_format)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else C.c_void_p(t.data_ptr())


def _mat(v) -> "Mat":
    """A matrix entry: a bf16 tensor, or (data, scale, global_scale) for FP8 / NVFP4."""
    if isinstance(v, tuple):
        d, sc, g = v
        return Mat(_p(d), _p(sc), float(g))
    return Mat(_p(v), None, 1.0)


def _stream():
    # the raw handle: torch.cuda.current_stream() builds a Stream object first (3 us against 0.2 us a call)
    return C.c_void_p(torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()))


def _chk(fn: str, st: int):
    if st != 0:
        raise DSparkError(fn, st)


class DSpark:
    """One drafter (geometry + device-resident weights) bound to libdspark.

    ``W`` maps names to device tensors (bf16 matrices row-major [out, in], fp32
    norm gains and confidence head), as produced by the seeded generators. With
    ``weight_format`` FP8 or NVFP4 the quantised matrices (fc, q_b, o, gate, up,
    down) are (data, scale, global_scale) triples.
    The workspace is allocated here, zero-filled, for up to ``max_bs``
    sequences and contexts of ``max_ctx`` tokens.
    """

    def __init__(self, G, W: Dict[str, torch.Tensor], max_bs: int = 1, max_ctx: int = 0,
                 weight_format: int = FMT_BF16):
        self.G = G
        self.W = W
        L = lib()
        self.geom = geom_struct(G, weight_format)
        w = Weights()
        w.w_fc = _mat(W["w_fc"])
        for l in range(G.n_layers):
            P = f"l{l}."
            lw = w.layers[l]
            lw.attn_norm = _p(W[P + "attn_norm"])
            lw.w_qkv_a = _p(W[P + "w_qkv_a"])
            lw.q_a_norm = _p(W[P + "q_a_norm"])
            lw.kv_a_norm = _p(W[P + "kv_a_norm"])
            lw.w_q_b = _mat(W[P + "w_q_b"])
            lw.w_kv_b = _p(W[P + "w_kv_b"])
            lw.w_o = _mat(W[P + "w_o"])
            lw.mlp_norm = _p(W[P + "mlp_norm"])
            lw.w_gate = _mat(W[P + "w_gate"])
            lw.w_up = _mat(W[P + "w_up"])
            lw.w_down = _mat(W[P + "w_down"])
        w.final_norm = _p(W["final_norm"])
        w.w_lm = _p(W["w_lm"])
        w.markov_w1 = _p(W["markov_w1"])
        w.markov_w2 = _p(W["markov_w2"])
        w.w_conf = _p(W["w_conf"])
        w.b_conf = float(W["b_conf"].item()) if torch.is_tensor(W["b_conf"]) else float(W["b_conf"])
        self.weights = w
        h = C.c_void_p()
        _chk("dspark_create", L.dspark_create(C.byref(self.geom), C.byref(w), C.byref(h)))
        self.h = h
        self.max_bs, self.max_ctx = max_bs, max_ctx
        self.ws_bytes = L.dspark_workspace_bytes(h, max_bs, max_ctx)
        if self.ws_bytes == 0:
            raise DSparkError("dspark_workspace_bytes", 3)
        self.ws = torch.zeros(self.ws_bytes, dtype=torch.uint8, device="cuda")

    def close(self):
        if getattr(self, "h", None):
            lib().dspark_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # --- the five calls ------------------------------------------------------------
    def fuse_ctx(self, aux: torch.Tensor, x: torch.Tensor, bs: int):
        _chk("dspark_fuse_ctx", lib().dspark_fuse_ctx(self.h, _p(aux), _p(x), bs, _p(self.ws), self.ws_bytes,
                                                       _stream()))

    def fuse_ctx_noalloc(self, aux: torch.Tensor, x: torch.Tensor, bs: int):
        """fc fusion with the library's own fixed scratch instead of the workspace."""
        _chk("dspark_fuse_ctx_noalloc", lib().dspark_fuse_ctx_noalloc(self.h, _p(aux), _p(x), bs, _stream()))

    def make_kv(self, pools: Sequence[torch.Tensor], page_table: torch.Tensor, ctx_len: torch.Tensor,
                max_ctx: int) -> KV:
        kv = KV()
        # the struct holds raw device pointers: keep the tensors alive as long as it lives
        kv._keep = (list(pools), page_table, ctx_len)
        for l, t in enumerate(pools):
            kv.pools[l] = t.data_ptr()
        kv.n_pages = int(pools[0].shape[0])
        kv.page_table = page_table.data_ptr()
        kv.max_pages = int(page_table.shape[1])
        kv.ctx_len = ctx_len.data_ptr()
        kv.max_ctx = int(max_ctx)
        return kv

    def draft_block(self, x: torch.Tensor, kv: KV, h_out: torch.Tensor, z: torch.Tensor, bs: int):
        _chk("dspark_draft_block", lib().dspark_draft_block(self.h, _p(x), C.byref(kv), _p(h_out), _p(z), bs,
                                                             _p(self.ws), self.ws_bytes, _stream()))

    def markov_rollout(self, z, anchor, sample: Sample, tokens, ell, bs: int):
        _chk("dspark_markov_rollout", lib().dspark_markov_rollout(self.h, _p(z), _p(anchor), C.byref(sample),
                                                                   _p(tokens), _p(ell), bs, _p(self.ws),
                                                                   self.ws_bytes, _stream()))

    def confidence(self, h_out, conf, bs: int):
        _chk("dspark_confidence", lib().dspark_confidence(self.h, _p(h_out), _p(conf), bs, _stream()))

    def verify(self, target_logits, ell, tokens, sample: Sample, accept_len, out_tokens, bs: int):
        _chk("dspark_verify", lib().dspark_verify(self.h, _p(target_logits), _p(ell), _p(tokens), C.byref(sample),
                                                   _p(accept_len), _p(out_tokens), bs, _p(self.ws), self.ws_bytes,
                                                   _stream()))

    def kv_append(self, x_new: torch.Tensor, n_new: torch.Tensor, kv: KV, bs: int):
        """Write the latent entries of newly verified tokens (x_new [bs, n_max, H]) into every
        layer's page pool at ctx_len + j, then advance ctx_len by n_new (device, in place)."""
        n_max = int(x_new.shape[1])
        _chk("dspark_kv_append", lib().dspark_kv_append(self.h, _p(x_new), n_max, _p(n_new), C.byref(kv), bs,
                                                         _p(self.ws), self.ws_bytes, _stream()))

    def check(self) -> int:
        """Synchronise and return (and clear) the device error word."""
        return lib().dspark_check(self.h, _p(self.ws), _stream())

    def check_noalloc(self) -> int:
        """Synchronise and return (and clear) the error word of the allocation-free fusion's fixed scratch."""
        return lib().dspark_check(self.h, None, _stream())


_I32 = torch.int32


def _int32(name: str, t: torch.Tensor, n: int, dev: int):
    """t holds at least n contiguous int32 values on GPU dev."""
    if t.dtype is not _I32 or t.get_device() != dev or not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"{name}: a contiguous int32 tensor of at least {n} elements on cuda:{dev}")


class QCache:
    """A paged latent cache in E4M3 with one power-of-two scale per page of 64 tokens.

    ``codes``: per layer uint8 (or float8_e4m3fn) [n_pages, 64, kv_lora + d_rope]; ``scales``: per layer fp32
    [n_pages]; ``page_table`` int32 [bs, max_pages]. All belong to the caller and are written in place; they and every
    call's tensors lie on one GPU, the current one at each call (kernels read no other GPU's memory). The three
    calls are the page plan, the quantising append (every layer) and the attention over one layer; they run on the
    current stream and do not wait. ``check()`` reads the error word that their kernels set. Without ``n_heads`` the
    workspace serves the plan and the append alone; a zero-filled ``workspace`` (uint8) may be given instead, and
    caches that run on one stream may share it.
    """

    def __init__(self, kv_lora: int, d_rope: int, codes: Sequence[torch.Tensor], scales: Sequence[torch.Tensor],
                 page_table: torch.Tensor, n_heads: int = 0, n_pages: Optional[int] = None,
                 workspace: Optional[torch.Tensor] = None):
        if len(codes) != len(scales) or len(codes) > MAX_LAYERS:
            raise ValueError("one code pool and one scale vector per layer, at most %d layers" % MAX_LAYERS)
        self.D, self.kv, self.layers, self.dev = kv_lora + d_rope, kv_lora, len(codes), page_table.get_device()
        if self.dev < 0:
            raise ValueError("page_table: a CUDA tensor")
        if n_pages is None:
            if not len(codes):
                raise ValueError("n_pages is needed without code pools")
            n_pages = int(codes[0].shape[0])
        for t, u in zip(codes, scales):
            if (t.dtype not in (torch.uint8, torch.float8_e4m3fn) or tuple(t.shape) != (n_pages, 64, self.D)
                    or not t.is_contiguous() or t.get_device() != self.dev):
                raise ValueError(f"codes: contiguous uint8 or float8_e4m3fn tensors [{n_pages}, 64, {self.D}] on cuda:{self.dev}")
            if u.dtype != torch.float32 or u.numel() != n_pages or not u.is_contiguous() or u.get_device() != self.dev:
                raise ValueError(f"scales: contiguous fp32 tensors [{n_pages}] on cuda:{self.dev}")
        if page_table.dim() != 2:
            raise ValueError("page_table: int32 [bs, max_pages]")
        _int32("page_table", page_table, 1, self.dev)
        c = QCacheStruct(kv_lora=kv_lora, d_rope=d_rope, page_size=64, n_layers=len(codes), n_pages=n_pages,
                         page_table=page_table.data_ptr(), max_pages=int(page_table.shape[1]))
        for l, (t, u) in enumerate(zip(codes, scales)):
            c.codes[l], c.scales[l] = t.data_ptr(), u.data_ptr()
        # the struct holds raw device pointers: keep the tensors alive as long as it lives
        self._keep = (list(codes), list(scales), page_table)
        self.c, self.ref, self.rows, self.n_pages = c, C.byref(c), int(page_table.shape[0]), n_pages
        need = lib().dspark_qcache_workspace_bytes(C.byref(c), n_heads)
        if need == 0:
            raise DSparkError("dspark_qcache_workspace_bytes", 3)
        if workspace is None:
            workspace = torch.zeros(need, dtype=torch.uint8, device=page_table.device)
        if workspace.dtype is not torch.uint8 or workspace.get_device() != self.dev or not workspace.is_contiguous():
            raise ValueError(f"workspace: a contiguous uint8 tensor on cuda:{self.dev}, zero-filled before its first use")
        self.ws, self.ws_ptr, self.ws_bytes = workspace, C.c_void_p(workspace.data_ptr()), workspace.numel()

    def _device(self) -> int:
        dev = torch._C._cuda_getDevice()
        if dev != self.dev:
            raise ValueError(f"the cache lies on cuda:{self.dev}, the current device is cuda:{dev}")
        return dev

    def plan(self, length: torch.Tensor, want: torch.Tensor, ring: torch.Tensor, ring_state: torch.Tensor,
             length_out: torch.Tensor, ring_state_out: torch.Tensor, cu_new: torch.Tensor,
             slots: Optional[torch.Tensor], positions: Optional[torch.Tensor], seg_row: torch.Tensor):
        """Pages, slots and positions for requests that go from ``length`` to ``want`` tokens (int32 [bs]).

        Free pages come from ``ring`` [n_pages] at ``ring_state`` [2] (first free, number). Outputs: ``length_out``
        [bs], ``ring_state_out`` [2], ``cu_new`` [bs + 1], ``slots`` and ``positions`` (one per new token, then -1;
        their size is the most new tokens served), ``seg_row`` (first new token of every touched page, then their
        number; its size less one is the most pages served)."""
        dev, bs, n, seg = self._device(), length.numel(), self.n_pages, seg_row.numel()
        max_new = 0 if slots is None else slots.numel()
        if bs > self.rows:
            raise ValueError("more requests than rows of the page table")
        _int32("length", length, bs, dev)
        _int32("want", want, bs, dev)
        _int32("ring", ring, n, dev)
        _int32("ring_state", ring_state, 2, dev)
        _int32("length_out", length_out, bs, dev)
        _int32("ring_state_out", ring_state_out, 2, dev)
        _int32("cu_new", cu_new, bs + 1, dev)
        _int32("seg_row", seg_row, 1, dev)
        ps = pp = None
        if max_new:
            _int32("slots", slots, 0, dev)
            _int32("positions", positions, max_new, dev)
            ps, pp = slots.data_ptr(), positions.data_ptr()
        a = QPlanArgs(length.data_ptr(), want.data_ptr(), ring.data_ptr(), ring_state.data_ptr(), length_out.data_ptr(),
                      ring_state_out.data_ptr(), cu_new.data_ptr(), ps, pp, seg_row.data_ptr())
        st = lib().dspark_qcache_plan(self.ref, C.byref(a), bs, max_new, seg - 1, self.ws_ptr, self.ws_bytes, _stream())
        if st:
            raise DSparkError("dspark_qcache_plan", st)

    def append(self, entries: torch.Tensor, slots: torch.Tensor, seg_row: torch.Tensor):
        """Quantise entries [n_layers, rows, kv_lora + d_rope] (bf16 or fp32, any row and layer stride) into the slots
        of dspark_qcache_plan, raising the scales of pages that need it."""
        dev, shape = self._device(), entries.shape
        if len(shape) != 3 or shape[0] != self.layers or shape[2] != self.D or entries.get_device() != dev:
            raise ValueError(f"entries: tensor [{self.layers}, rows, {self.D}] on cuda:{dev}")
        kind = 0 if entries.dtype is torch.bfloat16 else 1
        if kind and entries.dtype is not torch.float32:
            raise ValueError("entries: bf16 or fp32")
        layer_stride, row_stride, one = entries.stride()
        if one != 1:
            raise ValueError("entries: the elements of a row are contiguous")
        _int32("slots", slots, 0, dev)
        _int32("seg_row", seg_row, 1, dev)
        rows = min(shape[1], slots.numel())
        if shape[1] <= 1:
            row_stride = self.D  # torch leaves the stride of one row open
        st = lib().dspark_qcache_append(self.ref, entries.data_ptr(), kind, row_stride, layer_stride, slots.data_ptr(), rows,
                                        seg_row.data_ptr(), seg_row.numel() - 1, self.ws_ptr, self.ws_bytes, _stream())
        if st:
            raise DSparkError("dspark_qcache_append", st)

    def attend(self, layer: int, q: torch.Tensor, cu_q: torch.Tensor, length: torch.Tensor, o: torch.Tensor,
               lse: Optional[torch.Tensor] = None, causal: bool = True, scale: float = 1.0):
        """o = softmax(scale q k^T) v over one layer: q bf16 [total_q, n_heads, kv_lora + d_rope] (any token stride),
        request b's queries at cu_q[b] .. cu_q[b+1]-1, ``length`` cached tokens each; o bf16 [total_q, n_heads,
        kv_lora], lse fp32 [total_q, n_heads]."""
        dev, D, kv, shape = self._device(), self.D, self.kv, q.shape
        if len(shape) != 3 or shape[2] != D or q.dtype is not torch.bfloat16 or q.get_device() != dev:
            raise ValueError(f"q: bf16 tensor [total_q, n_heads, {D}] on cuda:{dev}")
        n, h, _ = shape
        if o.shape != (n, h, kv) or o.dtype is not torch.bfloat16 or o.get_device() != dev:
            raise ValueError(f"o: bf16 tensor [{n}, {h}, {kv}] on cuda:{dev}")
        qs, qh, q1 = q.stride()
        os, oh, o1 = o.stride()
        if n and (q1 != 1 or o1 != 1 or h > 1 and (qh != D or oh != kv)):
            raise ValueError("q and o: the heads of a token are contiguous")
        if n <= 1:  # torch leaves the stride of one token open
            qs, os = h * D, h * kv
        pl = None
        if lse is not None:
            if lse.dtype is not torch.float32 or lse.numel() != n * h or not lse.is_contiguous() or lse.get_device() != dev:
                raise ValueError(f"lse: contiguous fp32 tensor [{n}, {h}] on cuda:{dev}")
            pl = lse.data_ptr() or None
        bs = length.numel()
        if bs > self.rows:
            raise ValueError("more requests than rows of the page table")
        _int32("length", length, 1, dev)
        _int32("cu_q", cu_q, bs + 1, dev)
        a = QAttnArgs(q.data_ptr() or None, qs, cu_q.data_ptr(), length.data_ptr(), h, n, 1 if causal else 0, scale,
                      o.data_ptr() or None, os, pl)
        st = lib().dspark_qcache_attend(self.ref, layer, C.byref(a), bs, self.ws_ptr, self.ws_bytes, _stream())
        if st:
            raise DSparkError("dspark_qcache_attend", st)

    def check(self) -> int:
        """Synchronise and return (and clear) the device error word."""
        self._device()
        return lib().dspark_qcache_check(_p(self.ws), _stream())
