"""Python binding of libdsa.so -- the GLM-5 DSA attention hot path
(lightning indexer -> causal top-k -> sparse MLA) on one GB300.

Argument marshalling only: every step runs in the CUDA kernels of
``libdsa.so`` (C ABI in ``include/dsa.h``).  PyTorch supplies device memory
and the current stream.  There is no fallback: if the library is missing or
no CUDA device is present the calls raise.

    import sparse_attention_gb300 as dsa
    b  = dsa.make_batch(q_off, ctx_len, max_q, max_ctx, cache_stride)
    ws = dsa.workspace(b, k)
    dsa.forward(b, q_idx, w, k_idx, q, kv, k, sm_scale, out, lse, ws=ws)
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdsa.so")

H_IDX, D_IDX, H, D_QK, D_V, MAX_TOPK = 32, 128, 64, 576, 512, 2048
D_HEAD, D_EXP, D_HIDDEN, EXPANDED_ROOM = 256, 448, 6144, 128

STATUS = {
    0: "DSA_OK", 1: "DSA_ERR_INVALID_ARG", 2: "DSA_ERR_UNSUPPORTED", 3: "DSA_ERR_WORKSPACE",
    4: "DSA_ERR_CUDA", 5: "DSA_ERR_TIMEOUT", 6: "DSA_ERR_BAD_BATCH", 7: "DSA_ERR_BAD_INDEX", 8: "DSA_ERR_INTERNAL",
    9: "DSA_ERR_NO_PAGES",
}

EXPORTS = ("dsa_status_string", "dsa_last_cuda_error", "dsa_kernel_launch_count", "dsa_workspace_size", "dsa_reset_device_status", "dsa_read_device_status",
           "dsa_selftest_wait_timeout", "dsa_indexer_scores", "dsa_topk", "dsa_sparse_mla_fwd",
           "dsa_sparse_mla_fwd_noalloc", "dsa_forward", "dsa_mla_absorb_q", "dsa_mla_workspace_size", "dsa_mla_output", "dsa_index_key_workspace_size",
           "dsa_index_key_producer", "dsa_quantize_fp8", "dsa_indexer_scores_fp8", "dsa_forward_fp8",
           "dsa_tree_workspace_size", "dsa_step_tables", "dsa_latent_append", "dsa_tree_mla_fwd", "dsa_tree_topk",
           "dsa_tree_commit", "dsa_rope_table", "dsa_rope", "dsa_prompt_workspace_size", "dsa_mla_expand",
           "dsa_prompt_mla_fwd", "dsa_mla_o_proj", "dsa_prefix_workspace_size", "dsa_prefix_mla_fwd")


class DsaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = f"{where}: {STATUS.get(code, code)}"
        if code == 4 and _lib is not None:
            msg += f" ({_lib.dsa_last_cuda_error().decode()})"
        super().__init__(msg)


class DsaBatch(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("total_q", ctypes.c_int32), ("max_q", ctypes.c_int32),
                ("max_ctx", ctypes.c_int32), ("cache_stride", ctypes.c_int64),
                ("q_off", ctypes.c_void_p), ("ctx_len", ctypes.c_void_p)]


class DsaPages(ctypes.Structure):
    _fields_ = [("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("pool_pages", ctypes.c_int32),
                ("block_table", ctypes.c_void_p)]


class DsaGroups(ctypes.Structure):
    _fields_ = [("groups", ctypes.c_int32), ("off", ctypes.c_void_p), ("shared", ctypes.c_void_p)]


class DsaExpanded(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("off", ctypes.c_void_p), ("kv", ctypes.c_void_p),
                ("k_pe", ctypes.c_void_p)]


class DsaRopeScaling(ctypes.Structure):
    _fields_ = [("factor", ctypes.c_double), ("original_ctx", ctypes.c_int32), ("beta_fast", ctypes.c_float),
                ("beta_slow", ctypes.c_float), ("mscale", ctypes.c_float)]


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libdsa.so (build it first with ``python -m sparse_attention_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libdsa.so not found at {path}; build it with "
                           f"`python -m sparse_attention_gb300.build` (no CPU fallback exists)")
    lib = ctypes.CDLL(path)
    P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    BP = ctypes.POINTER(DsaBatch)
    lib.dsa_status_string.restype = ctypes.c_char_p
    lib.dsa_status_string.argtypes = [i32]
    lib.dsa_last_cuda_error.restype = ctypes.c_char_p
    lib.dsa_last_cuda_error.argtypes = []
    lib.dsa_kernel_launch_count.restype = ctypes.c_uint64
    lib.dsa_kernel_launch_count.argtypes = []
    lib.dsa_workspace_size.argtypes = [BP, i32, ctypes.POINTER(sz)]
    lib.dsa_reset_device_status.argtypes = [P, P]
    lib.dsa_read_device_status.argtypes = [P, P, ctypes.POINTER(ctypes.c_int)]
    lib.dsa_indexer_scores.argtypes = [BP, P, P, P, P, i64, P, sz, P]
    lib.dsa_topk.argtypes = [BP, P, i64, i32, P, P, sz, P]
    lib.dsa_sparse_mla_fwd.argtypes = [BP, P, P, P, i32, f32, P, P, P, sz, P]
    lib.dsa_sparse_mla_fwd_noalloc.argtypes = [BP, P, P, P, i32, f32, P, P, P, P]
    lib.dsa_selftest_wait_timeout.argtypes = [P, ctypes.c_uint32, P]
    lib.dsa_forward.argtypes = [BP, P, P, P, P, P, i32, f32, P, P, P, P, i64, P, sz, P]
    lib.dsa_mla_absorb_q.argtypes = [i32, P, P, P, P, P, sz, P]
    lib.dsa_mla_output.argtypes = [i32, P, P, P, P, P, P, sz, P]
    lib.dsa_mla_workspace_size.argtypes = [i32, ctypes.POINTER(sz)]
    lib.dsa_index_key_workspace_size.argtypes = [i32, ctypes.POINTER(sz)]
    lib.dsa_index_key_producer.argtypes = [BP, P, P, P, P, f32, P, P, P, P, P, P, sz, P]
    lib.dsa_quantize_fp8.argtypes = [i64, P, P, P, P]
    lib.dsa_indexer_scores_fp8.argtypes = [BP, P, P, P, P, P, P, i64, P, sz, P]
    lib.dsa_forward_fp8.argtypes = [BP, P, P, P, P, P, P, P, i32, f32, P, P, P, P, i64, P, sz, P]
    GP = ctypes.POINTER(DsaPages)
    lib.dsa_tree_workspace_size.argtypes = [BP, ctypes.POINTER(sz)]
    lib.dsa_step_tables.argtypes = [BP, GP, P, P, P, P, P, P, P, P, P, P, P, P, sz, P]
    lib.dsa_latent_append.argtypes = [i32, P, i64, P, f32, P, P, i32, P, P, i64, P, P, sz, P]
    lib.dsa_tree_mla_fwd.argtypes = [BP, GP, P, P, P, f32, P, P, P, sz, P]
    lib.dsa_tree_topk.argtypes = [BP, P, i64, P, i32, P, P, sz, P]
    lib.dsa_tree_commit.argtypes = [BP, GP, P, P, i32, i64, P, P, P, P, sz, P]
    lib.dsa_rope_table.argtypes = [i32, i32, i32, ctypes.c_double, ctypes.POINTER(DsaRopeScaling), P, P, P]
    lib.dsa_rope.argtypes = [i32, i32, i32, P, i64, i64, P, P, i32, P, i32, P, i64, i64, P, sz, P]
    XP = ctypes.POINTER(DsaExpanded)
    lib.dsa_prompt_workspace_size.argtypes = [BP, ctypes.POINTER(sz)]
    lib.dsa_mla_expand.argtypes = [BP, GP, P, P, P, XP, P, sz, P]
    lib.dsa_prompt_mla_fwd.argtypes = [BP, P, XP, f32, P, P, P, sz, P]
    lib.dsa_mla_o_proj.argtypes = [i32, P, P, P, P, sz, P]
    RP = ctypes.POINTER(DsaGroups)
    lib.dsa_prefix_workspace_size.argtypes = [BP, RP, ctypes.POINTER(sz)]
    lib.dsa_prefix_mla_fwd.argtypes = [BP, RP, GP, P, P, P, f32, P, P, P, sz, P]
    for name in EXPORTS:
        if name not in ("dsa_status_string", "dsa_last_cuda_error", "dsa_kernel_launch_count"):
            getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


class Batch:
    """Host handle of a dsa_batch.  Keeps the device q_off / ctx_len alive."""

    def __init__(self, q_off: torch.Tensor, ctx_len: torch.Tensor, max_q: int, max_ctx: int, cache_stride: int,
                 total_q: Optional[int] = None):
        assert q_off.dtype == torch.int32 and ctx_len.dtype == torch.int32
        assert q_off.is_cuda and ctx_len.is_cuda and q_off.is_contiguous() and ctx_len.is_contiguous()
        self.q_off, self.ctx_len = q_off, ctx_len
        B = ctx_len.numel()
        if total_q is None:
            total_q = int(q_off[-1].item())
        self.c = DsaBatch(B, int(total_q), int(max_q), int(max_ctx), int(cache_stride),
                          q_off.data_ptr(), ctx_len.data_ptr())

    @property
    def B(self) -> int:
        return self.c.batch

    @property
    def total_q(self) -> int:
        return self.c.total_q

    @property
    def max_q(self) -> int:
        return self.c.max_q

    @property
    def max_ctx(self) -> int:
        return self.c.max_ctx


def make_batch(q_off, ctx_len, max_q: int, max_ctx: int, cache_stride: int, total_q: Optional[int] = None,
               device="cuda") -> Batch:
    q_off = torch.as_tensor(q_off, dtype=torch.int32).to(device).contiguous()
    ctx_len = torch.as_tensor(ctx_len, dtype=torch.int32).to(device).contiguous()
    return Batch(q_off, ctx_len, max_q, max_ctx, cache_stride, total_q)


def _check(code: int, where: str) -> None:
    if code != 0:
        raise DsaError(code, where)


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("device tensor expected")
    if not t.is_contiguous():
        raise ValueError("contiguous tensor expected")
    return t.data_ptr()


def _bf16(t: torch.Tensor):
    if t.dtype != torch.bfloat16:
        raise TypeError(f"bf16 tensor expected, got {t.dtype}")
    return _p(t)


def _stream(stream) -> int:
    if stream is None:
        # the raw handle: building a Stream object takes 3 us of a 13 us call
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def kernel_launch_count() -> int:
    """Kernels launched by libdsa.so in this process so far."""
    return int(load_library().dsa_kernel_launch_count())


def workspace_size(batch: Batch, k: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().dsa_workspace_size(ctypes.byref(batch.c), int(k), ctypes.byref(n)), "dsa_workspace_size")
    return int(n.value)


def workspace(batch: Batch, k: int, device="cuda") -> torch.Tensor:
    """A fresh workspace (uint8 tensor) with a cleared status word."""
    ws = torch.empty(max(workspace_size(batch, k), 256), dtype=torch.uint8, device=device)
    reset_device_status(ws)
    return ws


def reset_device_status(ws: torch.Tensor, stream=None) -> None:
    _check(load_library().dsa_reset_device_status(_p(ws), _stream(stream)), "dsa_reset_device_status")


def read_device_status(ws: torch.Tensor, stream=None) -> int:
    v = ctypes.c_int(0)
    _check(load_library().dsa_read_device_status(_p(ws), _stream(stream), ctypes.byref(v)), "dsa_read_device_status")
    return int(v.value)


def selftest_wait_timeout(ws: torch.Tensor, limit_us: int = 2000, stream=None) -> None:
    """Launch the bounded-wait diagnostic (see dsa_selftest_wait_timeout)."""
    _check(load_library().dsa_selftest_wait_timeout(_p(ws), int(limit_us), _stream(stream)),
           "dsa_selftest_wait_timeout")


def indexer_scores(batch: Batch, q_idx, w, k_idx, scores, ld: Optional[int] = None, ws=None, stream=None):
    assert w.dtype == torch.float32 and scores.dtype == torch.float32
    ld = int(ld if ld is not None else scores.shape[-1])
    _check(load_library().dsa_indexer_scores(ctypes.byref(batch.c), _bf16(q_idx), _p(w), _bf16(k_idx), _p(scores),
                                             ld, _p(ws), ws.numel() if ws is not None else 0, _stream(stream)),
           "dsa_indexer_scores")
    return scores


def topk(batch: Batch, scores, k: int, idx, ld: Optional[int] = None, ws=None, stream=None):
    assert scores.dtype == torch.float32 and idx.dtype == torch.int32
    ld = int(ld if ld is not None else scores.shape[-1])
    _check(load_library().dsa_topk(ctypes.byref(batch.c), _p(scores), ld, int(k), _p(idx), _p(ws),
                                   ws.numel() if ws is not None else 0, _stream(stream)), "dsa_topk")
    return idx


def sparse_mla_fwd(batch: Batch, q, kv, idx, k: int, sm_scale: float, out, lse=None, ws=None, stream=None):
    assert idx.dtype == torch.int32 and (lse is None or lse.dtype == torch.float32)
    _check(load_library().dsa_sparse_mla_fwd(ctypes.byref(batch.c), _bf16(q), _bf16(kv), _p(idx), int(k),
                                             float(sm_scale), _bf16(out), _p(lse), _p(ws),
                                             ws.numel() if ws is not None else 0, _stream(stream)),
           "dsa_sparse_mla_fwd")
    return out


def sparse_mla_fwd_noalloc(batch: Batch, q, kv, idx, k: int, sm_scale: float, out, lse=None, device_status=None,
                           stream=None):
    """dsa_sparse_mla_fwd without a workspace: the split-K partials live in
    the library's static device scratch (for callers that cannot allocate).
    Calls that overlap on the GPU race; the first call on a device should
    come before any stream capture."""
    assert idx.dtype == torch.int32 and (lse is None or lse.dtype == torch.float32)
    assert device_status is None or device_status.dtype == torch.int32
    _check(load_library().dsa_sparse_mla_fwd_noalloc(ctypes.byref(batch.c), _bf16(q), _bf16(kv), _p(idx), int(k),
                                                     float(sm_scale), _bf16(out), _p(lse), _p(device_status),
                                                     _stream(stream)), "dsa_sparse_mla_fwd_noalloc")
    return out


def forward(batch: Batch, q_idx, w, k_idx, q, kv, k: int, sm_scale: float, out, lse=None, idx_out=None,
            scores_out=None, ld: int = 0, ws=None, stream=None):
    if scores_out is not None and not ld:
        ld = scores_out.shape[-1]
    _check(load_library().dsa_forward(ctypes.byref(batch.c), _bf16(q_idx), _p(w), _bf16(k_idx), _bf16(q), _bf16(kv),
                                      int(k), float(sm_scale), _bf16(out), _p(lse), _p(idx_out), _p(scores_out),
                                      int(ld), _p(ws), ws.numel() if ws is not None else 0, _stream(stream)),
           "dsa_forward")
    return out


def mla_absorb_q(q_nope, q_pe, w_kv_b, q_out, ws, stream=None):
    """q_out[t, h] = [W_UK[h]^T q_nope[t, h] | q_pe[t, h]] (see dsa_mla_absorb_q)."""
    total_q = q_nope.shape[0]
    assert q_pe.shape[0] == total_q and q_out.shape[0] == total_q
    _check(load_library().dsa_mla_absorb_q(int(total_q), _bf16(q_nope), _bf16(q_pe), _bf16(w_kv_b), _bf16(q_out),
                                           _p(ws), ws.numel(), _stream(stream)), "dsa_mla_absorb_q")
    return q_out


def mla_workspace(total_q: int, device="cuda") -> torch.Tensor:
    """A workspace for dsa_mla_output / dsa_mla_absorb_q with a cleared status word."""
    n = ctypes.c_size_t(0)
    _check(load_library().dsa_mla_workspace_size(int(total_q), ctypes.byref(n)), "dsa_mla_workspace_size")
    ws = torch.empty(max(int(n.value), 256), dtype=torch.uint8, device=device)
    reset_device_status(ws)
    return ws


def mla_output(o_lat, w_kv_b, w_o, o_mid, y, ws, stream=None):
    """o_mid[t, h] = W_UV[h] o_lat[t, h]; y[t] = w_o o_mid[t] (see dsa_mla_output)."""
    total_q = o_lat.shape[0]
    assert o_mid.shape[0] == total_q and y.shape[0] == total_q
    _check(load_library().dsa_mla_output(int(total_q), _bf16(o_lat), _bf16(w_kv_b), _bf16(w_o), _bf16(o_mid),
                                         _bf16(y), _p(ws), ws.numel(), _stream(stream)), "dsa_mla_output")
    return y


def index_key_workspace(total_q: int, device="cuda") -> torch.Tensor:
    n = ctypes.c_size_t(0)
    _check(load_library().dsa_index_key_workspace_size(int(total_q), ctypes.byref(n)),
           "dsa_index_key_workspace_size")
    ws = torch.empty(max(int(n.value), 256), dtype=torch.uint8, device=device)
    reset_device_status(ws)
    return ws


def index_key_producer(batch: Batch, x, wk, gamma, beta, eps: float, cos, sin, w_proj, k_idx, w_out, ws,
                       stream=None):
    """Index keys of the batch's new tokens appended to k_idx, and their head
    weights in w_out (see dsa_index_key_producer)."""
    for t in (gamma, beta, cos, sin, w_out):
        assert t.dtype == torch.float32
    _check(load_library().dsa_index_key_producer(ctypes.byref(batch.c), _bf16(x), _bf16(wk), _p(gamma), _p(beta),
                                                 float(eps), _p(cos), _p(sin), _bf16(w_proj), _bf16(k_idx),
                                                 _p(w_out), _p(ws), ws.numel(), _stream(stream)),
           "dsa_index_key_producer")
    return k_idx


def quantize_fp8(x, codes, scale, stream=None):
    """E4M3 codes and per-row scales of bf16 rows of 128 (see dsa_quantize_fp8)."""
    assert codes.dtype == torch.uint8 and scale.dtype == torch.float32
    rows = x.numel() // 128
    _check(load_library().dsa_quantize_fp8(int(rows), _bf16(x), _p(codes), _p(scale), _stream(stream)),
           "dsa_quantize_fp8")
    return codes, scale


def indexer_scores_fp8(batch: Batch, q8, qs, w, k8, ks, scores, ld: Optional[int] = None, ws=None, stream=None):
    ld = int(ld if ld is not None else scores.shape[-1])
    _check(load_library().dsa_indexer_scores_fp8(ctypes.byref(batch.c), _p(q8), _p(qs), _p(w), _p(k8), _p(ks),
                                                 _p(scores), ld, _p(ws), ws.numel() if ws is not None else 0,
                                                 _stream(stream)), "dsa_indexer_scores_fp8")
    return scores


def forward_fp8(batch: Batch, q8, qs, w, k8, ks, q, kv, k: int, sm_scale: float, out, lse=None, idx_out=None,
                scores_out=None, ld: int = 0, ws=None, stream=None):
    if scores_out is not None and not ld:
        ld = scores_out.shape[-1]
    _check(load_library().dsa_forward_fp8(ctypes.byref(batch.c), _p(q8), _p(qs), _p(w), _p(k8), _p(ks), _bf16(q),
                                          _bf16(kv), int(k), float(sm_scale), _bf16(out), _p(lse), _p(idx_out),
                                          _p(scores_out), int(ld), _p(ws), ws.numel() if ws is not None else 0,
                                          _stream(stream)), "dsa_forward_fp8")
    return out


# ---- A step of drafted tokens over a paged or contiguous cache --------------

class Pages:
    """Host handle of a dsa_pages.  Keeps the device block table alive."""

    def __init__(self, block_table: torch.Tensor, page_size: int, pool_pages: int):
        if block_table.dtype != torch.int32 or block_table.dim() != 2:
            raise TypeError("block_table: int32 [batch, max_pages] expected")
        self.block_table, self.page_size, self.pool_pages = block_table, int(page_size), int(pool_pages)
        self.c = DsaPages(self.page_size, block_table.shape[1], self.pool_pages, _p(block_table))


def make_pages(block_table: torch.Tensor, page_size: int, pool_pages: int) -> Pages:
    return Pages(block_table, page_size, pool_pages)


def tree_workspace(batch: Optional[Batch] = None, device="cuda") -> torch.Tensor:
    """A workspace of the drafted-step calls with a cleared status word (no
    batch: for latent_append alone)."""
    n = ctypes.c_size_t(0)
    _check(load_library().dsa_tree_workspace_size(ctypes.byref(batch.c) if batch is not None else None,
                                                  ctypes.byref(n)), "dsa_tree_workspace_size")
    ws = torch.empty(int(n.value), dtype=torch.uint8, device=device)
    reset_device_status(ws)
    return ws


def _typed(name: str, t: Optional[torch.Tensor], dtype: torch.dtype, numel: int, dev: int):
    """Pointer of a contiguous tensor of `dtype` with at least `numel` elements on device `dev` (None stays None)."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.numel() >= numel:
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name}: {dtype} tensor expected, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: expected on cuda:{dev}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: contiguous tensor expected")
    raise ValueError(f"{name}: {numel} elements expected, got {t.numel()}")


def _here(where: str, ws: Optional[torch.Tensor], stream) -> int:
    """The device of a call: the workspace's, which has to be the current one and the stream's."""
    if ws is None:
        raise DsaError(3, where)
    dev = ws.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice() or (stream is not None and stream.device_index != dev):
        raise ValueError(f"workspace on {ws.device}: expected on the current CUDA device, and the stream's")
    return dev


def _raw_stream(stream, dev: int) -> int:
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev)


def _paged(batch: Batch, pages: Optional[Pages], dev: int):
    """The dsa_pages argument, and the cache rows that a call may reach."""
    if batch.q_off.get_device() != dev or (pages is not None and pages.block_table.get_device() != dev):
        raise ValueError(f"batch or block table: expected on cuda:{dev}")
    if pages is None:
        return None, batch.c.batch * batch.c.cache_stride
    if pages.block_table.shape[0] < batch.c.batch:
        raise ValueError("block_table: a row for each sequence expected")
    return ctypes.byref(pages.c), pages.pool_pages * pages.page_size


def step_tables(batch: Batch, n_new, ctx_old, slots, positions, mask=None, parent=None, pages: Optional[Pages] = None,
                n_pages_old=None, n_pages=None, free_pages=None, free_range=None, free_range_out=None, ws=None,
                stream=None):
    """q_off and ctx_len of `batch`, block table, slot map, positions and
    masks of a step from its lengths (see dsa_step_tables).  mask: int64
    tensor holding the 64 bits."""
    dev, i32 = _here("dsa_step_tables", ws, stream), torch.int32
    c = batch.c
    pg, _ = _paged(batch, pages, dev)
    _check(load_library().dsa_step_tables(
        ctypes.byref(c), pg, _typed("n_new", n_new, i32, c.batch, dev), _typed("ctx_old", ctx_old, i32, c.batch, dev),
        _typed("parent", parent, i32, c.total_q, dev), _typed("n_pages_old", n_pages_old, i32, c.batch, dev),
        _typed("n_pages", n_pages, i32, c.batch, dev),
        _typed("free_pages", free_pages, i32, pages.pool_pages if pages is not None else 0, dev),
        _typed("free_range", free_range, i32, 2, dev), _typed("free_range_out", free_range_out, i32, 2, dev),
        _typed("slots", slots, i32, c.total_q, dev), _typed("positions", positions, i32, c.total_q, dev),
        _typed("mask", mask, torch.int64, c.total_q, dev), ws.data_ptr(), ws.numel(), _raw_stream(stream, dev)),
        "dsa_step_tables")
    return slots


def latent_append(x, gamma, eps: float, cos, sin, positions, slots, kv, ws, stream=None):
    """RMSNorm | RoPE of the new tokens' compressed rows x [total_q, >= 576]
    (rows may be strided), written to kv at slots (see dsa_latent_append)."""
    dev, f32, i32 = _here("dsa_latent_append", ws, stream), torch.float32, torch.int32
    if x.dtype is not torch.bfloat16 or x.get_device() != dev:
        raise TypeError(f"x: bf16 tensor on cuda:{dev} expected")
    if x.dim() != 2 or x.shape[1] != D_QK or x.stride(1) != 1:
        raise ValueError("x: [total_q, 576] with unit column stride expected")
    total_q, rows = x.shape[0], cos.shape[0]
    if kv.dim() < 2 or kv.shape[-1] != D_QK:
        raise ValueError("kv: [cache_rows, 576] expected")
    _check(load_library().dsa_latent_append(
        total_q, x.data_ptr(), x.stride(0) if total_q > 1 else D_QK, _typed("gamma", gamma, f32, D_V, dev), float(eps),
        _typed("cos", cos, f32, rows * 64, dev), _typed("sin", sin, f32, rows * 64, dev), rows,
        _typed("positions", positions, i32, total_q, dev), _typed("slots", slots, i32, total_q, dev),
        kv.numel() // D_QK, _typed("kv", kv, torch.bfloat16, 0, dev), ws.data_ptr(), ws.numel(), _raw_stream(stream, dev)),
        "dsa_latent_append")
    return kv


def tree_mla_fwd(batch: Batch, q, kv, mask, sm_scale: float, out, lse=None, pages: Optional[Pages] = None, ws=None,
                 stream=None):
    """Attention of every new row over the committed rows and the new rows of
    its mask (see dsa_tree_mla_fwd)."""
    dev, bf16 = _here("dsa_tree_mla_fwd", ws, stream), torch.bfloat16
    c = batch.c
    pg, rows = _paged(batch, pages, dev)
    _check(load_library().dsa_tree_mla_fwd(
        ctypes.byref(c), pg, _typed("q", q, bf16, c.total_q * H * D_QK, dev), _typed("kv", kv, bf16, rows * D_QK, dev),
        _typed("mask", mask, torch.int64, c.total_q, dev), float(sm_scale),
        _typed("out", out, bf16, c.total_q * H * D_V, dev), _typed("lse", lse, torch.float32, c.total_q * H, dev),
        ws.data_ptr(), ws.numel(), _raw_stream(stream, dev)), "dsa_tree_mla_fwd")
    return out


def tree_topk(batch: Batch, scores, mask, k: int, idx, ld: Optional[int] = None, ws=None, stream=None):
    """Causal top-k among what every new row sees (see dsa_tree_topk)."""
    dev = _here("dsa_tree_topk", ws, stream)
    c = batch.c
    ld = int(ld if ld is not None else scores.shape[-1])
    _paged(batch, None, dev)
    _check(load_library().dsa_tree_topk(
        ctypes.byref(c), _typed("scores", scores, torch.float32, c.total_q * ld, dev), ld,
        _typed("mask", mask, torch.int64, c.total_q, dev), int(k),
        _typed("idx", idx, torch.int32, c.total_q * int(k), dev), ws.data_ptr(), ws.numel(), _raw_stream(stream, dev)),
        "dsa_tree_topk")
    return idx


def _layered(name: str, t: torch.Tensor, width: int):
    """(layers, rows) of a cache [layers, rows, width] or [rows, width]."""
    s = t.shape
    if len(s) not in (2, 3) or s[-1] != width:
        raise ValueError(f"{name}: [layers, rows, {width}] expected, got {list(s)}")
    return (s[0], s[1]) if len(s) == 3 else (1, s[0])


def tree_commit(batch: Batch, mask, accepted, ctx_new, kv=None, k_idx=None, pages: Optional[Pages] = None, ws=None,
                stream=None):
    """Moves the accepted paths' rows behind the committed ones in every layer
    of kv [layers, rows, 576] and k_idx [layers, rows, 128] (one layer without
    the first dimension; see dsa_tree_commit)."""
    dev, bf16 = _here("dsa_tree_commit", ws, stream), torch.bfloat16
    c = batch.c
    pg, need = _paged(batch, pages, dev)
    layers, rows = _layered("kv", kv, D_QK) if kv is not None else (1, need)
    if k_idx is not None:
        other = _layered("k_idx", k_idx, D_IDX)
        if kv is not None and other != (layers, rows):
            raise ValueError("kv and k_idx: the same layers and rows expected")
        layers, rows = other
    _check(load_library().dsa_tree_commit(
        ctypes.byref(c), pg, _typed("mask", mask, torch.int64, c.total_q, dev),
        _typed("accepted", accepted, torch.int32, c.batch, dev), layers, rows,
        _typed("kv", kv, bf16, layers * rows * D_QK, dev), _typed("k_idx", k_idx, bf16, layers * rows * D_IDX, dev),
        _typed("ctx_new", ctx_new, torch.int32, c.batch, dev), ws.data_ptr(), ws.numel(), _raw_stream(stream, dev)),
        "dsa_tree_commit")
    return ctx_new


# ---- Prompts over the latent cache, and sequences behind a shared prefix ----

class RopeScaling:
    """Host handle of a dsa_rope_scaling: frequencies divided by `factor`, all
    of them (original_ctx 0) or by parts (YaRN), and cos and sin times mscale."""

    def __init__(self, factor: float, original_ctx: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                 mscale: float = 1.0):
        self.c = DsaRopeScaling(float(factor), int(original_ctx), float(beta_fast), float(beta_slow), float(mscale))


def rope_table(cos, sin, base: float, first: int = 0, scaling: Optional[RopeScaling] = None, stream=None):
    """Fills cos and sin fp32 [rows, dim] with the rotary rows of positions
    first, first + 1, .. (see dsa_rope_table)."""
    dev = cos.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice() or (stream is not None and stream.device_index != dev):
        raise ValueError(f"cos on {cos.device}: expected on the current CUDA device, and the stream's")
    if cos.dim() != 2 or sin.shape != cos.shape:
        raise ValueError("cos, sin: [rows, dim] of one shape expected")
    rows, dim = cos.shape
    _check(load_library().dsa_rope_table(
        rows, int(first), dim, float(base), ctypes.byref(scaling.c) if scaling is not None else None,
        _typed("cos", cos, torch.float32, rows * dim, dev), _typed("sin", sin, torch.float32, rows * dim, dev),
        _raw_stream(stream, dev)), "dsa_rope_table")
    return cos, sin


def _heads(name: str, t: torch.Tensor, dtype: torch.dtype, dev: int):
    """The shape of a tensor [total_q, heads, dim] of any strides but a unit one in its last dimension."""
    if t.dtype is not dtype or t.get_device() != dev:
        raise TypeError(f"{name}: {dtype} tensor on cuda:{dev} expected")
    if t.dim() != 3 or (t.stride(2) != 1 and t.shape[2] > 1):
        raise ValueError(f"{name}: [total_q, heads, dim] with unit stride in the last dimension expected")
    return t.shape


def rope(x, cos, sin, positions, out=None, interleaved: bool = False, inverse: bool = False, ws=None, stream=None):
    """Rotates x [total_q, heads, dim] (any strides, unit in the last
    dimension: a slice of wider heads) into out, or in place (see dsa_rope).
    interleaved: neighbours as pairs instead of the halves."""
    dev, f32, bf16 = _here("dsa_rope", ws, stream), torch.float32, torch.bfloat16
    if out is None:
        out = x
    total_q, heads, dim = shape = _heads("x", x, bf16, dev)
    if out is not x and _heads("out", out, bf16, dev) != shape:
        raise ValueError("x, out: one shape expected")
    rows = cos.shape[0]
    if cos.shape != (rows, dim) or sin.shape != (rows, dim):
        raise ValueError(f"cos, sin: [table_rows, {dim}] expected")
    if heads == 0:
        return out
    # the stride of a dimension of one element means nothing
    xt, xh, _ = x.stride()
    ot, oh, _ = out.stride()
    if total_q <= 1:
        xt = ot = 0
    if heads == 1:
        xh = oh = 0
    _check(load_library().dsa_rope(
        total_q, heads, dim, x.data_ptr(), xt, xh, _typed("cos", cos, f32, rows * dim, dev),
        _typed("sin", sin, f32, rows * dim, dev), rows, _typed("positions", positions, torch.int32, total_q, dev),
        (1 if interleaved else 0) | (2 if inverse else 0), out.data_ptr(), ot, oh, ws.data_ptr(), ws.numel(),
        _raw_stream(stream, dev)), "dsa_rope")
    return out


class Expanded:
    """Host handle of a dsa_expanded.  Keeps its buffers alive."""

    def __init__(self, off: torch.Tensor, kv: torch.Tensor, k_pe: torch.Tensor):
        dev = kv.get_device()
        rows = kv.shape[0] if kv.dim() >= 1 else 0
        if kv.numel() != rows * H * D_EXP or k_pe.numel() != rows * 64:
            raise ValueError("kv [rows, 64, 448] and k_pe [rows, 64] expected")
        if dev < 0:
            raise ValueError("device tensor expected")
        self.off, self.kv, self.k_pe = off, kv, k_pe
        self.c = DsaExpanded(rows, _typed("off", off, torch.int32, 1, dev), _typed("kv", kv, torch.bfloat16, 0, dev),
                             _typed("k_pe", k_pe, torch.bfloat16, 0, dev))


def make_expanded(off: torch.Tensor, kv: torch.Tensor, k_pe: torch.Tensor) -> Expanded:
    """Expanded rows: sequence b's begin at row off[b] (a multiple of 128) of kv [rows, 64, 448] and k_pe [rows, 64]."""
    return Expanded(off, kv, k_pe)


def prompt_workspace(batch: Batch, device="cuda") -> torch.Tensor:
    """A workspace of mla_expand and prompt_mla_fwd with a cleared status word."""
    n = ctypes.c_size_t(0)
    _check(load_library().dsa_prompt_workspace_size(ctypes.byref(batch.c), ctypes.byref(n)),
           "dsa_prompt_workspace_size")
    ws = torch.empty(int(n.value), dtype=torch.uint8, device=device)
    reset_device_status(ws)
    return ws


def _expanded(batch: Batch, x: Expanded, dev: int):
    if x.off.get_device() != dev:
        raise ValueError(f"expanded rows: expected on cuda:{dev}")
    if x.off.numel() <= batch.c.batch:
        raise ValueError("expanded rows: an offset for each sequence and one behind them expected")
    return ctypes.byref(x.c)


def mla_expand(batch: Batch, kv, w_kv_b, expanded: Expanded, first=None, pages: Optional[Pages] = None, ws=None,
               stream=None):
    """Expands cache rows first[b] .. ctx_len[b] - 1 of every sequence into
    each head's keys and values (see dsa_mla_expand)."""
    dev, bf16 = _here("dsa_mla_expand", ws, stream), torch.bfloat16
    pg, rows = _paged(batch, pages, dev)
    _check(load_library().dsa_mla_expand(
        ctypes.byref(batch.c), pg, _typed("kv", kv, bf16, rows * D_QK, dev),
        _typed("w_kv_b", w_kv_b, bf16, H * D_EXP * D_V, dev), _typed("first", first, torch.int32, batch.c.batch, dev),
        _expanded(batch, expanded, dev), ws.data_ptr(), ws.numel(), _raw_stream(stream, dev)), "dsa_mla_expand")
    return expanded


def prompt_mla_fwd(batch: Batch, q, expanded: Expanded, sm_scale: float, out, lse=None, ws=None, stream=None):
    """Causal attention of the new rows q [total_q, 64, 256] over expanded
    rows (see dsa_prompt_mla_fwd)."""
    dev, bf16 = _here("dsa_prompt_mla_fwd", ws, stream), torch.bfloat16
    c = batch.c
    _paged(batch, None, dev)
    _check(load_library().dsa_prompt_mla_fwd(
        ctypes.byref(c), _typed("q", q, bf16, c.total_q * H * D_HEAD, dev), _expanded(batch, expanded, dev),
        float(sm_scale), _typed("out", out, bf16, c.total_q * H * D_HEAD, dev),
        _typed("lse", lse, torch.float32, c.total_q * H, dev), ws.data_ptr(), ws.numel(), _raw_stream(stream, dev)),
        "dsa_prompt_mla_fwd")
    return out


def mla_o_proj(o_mid, w_o, y, ws, stream=None):
    """y[t] = w_o o_mid[t] for attention results [total_q, 64, 256] (see dsa_mla_o_proj; ws: mla_workspace)."""
    dev, bf16 = _here("dsa_mla_o_proj", ws, stream), torch.bfloat16
    total_q = o_mid.shape[0]
    _check(load_library().dsa_mla_o_proj(
        int(total_q), _typed("o_mid", o_mid, bf16, total_q * H * D_HEAD, dev),
        _typed("w_o", w_o, bf16, D_HIDDEN * H * D_HEAD, dev), _typed("y", y, bf16, total_q * D_HIDDEN, dev),
        ws.data_ptr(), ws.numel(), _raw_stream(stream, dev)), "dsa_mla_o_proj")
    return y


class Groups:
    """Host handle of a dsa_groups.  Keeps its device arrays alive."""

    def __init__(self, off: torch.Tensor, shared: torch.Tensor):
        dev, n = off.get_device(), shared.numel()
        if dev < 0:
            raise ValueError("device tensor expected")
        self.off, self.shared = off, shared
        self.c = DsaGroups(n, _typed("off", off, torch.int32, n + 1, dev), _typed("shared", shared, torch.int32, 0, dev))


def make_groups(off: torch.Tensor, shared: torch.Tensor) -> Groups:
    """Groups of consecutive sequences off[g] .. off[g + 1] - 1 whose first shared[g] cache rows are the same."""
    return Groups(off, shared)


def prefix_workspace(batch: Batch, groups: Groups, device="cuda") -> torch.Tensor:
    """A workspace of prefix_mla_fwd with a cleared status word."""
    n = ctypes.c_size_t(0)
    _check(load_library().dsa_prefix_workspace_size(ctypes.byref(batch.c), ctypes.byref(groups.c), ctypes.byref(n)),
           "dsa_prefix_workspace_size")
    ws = torch.empty(int(n.value), dtype=torch.uint8, device=device)
    reset_device_status(ws)
    return ws


def prefix_mla_fwd(batch: Batch, groups: Groups, q, kv, mask, sm_scale: float, out, lse=None,
                   pages: Optional[Pages] = None, ws=None, stream=None):
    """tree_mla_fwd for groups of sequences that share their first rows, which
    are read once a group (see dsa_prefix_mla_fwd).  mask None: a chain."""
    dev, bf16 = _here("dsa_prefix_mla_fwd", ws, stream), torch.bfloat16
    c = batch.c
    pg, rows = _paged(batch, pages, dev)
    if groups.off.get_device() != dev:
        raise ValueError(f"groups: expected on cuda:{dev}")
    _check(load_library().dsa_prefix_mla_fwd(
        ctypes.byref(c), ctypes.byref(groups.c), pg, _typed("q", q, bf16, c.total_q * H * D_QK, dev),
        _typed("kv", kv, bf16, rows * D_QK, dev), _typed("mask", mask, torch.int64, c.total_q, dev), float(sm_scale),
        _typed("out", out, bf16, c.total_q * H * D_V, dev), _typed("lse", lse, torch.float32, c.total_q * H, dev),
        ws.data_ptr(), ws.numel(), _raw_stream(stream, dev)), "dsa_prefix_mla_fwd")
    return out
