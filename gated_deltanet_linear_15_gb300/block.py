"""Operators that a hybrid stack puts next to its gated delta-rule layers: Python binding of include/gdn_block.h.

``paged_attention`` (attention of new tokens over a paged key/value cache), ``rotary_table`` / ``rotary`` /
``rotary_embedding`` / ``rotary_append`` (rotary positions, their gradient, and the write of new keys and values into
the cache), ``extend_pages`` / ``fork_pages`` / ``free_pages`` / ``compact_pages`` / ``copy_slots`` (the cache's
upkeep), ``rms_norm`` / ``rms_norm_bwd`` / ``residual_rms_norm`` (the residual stream's norm, optionally with an 8-bit
output).  As in the rest of the package, everything runs in the library's CUDA kernels on the current stream, and this
module only marshals arguments; bad arguments raise ``ValueError`` (found here) or ``RuntimeError`` (found by the
library, with its reason).
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple, Optional, Sequence

import torch

from . import _lib
from ._lib import GdnNormShape, GdnPagedShape, GdnPagesShape, GdnRotaryShape, GdnSlotPool

__all__ = ["paged_attention", "paged_attention_status", "rotary_frequencies", "rotary_table", "rotary", "rotary_embedding", "rotary_append",
           "extend_pages", "fork_pages", "free_pages", "compact_pages", "copy_slots", "rms_norm", "rms_norm_bwd",
           "residual_rms_norm", "NormOutput"]

_DTYPES = {torch.bfloat16: _lib.GDN_BF16, torch.float32: _lib.GDN_FP32}
_byref = ctypes.byref


def _check(rc: int, what: str):
    if rc != 0:
        lib = _lib.load()
        raise RuntimeError(f"{what}: {lib.gdn_status_string(rc).decode()} ({_lib.last_error()})")


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _dtype(t, what):
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ValueError(f"{what} must be bfloat16 or float32 (got {t.dtype})")
    return d


def _heads(t, what, dtype=None):
    """A [tokens, heads, features] tensor with contiguous features on the current GPU."""
    if t.dim() != 3:
        raise ValueError(f"{what} must have 3 dimensions [tokens, heads, features]")
    _features(t, what)
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype} like the others (got {t.dtype})")


def _features(t, what):
    if not t.is_cuda or t.device.index != torch.cuda.current_device():
        raise ValueError(f"{what} must be on the current CUDA device")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"the last dimension of {what} must be contiguous")


def _ints(t, what, shape=None):
    if t.dtype != torch.int32 or not t.is_cuda or t.device.index != torch.cuda.current_device():
        raise ValueError(f"{what} must be an int32 tensor on the current CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)} (got {tuple(t.shape)})")


def _workspace(nbytes, device):
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ paged cache
def _paged_shape(q, k_cache, v_cache, page_table, kv_lens, cu_q):
    _heads(q, "q")
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must have one shape [pages, page_size, kv heads, features]")
    _features(k_cache, "k_cache")
    _features(v_cache, "v_cache")
    dt = _dtype(q, "q")
    if k_cache.dtype != q.dtype or v_cache.dtype != q.dtype:
        raise ValueError("q, k_cache and v_cache must have one dtype")
    if k_cache.shape[3] != q.shape[2]:
        raise ValueError("q and the caches must have the same number of features")
    if page_table.dim() != 2 or page_table.dtype != torch.int32 or not page_table.is_cuda or \
            (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("page_table must be an int32 CUDA tensor [sequences, pages] with contiguous rows")
    n = page_table.shape[0]
    _ints(kv_lens, "kv_lens", (n,))
    if cu_q is not None:
        _ints(cu_q, "cu_q", (n + 1,))
    s = GdnPagedShape()
    s.num_seqs, s.total_q, s.num_heads, s.num_kv_heads, s.head_dim = n, q.shape[0], q.shape[1], k_cache.shape[2], q.shape[2]
    s.num_pages, s.page_size, s.max_pages, s.dtype = k_cache.shape[0], k_cache.shape[1], page_table.shape[1], dt
    s.table_stride = max(page_table.stride(0), s.max_pages)
    s.q_tok, s.q_head = q.stride(0), q.stride(1)
    s.k_page, s.k_tok, s.k_head = k_cache.stride()[:3]
    s.v_page, s.v_tok, s.v_head = v_cache.stride()[:3]
    return s


def paged_attention(q, k_cache, v_cache, page_table, kv_lens, cu_q=None, max_q: int = 0, scale: Optional[float] = None,
                    window: int = 0, return_lse: bool = False, out=None, workspace=None):
    """Causal attention of new tokens over a paged cache that already holds their keys and values.

    q [new tokens, heads, D]; k_cache, v_cache [pages, page_size, kv heads, D] (any strides with contiguous features);
    page_table int32 [sequences, pages]; kv_lens int32 [sequences], the tokens of each sequence with the new ones;
    cu_q int32 [sequences + 1], where each sequence's new tokens begin in q (None: as many for each).  max_q: the most
    new tokens of a sequence, if known on the host (it only picks the kernel).  window > 0: a query sees that many
    keys.  Returns o like q, or (o, lse) with lse fp32 [new tokens, heads]; a query without keys has o = 0 and
    lse = -inf.  Decoding is the case of one new token per sequence."""
    s = _paged_shape(q, k_cache, v_cache, page_table, kv_lens, cu_q)
    s.max_q, s.window = int(max_q), int(window)
    s.scale = 1.0 / math.sqrt(q.shape[2]) if scale is None else float(scale)
    o = torch.empty(q.shape, dtype=q.dtype, device=q.device) if out is None else out
    if out is not None:
        _heads(out, "out", q.dtype)
        if out.shape != q.shape:
            raise ValueError("out must have the shape of q")
    s.o_tok, s.o_head = o.stride(0), o.stride(1)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device) if return_lse else None
    lib = _lib.load()
    need = lib.gdn_paged_attn_workspace_size(_byref(s))
    if need == 0:
        _check(_lib.GDN_ERR_INVALID_ARG, "gdn_paged_attn_workspace_size")
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = _workspace(need, q.device)
    _check(lib.gdn_paged_attn_fwd(_byref(s), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(),
                                  None if cu_q is None else cu_q.data_ptr(), kv_lens.data_ptr(), o.data_ptr(),
                                  None if lse is None else lse.data_ptr(), workspace.data_ptr(),
                                  workspace.numel() * workspace.element_size(), _stream()), "gdn_paged_attn_fwd")
    return (o, lse) if return_lse else o


def paged_attention_status(q, k_cache, v_cache, page_table, kv_lens, workspace, cu_q=None, max_q: int = 0) -> int:
    """Status word of the last ``paged_attention`` call with these arguments and this workspace (0: clean; see
    gdn_paged_attn_status).  Synchronises the stream."""
    s = _paged_shape(q, k_cache, v_cache, page_table, kv_lens, cu_q)
    s.max_q, s.scale, s.o_tok, s.o_head = int(max_q), 1.0, q.stride(0), q.stride(1)
    return int(_lib.load().gdn_paged_attn_status(_byref(s), workspace.data_ptr(), _stream()))


# ------------------------------------------------------------------ rotary positions
def rotary_frequencies(rot: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                       context: int = 0, fast: float = 32.0, slow: float = 1.0):
    """(fp64 angles per position [rot / 2], amplitude) of a rotary embedding over `rot` features.

    scaling None: base^(-2 i / rot).  "linear": positions stretched by `factor`.  "base": the base raised so that the
    slowest pair is stretched by `factor` and the fastest is kept.  "parts": pairs that turn fewer than `slow` times over
    the original `context` are stretched, those that turn more than `fast` times are kept, the ones between are blended;
    the amplitude grows by 0.1 ln(factor) + 1."""
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and at least 2")
    if factor <= 0 or base <= 1:
        raise ValueError("need factor > 0 and base > 1")
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    if scaling is None:
        return base ** (-i / rot), 1.0
    if scaling == "linear":
        return base ** (-i / rot) / factor, 1.0
    if scaling == "base":
        if rot < 4:
            raise ValueError('scaling "base" needs rot >= 4')
        return (base * factor ** (rot / (rot - 2))) ** (-i / rot), 1.0
    if scaling == "parts":
        if context < 1 or not fast > slow > 0:
            raise ValueError('scaling "parts" needs context >= 1 and fast > slow > 0')
        freq = base ** (-i / rot)
        turns = context * freq / (2 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0, 1)
        return freq * keep + freq / factor * (1 - keep), 0.1 * math.log(factor) + 1 if factor > 1 else 1.0
    raise ValueError(f"unknown scaling {scaling!r}")


def rotary_table(positions: int, rot: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                 context: int = 0, fast: float = 32.0, slow: float = 1.0, device="cuda"):
    """The (cos, sin) table [positions, rot / 2, 2] fp32 of ``rotary_frequencies``, built once on the GPU in fp64."""
    freq, amplitude = rotary_frequencies(rot, base, scaling, factor, context, fast, slow)
    freq = freq.to(device)
    table = torch.empty(positions, rot // 2, 2, dtype=torch.float32, device=device)
    _check(_lib.load().gdn_rotary_table(freq.data_ptr(), rot // 2, positions, amplitude, table.data_ptr(), _stream()),
           "gdn_rotary_table")
    return table


def _rot_table(table):
    if table.dim() != 3 or table.shape[2] != 2 or table.dtype != torch.float32 or not table.is_cuda or not table.is_contiguous():
        raise ValueError("table must be a contiguous fp32 CUDA tensor [positions, rot / 2, 2]")


def rotary(q, k, table, positions, interleaved: bool = False, inverse: bool = False, inplace: bool = False):
    """q [T, heads, D] and k [T, heads, D] (or None) turned by the table's angles of positions int32 [T]; pairs of
    features (i, i + rot / 2), or (2 i, 2 i + 1) when interleaved, over the first rot = 2 table.shape[1] features.
    inverse turns back, which is also the gradient.  Returns (q, k)."""
    _rot_table(table)
    s = GdnRotaryShape()
    s.tokens, s.q_heads, s.k_heads = q.shape[0], q.shape[1], 0
    s.head_dim, s.rot, s.interleaved, s.inverse = q.shape[-1], 2 * table.shape[1], int(interleaved), int(inverse)
    s.table_rows, s.dtype = table.shape[0], _dtype(q, "q")
    _heads(q, "q")
    _ints(positions, "positions", (q.shape[0],))
    qo = q if inplace else torch.empty(q.shape, dtype=q.dtype, device=q.device)
    s.q_tok, s.q_head, s.qo_tok, s.qo_head = q.stride(0), q.stride(1), qo.stride(0), qo.stride(1)
    ko = None
    if k is not None:
        _heads(k, "k", q.dtype)
        if k.shape[0] != q.shape[0] or k.shape[2] != q.shape[2]:
            raise ValueError("q and k must have the same tokens and features")
        s.k_heads = k.shape[1]
        ko = k if inplace else torch.empty(k.shape, dtype=k.dtype, device=k.device)
        s.k_tok, s.k_head, s.ko_tok, s.ko_head = k.stride(0), k.stride(1), ko.stride(0), ko.stride(1)
    _check(_lib.load().gdn_rotary(_byref(s), q.data_ptr(), None if k is None else k.data_ptr(), table.data_ptr(),
                                  positions.data_ptr(), qo.data_ptr(), None if ko is None else ko.data_ptr(), _stream()),
           "gdn_rotary")
    return qo, ko


class RotaryFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, table, positions, interleaved):
        ctx.save_for_backward(table, positions)
        ctx.interleaved = interleaved
        return rotary(q, k, table, positions, interleaved)

    @staticmethod
    def backward(ctx, dq, dk):
        table, positions = ctx.saved_tensors
        dq, dk = rotary(dq.contiguous(), dk.contiguous(), table, positions, ctx.interleaved, inverse=True)
        return dq, dk, None, None, None


def rotary_embedding(q, k, table, positions, interleaved: bool = False):
    """``rotary`` with gradients for q and k."""
    return RotaryFunction.apply(q, k, table, positions, interleaved)


def rotary_append(q, k, v, table, k_cache, v_cache, page_table, kv_lens, cu_q=None, interleaved: bool = False, out=None):
    """Turns the new tokens' q and k by their positions, writes k and v into their cache slots and returns the turned q.

    q [new tokens, heads, D], k, v [new tokens, kv heads, D], as slices of one projection if need be.  The caches,
    page_table, kv_lens and cu_q are those of ``paged_attention``: kv_lens counts the new tokens already."""
    s = _paged_shape(q, k_cache, v_cache, page_table, kv_lens, cu_q)
    _heads(k, "k", q.dtype)
    _heads(v, "v", q.dtype)
    if k.shape != (q.shape[0], s.num_kv_heads, q.shape[2]) or v.shape != k.shape:
        raise ValueError("k and v must be [new tokens, kv heads, features]")
    _rot_table(table)
    o = torch.empty(q.shape, dtype=q.dtype, device=q.device) if out is None else out
    if out is not None:
        _heads(out, "out", q.dtype)
        if out.shape != q.shape:
            raise ValueError("out must have the shape of q")
    s.o_tok, s.o_head = o.stride(0), o.stride(1)
    s.kn_tok, s.kn_head, s.vn_tok, s.vn_head = k.stride(0), k.stride(1), v.stride(0), v.stride(1)
    s.rot, s.interleaved, s.table_rows = 2 * table.shape[1], int(interleaved), table.shape[0]
    _check(_lib.load().gdn_rotary_append(_byref(s), q.data_ptr(), k.data_ptr(), v.data_ptr(), table.data_ptr(),
                                         k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(),
                                         None if cu_q is None else cu_q.data_ptr(), kv_lens.data_ptr(), o.data_ptr(),
                                         _stream()), "gdn_rotary_append")
    return o


# ------------------------------------------------------------------ pages
def _pools(tensors: Sequence[torch.Tensor], what):
    arr = (GdnSlotPool * max(len(tensors), 1))()
    for i, t in enumerate(tensors):
        if not t.is_cuda or t.device.index != torch.cuda.current_device() or t.dim() < 1:
            raise ValueError(f"{what} must be tensors on the current CUDA device")
        n = t.shape[0]
        if n and not t[0].is_contiguous():
            raise ValueError(f"each slot of {what} must be contiguous")
        size = t.element_size()
        nbytes = t[0].numel() * size if n else 0
        arr[i].base, arr[i].bytes, arr[i].slots = t.data_ptr(), nbytes, n
        arr[i].stride = t.stride(0) * size if n > 1 else nbytes
    return arr


def _pages_shape(page_table, refcount, page_size):
    if page_table.dim() != 2 or page_table.dtype != torch.int32 or not page_table.is_cuda or \
            (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("page_table must be an int32 CUDA tensor [sequences, pages] with contiguous rows")
    _ints(refcount, "refcount")
    s = GdnPagesShape()
    s.num_seqs, s.max_pages = page_table.shape
    s.num_pages, s.page_size = refcount.numel(), int(page_size)
    s.table_stride = max(page_table.stride(0), s.max_pages)
    return s


def _pages_workspace(s, m, device):
    need = _lib.load().gdn_pages_workspace_size(_byref(s), m)
    if need == 0:
        _check(_lib.GDN_ERR_INVALID_ARG, "gdn_pages_workspace_size")
    return _workspace(need, device)


def extend_pages(page_table, seq_lens, refcount, seqs, add, page_size: int):
    """Grows sequences seqs int32 [m] by add int32 [m] tokens, taking the free pages of lowest number in list order.
    Returns ok int32 [m]: 1, or 0 where a sequence stays as it was (no room, no pages, a shared last page)."""
    s = _pages_shape(page_table, refcount, page_size)
    _ints(seq_lens, "seq_lens", (s.num_seqs,))
    _ints(seqs, "seqs")
    _ints(add, "add", seqs.shape)
    m = seqs.numel()
    ok = torch.empty_like(seqs)
    ws = _pages_workspace(s, m, seqs.device)
    _check(_lib.load().gdn_pages_extend(_byref(s), page_table.data_ptr(), seq_lens.data_ptr(), refcount.data_ptr(),
                                        seqs.data_ptr(), add.data_ptr(), m, ok.data_ptr(), ws.data_ptr(), ws.numel(),
                                        _stream()), "gdn_pages_extend")
    return ok


def fork_pages(page_table, seq_lens, refcount, parents, children, pools=(), page_size: int = 16, states=()):
    """Makes each (empty) child sequence a copy of its parent: full pages shared, a partly filled last page copied to a
    new page in every pool [pages, ...], slot `child` of every states tensor [sequences, ...] a copy of slot `parent`
    (the recurrent states of delta-rule layers).  Returns int32 [m]: the new page, -1 where none was needed, -2 where
    the fork was left out."""
    s = _pages_shape(page_table, refcount, page_size)
    _ints(seq_lens, "seq_lens", (s.num_seqs,))
    _ints(parents, "parents")
    _ints(children, "children", parents.shape)
    m = parents.numel()
    new = torch.empty_like(parents)
    ws = _pages_workspace(s, m, parents.device)
    _check(_lib.load().gdn_pages_fork(_byref(s), page_table.data_ptr(), seq_lens.data_ptr(), refcount.data_ptr(),
                                      parents.data_ptr(), children.data_ptr(), m, _pools(pools, "pools"), len(pools),
                                      _pools(states, "states"), len(states), new.data_ptr(), ws.data_ptr(), ws.numel(),
                                      _stream()), "gdn_pages_fork")
    return new


def free_pages(page_table, seq_lens, refcount, seqs):
    """Ends sequences: each of their pages loses one reference, their rows become -1 and their lengths 0."""
    s = _pages_shape(page_table, refcount, 1)
    _ints(seq_lens, "seq_lens", (s.num_seqs,))
    _ints(seqs, "seqs")
    _check(_lib.load().gdn_pages_free(_byref(s), page_table.data_ptr(), seq_lens.data_ptr(), refcount.data_ptr(),
                                      seqs.data_ptr(), seqs.numel(), _stream()), "gdn_pages_free")


def compact_pages(page_table, refcount, pools=(), inplace: bool = True):
    """Moves the pages in use to the lowest numbers, in every pool and in the table.  Returns (page_table, refcount,
    moves): the inputs themselves, updated, or with inplace=False new ones; moves int32 scalar tensor."""
    s = _pages_shape(page_table, refcount, 1)
    table = page_table if inplace else torch.empty_strided(page_table.shape, (s.table_stride, 1), dtype=torch.int32,
                                                           device=page_table.device)
    ref = refcount if inplace else torch.empty_like(refcount)
    moves = torch.empty((), dtype=torch.int32, device=refcount.device)
    ws = _pages_workspace(s, 0, refcount.device)
    _check(_lib.load().gdn_pages_compact(_byref(s), page_table.data_ptr(), refcount.data_ptr(), table.data_ptr(),
                                         ref.data_ptr(), _pools(pools, "pools"), len(pools), moves.data_ptr(),
                                         ws.data_ptr(), ws.numel(), _stream()), "gdn_pages_compact")
    return table, ref, moves


def copy_slots(pools, src, dst):
    """Copies slot src[i] to slot dst[i] (int32 [m]) in every tensor [slots, ...]; no dst twice or among the src."""
    _ints(src, "src")
    _ints(dst, "dst", src.shape)
    _check(_lib.load().gdn_slots_copy(_pools(pools, "pools"), len(pools), src.data_ptr(), dst.data_ptr(), src.numel(),
                                      _stream()), "gdn_slots_copy")


# ------------------------------------------------------------------ root-mean-square norm
class NormOutput(NamedTuple):
    y: torch.Tensor                   # the normed rows, e4m3 with fp8=True
    h: torch.Tensor                   # x + residual in x's dtype (x itself without a residual)
    scale: Optional[torch.Tensor]     # fp8: fp32 [rows, dim / group], or [rows, 1]
    rstd: torch.Tensor                # fp32 [rows]


def _rows(t, what, like=None):
    """(2-d view of [..., dim], row stride): copies nothing."""
    _features(t, what)
    if like is not None and (t.shape != like.shape or t.dtype != like.dtype):
        raise ValueError(f"{what} must have the shape and dtype of the other inputs")
    v = t.view(-1, t.shape[-1]) if t.dim() != 2 else t
    return v, v.stride(0)


def _norm_weight(weight, dim):
    if weight.dtype != torch.float32 or tuple(weight.shape) != (dim,) or not weight.is_cuda or not weight.is_contiguous():
        raise ValueError("weight must be a contiguous fp32 CUDA tensor [dim]")


def rms_norm(x, weight, residual=None, eps: float = 1e-6, fp8: bool = False, group: int = 0, weight_offset: float = 0.0,
             inplace: bool = False) -> NormOutput:
    """h = x + residual, y = h / sqrt(mean(h^2) + eps) * (weight + weight_offset) over the last dimension.

    x, residual [..., dim]; weight fp32 [dim].  fp8: y in e4m3 with one scale per row, or per `group` = 128 features;
    the normed values are y * scale.  inplace: h takes residual's place."""
    x2, xs = _rows(x, "x")
    T, D = x2.shape
    _norm_weight(weight, D)
    s = GdnNormShape()
    s.rows, s.dim, s.dtype, s.fp8, s.group = T, D, _dtype(x, "x"), int(fp8), int(group)
    s.eps, s.weight_offset, s.x_row = eps, weight_offset, xs
    h, r2 = x, None
    if residual is not None:
        r2, s.r_row = _rows(residual, "residual", x)
        h = residual if inplace else torch.empty(x.shape, dtype=x.dtype, device=x.device)
        s.h_row = r2.stride(0) if inplace else D
    y = torch.empty(x.shape, dtype=torch.float8_e4m3fn if fp8 else x.dtype, device=x.device)
    s.y_row = D
    scale = torch.empty(*x.shape[:-1], D // group if group else 1, dtype=torch.float32, device=x.device) if fp8 else None
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    _check(_lib.load().gdn_rmsnorm_fwd(_byref(s), x2.data_ptr(), None if r2 is None else r2.data_ptr(), weight.data_ptr(),
                                       None if r2 is None else h.data_ptr(), y.data_ptr(),
                                       None if scale is None else scale.data_ptr(), rstd.data_ptr(), _stream()),
           "gdn_rmsnorm_fwd")
    return NormOutput(y, h, scale, rstd)


def rms_norm_bwd(dy, h, weight, rstd, dh=None, weight_offset: float = 0.0):
    """(dx, dw): the gradient of x (and of residual), and of weight (fp32), from dy, the forward's h and rstd, and dh,
    the gradient that reaches h along the residual stream."""
    g2, gs = _rows(dy, "dy")
    h2, hs = _rows(h, "h", dy)
    T, D = g2.shape
    _norm_weight(weight, D)
    if rstd.dtype != torch.float32 or rstd.numel() != T or not rstd.is_contiguous():
        raise ValueError("rstd must be a contiguous fp32 tensor with one value per row")
    s = GdnNormShape()
    s.rows, s.dim, s.dtype, s.weight_offset = T, D, _dtype(dy, "dy"), weight_offset
    s.x_row, s.y_row, s.h_row = hs, gs, D
    e2 = None
    if dh is not None:
        e2, s.r_row = _rows(dh, "dh", dy)
    dx = torch.empty(dy.shape, dtype=dy.dtype, device=dy.device)
    dw = torch.empty(D, dtype=torch.float32, device=dy.device)
    lib = _lib.load()
    need = lib.gdn_rmsnorm_bwd_workspace_size(_byref(s))
    if need == 0:
        _check(_lib.GDN_ERR_INVALID_ARG, "gdn_rmsnorm_bwd_workspace_size")
    ws = _workspace(need, dy.device)
    _check(lib.gdn_rmsnorm_bwd(_byref(s), g2.data_ptr(), h2.data_ptr(), weight.data_ptr(), rstd.data_ptr(),
                               None if e2 is None else e2.data_ptr(), dx.data_ptr(), dw.data_ptr(), ws.data_ptr(),
                               ws.numel(), _stream()), "gdn_rmsnorm_bwd")
    return dx, dw


class ResidualRMSNormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps, weight_offset):
        r = rms_norm(x, weight, residual, eps, weight_offset=weight_offset)
        ctx.save_for_backward(r.h, weight, r.rstd)
        ctx.weight_offset, ctx.has_residual = weight_offset, residual is not None
        if residual is None:
            return r.y
        return r.y, r.h

    @staticmethod
    def backward(ctx, dy, dh=None):
        h, weight, rstd = ctx.saved_tensors
        dx, dw = rms_norm_bwd(dy.contiguous(), h, weight, rstd, None if dh is None else dh.contiguous(), ctx.weight_offset)
        return dx, dx if ctx.has_residual else None, dw, None, None


def residual_rms_norm(x, weight, residual=None, eps: float = 1e-6, weight_offset: float = 0.0):
    """``rms_norm`` with gradients: (y, h), or y alone without a residual."""
    return ResidualRMSNormFunction.apply(x, residual, weight, eps, weight_offset)
