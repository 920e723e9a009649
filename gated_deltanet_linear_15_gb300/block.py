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
_empty = torch.empty
_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream

# Checked arguments of earlier calls: sizes, strides, types and devices of a call -> its shape struct and workspace
# size (no addresses, no contents).  A decode step repeats the same sizes, and building and checking the struct anew
# costs more host time than the launch.
_known = {}


def _remember(key, value):
    if len(_known) >= 4096:
        _known.clear()
    _known[key] = value
    return value


def _meta(t):
    """What a call's checks depend on, of one tensor."""
    return t.shape, t.stride(), t.dtype, t.get_device()


def _check(rc: int, what: str):
    if rc != 0:
        lib = _lib.load()
        raise RuntimeError(f"{what}: {lib.gdn_status_string(rc).decode()} ({_lib.last_error()})")


def _dtype(t, what):
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ValueError(f"{what} must be bfloat16 or float32 (got {t.dtype})")
    return d


def _here(t, what):
    if not t.is_cuda or t.get_device() != _device():
        raise ValueError(f"{what} must be on the current CUDA device")


def _features(t, what):
    _here(t, what)
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"the last dimension of {what} must be contiguous")


def _heads(t, what, dtype=None):
    """A [tokens, heads, features] tensor with contiguous features on the current GPU."""
    if t.dim() != 3:
        raise ValueError(f"{what} must have 3 dimensions [tokens, heads, features]")
    _features(t, what)
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype} like the others (got {t.dtype})")


def _ints(t, what, shape=None):
    if t.dtype != torch.int32 or not t.is_cuda or t.get_device() != _device():
        raise ValueError(f"{what} must be an int32 tensor on the current CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)} (got {tuple(t.shape)})")


def _page_table(t):
    if t.dim() != 2 or t.dtype != torch.int32 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("page_table must be an int32 CUDA tensor [sequences, pages] with contiguous rows")
    _here(t, "page_table")


def _workspace(nbytes, device):
    return _empty(max(nbytes, 256), dtype=torch.uint8, device=device)


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
    _page_table(page_table)
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


def _like_q(out, q):
    if out is None:
        s = torch.empty(q.shape, dtype=q.dtype, device="meta").stride()
    else:
        _heads(out, "out", q.dtype)
        if out.shape != q.shape:
            raise ValueError("out must have the shape of q")
        s = out.stride()
    return s[0], s[1]


def paged_attention(q, k_cache, v_cache, page_table, kv_lens, cu_q=None, max_q: int = 0, scale: Optional[float] = None,
                    window: int = 0, return_lse: bool = False, out=None, workspace=None):
    """Causal attention of new tokens over a paged cache that already holds their keys and values.

    q [new tokens, heads, D]; k_cache, v_cache [pages, page_size, kv heads, D] (any strides with contiguous features);
    page_table int32 [sequences, pages]; kv_lens int32 [sequences], the tokens of each sequence with the new ones;
    cu_q int32 [sequences + 1], where each sequence's new tokens begin in q (None: as many for each).  max_q: the most
    new tokens of a sequence, if known on the host (it only picks the kernel).  window > 0: a query sees that many
    keys.  Returns o like q, or (o, lse) with lse fp32 [new tokens, heads]; a query without keys has o = 0 and
    lse = -inf.  Decoding is the case of one new token per sequence."""
    key = ("attn", _meta(q), _meta(k_cache), _meta(v_cache), _meta(page_table), _meta(kv_lens),
           None if cu_q is None else _meta(cu_q), None if out is None else _meta(out), max_q, scale, window, _device())
    known = _known.get(key)
    if known is None:
        s = _paged_shape(q, k_cache, v_cache, page_table, kv_lens, cu_q)
        s.max_q, s.window = int(max_q), int(window)
        s.scale = 1.0 / math.sqrt(q.shape[2]) if scale is None else float(scale)
        s.o_tok, s.o_head = _like_q(out, q)
        lib = _lib.load()
        need = lib.gdn_paged_attn_workspace_size(_byref(s))
        if need == 0:
            _check(_lib.GDN_ERR_INVALID_ARG, "gdn_paged_attn_workspace_size")
        known = _remember(key, (_byref(s), need, lib.gdn_paged_attn_fwd))
    shape, need, call = known
    dev = q.device
    o = _empty(q.shape, dtype=q.dtype, device=dev) if out is None else out
    lse = _empty(q.shape[:2], dtype=torch.float32, device=dev) if return_lse else None
    if workspace is None or workspace.nbytes < need:
        workspace = _empty(need, dtype=torch.uint8, device=dev)
    rc = call(shape, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(),
              None if cu_q is None else cu_q.data_ptr(), kv_lens.data_ptr(), o.data_ptr(),
              None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.nbytes, _raw_stream(dev.index))
    if rc:
        _check(rc, "gdn_paged_attn_fwd")
    return (o, lse) if return_lse else o


def paged_attention_status(q, k_cache, v_cache, page_table, kv_lens, workspace, cu_q=None, max_q: int = 0) -> int:
    """Status word of the last ``paged_attention`` call with these arguments and this workspace (0: clean; see
    gdn_paged_attn_status).  Synchronises the stream."""
    s = _paged_shape(q, k_cache, v_cache, page_table, kv_lens, cu_q)
    s.max_q, s.scale, s.o_tok, s.o_head = int(max_q), 1.0, q.stride(0), q.stride(1)
    return int(_lib.load().gdn_paged_attn_status(_byref(s), workspace.data_ptr(), _raw_stream(_device())))


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
    _check(_lib.load().gdn_rotary_table(freq.data_ptr(), rot // 2, positions, amplitude, table.data_ptr(),
                                        _raw_stream(_device())),
           "gdn_rotary_table")
    return table


def _rot_table(table):
    _here(table, "table")
    if table.dim() != 3 or table.shape[2] != 2 or table.dtype != torch.float32 or not table.is_contiguous():
        raise ValueError("table must be a contiguous fp32 CUDA tensor [positions, rot / 2, 2]")


def rotary(q, k, table, positions, interleaved: bool = False, inverse: bool = False, inplace: bool = False):
    """q [T, heads, D] and k [T, heads, D] (or None) turned by the table's angles of positions int32 [T]; pairs of
    features (i, i + rot / 2), or (2 i, 2 i + 1) when interleaved, over the first rot = 2 table.shape[1] features.
    inverse turns back, which is also the gradient.  Returns (q, k)."""
    key = ("rotary", _meta(q), None if k is None else _meta(k), _meta(table), _meta(positions), interleaved, inverse, inplace,
           _device())
    known = _known.get(key)
    if known is None:
        _rot_table(table)
        s = GdnRotaryShape()
        s.tokens, s.q_heads, s.k_heads = q.shape[0], q.shape[1], 0
        s.head_dim, s.rot, s.interleaved, s.inverse = q.shape[-1], 2 * table.shape[1], int(interleaved), int(inverse)
        s.table_rows, s.dtype = table.shape[0], _dtype(q, "q")
        _heads(q, "q")
        _ints(positions, "positions", (q.shape[0],))
        s.q_tok, s.q_head = q.stride(0), q.stride(1)
        s.qo_tok, s.qo_head = _like_q(q if inplace else None, q)
        if k is not None:
            _heads(k, "k", q.dtype)
            if k.shape[0] != q.shape[0] or k.shape[2] != q.shape[2]:
                raise ValueError("q and k must have the same tokens and features")
            s.k_heads, s.k_tok, s.k_head = k.shape[1], k.stride(0), k.stride(1)
            s.ko_tok, s.ko_head = _like_q(k if inplace else None, k)
        known = _remember(key, (_byref(s), _lib.load().gdn_rotary))
    shape, call = known
    dev = q.device
    qo = q if inplace else _empty(q.shape, dtype=q.dtype, device=dev)
    ko = k if inplace or k is None else _empty(k.shape, dtype=k.dtype, device=dev)
    rc = call(shape, q.data_ptr(), None if k is None else k.data_ptr(), table.data_ptr(), positions.data_ptr(),
              qo.data_ptr(), None if ko is None else ko.data_ptr(), _raw_stream(dev.index))
    if rc:
        _check(rc, "gdn_rotary")
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
    key = ("append", _meta(q), _meta(k), _meta(v), _meta(table), _meta(k_cache), _meta(v_cache), _meta(page_table),
           _meta(kv_lens), None if cu_q is None else _meta(cu_q), None if out is None else _meta(out), interleaved, _device())
    known = _known.get(key)
    if known is None:
        s = _paged_shape(q, k_cache, v_cache, page_table, kv_lens, cu_q)
        _heads(k, "k", q.dtype)
        _heads(v, "v", q.dtype)
        if k.shape != (q.shape[0], s.num_kv_heads, q.shape[2]) or v.shape != k.shape:
            raise ValueError("k and v must be [new tokens, kv heads, features]")
        _rot_table(table)
        s.o_tok, s.o_head = _like_q(out, q)
        s.kn_tok, s.kn_head, s.vn_tok, s.vn_head = k.stride(0), k.stride(1), v.stride(0), v.stride(1)
        s.rot, s.interleaved, s.table_rows = 2 * table.shape[1], int(interleaved), table.shape[0]
        known = _remember(key, (_byref(s), _lib.load().gdn_rotary_append))
    shape, call = known
    dev = q.device
    o = _empty(q.shape, dtype=q.dtype, device=dev) if out is None else out
    rc = call(shape, q.data_ptr(), k.data_ptr(), v.data_ptr(), table.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
              page_table.data_ptr(), None if cu_q is None else cu_q.data_ptr(), kv_lens.data_ptr(), o.data_ptr(),
              _raw_stream(dev.index))
    if rc:
        _check(rc, "gdn_rotary_append")
    return o


# ------------------------------------------------------------------ pages
def _pools(tensors: Sequence[torch.Tensor], what):
    arr = (GdnSlotPool * max(len(tensors), 1))()
    for i, t in enumerate(tensors):
        if t.dim() < 1:
            raise ValueError(f"{what} must be tensors of slots")
        _here(t, f"every tensor of {what}")
        n = t.shape[0]
        if n and not t[0].is_contiguous():
            raise ValueError(f"each slot of {what} must be contiguous")
        size = t.element_size()
        nbytes = t[0].numel() * size if n else 0
        arr[i].bytes, arr[i].slots = nbytes, n
        arr[i].stride = t.stride(0) * size if n > 1 else nbytes
    return arr


def _pool_bases(arr, tensors):
    """A call's own copy of a checked pool list, with the addresses of this call's tensors."""
    own = type(arr).from_buffer_copy(arr)
    for p, t in zip(own, tensors):
        p.base = t.data_ptr()
    return own


def _pages_shape(page_table, refcount, page_size):
    _page_table(page_table)
    _ints(refcount, "refcount")
    s = GdnPagesShape()
    s.num_seqs, s.max_pages = page_table.shape
    s.num_pages, s.page_size = refcount.numel(), int(page_size)
    s.table_stride = max(page_table.stride(0), s.max_pages)
    return s


def _pages_need(s, m):
    need = _lib.load().gdn_pages_workspace_size(_byref(s), m)
    if need == 0:
        _check(_lib.GDN_ERR_INVALID_ARG, "gdn_pages_workspace_size")
    return need


def extend_pages(page_table, seq_lens, refcount, seqs, add, page_size: int):
    """Grows sequences seqs int32 [m] by add int32 [m] tokens, taking the free pages of lowest number in list order.
    Returns ok int32 [m]: 1, or 0 where a sequence stays as it was (no room, no pages, a shared last page)."""
    key = ("extend", _meta(page_table), _meta(seq_lens), _meta(refcount), _meta(seqs), _meta(add), page_size, _device())
    known = _known.get(key)
    if known is None:
        s = _pages_shape(page_table, refcount, page_size)
        _ints(seq_lens, "seq_lens", (s.num_seqs,))
        _ints(seqs, "seqs")
        _ints(add, "add", seqs.shape)
        known = _remember(key, (_byref(s), _pages_need(s, seqs.numel()), _lib.load().gdn_pages_extend))
    shape, need, call = known
    ok = torch.empty_like(seqs)
    ws = _empty(need, dtype=torch.uint8, device=seqs.device)
    rc = call(shape, page_table.data_ptr(), seq_lens.data_ptr(), refcount.data_ptr(), seqs.data_ptr(), add.data_ptr(),
              seqs.numel(), ok.data_ptr(), ws.data_ptr(), need, _raw_stream(seqs.device.index))
    if rc:
        _check(rc, "gdn_pages_extend")
    return ok


def fork_pages(page_table, seq_lens, refcount, parents, children, pools=(), page_size: int = 16, states=()):
    """Makes each (empty) child sequence a copy of its parent: full pages shared, a partly filled last page copied to a
    new page in every pool [pages, ...], slot `child` of every states tensor [sequences, ...] a copy of slot `parent`
    (the recurrent states of delta-rule layers).  Returns int32 [m]: the new page, -1 where none was needed, -2 where
    the fork was left out."""
    key = ("fork", _meta(page_table), _meta(seq_lens), _meta(refcount), _meta(parents), _meta(children),
           tuple(map(_meta, pools)), page_size, tuple(map(_meta, states)), _device())
    known = _known.get(key)
    if known is None:
        s = _pages_shape(page_table, refcount, page_size)
        _ints(seq_lens, "seq_lens", (s.num_seqs,))
        _ints(parents, "parents")
        _ints(children, "children", parents.shape)
        known = _remember(key, (_byref(s), _pages_need(s, parents.numel()), _lib.load().gdn_pages_fork,
                                _pools(pools, "pools"), _pools(states, "states")))
    shape, need, call, p, st = known
    new = torch.empty_like(parents)
    ws = _empty(need, dtype=torch.uint8, device=parents.device)
    rc = call(shape, page_table.data_ptr(), seq_lens.data_ptr(), refcount.data_ptr(), parents.data_ptr(),
              children.data_ptr(), parents.numel(), _pool_bases(p, pools), len(pools), _pool_bases(st, states), len(states),
              new.data_ptr(), ws.data_ptr(), need, _raw_stream(parents.device.index))
    if rc:
        _check(rc, "gdn_pages_fork")
    return new


def free_pages(page_table, seq_lens, refcount, seqs):
    """Ends sequences: each of their pages loses one reference, their rows become -1 and their lengths 0."""
    key = ("free", _meta(page_table), _meta(seq_lens), _meta(refcount), _meta(seqs), _device())
    known = _known.get(key)
    if known is None:
        s = _pages_shape(page_table, refcount, 1)
        _ints(seq_lens, "seq_lens", (s.num_seqs,))
        _ints(seqs, "seqs")
        known = _remember(key, (_byref(s), _lib.load().gdn_pages_free))
    shape, call = known
    rc = call(shape, page_table.data_ptr(), seq_lens.data_ptr(), refcount.data_ptr(), seqs.data_ptr(), seqs.numel(),
              _raw_stream(seqs.device.index))
    if rc:
        _check(rc, "gdn_pages_free")


def compact_pages(page_table, refcount, pools=(), inplace: bool = True):
    """Moves the pages in use to the lowest numbers, in every pool and in the table.  Returns (page_table, refcount,
    moves): the inputs themselves, updated, or with inplace=False new ones; moves int32 scalar tensor."""
    key = ("compact", _meta(page_table), _meta(refcount), tuple(map(_meta, pools)), _device())
    known = _known.get(key)
    if known is None:
        s = _pages_shape(page_table, refcount, 1)
        known = _remember(key, (_byref(s), _pages_need(s, 0), _lib.load().gdn_pages_compact, _pools(pools, "pools"),
                                (s.table_stride, 1)))
    shape, need, call, p, stride = known
    dev = refcount.device
    table = page_table if inplace else torch.empty_strided(page_table.shape, stride, dtype=torch.int32, device=dev)
    ref = refcount if inplace else torch.empty_like(refcount)
    moves = _empty((), dtype=torch.int32, device=dev)
    ws = _empty(need, dtype=torch.uint8, device=dev)
    rc = call(shape, page_table.data_ptr(), refcount.data_ptr(), table.data_ptr(), ref.data_ptr(), _pool_bases(p, pools),
              len(pools), moves.data_ptr(), ws.data_ptr(), need, _raw_stream(dev.index))
    if rc:
        _check(rc, "gdn_pages_compact")
    return table, ref, moves


def copy_slots(pools, src, dst):
    """Copies slot src[i] to slot dst[i] (int32 [m]) in every tensor [slots, ...]; no dst twice or among the src."""
    _ints(src, "src")
    _ints(dst, "dst", src.shape)
    _check(_lib.load().gdn_slots_copy(_pool_bases(_pools(pools, "pools"), pools), len(pools), src.data_ptr(), dst.data_ptr(),
                                      src.numel(), _raw_stream(_device())), "gdn_slots_copy")


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
    v = t.view(-1, t.shape[-1]) if t.dim() != 2 else t  # raises where the rows have no common stride
    return v, v.stride(0)


def _norm_weight(weight, dim):
    if weight.dtype != torch.float32 or tuple(weight.shape) != (dim,) or not weight.is_contiguous():
        raise ValueError("weight must be a contiguous fp32 CUDA tensor [dim]")
    _here(weight, "weight")


def rms_norm(x, weight, residual=None, eps: float = 1e-6, fp8: bool = False, group: int = 0, weight_offset: float = 0.0,
             inplace: bool = False) -> NormOutput:
    """h = x + residual, y = h / sqrt(mean(h^2) + eps) * (weight + weight_offset) over the last dimension.

    x, residual [..., dim]; weight fp32 [dim].  fp8: y in e4m3 with one scale per row, or per `group` = 128 features;
    the normed values are y * scale.  inplace: h takes residual's place."""
    key = ("norm", _meta(x), _meta(weight), None if residual is None else _meta(residual), eps, fp8, group, weight_offset,
           inplace, _device())
    known = _known.get(key)
    if known is None:
        x2, xs = _rows(x, "x")
        T, D = x2.shape
        _norm_weight(weight, D)
        s = GdnNormShape()
        s.rows, s.dim, s.dtype, s.fp8, s.group = T, D, _dtype(x, "x"), int(fp8), int(group)
        s.eps, s.weight_offset, s.x_row, s.y_row = eps, weight_offset, xs, D
        if residual is not None:
            _, s.r_row = _rows(residual, "residual", x)
            s.h_row = s.r_row if inplace else D
        known = _remember(key, (_byref(s), _lib.load().gdn_rmsnorm_fwd, torch.float8_e4m3fn if fp8 else x.dtype,
                                (*x.shape[:-1], D // group if group else 1), x.shape[:-1]))
    shape, call, y_type, scale_shape, row_shape = known
    dev = x.device
    h, hp, rp = x, None, None
    if residual is not None:
        h = residual if inplace else _empty(x.shape, dtype=x.dtype, device=dev)
        hp, rp = h.data_ptr(), residual.data_ptr()
    y = _empty(x.shape, dtype=y_type, device=dev)
    scale = _empty(scale_shape, dtype=torch.float32, device=dev) if fp8 else None
    rstd = _empty(row_shape, dtype=torch.float32, device=dev)
    rc = call(shape, x.data_ptr(), rp, weight.data_ptr(), hp, y.data_ptr(), None if scale is None else scale.data_ptr(),
              rstd.data_ptr(), _raw_stream(dev.index))
    if rc:
        _check(rc, "gdn_rmsnorm_fwd")
    return NormOutput(y, h, scale, rstd)


def rms_norm_bwd(dy, h, weight, rstd, dh=None, weight_offset: float = 0.0):
    """(dx, dw): the gradient of x (and of residual), and of weight (fp32), from dy, the forward's h and rstd, and dh,
    the gradient that reaches h along the residual stream."""
    key = ("norm_bwd", _meta(dy), _meta(h), _meta(weight), _meta(rstd), None if dh is None else _meta(dh), weight_offset,
           _device())
    known = _known.get(key)
    if known is None:
        g2, gs = _rows(dy, "dy")
        _, hs = _rows(h, "h", dy)
        T, D = g2.shape
        _norm_weight(weight, D)
        if rstd.dtype != torch.float32 or rstd.numel() != T or not rstd.is_contiguous():
            raise ValueError("rstd must be a contiguous fp32 tensor with one value per row")
        _here(rstd, "rstd")
        s = GdnNormShape()
        s.rows, s.dim, s.dtype, s.weight_offset = T, D, _dtype(dy, "dy"), weight_offset
        s.x_row, s.y_row, s.h_row = hs, gs, D
        if dh is not None:
            _, s.r_row = _rows(dh, "dh", dy)
        lib = _lib.load()
        need = lib.gdn_rmsnorm_bwd_workspace_size(_byref(s))
        if need == 0:
            _check(_lib.GDN_ERR_INVALID_ARG, "gdn_rmsnorm_bwd_workspace_size")
        known = _remember(key, (_byref(s), need, lib.gdn_rmsnorm_bwd))
    shape, need, call = known
    dev = dy.device
    dx = _empty(dy.shape, dtype=dy.dtype, device=dev)
    dw = _empty(dy.shape[-1], dtype=torch.float32, device=dev)
    ws = _empty(need, dtype=torch.uint8, device=dev)
    rc = call(shape, dy.data_ptr(), h.data_ptr(), weight.data_ptr(), rstd.data_ptr(), None if dh is None else dh.data_ptr(),
              dx.data_ptr(), dw.data_ptr(), ws.data_ptr(), need, _raw_stream(dev.index))
    if rc:
        _check(rc, "gdn_rmsnorm_bwd")
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
