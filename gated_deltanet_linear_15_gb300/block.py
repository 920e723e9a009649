"""Operators that a hybrid stack puts next to its gated delta-rule layers: the functions of include/gdn_block.h on tensors.

``paged_attention`` (attention of new tokens over a paged key/value cache), ``prefix_attention`` (the same of sequences that
share a prefix), ``rotary_table`` / ``rotary`` / ``rotary_embedding`` / ``rotary_append`` (rotary positions, their gradient,
and the write of new keys and values into the cache), ``norm_rotary`` / ``norm_rotary_bwd`` / ``norm_rotary_embedding`` /
``norm_rotary_append`` (the same behind a norm of every head), ``extend_pages`` / ``fork_pages`` / ``free_pages`` /
``compact_pages`` / ``copy_slots`` (the cache's upkeep), ``rms_norm`` / ``rms_norm_bwd`` / ``residual_rms_norm`` (the residual
stream's norm, optionally with an 8-bit output), ``gated_scan`` / ``gated_scan_bwd`` / ``gated_linear_recurrence`` /
``gated_scan_step`` (a gated linear recurrence with one state per channel: forward, backward, with gradients, and for single
tokens).  As in the rest of the package, everything runs in the library's CUDA kernels on the current stream; the
arguments are checked, and outputs and workspaces allocated, by the extension csrc/block_py.cpp.  Bad arguments raise
``ValueError`` (found there) or ``RuntimeError`` (found by the library, with its reason), a lack of memory
``torch.OutOfMemoryError``.

Gradients come from ``rotary_embedding``, ``residual_rms_norm``, ``norm_rotary_embedding`` and ``gated_linear_recurrence``.
Every other function computes outside autograd, as
the ``_fwd`` / ``_bwd`` functions of the delta rule do: its outputs carry no graph, whatever its inputs require.  What a
function writes in place counts as an in-place operation (its version moves on).

Attention, rotary positions, norms and the recurrence (but not ``rotary_table`` and the ``_status`` functions) can be captured
into a CUDA graph; two graphs that may run at once need a workspace each.  A captured
``backward()`` adds to leaves whose accumulation PyTorch ties to the stream that first used them: let no eager graph of the
same leaves live then, or take ``torch.autograd.grad``.
"""
from __future__ import annotations

import math
from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import _lib

__all__ = ["paged_attention", "paged_attention_status", "prefix_attention", "prefix_attention_status", "rotary_frequencies",
           "rotary_table", "rotary", "rotary_embedding", "rotary_append", "extend_pages", "fork_pages", "free_pages", "compact_pages", "copy_slots", "rms_norm",
           "rms_norm_bwd", "residual_rms_norm", "NormOutput", "norm_rotary", "norm_rotary_bwd",
           "norm_rotary_embedding", "norm_rotary_append", "gated_scan", "gated_scan_bwd", "gated_scan_step",
           "gated_linear_recurrence"]


class _Extension:
    """The extension module, loaded at the first call."""

    def __getattr__(self, name):
        global _py
        _py = _lib.load_py()
        return getattr(_py, name)


_py = _Extension()


# ------------------------------------------------------------------ paged cache
def paged_attention(q, k_cache, v_cache, page_table, kv_lens, cu_q=None, max_q: int = 0, scale: Optional[float] = None,
                    window: int = 0, return_lse: bool = False, out=None, workspace=None, sinks: int = 0):
    """Causal attention of new tokens over a paged cache that already holds their keys and values.

    q [new tokens, heads, D]; k_cache, v_cache [pages, page_size, kv heads, D] (any strides with contiguous features);
    page_table int32 [sequences, pages] (one row may be expanded over all sequences); kv_lens int32 [sequences], the tokens
    of each sequence with the new ones;
    cu_q int32 [sequences + 1], where each sequence's new tokens begin in q (None: as many for each).  max_q: the most
    new tokens of a sequence, if known on the host (it only picks the kernel).  window > 0: a query sees that many
    keys, and with sinks > 0 the sequence's first `sinks` keys too.  Returns o like q, or (o, lse) with lse fp32 [new tokens,
    heads]; a query without keys has o = 0 and lse = -inf.  workspace: a tensor to use as scratch memory (contiguous, 32-byte
    aligned, refused when it is too small).  Decoding is the case of one new token per sequence."""
    return _py.paged_attention(q, k_cache, v_cache, page_table, kv_lens, cu_q, max_q, scale, window, return_lse, out, workspace,
                               sinks)


def paged_attention_status(q, k_cache, v_cache, page_table, kv_lens, workspace, cu_q=None, max_q: int = 0) -> int:
    """Status word of the last ``paged_attention`` call with these arguments and this workspace, which that call must have
    been given (0: clean; see gdn_paged_attn_status).  Synchronises the stream."""
    return _py.paged_attention_status(q, k_cache, v_cache, page_table, kv_lens, workspace, cu_q, max_q)


def prefix_attention(q, k_cache, v_cache, page_table, kv_lens, prefix_lens, cu_seqs=None, cu_q=None, max_q: int = 0,
                     max_group: int = 0, scale: Optional[float] = None, return_lse: bool = False, out=None, workspace=None):
    """``paged_attention`` of groups of sequences that share a prefix, whose keys are read once for each group.

    prefix_lens int32 [groups]: tokens that all sequences of a group with new tokens have in common; their rows of page_table
    name the same pages there, as after ``fork_pages``.  Those without new tokens may have ended (``free_pages``).  A prefix
    longer than what some sequence with new tokens had cached before them is cut to that.  cu_seqs int32 [groups + 1]: where
    each group's sequences begin (None: as many for each; sequences outside share nothing).  max_group: the most new tokens of
    a group, if known on the host (it only picks the kernel).  The rest as in ``paged_attention``, without a window.

    Where sharing saves too little, the call is ``paged_attention`` of the same arguments: many new tokens to a sequence, or
    little room in the rows of page_table (the host knows no lengths, so a table as wide as need be is best for few sequences)."""
    return _py.prefix_attention(q, k_cache, v_cache, page_table, kv_lens, prefix_lens, cu_seqs, cu_q, max_q, max_group, scale,
                                return_lse, out, workspace)


def prefix_attention_status(q, k_cache, v_cache, page_table, kv_lens, prefix_lens, workspace, cu_seqs=None, cu_q=None,
                            max_q: int = 0, max_group: int = 0) -> int:
    """``paged_attention_status`` of the last ``prefix_attention`` call with these arguments and this workspace."""
    return _py.prefix_attention_status(q, k_cache, v_cache, page_table, kv_lens, prefix_lens, workspace, cu_seqs, cu_q, max_q,
                                       max_group)


# ------------------------------------------------------------------ rotary positions
def rotary_frequencies(rot: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                       context: int = 0, fast: float = 32.0, slow: float = 1.0):
    """(fp64 angles per position [rot / 2], amplitude) of a rotary embedding over `rot` features.

    scaling None: base^(-2 i / rot).  "linear": positions stretched by `factor`.  "base": the base raised so that the
    slowest pair is stretched by `factor` and the fastest is kept.  "parts": pairs that turn fewer than `slow` times over
    the original `context` are stretched, those that turn more than `fast` times are kept, and the share that is kept of
    those between grows linearly with their turns (not with their index); for factor > 1 the amplitude is
    0.1 ln(factor) + 1.  With another blend or amplitude a program forms the table itself: any fp32 tensor [positions,
    rot / 2, 2] of (amplitude cos, amplitude sin)."""
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
    with torch.cuda.device(table.device):
        lib, stream = _lib.load(), torch.cuda.current_stream().cuda_stream
        rc = lib.gdn_rotary_table(freq.data_ptr(), rot // 2, positions, amplitude, table.data_ptr(), stream)
    if rc != 0:
        raise RuntimeError(f"gdn_rotary_table: {lib.gdn_status_string(rc).decode()} ({_lib.last_error()})")
    return table


def rotary(q, k, table, positions, interleaved: bool = False, inverse: bool = False, inplace: bool = False):
    """q [T, heads, D] and k [T, heads, D] (or None) turned by the table's angles of positions int32 [T]; pairs of
    features (i, i + rot / 2), or (2 i, 2 i + 1) when interleaved, over the first rot = 2 table.shape[1] features.
    inverse turns back, which is also the gradient.  Returns (q, k)."""
    return _py.rotary(q, k, table, positions, interleaved, inverse, inplace)


class RotaryFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, table, positions, interleaved, inverse):
        ctx.save_for_backward(table, positions)
        ctx.interleaved, ctx.inverse = interleaved, inverse
        return rotary(q, k, table, positions, interleaved, inverse)

    @staticmethod
    def backward(ctx, dq, dk):
        table, positions = ctx.saved_tensors
        dk = None if dk is None else dk.contiguous()  # there is none without k
        # linear in q and k, so its own gradient is the function again, the other way round
        dq, dk = RotaryFunction.apply(dq.contiguous(), dk, table, positions, ctx.interleaved, not ctx.inverse)
        return dq, dk, None, None, None, None


def rotary_embedding(q, k, table, positions, interleaved: bool = False):
    """``rotary`` with gradients of any order for q and k (or q alone, with k None)."""
    return RotaryFunction.apply(q, k, table, positions, interleaved, False)


def rotary_append(q, k, v, table, k_cache, v_cache, page_table, kv_lens, cu_q=None, interleaved: bool = False, out=None):
    """Turns the new tokens' q and k by their positions, writes k and v into their cache slots and returns the turned q.

    q [new tokens, heads, D], k, v [new tokens, kv heads, D], as slices of one projection if need be.  The caches,
    page_table, kv_lens and cu_q are those of ``paged_attention``: kv_lens counts the new tokens already."""
    return _py.rotary_append(q, k, v, table, k_cache, v_cache, page_table, kv_lens, cu_q, interleaved, out)


# ------------------------------------------------------------------ norm of heads with rotary positions
def norm_rotary(q, k, q_weight, k_weight, table, positions, eps: float = 1e-6, weight_offset: float = 0.0,
                interleaved: bool = False):
    """The root-mean-square norm of every head of q and k, then ``rotary``, in one pass.

    q [T, heads, D] and k [T, heads, D] (or None, with its weight), D at most 1024; q_weight, k_weight fp32 [D] (one for all
    heads of q, one for those of k): head / sqrt(mean(head^2) + eps) * (weight + weight_offset).  table, positions and
    interleaved as in ``rotary``.  Returns (q, k)."""
    return _py.norm_rotary(q, k, q_weight, k_weight, table, positions, eps, weight_offset, interleaved)


def norm_rotary_bwd(dq, dk, q, k, q_weight, k_weight, table, positions, eps: float = 1e-6, weight_offset: float = 0.0,
                    interleaved: bool = False):
    """(dq, dk, dq_weight, dk_weight): the gradients of ``norm_rotary``'s inputs from those of its outputs and the inputs."""
    return _py.norm_rotary_bwd(dq, dk, q, k, q_weight, k_weight, table, positions, eps, weight_offset, interleaved)


class NormRotaryFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, table, positions, eps, weight_offset, interleaved):
        ctx.save_for_backward(q, k, q_weight, k_weight, table, positions)
        ctx.how = (eps, weight_offset, interleaved)
        return norm_rotary(q, k, q_weight, k_weight, table, positions, *ctx.how)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        q, k, q_weight, k_weight, table, positions = ctx.saved_tensors
        dk = None if dk is None else dk.contiguous()  # there is none without k
        grads = norm_rotary_bwd(dq.contiguous(), dk, q, k, q_weight, k_weight, table, positions, *ctx.how)
        return (*grads, None, None, None, None, None)


def norm_rotary_embedding(q, k, q_weight, k_weight, table, positions, eps: float = 1e-6, weight_offset: float = 0.0,
                          interleaved: bool = False):
    """``norm_rotary`` with (first) gradients for q, k and both weights (or q and its weight alone, with k None)."""
    return NormRotaryFunction.apply(q, k, q_weight, k_weight, table, positions, eps, weight_offset, interleaved)


def norm_rotary_append(q, k, v, q_weight, k_weight, table, k_cache, v_cache, page_table, kv_lens, cu_q=None, eps: float = 1e-6,
                       weight_offset: float = 0.0, interleaved: bool = False, out=None):
    """``rotary_append`` with the heads of q and k normed first, as in ``norm_rotary``, in the same pass."""
    return _py.norm_rotary_append(q, k, v, q_weight, k_weight, table, k_cache, v_cache, page_table, kv_lens, cu_q, eps,
                                  weight_offset, interleaved, out)


# ------------------------------------------------------------------ pages
def extend_pages(page_table, seq_lens, refcount, seqs, add, page_size: int):
    """Grows sequences seqs int32 [m] by add int32 [m] tokens, taking the free pages of lowest number in list order.
    Returns ok int32 [m]: 1, or 0 where a sequence stays as it was (no room, no pages, a shared last page)."""
    return _py.extend_pages(page_table, seq_lens, refcount, seqs, add, page_size)


def fork_pages(page_table, seq_lens, refcount, parents, children, pools=(), page_size: int = 16, states=()):
    """Makes each (empty) child sequence a copy of its parent: full pages shared, a partly filled last page copied to a
    new page in every pool [pages, ...], slot `child` of every states tensor [sequences, ...] a copy of slot `parent`
    (the recurrent states of delta-rule layers).  Pools and states with fewer slots than that are refused.  Returns int32 [m]: the new page, -1 where none was needed, -2 where
    the fork was left out."""
    return _py.fork_pages(page_table, seq_lens, refcount, parents, children, pools, page_size, states)


def free_pages(page_table, seq_lens, refcount, seqs):
    """Ends sequences: each of their pages loses one reference, their rows become -1 and their lengths 0."""
    _py.free_pages(page_table, seq_lens, refcount, seqs)


def compact_pages(page_table, refcount, pools=(), inplace: bool = True):
    """Moves the pages in use to the lowest numbers, in every pool and in the table.  Returns (page_table, refcount,
    moves): the inputs themselves, updated, or with inplace=False new ones; moves int32 scalar tensor."""
    return _py.compact_pages(page_table, refcount, pools, inplace)


def copy_slots(pools, src, dst):
    """Copies slot src[i] to slot dst[i] (int32 [m]) in every tensor [slots, ...]; no dst twice or among the src."""
    _py.copy_slots(pools, src, dst)


# ------------------------------------------------------------------ root-mean-square norm
class NormOutput(NamedTuple):
    y: torch.Tensor                   # the normed rows, e4m3 with fp8=True
    h: torch.Tensor                   # x + residual in x's dtype (x itself without a residual)
    scale: Optional[torch.Tensor]     # fp8: fp32 [rows, dim / group], or [rows, 1]
    rstd: torch.Tensor                # fp32 [rows]


def rms_norm(x, weight, residual=None, eps: float = 1e-6, fp8: bool = False, group: int = 0, weight_offset: float = 0.0,
             inplace: bool = False) -> NormOutput:
    """h = x + residual, y = h / sqrt(mean(h^2) + eps) * (weight + weight_offset) over the last dimension.

    x, residual [..., dim]; weight fp32 [dim].  fp8: y in e4m3 with one scale per row, or per `group` = 128 features;
    the normed values are y * scale.  inplace: h takes residual's place."""
    return NormOutput._make(_py.rms_norm(x, weight, residual, eps, fp8, group, weight_offset, inplace))


def rms_norm_bwd(dy, h, weight, rstd, dh=None, weight_offset: float = 0.0):
    """(dx, dw): the gradient of x (and of residual), and of weight (fp32), from dy, the forward's h and rstd, and dh,
    the gradient that reaches h along the residual stream."""
    return _py.rms_norm_bwd(dy, h, weight, rstd, dh, weight_offset)


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
    @once_differentiable
    def backward(ctx, dy, dh=None):
        h, weight, rstd = ctx.saved_tensors
        dx, dw = rms_norm_bwd(dy.contiguous(), h, weight, rstd, None if dh is None else dh.contiguous(), ctx.weight_offset)
        return dx, dx if ctx.has_residual else None, dw, None, None


def residual_rms_norm(x, weight, residual=None, eps: float = 1e-6, weight_offset: float = 0.0):
    """``rms_norm`` with (first) gradients: (y, h), or y alone without a residual."""
    return ResidualRMSNormFunction.apply(x, residual, weight, eps, weight_offset)


# ------------------------------------------------------------------ gated linear recurrence
def gated_scan(x, g, initial_state=None, cu_seqlens=None, output_final_state: bool = True, save_states: bool = False):
    """h_t = exp(g_t) h_{t-1} + x_t in every channel; y_t = h_t.

    x [sequences, tokens, D] (rows of one stride), g like x in its dtype or fp32: the log-gates, meant to be <= 0 (-inf
    forgets).  Packed sequences: x [1, tokens, D] and cu_seqlens int32 [sequences + 1] on the device; rows in front of the
    first and behind the last one are padding, zeros in y and in the gradients.  initial_state fp32 [sequences, D] (None: zeros).  Returns (y, final state fp32 [sequences,
    D], or None without output_final_state), and with save_states the states that ``gated_scan_bwd`` reads."""
    y, final, states = _py.gated_scan(x, g, initial_state, cu_seqlens, output_final_state, save_states)
    return (y, final, states) if save_states else (y, final)


def gated_scan_bwd(dy, x, g, states, initial_state=None, d_final=None, cu_seqlens=None):
    """(dx, dg, gradient of initial_state or None) from dy, d_final (fp32 [sequences, D], the gradient of the final states;
    None: zero) and the forward's inputs and ``save_states`` output."""
    return _py.gated_scan_bwd(dy, x, g, states, initial_state, d_final, cu_seqlens)


def gated_scan_step(x, g, state):
    """One token of each sequence: state fp32 [sequences, D] becomes exp(g) state + x in place.  x, g [sequences, D].
    Returns (y, state), y the new state in x's dtype."""
    return _py.gated_scan_step(x, g, state), state


class GatedLinearRecurrenceFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, g, initial_state, cu_seqlens):
        y, final, states = gated_scan(x, g, initial_state, cu_seqlens, save_states=True)
        ctx.save_for_backward(x, g, states, initial_state, cu_seqlens)
        ctx.set_materialize_grads(False)
        return y, final

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, d_final):
        x, g, states, initial_state, cu_seqlens = ctx.saved_tensors
        dy = torch.zeros_like(x) if dy is None else dy.contiguous()
        d_final = None if d_final is None else d_final.contiguous()
        dx, dg, dh0 = gated_scan_bwd(dy, x, g, states, initial_state, d_final, cu_seqlens)
        return dx, dg, dh0, None


def gated_linear_recurrence(x, g, initial_state=None, cu_seqlens=None):
    """``gated_scan`` with (first) gradients for x, g and initial_state: (y, final state)."""
    return GatedLinearRecurrenceFunction.apply(x, g, initial_state, cu_seqlens)
