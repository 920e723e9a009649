"""Attention behind a shared prefix: which batches are computed in two parts, seen by the workspace that they need, and right
results on both sides of the rule.  Against the definition in 64 bits, with its bounds (tests/test_block_attention_parts.py)."""
import ctypes

import pytest
import torch

from gated_deltanet_linear_15_gb300 import _lib
from tests import block_ref as ref
from tests.test_block_attention_parts import BF, DEV, F32, _shape, close, lib, shared  # noqa: F401

gpu = pytest.mark.gpu


def in_two_parts(lib, groups=4, max_group=0, **kw):  # noqa: F811
    s = ctypes.byref(_shape(**kw))
    both, one = lib.gdn_prefix_attn_workspace_size(s, groups, max_group), lib.gdn_paged_attn_workspace_size(s)
    assert both >= one > 0
    return both > one


@pytest.mark.parametrize("dtype,most", [(_lib.GDN_BF16, 128), (_lib.GDN_FP32, 32)])
@pytest.mark.parametrize("heads", [2, 8, 32])  # 1, 4, 16 to a key head
@pytest.mark.parametrize("max_q", [0, 1, 1000])
def test_many_new_tokens_are_computed_in_one_part(lib, dtype, most, heads, max_q):  # noqa: F811
    """From half a tile of query rows to a sequence on (fp32: a tile) two parts only add their sums (up to 2.2 times the time)."""
    new = most // (heads // 2)
    for total, two in ((64, True), (64 * new - 1, True), (64 * new, False), (64 * new * 30, False)):
        assert in_two_parts(lib, dtype=dtype, num_heads=heads, total_q=total, max_q=max_q) == two, total


@pytest.mark.parametrize("dtype,least", [(_lib.GDN_BF16, 128e6), (_lib.GDN_FP32, 80e6)])
def test_room_of_the_table_decides(lib, dtype, least):  # noqa: F811
    page = 60 * 64 * 2 * 128 * 2 * (2 if dtype == _lib.GDN_BF16 else 4)  # what 60 sequences more than groups have in a page each
    for pages in (1, int(least / page), int(least / page) + 1, 100000):
        assert in_two_parts(lib, dtype=dtype, max_pages=pages, table_stride=pages) == (pages * page > least), pages


@gpu
@pytest.mark.parametrize("dtype,D,G,new", [(BF, 128, 4, 31), (BF, 128, 4, 32), (BF, 64, 1, 127), (BF, 64, 1, 128), (F32, 128, 4, 7),
                                           (F32, 128, 4, 8), (F32, 64, 1, 31), (F32, 64, 1, 32), (BF, 128, 2, 150)])
def test_both_sides_of_the_rule(dtype, D, G, new):
    import gated_deltanet_linear_15_gb300 as g
    x, qs, pre, cu = shared([(300, [(new, new + 3 * i) for i in range(5)]), (90, [(new, new + 11)] * 3)], dtype, D, 2, G, 16)
    for args in (dict(max_q=new, max_group=5 * new), dict()):
        o, lse = g.prefix_attention(**x, prefix_lens=pre, cu_seqs=cu, cu_q=ref.lens_to_cu(qs, DEV), return_lse=True, **args)
        close(o, lse, x, qs, D ** -0.5)


@gpu
@pytest.mark.parametrize("dtype,D,G", [(BF, 128, 2), (BF, 64, 8), (F32, 64, 1), (F32, 128, 2)])
def test_a_long_chunk_among_decoding_sequences(dtype, D, G):
    """Few rows on the mean, so in two parts, but several tiles for one sequence in either of them."""
    import gated_deltanet_linear_15_gb300 as g
    x, qs, pre, cu = shared([(500, [(1, 5 + i) for i in range(20)] + [(270, 290)] + [(1, 9)] * 20)], dtype, D, 1, G, 16)
    for args in (dict(max_q=270, max_group=310), dict(max_q=1, max_group=1)):
        o, lse = g.prefix_attention(**x, prefix_lens=pre, cu_seqs=cu, cu_q=ref.lens_to_cu(qs, DEV), return_lse=True, **args)
        close(o, lse, x, qs, D ** -0.5)


@gpu
def test_status_of_an_expired_wait_in_two_chunk_kernels(lib):  # noqa: F811
    """A call that is made to wait, with a short limit, for what never comes returns, leaves 4 and no output."""
    import gated_deltanet_linear_15_gb300 as g
    new, seqs = 12, 12
    x, qs, pre, cu = shared([(700, [(new, 20 + new)] * seqs)], BF, 128, 2, 4, 16)
    ws, out = torch.empty(256 << 20, dtype=torch.uint8, device=DEV), torch.full_like(x["q"], 7.0)
    s = _shape(num_seqs=seqs, total_q=seqs * new, page_size=16, num_pages=x["k_cache"].shape[0], max_pages=x["page_table"].shape[1],
               max_q=new, table_stride=x["page_table"].shape[1], k_page=16 * 256, v_page=16 * 256)
    assert lib.gdn_prefix_attn_workspace_size(ctypes.byref(s), 1, 0) > lib.gdn_paged_attn_workspace_size(ctypes.byref(s))
    p, st = lambda t: t.data_ptr(), torch.cuda.current_stream().cuda_stream  # noqa: E731

    def call():
        return lib.gdn_prefix_attn_fwd(ctypes.byref(s), 1, 0, p(x["q"]), p(x["k_cache"]), p(x["v_cache"]), p(x["page_table"]), None,
                                       p(x["kv_lens"]), p(cu), p(pre), p(out), None, p(ws), ws.numel(), st)

    s.reserved = _lib.GDN_DEBUG_WAIT_TIMEOUT - (1 << 32)
    assert call() == 0
    assert lib.gdn_prefix_attn_status(ctypes.byref(s), 1, 0, p(ws), st) == 4 and (out == 7).all()
    s.reserved = 0
    assert call() == 0 and lib.gdn_prefix_attn_status(ctypes.byref(s), 1, 0, p(ws), st) == 0
    assert torch.equal(out, g.prefix_attention(**x, prefix_lens=pre, cu_seqs=cu, max_q=new, scale=0.1))
