"""Attention of groups of sequences behind a shared prefix some of which have no new tokens: branches that have ended, or that
hold fewer tokens than the prefix.  They see nothing and limit nothing, and what their rows of the page table hold does not
matter, wherever they stand in their group.  Against the definition in 64 bits, with its bounds (tests/test_block_attention_parts.py)."""
import pytest
import torch

from tests import block_ref as ref
from tests.test_block_attention_parts import BF, DEV, F32, close, lib, shared  # noqa: F401

pytestmark = pytest.mark.gpu


def end(x, seqs):
    """The sequences end: free_pages takes their pages and tokens, as a server does when a branch is done."""
    import gated_deltanet_linear_15_gb300 as g
    table, pages = x["page_table"], x["k_cache"].shape[0]
    ref_count = torch.bincount(table[table >= 0].flatten().long().cpu(), minlength=pages).to(torch.int32).to(DEV)
    g.free_pages(table, x["kv_lens"], ref_count, torch.tensor(seqs, dtype=torch.int32, device=DEV))
    assert (x["kv_lens"][seqs] == 0).all() and (table[seqs] == -1).all()


def shorten(x, seqs, tokens):
    """The sequences hold only the first few tokens of the prefix; behind their page the rows name pages of others."""
    x["kv_lens"][seqs] = tokens
    others = x["page_table"][:, :2].flatten().flip(0)
    width = min(x["page_table"].shape[1], 200)
    for n in seqs:
        x["page_table"][n, 1:width] = others.repeat(width // others.numel() + 1)[:width - 1]


# prefix, sequences with new tokens of a group, new tokens of each, dtype, D, Hkv, G: the row kernel for both parts, the
# chunk kernel for the prefix, and for both
KINDS = [(1000, 4, 1, BF, 128, 2, 4), (300, 40, 1, BF, 128, 2, 4), (700, 6, 12, BF, 64, 2, 4), (250, 3, 2, F32, 64, 2, 2),
         (600, 12, 3, F32, 128, 1, 3)]


@pytest.mark.parametrize("prefix,count,new,dtype,D,Hkv,G", KINDS)
@pytest.mark.parametrize("idle", [[0], [0, 1], [2], [0, 3]])
@pytest.mark.parametrize("how", ["ended", "short", "cached"])
@pytest.mark.parametrize("wide", [True, False])
def test_sequences_without_new_tokens(prefix, count, new, dtype, D, Hkv, G, idle, how, wide):
    import gated_deltanet_linear_15_gb300 as g
    own = [(new, new + 3 * i) for i in range(count)]
    for n in idle:
        own.insert(n, (0, 1 + n))
    x, qs, pre, cu = shared([(prefix, own), (64, [(1, 2), (1, 9)])], dtype, D, Hkv, G, 16, seed=len(idle), wide=wide)
    if how == "ended":
        end(x, idle)
    elif how == "short":
        shorten(x, idle, 5)
    else:
        x["kv_lens"][idle] = prefix - 30  # most of the prefix, in the pages that all share
    args = dict(prefix_lens=pre, cu_seqs=cu, cu_q=ref.lens_to_cu(qs, DEV), return_lse=True)
    o, lse = g.prefix_attention(**x, **args)
    close(o, lse, x, qs, D ** -0.5)
    args.update(max_q=new, max_group=sum(qs))
    o, lse = g.prefix_attention(**x, **args)
    close(o, lse, x, qs, D ** -0.5)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("active", range(4))
def test_one_sequence_of_a_group_is_left(dtype, active):
    """All branches but one have ended: it shares with nobody."""
    import gated_deltanet_linear_15_gb300 as g
    own = [(1 if n == active else 0, 5 + n) for n in range(4)]
    x, qs, pre, cu = shared([(500, own), (100, [(1, 3), (2, 5)])], dtype, 64, 2, 2, 16)
    end(x, [n for n in range(4) if n != active])
    o, lse = g.prefix_attention(**x, prefix_lens=pre, cu_seqs=cu, cu_q=ref.lens_to_cu(qs, DEV), return_lse=True)
    close(o, lse, x, qs, 64 ** -0.5)
