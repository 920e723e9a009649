"""Upkeep of a paged cache against the rules in plain Python: tables, counts and lengths have to be equal, copies exact."""
import ctypes
import random

import pytest
import torch

from gated_deltanet_linear_15_gb300 import _lib
from tests.block_ref import Pages

gpu = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return _lib.load()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Device:
    """The tensors of a cache beside their Python model; two pools and a state tensor whose slots are told apart by value."""

    def __init__(self, seqs, width, pages, page, strided=False):
        self.m = Pages(seqs, width, pages, page)
        wide = torch.full((seqs, width + (3 if strided else 0)), -1, dtype=torch.int32, device=DEV)
        self.table = wide[:, :width]
        self.lens, self.ref = ints([0] * seqs), ints([0] * pages)
        gen = torch.Generator(device=DEV).manual_seed(pages)
        self.pools = [torch.randn(pages, page, 2, 24, generator=gen, device=DEV).bfloat16(),
                      torch.randn(pages, 3 if not strided else 5, 8, generator=gen, device=DEV)[:, :3]]
        self.states = torch.randn(seqs, 2, 6, 10, generator=gen, device=DEV)

    def same(self):
        assert self.table.tolist() == self.m.table
        assert self.lens.tolist() == self.m.lens
        assert self.ref.tolist() == self.m.ref

    def extend(self, g, seqs, add):
        ok = g.extend_pages(self.table, self.lens, self.ref, ints(seqs), ints(add), self.m.page)
        assert ok.tolist() == self.m.extend(seqs, add)
        self.same()

    def fork(self, g, parents, children):
        pools, states = [p.clone() for p in self.pools], self.states.clone()
        new = g.fork_pages(self.table, self.lens, self.ref, ints(parents), ints(children), self.pools, self.m.page, [self.states])
        want, copies, moved = self.m.fork(parents, children)
        assert new.tolist() == want
        for a, b in copies:
            for p in pools:
                p[b] = p[a]
        for a, b in moved:
            states[b] = states[a]
        assert all(torch.equal(x, y) for x, y in zip(pools, self.pools)) and torch.equal(states, self.states)
        self.same()

    def free(self, g, seqs):
        g.free_pages(self.table, self.lens, self.ref, ints(seqs))
        self.m.free(seqs)
        self.same()

    def compact(self, g, inplace):
        pools = [p.clone() for p in self.pools]
        old = self.table.clone(), self.ref.clone()
        table, ref, moves = g.compact_pages(self.table, self.ref, self.pools, inplace=inplace)
        if not inplace:
            assert torch.equal(self.table, old[0]) and torch.equal(self.ref, old[1])
            self.table, self.ref = table, ref
        pairs = self.m.compact()
        assert int(moves) == len(pairs)
        for s, d in pairs:
            for p in pools:
                p[d] = p[s]
        assert all(torch.equal(x, y) for x, y in zip(pools, self.pools))
        self.same()


@gpu
@pytest.mark.parametrize("seqs,width,pages,page,strided", [(4, 3, 8, 4, False), (9, 40, 200, 16, True), (30, 300, 9000, 16, False),
                                                          (1, 1, 1, 16, False), (1500, 4, 5000, 8, True)])
def test_a_life_of_requests(seqs, width, pages, page, strided):
    import gated_deltanet_linear_15_gb300 as g
    r = random.Random(seqs * 31 + pages)
    d = Device(seqs, width, pages, page, strided)
    for step in range(14):
        some = r.sample(range(seqs), r.randint(1, seqs))
        d.extend(g, some, [r.choice([0, 1, page - 1, page, r.randint(0, width * page)]) for _ in some])
        empty = [s for s in range(seqs) if d.m.lens[s] == 0]
        full = [s for s in range(seqs) if d.m.lens[s]]
        if empty and full:
            children = r.sample(empty, r.randint(1, len(empty)))
            d.fork(g, [r.choice(full) for _ in children], children)
        d.free(g, r.sample(range(seqs), r.randint(0, seqs // 2)) or [0])
        if step % 3 == 2:
            d.compact(g, inplace=step % 2 == 0)


@gpu
def test_fork_shares_full_pages_only():
    import gated_deltanet_linear_15_gb300 as g
    d = Device(5, 6, 20, 16)
    d.extend(g, [0, 1], [40, 32])
    d.fork(g, [0, 1, 0], [2, 3, 4])
    assert d.m.ref[:3] == [3, 3, 1] and d.m.table[3] == d.m.table[1]
    d.extend(g, [0, 2, 4], [3, 9, 1])     # each writes into a last page of its own
    d.free(g, [0, 1])
    d.compact(g, True)


@gpu
def test_out_of_pages_and_bad_requests():
    import gated_deltanet_linear_15_gb300 as g
    d = Device(6, 4, 5, 16)
    d.extend(g, [0, 1, 2, 3], [33, 20, 0, 5])          # 3 + 2 pages, then one that is not there
    d.extend(g, [4, 0], [1, 15])                       # no page, but room in a last page
    d.extend(g, [7, -1, 0, 5], [1, 1, -4, 65])         # bad numbers, a row that is too short
    d.fork(g, [0, 0, 9, 1], [4, 1, 5, -2])             # no page; child not empty; bad parent; bad child
    d.free(g, [1])
    d.fork(g, [0, 0, 0, 3], [1, 4, 5, 2])              # two pages for three children; an empty parent
    d.free(g, [0, -1, 77])


@gpu
def test_shared_partial_page_is_not_extended():
    """A table that shares a partly filled page (no fork makes one) cannot grow into it."""
    import gated_deltanet_linear_15_gb300 as g
    table, lens, ref = ints([[0, -1], [0, -1]]), ints([5, 5]), ints([2, 0])
    assert g.extend_pages(table, lens, ref, ints([0, 1]), ints([1, 0]), 16).tolist() == [0, 1]
    assert lens.tolist() == [5, 5] and ref.tolist() == [2, 0]


@gpu
def test_lengths_end_at_31_bits():
    """A table row may have room for more tokens than a length can count."""
    import gated_deltanet_linear_15_gb300 as g
    P, start = 1 << 20, (1 << 31) - (1 << 20)
    table, lens, ref = torch.full((2, 4096), -1, dtype=torch.int32, device=DEV), ints([start, 0]), ints([0] * 4)
    assert g.extend_pages(table, lens, ref, ints([0, 1]), ints([P, P + 1]), P).tolist() == [0, 1]
    assert lens.tolist() == [start, P + 1] and ref.tolist() == [1, 1, 0, 0] and (table[0] == -1).all()
    assert g.extend_pages(table, lens, ref, ints([0]), ints([P - 1]), P).tolist() == [1]
    assert lens.tolist() == [2 ** 31 - 1, P + 1] and ref.tolist() == [1, 1, 1, 0] and int(table[0, 2047]) == 2
    assert g.extend_pages(table, lens, ref, ints([0]), ints([1]), P).tolist() == [0]


@gpu
def test_requests_for_more_pages_than_30_bits_count():
    """Together the requests ask for more than 2^30 pages: none of those that need pages is granted, the later ones included."""
    import gated_deltanet_linear_15_gb300 as g
    NP, m = 1 << 20, 1027
    table = torch.full((m, NP + 1), -1, dtype=torch.int32, device=DEV)
    lens, ref = ints([0] * m), torch.zeros(NP, dtype=torch.int32, device=DEV)
    add = [NP + 1] * m
    add[-1] = 0
    assert g.extend_pages(table, lens, ref, ints(list(range(m))), ints(add), 1).tolist() == [0] * (m - 1) + [1]
    assert not lens.any() and not ref.any()


@gpu
def test_sequence_named_twice_is_freed_once():
    import gated_deltanet_linear_15_gb300 as g
    table, lens, ref = ints([[0, 1], [0, -1]]), ints([20, 16]), ints([2, 1])
    g.free_pages(table, lens, ref, ints([0, 0, 0]))
    assert ref.tolist() == [1, 0] and table.tolist() == [[-1, -1], [0, -1]] and lens.tolist() == [0, 16]


@gpu
@pytest.mark.parametrize("slots,inner,dtype", [(7, 8, torch.float32), (40, 50000, torch.bfloat16), (3, 16384, torch.int8)])
def test_copy_slots(slots, inner, dtype):
    import gated_deltanet_linear_15_gb300 as g
    gen = torch.Generator(device=DEV).manual_seed(slots)
    pools = [torch.randint(-100, 100, (slots, inner + 16 * i), generator=gen, device=DEV).to(dtype) for i in range(70)]
    src, dst = [0, 2, -1, 1, slots], [slots - 1, 1 if slots < 5 else 4, 0, -5, 0]
    src, dst = (src, dst) if slots > 3 else ([0, -1], [2, 1])
    want = [p.clone() for p in pools]
    for p in want:
        for a, b in zip(src, dst):
            if 0 <= a < slots and 0 <= b < slots:
                p[b] = p[a]
    g.copy_slots(pools, ints(src), ints(dst))
    assert all(torch.equal(a, b) for a, b in zip(want, pools))
    g.copy_slots(pools, ints([]), ints([]))
    g.copy_slots([], ints(src), ints(dst))


@gpu
def test_offsets_past_32_bits():
    import gated_deltanet_linear_15_gb300 as g
    pool = torch.empty(1300, 1 << 22, dtype=torch.int8, device=DEV)
    pool[1299], pool[700], pool[0] = 3, 2, 1
    g.copy_slots([pool], ints([1299, 0]), ints([600, 1298]))
    assert (pool[600] == 3).all() and (pool[1298] == 1).all() and (pool[700] == 2).all()


@gpu
def test_binding_refuses():
    import gated_deltanet_linear_15_gb300 as g
    table, lens, ref = ints([[-1, -1]]), ints([0]), ints([0, 0])
    pool = torch.zeros(2, 16, device=DEV)
    with pytest.raises(ValueError):
        g.extend_pages(table, lens, ref, ints([0]), ints([1, 2]), 16)
    with pytest.raises(ValueError):
        g.free_pages(table.long(), lens, ref, ints([0]))
    with pytest.raises(ValueError):
        g.fork_pages(table, ints([0, 0]), ref, ints([0]), ints([0]), [pool], 16)
    with pytest.raises(ValueError):
        g.copy_slots([torch.zeros(4, 4, 4, device=DEV).transpose(1, 2)], ints([0]), ints([1]))
    with pytest.raises(RuntimeError):
        g.copy_slots([torch.zeros(4, 3, device=DEV)], ints([0]), ints([1]))       # 12 bytes
    with pytest.raises(RuntimeError):
        g.extend_pages(table, lens, ref, ints([0]), ints([1]), 0)
    with pytest.raises(ValueError):
        g.compact_pages(table, ref.cpu())


@gpu
def test_tables_whose_rows_share_memory_are_refused():
    """The page functions write rows, so an expanded row or rows that overlap are refused; nothing is written."""
    import gated_deltanet_linear_15_gb300 as g
    whole, lens, ref = ints([[-1] * 4] * 6), ints([0] * 3), ints([0] * 8)
    pool = torch.zeros(8, 16, device=DEV)
    for table in (whole[:1].expand(3, -1), whole.as_strided((3, 4), (2, 1))):
        for call in (lambda: g.extend_pages(table, lens, ref, ints([0, 1, 2]), ints([5, 5, 5]), 16),
                     lambda: g.fork_pages(table, lens, ref, ints([0]), ints([1]), [pool], 16),
                     lambda: g.free_pages(table, lens, ref, ints([2])), lambda: g.compact_pages(table, ref, [pool]),
                     lambda: g.compact_pages(table, ref, [pool], inplace=False)):
            with pytest.raises(RuntimeError, match="table_stride"):
                call()
    assert (whole == -1).all() and not lens.any() and not ref.any()
    one = whole.as_strided((1, 4), (1, 1))    # a single row has no stride to speak of
    assert g.extend_pages(one, lens[:1], ref, ints([0]), ints([20]), 16).tolist() == [1]
    assert one.tolist() == [[0, 1, -1, -1]]


@gpu
def test_what_is_written_has_a_new_version():
    """Autograd compares versions before it uses a saved tensor; every function counts its writes, also for inference
    tensors (which have none) and pools that come from a generator."""
    import gated_deltanet_linear_15_gb300 as g
    d = Device(4, 6, 20, 16)

    def moved(call, written, kept=()):
        old = [t._version for t in written], [t._version for t in kept]
        call()
        assert all(t._version > v for t, v in zip(written, old[0])) and [t._version for t in kept] == old[1]

    book, caches = [d.table, d.lens, d.ref], d.pools
    moved(lambda: g.extend_pages(d.table, d.lens, d.ref, ints([0]), ints([20]), 16), book, caches)
    moved(lambda: g.fork_pages(*book, ints([0]), ints([1]), (p for p in caches), 16, (s for s in [d.states])),
          book + caches + [d.states])
    moved(lambda: g.free_pages(*book, ints([0])), book, caches)
    moved(lambda: g.compact_pages(d.table, d.ref, caches, inplace=False), caches, [d.table, d.ref])
    moved(lambda: g.compact_pages(d.table, d.ref, caches), [d.table, d.ref] + caches, [d.lens])
    moved(lambda: g.copy_slots(caches, ints([0]), ints([3])), caches)
    q, k, v = (torch.randn(2, 2, 64, device=DEV) for _ in range(3))
    kc, vc, out = torch.zeros(4, 16, 2, 64, device=DEV), torch.zeros(4, 16, 2, 64, device=DEV), torch.zeros_like(q)
    cs, table, lens, pos = torch.ones(8, 32, 2, device=DEV), ints([[0], [1]]), ints([1, 1]), ints([0, 1])
    moved(lambda: g.rotary(q, k, cs, pos, inplace=True), [q, k], [cs, pos])
    moved(lambda: g.rotary(q, k, cs, pos), [], [q, k])
    moved(lambda: g.rotary_append(q, k, v, cs, kc, vc, table, lens), [kc, vc], [q, k, v, table, lens])
    moved(lambda: g.paged_attention(q, kc, vc, table, lens, out=out), [out], [q, kc, vc])
    x, r, w = torch.randn(3, 64, device=DEV), torch.randn(3, 64, device=DEV), torch.ones(64, device=DEV)
    moved(lambda: g.rms_norm(x, w, r), [], [x, r, w])
    moved(lambda: g.rms_norm(x, w, r, inplace=True), [r], [x, w])
    a = torch.randn(3, 64, device=DEV, requires_grad=True)
    y = (a * r).sum()                            # saves r
    g.rms_norm(x, w, r, inplace=True)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():
        x, r = torch.randn(3, 64, device=DEV), torch.randn(3, 64, device=DEV)
        g.rms_norm(x, w, r, inplace=True)
    g.rms_norm(x, w, r, inplace=True)


@gpu
def test_binding_refuses_pools_of_too_few_slots():
    """[layers, pages, ...] in place of one tensor for each layer, or states of another batch; more slots are no fault."""
    import gated_deltanet_linear_15_gb300 as g
    table, lens, ref = ints([[0, -1], [-1, -1]]), ints([3, 0]), ints([1, 0, 0])
    good, layers = torch.zeros(4, 16, device=DEV), torch.zeros(2, 3, 16, device=DEV)
    for pools, states in (([layers], []), ([good, good[:2]], []), ([good], [good[:1]]), ([good[:0]], [])):
        with pytest.raises(ValueError, match="slots"):
            g.fork_pages(table, lens, ref, ints([0]), ints([1]), pools, 16, states)
        if not states:
            with pytest.raises(ValueError, match="slots"):
                g.compact_pages(table, ref, pools)
    assert table.tolist() == [[0, -1], [-1, -1]] and ref.tolist() == [1, 0, 0] and lens.tolist() == [3, 0]
    good[0] = 5
    assert g.fork_pages(table, lens, ref, ints([0]), ints([1]), [good], 16, [good]).tolist() == [1]
    assert (good[1] == 5).all() and table.tolist() == [[0, -1], [1, -1]]


# ------------------------------------------------------------------ refusals of the C entry points (no GPU needed)
def _shape(**kw):
    s = _lib.GdnPagesShape()
    s.num_seqs, s.max_pages, s.num_pages, s.page_size, s.table_stride = 4, 8, 100, 16, 8
    for k, v in kw.items():
        if k == "reserved":
            s.reserved[1] = v
        else:
            setattr(s, k, v)
    return s


@pytest.mark.parametrize("kw", [dict(num_seqs=0), dict(max_pages=0), dict(num_pages=0), dict(num_pages=(1 << 20) + 1),
                                dict(page_size=0), dict(table_stride=7), dict(reserved=1)])
def test_c_entries_refuse_shapes(lib, kw):
    s, p, big = _shape(**kw), 0x10000, 1 << 40
    ref = ctypes.byref(s)
    assert lib.gdn_pages_extend(ref, p, p, p, p, p, 1, p, p, big, None) != 0
    assert lib.gdn_pages_fork(ref, p, p, p, p, p, 1, None, 0, None, 0, p, p, big, None) != 0
    assert lib.gdn_pages_free(ref, p, p, p, p, 1, None) != 0
    assert lib.gdn_pages_compact(ref, p, p, p, p, None, 0, None, p, big, None) != 0
    assert lib.gdn_pages_workspace_size(ref, 4) == 0
    assert lib.gdn_last_error_string() != b""


def test_c_entries_refuse_pools_of_too_few_slots(lib):
    """A pool that lacks the slots would lose what the tables go on to name."""
    s, p, big = _shape(), 0x10000, 1 << 40
    ref, pool = ctypes.byref(s), (_lib.GdnSlotPool * 1)()
    pool[0].base, pool[0].stride, pool[0].bytes = 0x10000, 32, 32
    for slots, least in ((99, b"100"), (2, b"100"), (0, b"100")):
        pool[0].slots = slots
        assert lib.gdn_pages_fork(ref, p, p, p, p, p, 1, pool, 1, None, 0, p, p, big, None) == 1
        assert least in lib.gdn_last_error_string()
        assert lib.gdn_pages_compact(ref, p, p, p, p, pool, 1, None, p, big, None) == 1
        assert least in lib.gdn_last_error_string()
    pool[0].slots = 3
    assert lib.gdn_pages_fork(ref, p, p, p, p, p, 1, None, 0, pool, 1, p, p, big, None) == 1
    assert b"states" in lib.gdn_last_error_string()


def test_c_entries_refuse_arguments(lib):
    s, p, big = _shape(), 0x10000, 1 << 40
    ref = ctypes.byref(s)
    need = lib.gdn_pages_workspace_size(ref, 5)
    assert need > 0 and lib.gdn_pages_workspace_size(ref, -1) == 0
    for i in range(5):
        a = [p] * 5
        a[i] = None
        assert lib.gdn_pages_extend(ref, *a, 5, p, p, big, None) == 1
        assert lib.gdn_pages_fork(ref, *a, 5, None, 0, None, 0, p, p, big, None) == 1
    for i in range(4):
        a = [p] * 4
        a[i] = None
        assert lib.gdn_pages_free(ref, *a, 5, None) == 1
        assert lib.gdn_pages_compact(ref, *a, None, 0, None, p, big, None) == 1
    assert lib.gdn_pages_extend(ref, p, p, p, p, p, 5, None, p, big, None) == 1
    assert lib.gdn_pages_extend(ref, p, p, p, p, p, 5, p, p, need - 1, None) == 3
    assert lib.gdn_pages_extend(ref, p, p, p, p, p, 5, p, None, big, None) == 3
    assert lib.gdn_pages_extend(ref, p, p, p, p, p, -1, p, p, big, None) == 1
    assert lib.gdn_pages_extend(ref, p, p, p, p, p, 0, p, p, big, None) == 0
    assert lib.gdn_pages_free(ref, p, p, p, p, 0, None) == 0
    pool = (_lib.GdnSlotPool * 1)()
    for kw in (dict(base=None), dict(base=0x10008), dict(stride=24), dict(bytes=40), dict(bytes=8), dict(bytes=-16), dict(slots=-1)):
        pool[0].base, pool[0].stride, pool[0].bytes, pool[0].slots = 0x10000, 32, 32, 4
        for k, v in kw.items():
            setattr(pool[0], k, v)
        assert lib.gdn_slots_copy(pool, 1, p, p, 1, None) == 1, kw
        assert lib.gdn_pages_fork(ref, p, p, p, p, p, 1, pool, 1, None, 0, p, p, big, None) == 1, kw
    assert lib.gdn_slots_copy(None, 1, p, p, 1, None) == 1
    assert lib.gdn_slots_copy(None, -1, p, p, 1, None) == 1
    assert lib.gdn_slots_copy(None, 0, p, p, -1, None) == 1
