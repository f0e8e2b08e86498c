"""Operations on a cache's pages against the oracle, whole number for whole
number, and the bytes they move; then a serving loop of all of them together
with the attention that reads the cache."""
import numpy as np
import pytest
import torch

import oracle
import paged_cases as P
from block_sparse_attention_slice_gb300 import (attn_cache_compact, attn_cache_copy_pages, attn_cache_extend, attn_cache_fork,
                                                attn_cache_free, attn_cache_trim, attn_cache_write, attn_last_device_error,
                                                attn_paged_fwd, attn_prefix_fwd)
from block_sparse_attention_slice_gb300 import binding as B

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Both:
    """A cache on the GPU and the oracle's, changed alike and compared."""

    def __init__(self, n_slots, max_pages, n_pages, page, stride=0):
        self.o = oracle.CacheOracle(n_slots, max_pages, n_pages, page)
        self.page = page
        self.table = torch.full((n_slots, max_pages + stride), -1, dtype=torch.int32, device="cuda")[:, :max_pages]
        self.lens = torch.zeros(n_slots, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")

    @property
    def c(self):
        return self.table, self.lens, self.refs

    def same(self, status=0):
        assert attn_last_device_error() == status
        assert self.lens.tolist() == self.o.lens
        assert self.table.tolist() == self.o.table()
        assert self.refs.tolist() == self.o.refs

    def extend(self, seqs, counts):
        attn_cache_extend(*self.c, ints(seqs), ints(counts), self.page)
        self.same(0 if self.o.extend(seqs, counts) else B.ATTN_ERR_CAPACITY)

    def free(self, seqs):
        attn_cache_free(*self.c, ints(seqs), self.page)
        self.o.free(seqs)
        self.same()

    def trim(self, window, sinks, seqs=None):
        attn_cache_trim(*self.c, self.page, window, sinks, None if seqs is None else ints(seqs))
        self.o.trim(range(len(self.o.rows)) if seqs is None else seqs, window, sinks)
        self.same()

    def _list(self, copies, want):
        n = (len(copies) - 1) // 2
        got = copies.tolist()
        assert got[0] == len(want)
        assert list(zip(got[1:1 + n], got[1 + n:])) == want + [(-1, -1)] * (n - len(want))
        return copies

    def fork(self, src, dst):
        copies = attn_cache_fork(*self.c, ints(src), ints(dst), self.page)
        want = self.o.fork(src, dst)
        self.same(0 if want is not None else B.ATTN_ERR_CAPACITY)
        if want is None:
            assert int(copies[0]) == 0
            return copies
        return self._list(copies, want)

    def compact(self):
        copies = attn_cache_compact(*self.c, self.page)
        want = self.o.compact()
        self.same()
        return self._list(copies, want)


SIZES = [(4, 5, 12, 16, 0), (50, 40, 1000, 16, 3), (7, 300, 1501, 64, 0), (300, 9, 2000, 128, 1), (1000, 20, 40000, 16, 0),
         (20, 2000, 33333, 32, 0), (4096, 3, 9001, 16, 0)]


@pytest.mark.parametrize("n_slots,max_pages,n_pages,page,stride", SIZES)
@pytest.mark.parametrize("seed", range(2))
def test_random_rounds(n_slots, max_pages, n_pages, page, stride, seed):
    rng = np.random.default_rng(seed)
    b = Both(n_slots, max_pages, n_pages, page, stride)
    for _ in range(14):
        n = int(rng.integers(0, n_slots + 1))
        seqs = rng.permutation(n_slots)[:n].tolist()
        what = rng.integers(0, 6)
        if what <= 1:
            room = [max_pages * page - b.o.lens[s] for s in seqs]
            most = [int(min(r, 1 + 1.5 * n_pages * page / n_slots)) for r in room]
            b.extend(seqs, [int(rng.integers(0, m + 1)) for m in most])
        elif what == 2:
            b.free(seqs[:len(seqs) // 2])
        elif what == 3:
            b.fork(rng.integers(0, n_slots, n).tolist(), seqs)
        elif what == 4:
            b.trim(int(rng.integers(1, max_pages * page)), int(rng.integers(0, 3 * page)), seqs if rng.integers(2) else None)
        else:
            b.compact()


def test_growth_of_a_partial_page_and_by_nothing():
    b = Both(3, 4, 8, 16)
    b.extend([2, 0], [5, 16])
    b.extend([2], [11])           # up to the page's end: no page is taken
    b.extend([2, 1, 0], [1, 0, 0])
    b.extend([], [])
    b.extend([0], [16 * 4 - 16])  # up to the table's end
    b.extend([0], [1])            # past it: refused
    b.extend([1], [3 * 16])       # more than the free pages: refused
    b.extend([1], [2 * 16])


def test_fork_in_place_swap_and_capacity():
    b = Both(4, 4, 8, 16)
    b.extend([0, 1], [20, 33])
    b.fork([1, 0], [0, 1])                    # swapped: nothing copied
    b.fork([0, 0, 0], [0, 2, 3])              # the source goes on as its first child
    b.fork([0, 0], [1, 1 + 1])                # more copies than free pages: see same()
    b.fork([3, 3, 3, 3], [0, 1, 2, 3])
    b.free([0, 1, 2, 3])


@pytest.mark.parametrize("what", ["twice", "below", "above"])
def test_bad_lists_change_nothing(what):
    b = Both(5, 4, 30, 16)
    b.extend([0, 1, 2, 3, 4], [20, 33, 0, 64, 1])
    bad = {"twice": [1, 3, 1], "below": [1, -1, 2], "above": [1, 2, 5]}[what]
    c = b.c
    for call in (lambda: attn_cache_extend(*c, ints(bad), ints([1, 1, 1]), 16), lambda: attn_cache_free(*c, ints(bad), 16),
                 lambda: attn_cache_trim(*c, 16, 1, 0, ints(bad)), lambda: attn_cache_fork(*c, ints([0, 1, 2]), ints(bad), 16)):
        copies = call()
        b.same(B.ATTN_ERR_INVALID_ARG)
        assert copies is None or int(copies[0]) == 0
    if what != "twice":                       # a source may be named twice
        attn_cache_fork(*c, ints(bad), ints([2, 3, 4]), 16)
        b.same(B.ATTN_ERR_INVALID_ARG)
    attn_cache_extend(*c, ints([0, 1]), ints([1, -1]), 16)
    b.same(B.ATTN_ERR_INVALID_ARG)


def test_lists_of_more_entries_than_32_bits_count_are_refused():
    b = Both(2, 2, 4, 16)
    x = torch.empty(2 ** 31, dtype=torch.int32, device="cuda")
    for call in (lambda: attn_cache_extend(*b.c, x, x, b.page), lambda: attn_cache_free(*b.c, x, b.page),
                 lambda: attn_cache_trim(*b.c, b.page, 1, 0, x), lambda: attn_cache_fork(*b.c, x, x, b.page)):
        with pytest.raises(ValueError, match="out of range"):
            call()
    b.same()


def test_bad_lengths_and_pages_are_not_followed():
    b = Both(4, 4, 10, 16)
    b.extend([0, 1], [40, 16])
    for bad in (-3, 65):
        keep = b.lens.clone()
        b.lens[0] = bad
        table, refs = b.table.clone(), b.refs.clone()
        attn_cache_free(*b.c, ints([1, 0]), 16)
        attn_cache_extend(*b.c, ints([0]), ints([1]), 16)
        attn_cache_fork(*b.c, ints([0]), ints([2]), 16)
        attn_cache_compact(*b.c, 16)
        assert attn_last_device_error() == B.ATTN_ERR_INVALID_ARG
        assert torch.equal(table, b.table) and torch.equal(refs, b.refs)
        b.lens.copy_(keep)
    b.table[0, 1] = 10 ** 8
    attn_cache_free(*b.c, ints([0]), 16)
    assert attn_last_device_error() == B.ATTN_ERR_INVALID_ARG
    assert b.refs.tolist() == [0, 1, 0, 1] + [0] * 6 and b.lens.tolist() == [0, 16, 0, 0]


@pytest.mark.parametrize("shape,dtype", [((16, 2, 64), torch.bfloat16), ((16, 1, 128), torch.float32), ((5, 8), torch.int16),
                                         ((64, 8, 128), torch.bfloat16), ((33, 8, 24), torch.int32)])
@pytest.mark.parametrize("n_pools", [1, 3, 256])
def test_copies(shape, dtype, n_pools):
    n = 20
    make = lambda: torch.randint(-100, 100, (n, *shape), device="cuda").to(dtype)  # noqa: E731
    # every other pool's pages are the inner part of wider ones would differ in
    # stride, so all are alike: a column of a wider array
    pools = [torch.stack([make(), make()], 1)[:, 0] for _ in range(n_pools)]
    want = [x.clone() for x in pools]
    pairs = [(3, 0), (3, 19), (7, 1), (18, 4)]
    for x in want:
        for a, b in pairs:
            x[b] = x[a]
    cap = 6
    copies = ints([len(pairs)] + [a for a, _ in pairs] + [9, 9] + [b for _, b in pairs] + [10, 10])
    assert copies.shape[0] == 1 + 2 * cap
    attn_cache_copy_pages(pools, copies)
    assert attn_last_device_error() == 0
    for x, y in zip(pools, want):
        assert torch.equal(x, y)
    # pairs out of range are left out, and a count beyond the list is cut
    want = [x.clone() for x in pools]
    for x in want:
        x[2] = x[5]
    copies = ints([99, n, 5, 4, 1, 2, -1])
    attn_cache_copy_pages(pools, copies)
    assert attn_last_device_error() == B.ATTN_ERR_INVALID_ARG
    for x, y in zip(pools, want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("hk,d,page", [(1, 64, 16), (8, 128, 64), (3, 64, 32), (16, 128, 16)])
@pytest.mark.parametrize("packed", [False, True])
def test_writes(hk, d, page, packed):
    lens, news, T = [40, 0, 17, 100], [5, 0, 17, 1], 26
    c = P.make(lens, news, page, hk, hk, d, seed=1, slots=[3, 0, 1, 5], garbage=0.0)
    x = torch.randn((T, 3 * hk, d), device="cuda").bfloat16()
    k_new, v_new = (x[:, hk:2 * hk], x[:, 2 * hk:]) if packed else (x[:, :hk].contiguous(), x[:, hk:2 * hk].contiguous())
    want = [c["k"].clone(), c["v"].clone()]
    t = 0
    for b, (n, new) in enumerate(zip(lens, news)):
        for j in range(n - new, n):
            at = int(c["table"][c["seqs"][b], j // page])
            want[0][at, j % page], want[1][at, j % page] = k_new[t], v_new[t]
            t += 1
    attn_cache_write(c["k"], c["v"], k_new, v_new, c["d_table"], c["d_lens"], q_ptr=c["d_q_ptr"], seqs=c["d_seqs"])
    assert attn_last_device_error() == 0
    assert torch.equal(c["k"], want[0]) and torch.equal(c["v"], want[1])
    # a page out of range, a slot out of range, a sequence shorter than its new tokens
    c["d_table"][3, 2 if page == 16 else 32 // page if page == 32 else 0] = -7
    c["d_seqs"][2] = 6
    c["d_lens"][5] = 0
    keep = c["k"].clone()
    attn_cache_write(c["k"], c["v"], -k_new, -v_new, c["d_table"], c["d_lens"], q_ptr=c["d_q_ptr"], seqs=c["d_seqs"])
    assert attn_last_device_error() == B.ATTN_ERR_INVALID_ARG
    changed = (c["k"] != keep).flatten(2).any(-1).nonzero()
    assert all(int(p) in c["table"][3] for p, _ in changed)


def test_one_write_a_sequence_for_many_sequences():
    n, page, hk, d = 4000, 16, 2, 64
    b = Both(n, 2, 8100, page)
    lens = (torch.arange(n) % 20 + 1).tolist()
    b.extend(list(range(n)), lens)
    k, v = (torch.zeros((8100, page, hk, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    new = torch.randn((n, hk, d), device="cuda").bfloat16()
    attn_cache_write(k, v, new, -new, b.table, b.lens)
    at = torch.tensor([b.o.rows[i][(m - 1) // page] for i, m in enumerate(lens)], device="cuda")
    pos = torch.tensor([(m - 1) % page for m in lens], device="cuda")
    assert torch.equal(k[at, pos], new) and torch.equal(v[at, pos], -new)
    assert attn_last_device_error() == 0


def test_captured_operations_read_their_lists_when_replayed():
    b = Both(6, 8, 60, 16)
    b.extend([0, 1, 2], [50, 60, 70])
    seqs, counts = ints([3, 4]), ints([20, 40])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attn_cache_free(*b.c, seqs, 16)
        attn_cache_extend(*b.c, seqs, counts, 16)
        copies = attn_cache_compact(*b.c, 16)
    for step in range(3):
        s, n = [[3, 4], [0, 1], [2, 5]][step], [[20, 40], [3, 0], [64, 17]][step]
        seqs.copy_(ints(s))
        counts.copy_(ints(n))
        g.replay()
        b.o.free(s)
        assert b.o.extend(s, n)
        want = b.o.compact()
        b.same()
        b._list(copies, want)


def test_a_serving_loop_of_all_of_them():
    """Prompts are admitted and written, forked, decoded token by token through
    a window, trimmed, compacted and retired; each step's attention is that of
    the tokens that every sequence was really given."""
    rng = np.random.default_rng(0)
    page, hq, hk, d, window, sinks, n_slots, n_pages = 16, 4, 2, 64, 40, 3, 8, 60
    b = Both(n_slots, 16, n_pages, page)
    kv = [torch.full((n_pages, page, hk, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    given = {}                                             # slot -> keys, values of every token so far

    def append(slots, counts):
        b.extend(slots, counts)
        new = torch.from_numpy(rng.standard_normal((2, sum(counts), hk, d)).astype(np.float32)).bfloat16().cuda()
        ptr = np.concatenate([[0], np.cumsum(counts)])
        attn_cache_write(kv[0], kv[1], new[0], new[1], b.table, b.lens, q_ptr=ints(ptr), seqs=ints(slots))
        for i, s in enumerate(slots):
            old = given.get(s, torch.zeros((2, 0, hk, d), dtype=torch.bfloat16, device="cuda"))
            given[s] = torch.cat([old, new[:, ptr[i]:ptr[i + 1]]], 1)
        attend(slots, counts)

    def attend(slots, counts):
        q = torch.from_numpy(rng.standard_normal((sum(counts), hq, d)).astype(np.float32)).bfloat16().cuda()
        ptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        out, lse = attn_paged_fwd(q, kv[0], kv[1], b.table, b.lens, 0.2, q_ptr=ints(ptr), seqs=ints(slots), window=window, sinks=sinks)
        assert attn_last_device_error() == 0
        longest = max(given[s].shape[1] for s in slots)
        k, v = np.zeros((2, len(slots), longest, hk, d))
        for i, s in enumerate(slots):
            k[i, :given[s].shape[1]], v[i, :given[s].shape[1]] = given[s].double().cpu().numpy()
        lens = [given[s].shape[1] for s in slots]
        ref = oracle.oracle_paged(q.double().cpu().numpy(), k, v, np.arange(len(slots))[:, None], lens, ptr, 0.2, window, sinks)
        P.check({"lens": lens, "plens": []}, out, lse, ref)

    append([5, 1, 2], [70, 16, 33])
    attn_cache_copy_pages(kv, b.fork([5, 5, 2], [0, 3, 4]))
    given.update({0: given[5], 3: given[5], 4: given[2]})
    for step in range(6):
        append([0, 1, 3, 4, 5], [1, 2, 1, 1 + step, 1])
        if step == 2:
            attn_cache_copy_pages(kv, b.fork([3, 3, 0], [3, 5, 7]))     # a beam search's step
            given.update({5: given[3], 7: given[0]})
        if step == 3:
            b.trim(window, sinks)
            b.free([1, 2])
            given[1] = given[2] = None
            attn_cache_copy_pages(kv, b.compact())
            given.pop(1)
            given.pop(2)
    append([2, 7], [100, 3])
    attend([7, 2, 0, 3], [1, 1, 1, 1])
    b.free(list(range(8)))
    assert b.refs.sum() == 0


def test_a_shared_prefix_is_that_of_forked_rows():
    """Rows forked from one prompt see the same through their own tables as
    through the prompt's pages as a shared prefix."""
    page, hq, hk, d, n = 16, 8, 2, 128, 20
    b = Both(n + 1, 40, 400, page)
    kv = [torch.zeros((400, page, hk, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    prompt = torch.randn((2, 320, hk, d), device="cuda").bfloat16()
    b.extend([n], [320])                                   # whole pages: the tables' next column starts the answers
    attn_cache_write(kv[0], kv[1], prompt[0], prompt[1], b.table, b.lens, q_ptr=ints([0, 320]), seqs=ints([n]))
    b.fork([n] * n, list(range(n)))
    more = [1 + i for i in range(n)]
    b.extend(list(range(n)), more)
    new = torch.randn((2, sum(more), hk, d), device="cuda").bfloat16()
    ptr = ints(np.concatenate([[0], np.cumsum(more)]))
    attn_cache_write(kv[0], kv[1], new[0], new[1], b.table, b.lens, q_ptr=ptr, seqs=ints(list(range(n))))
    q = torch.randn((n, hq, d), device="cuda").bfloat16()
    a = attn_paged_fwd(q, *kv, b.table[:n], b.lens[:n], 0.1, out_dtype=torch.float32)
    c = attn_prefix_fwd(q, *kv, b.table[n:], b.lens[n:], ints([0, n]), b.table[:n, 20:], b.lens[:n] - 320, 0.1, out_dtype=torch.float32)
    assert attn_last_device_error() == 0
    # P's roundings fall differently only where the running maxima differ: 2^-8 of sum p |v| on each side
    assert (a[0] - c[0]).abs().max() <= 2 * 2.0 ** -8 * float(kv[1].abs().max())
    assert torch.allclose(a[1], c[1], atol=1e-5, rtol=1e-6)


@pytest.mark.parametrize("n", [33, 64, 1000, 1025, 4096])
@pytest.mark.parametrize("bad", [-1, 16 * 3 + 1])
def test_one_bad_length_in_a_long_list_changes_nothing(n, bad):
    # the row with the bad length in the first warp of the list, in the middle and in the last one
    b = Both(n, 3, 4096, 16)
    b.extend(list(range(0, n, 7)), [1 + i % 40 for i in range(0, n, 7)])
    rows = np.random.default_rng(n).permutation(n).tolist()
    for at in (0, n // 2, n - 1):
        good = int(b.lens[rows[at]])
        calls = [lambda: attn_cache_free(*b.c, ints(rows), 16), lambda: attn_cache_trim(*b.c, 16, 1, 0, ints(rows)),
                 lambda: attn_cache_trim(*b.c, 16, 1, 0), lambda: attn_cache_extend(*b.c, ints(rows), ints([1] * n), 16),
                 lambda: attn_cache_fork(*b.c, ints(rows), ints(rows[1:] + rows[:1]), 16), lambda: attn_cache_compact(*b.c, 16)]
        for call in calls:
            b.lens[rows[at]] = bad
            call()
            assert attn_last_device_error() == B.ATTN_ERR_INVALID_ARG
            assert int(b.lens[rows[at]]) == bad
            b.lens[rows[at]] = good
            b.same()


@pytest.mark.parametrize("n,hq,hk,d,new", [(6, 8, 2, 128, 1), (40, 4, 4, 64, 1), (6, 8, 1, 128, 40)])
def test_calls_behind_one_another_read_what_the_one_before_wrote(n, hq, hk, d, new):
    # each call starts while the one before drains; the same rounds with the
    # GPU waited for behind every call, one after the other, and in one graph
    rng, page, n_pages, rounds = np.random.default_rng(n), 16, 40 * n, 24
    start = Both(2 * n, 20, n_pages, page)
    kv = [torch.zeros((n_pages, page, hk, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    plans = []
    for _ in range(rounds):
        ids = rng.permutation(2 * n)[:n]
        counts = rng.integers(new, 200, n)
        x = torch.from_numpy(rng.standard_normal((2, int(counts.sum()), hk, d)).astype(np.float32)).bfloat16().cuda()
        q = torch.from_numpy(rng.standard_normal((2, n * new, hq, d)).astype(np.float32)).bfloat16().cuda()
        src, dst = rng.permutation(2 * n)[:n // 2], rng.permutation(2 * n)[:n // 2]
        plans.append([ints(ids), ints(counts), ints(np.concatenate([[0], np.cumsum(counts)])), x, q, ints(src), ints(dst)])
    ptr, groups = ints(list(range(0, n * new + 1, new))), ints([0, n // 2, n])

    def go(table, lens, refs, pools, wait):
        got = []
        for ids, counts, starts, x, q, src, dst in plans:
            attn_cache_free(table, lens, refs, ids, page)
            wait()
            attn_cache_extend(table, lens, refs, ids, counts, page)
            wait()
            attn_cache_write(pools[0], pools[1], x[0], x[1], table, lens, q_ptr=starts, seqs=ids)
            wait()
            got += attn_paged_fwd(q[0], *pools, table, lens, 0.1, q_ptr=ptr, seqs=ids, max_q=new, out_dtype=torch.float32)
            wait()
            copies = attn_cache_fork(table, lens, refs, src, dst, page)
            wait()
            attn_cache_copy_pages(pools, copies)
            wait()
            got += attn_prefix_fwd(q[1], *pools, table[:2], lens[:2], groups, table, lens, 0.1, q_ptr=ptr, seqs=ids, max_q=new,
                                   out_dtype=torch.float32)
            wait()
        return got + [copies]

    def fresh():
        return [x.clone() for x in start.c] + [[x.clone() for x in kv]]

    want_state = fresh()
    want = go(*want_state, torch.cuda.synchronize)
    assert attn_last_device_error() == 0
    state = fresh()
    torch.cuda.synchronize()
    got = go(*state, lambda: None)
    captured = fresh()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        replayed = go(*captured, lambda: None)
    g.replay()
    assert attn_last_device_error() == 0
    for mine, s in ((got, state), (replayed, captured)):
        for a, b in zip(mine + s[:3] + s[3], want + want_state[:3] + want_state[3]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("bad_page", [-7, -1, 10 ** 8, "n_pages"])
@pytest.mark.parametrize("bad_slot", [-1, "n_slots", 2 ** 31 - 1])
@pytest.mark.parametrize("hk,d", [(3, 64), (8, 128)])
def test_a_write_leaves_out_just_the_tokens_that_have_no_place(bad_page, bad_slot, hk, d):
    # sequence 0: its second page is good, its third not; 1: a slot that is none;
    # 2: as it should be; 3: two new tokens, but one in its length
    page, lens, news = 16, [40, 20, 17, 1], [20, 5, 17, 2]
    c = P.make(lens, news, page, hk, hk, d, seed=1, slots=[3, 0, 1, 5], garbage=0.0)
    n_pages, n_slots = c["k"].shape[0], c["table"].shape[0]
    k_new, v_new = torch.randn((2, sum(news), hk, d), device="cuda").bfloat16()
    want = [c["k"].clone(), c["v"].clone()]
    t = 0
    for b, (n, new) in enumerate(zip(lens, news)):
        for j in range(n - new, n):
            if j >= 0 and b != 1 and (b, j // page) != (0, 2):
                at = int(c["table"][c["seqs"][b], j // page])
                want[0][at, j % page], want[1][at, j % page] = k_new[t], v_new[t]
            t += 1
    c["d_table"][3, 2] = n_pages if bad_page == "n_pages" else bad_page
    c["d_seqs"][1] = n_slots if bad_slot == "n_slots" else bad_slot
    attn_cache_write(c["k"], c["v"], k_new, v_new, c["d_table"], c["d_lens"], q_ptr=c["d_q_ptr"], seqs=c["d_seqs"])
    assert attn_last_device_error() == B.ATTN_ERR_INVALID_ARG
    assert torch.equal(c["k"], want[0]) and torch.equal(c["v"], want[1])


def test_lists_of_no_rows_change_nothing():
    b = Both(3, 6, 20, 16)
    b.extend([0, 2], [70, 33])
    b.extend([], [])
    b.free([])
    b.trim(5, 0, [])
    b.fork([], [])
    empty = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros((2, 20, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = attn_paged_fwd(empty, kv[0], kv[1], b.table, b.lens, 0.1, seqs=ints([]))
    assert out.shape == (0, 2, 64) and lse.shape == (2, 0)
    out, lse = attn_prefix_fwd(empty, kv[0], kv[1], b.table[:1], b.lens[:1], ints([0, 0]), b.table, b.lens, 0.1, seqs=ints([]))
    assert out.shape == (0, 2, 64) and lse.shape == (2, 0)
    attn_cache_write(kv[0], kv[1], empty, empty, b.table, b.lens, seqs=ints([]))
    attn_cache_copy_pages([], ints([0]))
    attn_cache_copy_pages([kv[0]], ints([0]))
    b.same()
    assert not kv.any()
    with pytest.raises(B.AttnError):
        attn_cache_trim(*b.c, 16, 0, 0, ints([]))      # its other arguments are looked at all the same
    b.trim(5, 0)
