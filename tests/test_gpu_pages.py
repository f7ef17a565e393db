"""The page calls on the GPU against their definitions as plain lists (tests/serve_ref.py)."""
import pytest
import torch

from kv_cache_compression_02_gb300 import cachegen as cg
from tests import gpu_util as gu
from tests import serve_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    gu.ready()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Setup:
    """A cache with pools of random bytes, its bookkeeping, and the plain lists beside it."""

    def __init__(self, n_blocks, bt, lens, n_seqs, width, L=2, H=2, d=16, fmt=cg.CG_CACHE_E4M3, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.cache = cg.Cache(L, H, d, bt, n_blocks, fmt)
        size = 2 if fmt == cg.CG_CACHE_F16 else 1
        self.pools = [torch.randint(0, 256, (n_blocks, H, bt, d * size), generator=g, dtype=torch.uint8).cuda() for _ in range(2 * L)]
        self.scales = [torch.rand(n_blocks, H, generator=g).cuda() for _ in range(2 * L)]
        self.was = [t.clone() for t in self.pools], [t.clone() for t in self.scales]
        self.pool_ptrs = torch.tensor([t.data_ptr() for t in self.pools], dtype=torch.int64).cuda()
        self.scale_ptrs = None if fmt == cg.CG_CACHE_F16 else torch.tensor([t.data_ptr() for t in self.scales], dtype=torch.int64).cuda()
        order, at = torch.randperm(n_blocks, generator=g).tolist(), 0
        refs, table = [0] * n_blocks, [[-1] * width for _ in range(n_seqs)]
        for s, n in enumerate(lens):
            for j in range(-(-n // bt)):
                table[s][j], refs[order[at]], at = order[at], 1, at + 1
        self.book = ref.Book(refs, table, lens + [0] * (n_seqs - len(lens)), bt)
        self.refs, self.table, self.lens = i32(refs), i32(table), i32(self.book.lens)
        self.pages = cg.Pages(self.refs, self.table, self.lens)
        self.ws = cg.empty_u8(cg.cg_pages_workspace_bytes(self.cache, self.pages, 64))
        self.ws.fill_(0xA5)

    def status(self, rc):
        assert rc == cg.CG_OK
        torch.cuda.synchronize()
        return cg.cg_read_status(self.ws)

    def fork(self, parents, children):
        return self.status(cg.cg_pages_fork(self.cache, self.pages, self.pool_ptrs, self.scale_ptrs, i32(parents), i32(children), self.ws))

    def extend(self, seqs, lens):
        return self.status(cg.cg_pages_extend(self.cache, self.pages, i32(seqs), i32(lens), self.ws))

    def free(self, seqs):
        return self.status(cg.cg_pages_free(self.cache, self.pages, i32(seqs), self.ws))

    def same_book(self):
        assert self.refs.tolist() == self.book.refs
        assert self.table.tolist() == self.book.table
        assert self.lens.tolist() == self.book.lens

    def same_pools(self, moves):
        for kept, now in zip(self.was, (self.pools, self.scales if self.scale_ptrs is not None else [])):
            for w, t in zip(kept, now):
                for s, d in moves:
                    w[d] = w[s]
                assert torch.equal(w.view(torch.uint8), t.view(torch.uint8))


@pytest.mark.parametrize("bt,d,fmt", [(16, 16, cg.CG_CACHE_E4M3), (7, 8, cg.CG_CACHE_INT8), (1, 8, cg.CG_CACHE_E4M3), (64, 128, cg.CG_CACHE_F16)])
def test_a_life_of_pages(bt, d, fmt):
    """Extend, fork, extend, free, fork again, compact: the lists, and every byte of the pools, as defined."""
    H = 1 if bt == 1 else 2
    s = Setup(200, bt, [3 * bt + 1 if bt > 1 else 4, 2 * bt, 1], n_seqs=12, width=9, H=H, d=d, fmt=fmt)
    b, moves = s.book, []
    assert s.extend([3, 0], [5 * bt, 4 * bt + (bt > 1)]) == cg.CG_OK and b.extend([3, 0], [5 * bt, 4 * bt + (bt > 1)])
    s.same_book()
    assert s.fork([0, 0, 1, 2, 0], [4, 5, 6, 7, 11]) == cg.CG_OK
    m = b.fork([0, 0, 1, 2, 0], [4, 5, 6, 7, 11])
    s.same_book()
    s.same_pools(m)
    assert s.extend([4, 7], [6 * bt, 1]) == cg.CG_OK and b.extend([4, 7], [6 * bt, 1])
    assert s.free([0, 5, 8]) == cg.CG_OK
    b.free([0, 5, 8])
    s.same_book()
    assert s.fork([4, 11], [0, 5]) == cg.CG_OK
    s.same_pools(b.fork([4, 11], [0, 5]))
    s.same_book()
    refs, table, n_live = torch.full_like(s.refs, -9), torch.full_like(s.table, -9), i32([-9])
    rc = cg.cg_pages_compact(s.cache, s.pages, s.pool_ptrs, s.scale_ptrs, refs, table, n_live, s.ws)
    assert s.status(rc) == cg.CG_OK
    s.same_book()  # the input stays
    live, m = b.compact()
    assert (n_live.tolist(), refs.tolist(), table.tolist()) == ([live], b.refs, b.table)
    s.same_pools(m)


def test_compact_in_place_large():
    """50,000 pages, the counts and table written over themselves."""
    lens = [i % 40 for i in range(600)]
    s = Setup(50000, 4, lens, n_seqs=700, width=11, L=1, H=1, d=8)
    s.fork([5, 5, 39], [650, 651, 652])
    s.same_pools(s.book.fork([5, 5, 39], [650, 651, 652]))
    n_live = i32([0])
    rc = cg.cg_pages_compact(s.cache, s.pages, s.pool_ptrs, s.scale_ptrs, s.refs, s.table, n_live, s.ws)
    assert s.status(rc) == cg.CG_OK
    live, m = s.book.compact()
    assert n_live.tolist() == [live]
    s.same_book()
    s.same_pools(m)


def test_compact_full_and_empty():
    for lens, n in (([], 33), ([16] * 33, 33)):
        s = Setup(n, 16, lens, n_seqs=40, width=2)
        n_live = i32([7])
        rc = cg.cg_pages_compact(s.cache, s.pages, s.pool_ptrs, s.scale_ptrs, s.refs, s.table, n_live, s.ws)
        assert s.status(rc) == cg.CG_OK and n_live.tolist() == [len(lens)]
        s.same_book()
        s.same_pools([])


def test_extend_many_and_to_the_last_page():
    s = Setup(5000, 16, [5], n_seqs=1500, width=4)
    seqs, lens = list(range(1499, -1, -1)), [(i * 13) % 60 + (5 if i == 1499 else 0) for i in range(1500)]
    s.ws = cg.empty_u8(cg.cg_pages_workspace_bytes(s.cache, s.pages, 1500))
    assert s.extend(seqs, lens) == cg.CG_OK and s.book.extend(seqs, lens)
    s.same_book()
    left = len(s.book.free_pages())
    room = [i for i in range(1500) if s.book.lens[i] <= 16][:]
    # one page more than there are: nothing changes
    grow = []
    for q in room:
        take = 4 - s.book.pages(s.book.lens[q])
        grow.append((q, 64))
        left -= take
        if left < 0:
            break
    if left < 0:
        assert s.extend([a for a, _ in grow], [b for _, b in grow]) == cg.CG_ERR_CAPACITY
        assert not s.book.extend([a for a, _ in grow], [b for _, b in grow])
        s.same_book()


def test_refusals_on_the_device_change_nothing():
    bad = cg.CG_ERR_INVALID_ARG
    for what, want in ((lambda s: s.extend([0, 0], [40, 41]), bad), (lambda s: s.extend([12], [3]), bad), (lambda s: s.extend([-1], [3]), bad),
                       (lambda s: s.extend([0], [1]), bad), (lambda s: s.extend([0], [9 * 16 + 1]), bad),
                       (lambda s: s.extend([0, 5, 6], [40, 9 * 16, 9 * 16]), cg.CG_ERR_CAPACITY),
                       (lambda s: s.fork([0, 0], [4, 4]), bad), (lambda s: s.fork([0], [1]), bad), (lambda s: s.fork([0], [12]), bad),
                       (lambda s: s.fork([-1], [4]), bad), (lambda s: s.fork([4], [4]), bad), (lambda s: s.fork([0, 4], [4, 5]), bad),
                       (lambda s: s.fork([0] * 7, [4, 5, 6, 7, 8, 9, 10]), cg.CG_ERR_CAPACITY)):
        s = Setup(12, 16, [35, 20, 1], n_seqs=12, width=9)
        assert what(s) == want
        s.same_book()
        s.same_pools([])


def test_free_twice_bad_ids_and_pages():
    s = Setup(40, 16, [35, 20, 1], n_seqs=6, width=9)
    assert s.free([1, 1, 4, 1]) == cg.CG_OK
    s.book.free([1])
    s.same_book()
    assert s.free([6, 0, -3]) == cg.CG_ERR_INVALID_ARG
    s.book.free([0])
    s.same_book()
    s.table[2, 0] = 40  # a page that is none
    assert s.free([2]) == cg.CG_ERR_INVALID_ARG and s.lens[2].item() == 0 and s.table[2, 0].item() == -1
    s = Setup(40, 16, [35], n_seqs=2, width=9)
    s.refs[s.book.table[0][1]] = 0  # a page that nobody should have
    assert s.free([0]) == cg.CG_ERR_CORRUPT and int(s.refs.min()) == 0


def test_calls_for_nothing():
    s = Setup(12, 16, [35, 20, 1], n_seqs=12, width=9)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    for rc in (cg.cg_pages_extend(s.cache, s.pages, none, none, s.ws), cg.cg_pages_free(s.cache, s.pages, none, s.ws),
               cg.cg_pages_fork(s.cache, s.pages, s.pool_ptrs, s.scale_ptrs, none, none, s.ws),
               cg.cg_pages_copy(s.cache, s.pool_ptrs, s.scale_ptrs, none, none, s.ws)):
        assert s.status(rc) == cg.CG_OK
    s.same_book()
    s.same_pools([])


def test_copy():
    s = Setup(64, 7, [], n_seqs=1, width=1, L=3, H=3, d=24)
    src, dst = [5, 9, 5, 63], [1, 0, 62, 30]
    rc = cg.cg_pages_copy(s.cache, s.pool_ptrs, s.scale_ptrs, i32(src), i32(dst), s.ws)
    assert s.status(rc) == cg.CG_OK
    s.same_pools(list(zip(src, dst)))
    rc = cg.cg_pages_copy(s.cache, s.pool_ptrs, s.scale_ptrs, i32([64, 3, 4]), i32([2, -1, 6]), s.ws)
    assert s.status(rc) == cg.CG_ERR_INVALID_ARG
    s.same_pools([(4, 6)])
    s.pool_ptrs[1] = 0  # a null pool is left out and reported
    rc = cg.cg_pages_copy(s.cache, s.pool_ptrs, s.scale_ptrs, i32([8]), i32([10]), s.ws)
    assert s.status(rc) == cg.CG_ERR_INVALID_ARG
    assert torch.equal(s.pools[0][10], s.pools[0][8]) and not torch.equal(s.pools[1][10], s.pools[1][8])


def test_copy_offsets_past_32_bits():
    H, bt, d = 8, 64, 128
    n_blocks = (1 << 31) // (H * bt * d) + 5
    pool = torch.empty(2, n_blocks, H, bt, d, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(2, n_blocks, H, device="cuda")
    pool[:, 3] = 7
    pool[:, n_blocks - 2] = 1
    ptrs = [torch.tensor([t[i].data_ptr() for i in range(2)], dtype=torch.int64).cuda() for t in (pool, scale)]
    ws = cg.empty_u8(256)
    rc = cg.cg_pages_copy(cg.Cache(1, H, d, bt, n_blocks), ptrs[0], ptrs[1], i32([3]), i32([n_blocks - 2]), ws)
    assert rc == cg.CG_OK
    torch.cuda.synchronize()
    assert cg.cg_read_status(ws) == cg.CG_OK and bool((pool[:, n_blocks - 2] == 7).all())


def test_graph_of_a_branch_step():
    """Free, fork and extend captured once: each replay drops the branches and makes them again."""
    s = Setup(60, 16, [35, 20], n_seqs=8, width=9)
    parents, children, grown = i32([0, 1, 0]), i32([4, 5, 6]), i32([40, 49, 36])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert cg.cg_pages_free(s.cache, s.pages, children, s.ws) == cg.CG_OK
        assert cg.cg_pages_fork(s.cache, s.pages, s.pool_ptrs, s.scale_ptrs, parents, children, s.ws) == cg.CG_OK
        assert cg.cg_pages_extend(s.cache, s.pages, children, grown, s.ws) == cg.CG_OK
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert cg.cg_read_status(s.ws) == cg.CG_OK
        s.book.free([4, 5, 6])
        m = s.book.fork([0, 1, 0], [4, 5, 6])
        assert s.book.extend([4, 5, 6], [40, 49, 36])
        s.same_book()
        s.same_pools(m)


BAD_POOLS = {
    # what: (which array, the entry, its value from the right one)
    "null_pool": ("pool_ptrs", -1, lambda x: 0),
    "misaligned_pool": ("pool_ptrs", 1, lambda x: x + 8),
    "null_scale": ("scale_ptrs", -1, lambda x: 0),
    "misaligned_scale": ("scale_ptrs", 2, lambda x: x + 2),
}


@pytest.mark.parametrize("what", list(BAD_POOLS))
def test_fork_and_compact_with_a_bad_pool_change_nothing(what):
    """A null or misaligned entry among the pools or scales is found before a count, a row, a length or a page changes;
    where no page is copied or moved the entry does not matter."""
    name, at, wrong = BAD_POOLS[what]
    s = Setup(40, 16, [35, 32, 1], n_seqs=8, width=5)
    good = getattr(s, name)[at].item()
    getattr(s, name)[at] = wrong(good)
    assert s.fork([1, 0], [5, 6]) == cg.CG_ERR_INVALID_ARG
    s.same_book()
    s.same_pools([])
    assert s.fork([1], [5]) == cg.CG_OK and s.book.fork([1], [5]) == []
    s.same_book()
    n_live = i32([-9])
    rc = cg.cg_pages_compact(s.cache, s.pages, s.pool_ptrs, s.scale_ptrs, s.refs, s.table, n_live, s.ws)
    assert s.status(rc) == cg.CG_ERR_INVALID_ARG and n_live.tolist() == [-9]
    s.same_book()
    s.same_pools([])
    refs, table = torch.full_like(s.refs, -9), torch.full_like(s.table, -9)
    rc = cg.cg_pages_compact(s.cache, s.pages, s.pool_ptrs, s.scale_ptrs, refs, table, n_live, s.ws)
    assert s.status(rc) == cg.CG_ERR_INVALID_ARG
    assert bool((refs == -9).all()) and bool((table == -9).all()) and n_live.tolist() == [-9]
    # once the entry is right the same calls go through
    getattr(s, name)[at] = good
    assert s.fork([0], [6]) == cg.CG_OK
    s.same_pools(s.book.fork([0], [6]))
    rc = cg.cg_pages_compact(s.cache, s.pages, s.pool_ptrs, s.scale_ptrs, s.refs, s.table, n_live, s.ws)
    assert s.status(rc) == cg.CG_OK
    live, m = s.book.compact()
    assert n_live.tolist() == [live] and m
    s.same_book()
    s.same_pools(m)
    # nothing left to move
    getattr(s, name)[at] = wrong(good)
    rc = cg.cg_pages_compact(s.cache, s.pages, s.pool_ptrs, s.scale_ptrs, s.refs, s.table, n_live, s.ws)
    assert s.status(rc) == cg.CG_OK and n_live.tolist() == [live]
    s.same_book()
    s.same_pools([])


def test_a_bad_pool_among_more_than_a_plan_has_threads():
    """Layer 700's V pool of 800 layers: fork and compact look at every entry."""
    L = 800
    s = Setup(12, 4, [6], n_seqs=4, width=3, L=L, H=1, d=8)
    good = s.pool_ptrs[1401].item()
    s.pool_ptrs[1401] = 0
    assert s.fork([0], [1]) == cg.CG_ERR_INVALID_ARG
    s.same_book()
    s.same_pools([])
    s.pool_ptrs[1401] = good
    assert s.fork([0], [1]) == cg.CG_OK
    s.same_pools(s.book.fork([0], [1]))
    s.same_book()


def test_extend_takes_the_last_of_many_pages_and_not_one_more():
    """9000 pages, more than two rounds of the search for free ones: refused by one page with nothing changed, then to
    the last page, then refused once more."""
    n, width = 9000, 6
    lens = [16 * (1 + i % 3) for i in range(2000)]  # whole pages, strewn over the pool
    s = Setup(n, 16, lens, n_seqs=2500, width=width)
    s.ws = cg.empty_u8(cg.cg_pages_workspace_bytes(s.cache, s.pages, 2500))
    left = len(s.book.free_pages())
    assert left == n - sum(-(-m // 16) for m in lens)
    grow, take = [], 0
    for q in range(2499, -1, -1):
        more = min(width - s.book.pages(s.book.lens[q]), left - take)
        grow.append((q, s.book.lens[q] + 16 * more))
        take += more
        if take == left:
            break
    assert take == left > 4096
    spare = next(q for q in range(2500) if q not in dict(grow) and s.book.pages(s.book.lens[q]) < width)
    seqs, new = [q for q, _ in grow], [m for _, m in grow]
    over = seqs + [spare], new + [s.book.lens[spare] + 1]
    assert s.extend(*over) == cg.CG_ERR_CAPACITY and not s.book.extend(*over)
    s.same_book()
    assert s.extend(seqs, new) == cg.CG_OK and s.book.extend(seqs, new)
    assert s.book.free_pages() == [] and s.book.refs[n - 1] == 1
    s.same_book()
    assert s.extend([spare], [s.book.lens[spare] + 1]) == cg.CG_ERR_CAPACITY
    s.same_book()
    s.same_pools([])
