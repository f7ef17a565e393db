"""cg_shared_attend on the GPU against its 64-bit definition (tests/serve_ref.py): each sequence by itself, over its own row of the table.

Beside the tolerances there, a small weight has an absolute one.  A weight of the second product is W = p s / u in f16, with p = 2^(score - m + 7),
m at most 8 under the maximum, s its page's V scale and u a power of two, s < u <= 2 max s.  f16 rounds W by 2^-11 of itself at most, or by half of
the spacing of its subnormals, 2^-25.  The output is u sum(W c) / sum(p), c the codes, and sum(p) >= 2^7, for the maximum itself is in the sum: what
the subnormals' spacing moves is at most 2^-25 u sum|c| / 2^7 <= 2^-31 max(s) sum|c|.  (It is seen where the positions that have the weight have
code 0 in a channel.)
"""
import math
import random

import pytest
import torch

from kv_cache_compression_02_gb300 import cachegen as cg
from tests import gpu_util as gu
from tests import serve_ref as ref

pytestmark = pytest.mark.gpu

FMT = {"e4m3": cg.CG_CACHE_E4M3, "int8": cg.CG_CACHE_INT8}
DT = {torch.float16: cg.CG_F16, torch.bfloat16: cg.CG_BF16}
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    gu.ready()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Setup:
    """A cache on the CPU whose sequences branch off prefixes.  groups: [(pages of the prefix, own tokens of each reader)], loose: tokens of
    sequences without a prefix.  Sequences lie mixed in the table; bytes that no token has are 0x7f (e4m3's NaN), scales of unused pages NaN."""

    def __init__(self, fmt, dt, T, Hq, H, d, bt, groups, loose=(), seed=0, grown=False):
        g = torch.Generator().manual_seed(seed)
        self.fmt, self.H, self.bt, self.T, self.scale = fmt, H, bt, T, d ** -0.5
        kinds = [(i, n) for i, (_, own) in enumerate(groups) for n in own] + [(-1, n) for n in loose]
        random.Random(seed).shuffle(kinds)
        self.lens = [(groups[i][0] * bt if i >= 0 else 0) + n for i, n in kinds]
        width = max(1, max(-(-n // bt) for n in self.lens))
        n_blocks = sum(p for p, _ in groups) + sum(-(-n // bt) for _, n in kinds) + 3
        order = torch.randperm(n_blocks, generator=g).tolist()
        stems = [[order.pop() for _ in range(p)] for p, _ in groups]
        self.table = torch.full((len(kinds), width), -1, dtype=torch.int32)
        stale = torch.ones(n_blocks, bt, dtype=torch.bool)
        for b, (i, n) in enumerate(kinds):
            row = (stems[i] if i >= 0 else []) + [order.pop() for _ in range(-(-n // bt))]
            self.table[b, :len(row)] = torch.tensor(row, dtype=torch.int32)
            for j in range(len(row)):
                stale[row[j], :min(bt, self.lens[b] - j * bt)] = False
        self.members = [[b for b, (i, _) in enumerate(kinds) if i == k] for k in range(len(groups))]
        self.pages = [p for p, _ in groups]
        x = torch.randn(2, n_blocks, H, bt, d, generator=g)
        x[0, ..., 3::16] *= 10.0
        size = 1.0 + 3.0 * torch.rand(n_blocks, H, 1, 1, generator=g)
        if grown:  # V's scales span many powers of two
            size = size * 2.0 ** torch.randint(-30, 30, (n_blocks, H, 1, 1), generator=g)
            x[0] /= size
        self.pools, self.scales = [], []
        for i in range(2):
            p, s = ref.quantise(x[i] * size, fmt)
            p.view(torch.uint8).masked_fill_(stale[:, None, :, None], 0x7F)
            s[stale.all(1)] = math.nan
            self.pools.append(p)
            self.scales.append(s)
        self.q = torch.randn(len(kinds), T, Hq, d, generator=g).to(dt)

    def groups(self):
        cu = [0]
        for m in self.members:
            cu.append(cu[-1] + len(m))
        return cg.Groups(i32(cu), i32([b for m in self.members for b in m]), i32(self.pages))

    def shapes(self, q_stride=None, lse=True):
        B, T, Hq, d = self.q.shape
        cache = cg.Cache(1, self.H, d, self.bt, self.pools[0].shape[0], FMT[self.fmt])
        return cache, cg.Attend(B, T, Hq, DT[self.q.dtype], self.table.shape[1], self.scale, q_stride)

    def on_gpu(self):
        """What a call takes behind its descriptions: q, pools, scales, table, lengths."""
        return [self.q.cuda(), *(t.cuda() for t in self.pools), *(t.cuda() for t in self.scales), self.table.cuda(), i32(self.lens)]

    def run(self, groups=None, args=None, stream=None, lse=True, q_stride=None, fill=0xA5):
        cache, att = self.shapes(q_stride)
        groups = self.groups() if groups is None else groups
        ws = cg.empty_u8(cg.cg_shared_workspace_bytes(cache, att, groups))
        ws.fill_(fill)  # a workspace may hold anything
        out = torch.full(self.q.shape, math.nan, dtype=self.q.dtype, device="cuda")
        z = torch.full(self.q.shape[:3], math.nan, device="cuda") if lse else None
        args = self.on_gpu() if args is None else args
        torch.cuda.synchronize()
        assert cg.cg_shared_attend(cache, att, groups, *args, out, z, ws, stream) == cg.CG_OK
        torch.cuda.synchronize()
        return out, z, cg.cg_read_status(ws)

    def tokens(self, i, b, h, n):
        j = torch.arange(n)
        page = self.table[b, j // self.bt].long()
        codes = self.pools[i].view(torch.uint8)[page, h, j % self.bt].view(self.pools[i].dtype).to(torch.float64)
        return codes * self.scales[i][page, h].double()[:, None], codes.abs().sum(0) * self.scales[i][page, h].double().amax() if n else 0.0

    def tolerances(self, o, l, A, X, n, small):
        to, tl = ref.tolerances(o, l, A, X, self.q.shape[3], n, self.q.dtype, 11)  # weights go into the second product with 11 bits
        return to + 2.0 ** -31 * small, tl

    def check(self, out, z, only=None):
        B, T, Hq, d = self.q.shape
        G = Hq // self.H
        for b in range(B) if only is None else only:
            n = self.lens[b]
            last = (torch.arange(T) + n - T).repeat_interleave(G)
            for h in range(self.H):
                (k, _), (v, small) = (self.tokens(i, b, h, n) for i in range(2))
                o, l, A, X = ref.attend_rows(self.q[b, :, h * G:(h + 1) * G].reshape(T * G, d), k, v, last, self.scale)
                to, tl = self.tolerances(o, l, A, X, n, small)
                ref.assert_close(out[b, :, h * G:(h + 1) * G].reshape(T * G, d), o, to, f"out of sequence {b}, head {h}")
                ref.assert_close(z[b, :, h * G:(h + 1) * G].reshape(-1), l, tl, f"lse of sequence {b}, head {h}")


CASES = {
    # name: (format, q dtype, T, Hq, H, d, block tokens, groups, loose)
    "two_readers": ("e4m3", F16, 1, 8, 2, 128, 16, [(8, [5, 1])], []),
    "one_page": ("int8", BF16, 1, 4, 4, 128, 16, [(1, [3, 16, 1])], []),
    "nothing_of_their_own": ("e4m3", F16, 1, 8, 2, 128, 16, [(9, [0, 0, 7])], [0]),
    "ragged_end": ("e4m3", BF16, 1, 16, 2, 128, 16, [(21, [1, 30, 200])], [40]),
    "long_split": ("int8", F16, 1, 8, 1, 128, 64, [(80, [9, 1, 100])], []),
    "two_row_tiles": ("e4m3", F16, 1, 32, 1, 128, 64, [(9, [1, 2, 3, 4, 70, 6, 7])], []),
    "two_row_tiles_long": ("int8", BF16, 1, 32, 1, 128, 64, [(50, [1, 2, 3, 4, 70, 6, 7])], []),
    "many_rows": ("e4m3", BF16, 1, 64, 2, 128, 32, [(11, [1 + i % 3 for i in range(21)])], [5]),
    "three_groups": ("int8", F16, 1, 8, 2, 128, 16, [(40, [1, 2]), (3, [4, 5, 6]), (17, [20, 1, 1, 1])], [7, 0, 100]),
    "drafts_odd": ("int8", BF16, 5, 12, 4, 80, 24, [(13, [5, 9, 77]), (5, [6, 5])], [5, 0, 60]),
    "drafts_behind": ("e4m3", F16, 4, 8, 2, 64, 16, [(20, [4, 3, 2, 0, 9])], [1]),  # some see the prefix in part: they go alone
    "d8_page_1": ("int8", BF16, 1, 3, 1, 8, 1, [(150, [5, 1, 9])], []),
    "d16_page_7": ("e4m3", BF16, 2, 4, 4, 16, 7, [(30, [2, 5]), (4, [3, 2])], [6]),
    "d40": ("int8", F16, 3, 6, 3, 40, 24, [(12, [3, 49, 3])], [2]),
    "d64": ("e4m3", F16, 1, 16, 2, 64, 32, [(10, [700, 3])], [64]),
    "d72_page_16": ("e4m3", F16, 1, 8, 1, 72, 16, [(33, [3, 4])], []),
    "page_8": ("e4m3", BF16, 1, 16, 2, 128, 8, [(37, [3, 4, 9])], [17]),
    "page_24_rows_over_128": ("int8", F16, 1, 32, 1, 128, 24, [(31, [1, 2, 3, 4, 70, 6, 7])], []),
    "page_40_d64": ("e4m3", F16, 2, 8, 2, 64, 40, [(23, [2, 50, 3]), (3, [2, 9])], [5]),
    "page_8_d40": ("int8", BF16, 1, 4, 2, 40, 8, [(150, [1, 2])], []),
    "d96": ("e4m3", F16, 1, 40, 2, 96, 16, [(33, [3, 4, 5])], [20]),
    "d120_page_128": ("int8", BF16, 8, 16, 2, 120, 128, [(3, [13, 8, 30])], []),
    "group_7": ("e4m3", F16, 3, 35, 5, 128, 16, [(25, [30, 3])], [61]),
    "page_longer_than_a_tile": ("int8", F16, 1, 8, 8, 64, 512, [(2, [50, 1])], []),
    "many_groups": ("e4m3", F16, 1, 4, 2, 64, 16, [(1 + i % 9, [1 + i % 4, 2]) for i in range(120)], [3] * 10),
    "groups_of_one": ("int8", F16, 1, 4, 2, 128, 16, [(12, [4]), (1, [1])], []),
    "more_sequences_than_are_kept": ("int8", BF16, 1, 2, 1, 16, 16, [(2 + i % 3, [(i * k) % 5 for k in range(14)]) for i in range(50)], [3, 0]),
    "more_groups_than_threads": ("e4m3", F16, 1, 1, 1, 8, 16, [(1 + i % 2, [1, 2]) for i in range(1100)], []),
    "more_sequences_than_the_plan_keeps": ("int8", F16, 1, 1, 1, 8, 4, [(3, [i % 3 for i in range(4200)]), (9, [1] * 4000)], [1, 2]),
    "rows_of_one_reader_in_many_blocks": ("e4m3", BF16, 40, 16, 1, 64, 16, [(20, [40, 55])], []),
}


@pytest.mark.parametrize("name", list(CASES))
def test_shared(name):
    fmt, dt, T, Hq, H, d, bt, groups, loose = CASES[name]
    s = Setup(fmt, dt, T, Hq, H, d, bt, groups, loose, seed=len(name))
    out, z, st = s.run()
    assert st == cg.CG_OK
    n = len(s.lens)
    s.check(out, z, range(0, n, 9) if n > 60 else None)
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("name", list(CASES))
def test_what_the_workspace_held_does_not_matter(name):
    """0xff bytes are NaN as floats: a part that nothing has written shows in the results."""
    fmt, dt, T, Hq, H, d, bt, groups, loose = CASES[name]
    s = Setup(fmt, dt, T, Hq, H, d, bt, groups, loose, seed=len(name))
    args = s.on_gpu()
    (out, z, st), (want, zw, _) = s.run(None, args, fill=0xFF), s.run(None, args)
    assert st == cg.CG_OK and torch.equal(out, want) and torch.equal(z, zw)


@pytest.mark.parametrize("pages", [3, 4, 5, 6, 17, 18, 30, 31, 32, 33, 34])
@pytest.mark.parametrize("readers,H", [(17, 1), (20, 3), (33, 1), (48, 1)])
def test_little_work_in_runs_of_odd_lengths(pages, readers, H):
    """Blocks of 256 rows and of up to 128 behind one another, less work than every CTA could have: 8 rows a reader and KV head, a tile a page."""
    s = Setup("int8", BF16, 1, 8 * H, H, 40, 128, [(pages, [i % 3 for i in range(readers)])], seed=pages)
    out, z, st = s.run(fill=0xFF)
    assert st == cg.CG_OK
    s.check(out, z, range(0, readers, 11))
    assert torch.isfinite(out).all() and torch.isfinite(z).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_scales_of_many_sizes(fmt):
    """V's page scales span 60 powers of two (K's the inverse, so that scores stay as they are), and a page of zeros lies among them."""
    s = Setup(fmt, BF16, 1, 16, 1, 128, 16, [(60, [5, 20, 3])], seed=3, grown=True)
    zero = int(s.table[s.members[0][0], 7])
    for i in range(2):
        s.pools[i][zero] = torch.zeros_like(s.pools[i][zero])
        s.scales[i][zero] = 0.0
    out, z, st = s.run()
    assert st == cg.CG_OK
    s.check(out, z)


def test_large_scores_and_rows():
    """Scores of thousands (one weight is all), and query rows of very different sizes, bf16 ones among them beyond f16's range."""
    s = Setup("int8", BF16, 1, 8, 1, 128, 16, [(40, [5, 20])], seed=5)
    s.q[0, 0, 0] *= 1e6
    s.q[1, 0, 3] *= 2.0 ** -40
    s.q[0, 0, 5] *= 300.0
    s.q[0, 0, 6] = 0.0
    out, z, st = s.run()
    assert st == cg.CG_OK
    s.check(out, z)


def test_without_groups_it_is_cache_attend():
    s = Setup("e4m3", F16, 1, 8, 2, 128, 16, [(9, [4, 5])], [30], seed=1)
    args = s.on_gpu()
    cache, att = s.shapes()
    ws = cg.empty_u8(cg.cg_cache_workspace_bytes(cache, att))
    want, zw = torch.empty_like(args[0]), torch.empty(s.q.shape[:3], device="cuda")
    cg.check(cg.cg_cache_attend(cache, att, *args, want, zw, ws), "attend")
    none, empty = cg.Groups(i32([0]), i32([]), i32([])), cg.Groups(i32([0, 0, 0]), i32([-1, -1]), i32([0, 0]))
    for groups in (none, empty):
        out, z, st = s.run(groups, args)
        assert st == cg.CG_OK and torch.equal(out, want) and torch.equal(z, zw)


def test_bad_groups():
    s = Setup("e4m3", F16, 1, 8, 2, 128, 16, [(9, [4, 5]), (20, [3, 1, 2])], [30], seed=2)
    (m0, m1), wide = s.members, s.table.shape[1]
    big = 2 ** 31 - 1
    bad = [([0, 2, 1], m0 + m1, s.pages), ([-1, 2, 5], m0 + m1, s.pages), ([0, 2, 6], m0 + m1, s.pages), ([0, big, 5], m0 + m1, s.pages),
           ([0, 2, 5], m0 + [6, m1[1], m1[2]], s.pages), ([0, 2, 5], [-1, m0[1]] + m1, s.pages), ([0, 2, 5], m0 + [m1[0], m1[1], m1[0]], s.pages),
           ([0, 2, 5], [big, m0[1]] + m1, s.pages), ([0, 2, 5], m0 + m1, [-1, 20]), ([0, 2, 5], m0 + m1, [9, wide + 1]), ([0, 2, 5], m0 + m1, [9, big])]
    for cu, member, pages in bad:
        out, z, st = s.run(cg.Groups(i32(cu), i32(member), i32(pages)))
        assert st == cg.CG_ERR_INVALID_ARG, (cu, member, pages)
        s.check(out, z)  # who is in no group reads everything alone
    # fewer pages than are shared are right as well, and empty groups between
    out, z, st = s.run(cg.Groups(i32([0, 0, 2, 2, 5, 5]), i32(m0 + m1 + [-1]), i32([3, 4, 0, 15, 7])))
    assert st == cg.CG_OK
    s.check(out, z)


def test_bad_pages_and_lengths():
    s = Setup("int8", BF16, 1, 16, 2, 128, 16, [(20, [3, 1, 2])], [30], seed=4)
    lead, bt = s.members[0][0], s.bt
    whole, _, _ = s.run()
    for bad in (-1, s.pools[0].shape[0], 2 ** 31 - 1, -2 ** 31):
        s2 = Setup("int8", BF16, 1, 16, 2, 128, 16, [(20, [3, 1, 2])], [30], seed=4)
        for b in s2.members[0]:
            s2.table[b, 5] = bad
        out, z, st = s2.run()
        assert st == cg.CG_ERR_INVALID_ARG and torch.isfinite(out).all()
        keep = [b for b in range(4) if b not in s2.members[0]]
        assert torch.equal(out[keep], whole[keep])
        # as if the positions of that page were not there
        s2.table[s2.members[0], 5] = s.table[s.members[0], 5]
        there = torch.arange(max(s2.lens)) // bt != 5
        for b in s2.members[0]:
            for h in range(2):
                n = s2.lens[b]
                (k, _), (v, small) = (s2.tokens(i, b, h, n) for i in range(2))
                o, l, A, X = ref.attend_rows(s2.q[b, 0, h * 8:h * 8 + 8], k[there[:n]], v[there[:n]], torch.full((8,), n), s2.scale)
                to, tl = s2.tolerances(o, l, A, X, n, small)
                ref.assert_close(out[b, 0, h * 8:h * 8 + 8], o, to, "out")
                ref.assert_close(z[b, 0, h * 8:h * 8 + 8], l, tl, "lse")
    args = s.on_gpu()
    lens = list(s.lens)
    lens[lead] = -5
    args[6] = i32(lens)
    out, z, st = s.run(args=args)
    assert st == cg.CG_ERR_INVALID_ARG and (out[lead] == 0).all() and (z[lead] == -math.inf).all()
    s.check(out, z, [b for b in range(4) if b != lead])


def test_strided_q_and_no_lse():
    s = Setup("e4m3", F16, 2, 8, 2, 128, 16, [(9, [4, 5, 2])], [30], seed=6)
    B, T, Hq, d = s.q.shape
    wide = torch.full((T, B, Hq + 3, d), math.nan, dtype=F16)
    wide[:, :, 1:1 + Hq] = s.q.transpose(0, 1)
    w = wide.cuda()
    view = w[:, :, 1:1 + Hq].transpose(0, 1)
    want, _, _ = s.run()
    args = s.on_gpu()
    args[0] = view
    got, _, st = s.run(args=args, lse=False, q_stride=view.stride()[:3])
    assert st == cg.CG_OK and torch.equal(got, want)


def test_repeats_other_stream_graph_and_two_calls_at_once():
    s = Setup("int8", BF16, 1, 16, 2, 128, 64, [(60, [40, 5, 7]), (9, [1, 2])], [70], seed=7)
    args, groups = s.on_gpu(), s.groups()
    want, zw, _ = s.run(groups, args)
    side = torch.cuda.Stream()
    got, z, st = s.run(groups, args, stream=side)
    assert st == cg.CG_OK and torch.equal(got, want) and torch.equal(z, zw)
    cache, att = s.shapes()
    ws = [cg.empty_u8(cg.cg_shared_workspace_bytes(cache, att, groups)) for _ in range(2)]
    outs = [torch.zeros_like(args[0]) for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            cg.check(cg.cg_shared_attend(cache, att, groups, *args, outs[0], None, ws[0]), "shared")
    for _ in range(5):
        outs[0].zero_(), outs[1].zero_()
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            cg.check(cg.cg_shared_attend(cache, att, groups, *args, outs[1], None, ws[1]), "shared")
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    # other lengths and groups in the captured call: one sequence leaves its group
    s.lens[s.members[0][0]] -= 30
    args[6].copy_(i32(s.lens))
    groups.tensors[2].copy_(i32([50, 4]))
    graph.replay()
    torch.cuda.synchronize()
    again, z, st = s.run(groups, args)
    assert st == cg.CG_OK and torch.equal(outs[0], again)
    s.check(again, z)


@pytest.mark.parametrize("seed", range(6))
def test_random_shapes(seed):
    rng = random.Random(100 + seed)
    T, H, d = rng.choice([1, 1, 2, 5]), rng.choice([1, 2, 3]), 8 * rng.randint(1, 16)
    G, bt = rng.choice([1, 2, 5, 8, 16]), rng.choice([1, 5, 16, 48, 64, 128])
    groups = [(rng.randint(1, max(1, 900 // bt)), [rng.randint(0, 40) for _ in range(rng.randint(1, 9))]) for _ in range(rng.randint(1, 4))]
    s = Setup(rng.choice(["e4m3", "int8"]), rng.choice([F16, BF16]), T, G * H, H, d, bt, groups, [rng.randint(0, 300) for _ in range(3)], seed=seed)
    out, z, st = s.run()
    assert st == cg.CG_OK
    s.check(out, z)


def test_groups_as_the_table_gives_them():
    """fork, extend, write, groups and attention, as a server calls them, for the same result as attention of each sequence alone."""
    H, Hq, d, bt, readers, n_blocks, per = 2, 16, 128, 16, 5, 200, 40
    g = torch.Generator(device="cuda").manual_seed(1)
    cache = cg.Cache(1, H, d, bt, n_blocks, cg.CG_CACHE_E4M3)
    pools = torch.zeros(2, n_blocks, H, bt, d, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(2, n_blocks, H, device="cuda")
    addr = [torch.tensor([t[i].data_ptr() for i in range(2)], dtype=torch.int64, device="cuda") for t in (pools, scales)]
    n_seqs = readers + 2
    pages = cg.Pages(i32([0] * n_blocks), torch.full((n_seqs, per), -1, dtype=torch.int32, device="cuda"), i32([0] * n_seqs))
    refs, table, lens = pages.tensors
    ws = cg.empty_u8(cg.cg_pages_workspace_bytes(cache, pages, n_seqs))
    ws_rows = cg.empty_u8(256)
    n = 503
    cu, start, new = i32([0] * (n_seqs + 1)), i32([0] * n_seqs), i32([n, 20] + [0] * readers)

    def write(n_rows, most):
        cg.check(cg.cg_pages_slots(cache, pages, n_rows, new, cu, start, None, None, None, ws_rows), "slots")
        k, v = (torch.randn(n_rows, H, d, generator=g, device="cuda").half() for _ in range(2))
        rows = cg.Rows(n_seqs, n_rows, most, cg.CG_F16, per, H * d, d)
        w = cg.empty_u8(256)
        cg.check(cg.cg_cache_write(cache, rows, k, v, cu, start, table, pools[0], pools[1], scales[0], scales[1], w), "write")
        torch.cuda.synchronize()
        assert cg.cg_read_status(w) == cg.cg_read_status(ws_rows) == cg.CG_OK

    cg.check(cg.cg_pages_extend(cache, pages, i32([0, 1]), i32([n, 20]), ws), "extend")
    write(n + 20, n)
    ids = list(range(2, n_seqs))
    cg.check(cg.cg_pages_fork(cache, pages, addr[0], addr[1], i32([0] * readers), i32(ids), ws), "fork")
    groups = cg.Groups(i32([0] * (n_seqs // 2 + 1)), i32([0] * n_seqs), i32([0] * (n_seqs // 2)))
    att = cg.Attend(n_seqs, 1, Hq, cg.CG_BF16, per, d ** -0.5)
    ws_all, ws_one = cg.empty_u8(cg.cg_shared_workspace_bytes(cache, att, groups)), cg.empty_u8(cg.cg_cache_workspace_bytes(cache, att))
    new.copy_(i32([0, 1] + [1] * readers))
    for _ in range(20):
        cg.check(cg.cg_pages_extend(cache, pages, i32([1] + ids), lens[1:] + 1, ws), "extend")
        write(readers + 1, 1)
        cg.check(cg.cg_pages_groups(cache, pages, 4, *groups.tensors, ws), "groups")
        q = torch.randn(n_seqs, 1, Hq, d, generator=g, device="cuda").bfloat16()
        outs, z = [torch.empty_like(q) for _ in range(2)], [torch.empty(n_seqs, 1, Hq, device="cuda") for _ in range(2)]
        args = (q, pools[0], pools[1], scales[0], scales[1], table, lens)
        cg.check(cg.cg_shared_attend(cache, att, groups, *args, outs[0], z[0], ws_all), "shared")
        cg.check(cg.cg_cache_attend(cache, att, *args, outs[1], z[1], ws_one), "attend")
        torch.cuda.synchronize()
        assert cg.cg_read_status(ws) == cg.cg_read_status(ws_all) == cg.cg_read_status(ws_one) == cg.CG_OK
        # both round once to bf16; before that a weight of the one has 11 bits: 2^-9 + 2^-9 + 2^-11 of the largest value, and more than that spare
        top = 448.0 * scales[1][refs > 0].max().item()
        assert (outs[0].double() - outs[1].double()).abs().max() <= 2.0 ** -7 * top
        assert (z[0] - z[1]).abs().max() <= 1e-4
    assert groups.tensors[0].tolist() == [0, 1 + readers, 1 + readers, 1 + readers] and groups.tensors[2].tolist() == [n // bt, 0, 0]


def test_heads_and_tokens_in_reverse():
    """Strides may be negative: query heads and tokens from the last to the first."""
    s = Setup("int8", BF16, 3, 8, 2, 64, 16, [(12, [5, 9, 3])], [20], seed=8)
    B, T, Hq, d = s.q.shape
    want, zw, _ = s.run()
    args = s.on_gpu()
    back = s.q.flip(1, 2).contiguous().cuda()
    args[0] = back[:, -1:, -1:]  # the address of what is first now
    got, z, st = s.run(args=args, q_stride=(T * Hq * d, -Hq * d, -d))
    assert st == cg.CG_OK and torch.equal(got, want) and torch.equal(z, zw)
