"""cg_cache_write and cg_cache_attend on the GPU against their 64-bit definitions (tests/serve_ref.py)."""
import math

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


def make_cache(fmt, H, d, bt, lens, seed, spare=3, width=None):
    """A shuffled cache on the CPU: pools, scales, table; every byte that no token has is 0x7f (e4m3's NaN), every
    scale of a page that no sequence has is NaN."""
    g = torch.Generator().manual_seed(seed)
    need = sum(-(-n // bt) for n in lens)
    n_blocks = need + spare
    order = torch.randperm(n_blocks, generator=g).tolist()
    width = max(1, max(-(-n // bt) for n in lens)) if width is None else width
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    stale = torch.ones(n_blocks, bt, dtype=torch.bool)
    at = 0
    for b, n in enumerate(lens):
        for j in range(-(-n // bt)):
            table[b, j] = order[at]
            stale[order[at], :min(bt, n - j * bt)] = False
            at += 1
    x = torch.randn(2, n_blocks, H, bt, d, generator=g)
    x[0, ..., 3::16] *= 10.0
    pools, scales = [], []
    for i in range(2):
        p, s = ref.quantise(x[i] * (1.0 + 3.0 * torch.rand(n_blocks, H, 1, 1, generator=g)), fmt)
        p.view(torch.uint8).masked_fill_(stale[:, None, :, None], 0x7F)
        s[stale.all(1)] = math.nan
        pools.append(p)
        scales.append(s)
    return pools, scales, table


def tokens_of(pool, scale, table_row, n, bt, h):
    """The first n tokens' values of head h, in float64."""
    rows = [pool[int(table_row[j // bt]), h, j % bt].to(torch.float64) * float(scale[int(table_row[j // bt]), h])
            for j in range(n)]
    return torch.stack(rows) if rows else torch.zeros(0, pool.shape[-1], dtype=torch.float64)


def run_attend(fmt, q, pools, scales, table, lens, H, bt, scale, q_stride=None, lse=True, stream=None):
    B, T, Hq, d = q.shape
    cache = cg.Cache(1, H, d, bt, pools[0].shape[0], FMT[fmt])
    att = cg.Attend(B, T, Hq, DT[q.dtype], table.shape[1], scale, q_stride)
    ws = cg.empty_u8(cg.cg_cache_workspace_bytes(cache, att))
    ws.fill_(0xA5)  # a workspace may hold anything
    out = torch.full((B, T, Hq, d), math.nan, dtype=q.dtype, device="cuda")
    z = torch.full((B, T, Hq), math.nan, device="cuda") if lse else None
    torch.cuda.synchronize()
    rc = cg.cg_cache_attend(cache, att, q, pools[0], pools[1], scales[0], scales[1], table, lens, out, z, ws, stream)
    assert rc == cg.CG_OK
    torch.cuda.synchronize()
    return out, z, cg.cg_read_status(ws)


def dev(x):
    return [t.cuda() for t in x]


CASES = {
    # name: (format, q dtype, T, Hq, H, d, block tokens, lengths)
    "one_token_of_one": ("e4m3", F16, 1, 8, 8, 128, 16, [1]),
    "short_gqa": ("e4m3", BF16, 1, 32, 8, 128, 16, [500]),
    "ragged": ("int8", F16, 1, 16, 2, 128, 64, [1, 63, 64, 65, 0, 127, 129, 1000, 16, 17]),
    "d64": ("e4m3", F16, 1, 8, 2, 64, 32, [700, 3, 64]),
    "d8_page_1": ("int8", BF16, 1, 3, 1, 8, 1, [77, 5]),
    "d16_page_7": ("e4m3", BF16, 2, 4, 4, 16, 7, [90, 1, 0, 33]),
    "d40": ("int8", F16, 3, 6, 3, 40, 24, [200, 2, 3, 49]),
    "d80_drafts": ("int8", BF16, 5, 12, 4, 80, 24, [301, 4, 5, 0, 24, 25]),
    "d96_wide_group": ("e4m3", F16, 1, 40, 2, 96, 16, [333, 20]),
    "d120_drafts_wide": ("e4m3", BF16, 8, 16, 2, 120, 128, [513, 8, 7, 1]),
    "group_7": ("e4m3", F16, 3, 35, 5, 128, 16, [130, 61]),
    "page_longer_than_all": ("int8", F16, 1, 8, 8, 64, 512, [250, 1]),
    "many_sequences": ("e4m3", F16, 1, 2, 1, 64, 16, [(37 * i) % 90 for i in range(300)]),
    "more_sequences_than_are_kept": ("int8", BF16, 1, 1, 1, 16, 8, [(7 * i) % 23 for i in range(700)]),
    "long": ("int8", BF16, 1, 8, 1, 128, 64, [9000]),
    "long_drafts": ("e4m3", F16, 4, 16, 2, 128, 64, [5001, 2]),
}


@pytest.mark.parametrize("name", list(CASES))
def test_attend(name):
    fmt, dt, T, Hq, H, d, bt, lens = CASES[name]
    pools, scales, table = make_cache(fmt, H, d, bt, lens, seed=len(name))
    q = torch.randn(len(lens), T, Hq, d, generator=torch.Generator().manual_seed(9)).to(dt)
    scale = d ** -0.5
    out, z, st = run_attend(fmt, q.cuda(), dev(pools), dev(scales), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), H, bt, scale)
    assert st == cg.CG_OK
    G = Hq // H
    for b, n in enumerate(lens):
        last = (torch.arange(T) + n - T).repeat_interleave(G)
        for h in range(H):
            k, v = (tokens_of(pools[i], scales[i], table[b], n, bt, h) for i in range(2))
            o, l, A, X = ref.attend_rows(q[b, :, h * G:(h + 1) * G].reshape(T * G, d), k, v, last, scale)
            # probabilities go into the second product with 11 bits whatever the type of q
            to, tl = ref.tolerances(o, l, A, X, d, n, dt, 11)
            ref.assert_close(out[b, :, h * G:(h + 1) * G].reshape(T * G, d), o, to, f"out of sequence {b}, head {h}")
            ref.assert_close(z[b, :, h * G:(h + 1) * G].reshape(-1), l, tl, f"lse of sequence {b}, head {h}")


def _small(fmt="e4m3", T=1, lens=(200, 40), dt=F16, H=2, Hq=8, d=128, bt=16, **kw):
    pools, scales, table = make_cache(fmt, H, d, bt, list(lens), seed=3, **kw)
    q = torch.randn(len(lens), T, Hq, d, generator=torch.Generator().manual_seed(4)).to(dt)
    return q, pools, scales, table, torch.tensor(lens, dtype=torch.int32)


def test_attend_strided_q_and_no_lse():
    q, pools, scales, table, lens = _small(T=2)
    B, T, Hq, d = q.shape
    wide = torch.full((T, B, Hq + 3, d), math.nan, dtype=q.dtype)  # tokens first, other heads between
    wide[:, :, 1:1 + Hq] = q.transpose(0, 1)
    w = wide.cuda()
    view = w[:, :, 1:1 + Hq].transpose(0, 1)
    args = (dev(pools), dev(scales), table.cuda(), lens.cuda(), 2, 16, 0.1)
    want, _, _ = run_attend("e4m3", q.cuda(), *args)
    got, _, st = run_attend("e4m3", view, *args, q_stride=view.stride()[:3], lse=False)
    assert st == cg.CG_OK and torch.equal(got, want)


def test_attend_repeats_and_other_stream_and_graph():
    q, pools, scales, table, lens = _small(lens=(3000, 40, 0), T=2)
    args = (q.cuda(), dev(pools), dev(scales), table.cuda(), lens.cuda(), 2, 16, 0.1)
    want, zw, _ = run_attend("e4m3", *args)
    for _ in range(3):
        got, z, _ = run_attend("e4m3", *args)
        assert torch.equal(got, want) and torch.equal(z, zw)
    s = torch.cuda.Stream()
    got, z, _ = run_attend("e4m3", *args, stream=s)
    assert torch.equal(got, want) and torch.equal(z, zw)
    # a captured call follows the lengths that stand in memory when it runs
    qd, pd, sd, td, ld = args[:5]
    cache, att = cg.Cache(1, 2, 128, 16, pools[0].shape[0], FMT["e4m3"]), cg.Attend(3, 2, 8, cg.CG_F16, table.shape[1], 0.1)
    ws, out = cg.empty_u8(cg.cg_cache_workspace_bytes(cache, att)), torch.zeros_like(qd)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert cg.cg_cache_attend(cache, att, qd, pd[0], pd[1], sd[0], sd[1], td, ld, out, None, ws) == cg.CG_OK
    for n in (3000, 17, 1):
        ld[0] = n
        graph.replay()
        torch.cuda.synchronize()
        again, _, _ = run_attend("e4m3", qd, pd, sd, td, ld, 2, 16, 0.1)
        assert torch.equal(out, again)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_attend_bad_pages_and_lengths(fmt):
    """A bad page is reported and its positions are left out; a length outside the table is cut to it."""
    q, pools, scales, table, lens = _small(fmt, lens=(200, 40, 33))
    bad = table.clone()
    bad[0, 3], bad[1, 0] = pools[0].shape[0], -7
    out, z, st = run_attend(fmt, q.cuda(), dev(pools), dev(scales), bad.cuda(), lens.cuda(), 2, 16, 0.1)
    assert st == cg.CG_ERR_INVALID_ARG
    for b, n in enumerate(lens.tolist()):
        for h in range(2):
            ok = [j for j in range(n) if 0 <= int(bad[b, j // 16]) < pools[0].shape[0]]
            k, v = (tokens_of(pools[i], scales[i], table[b], n, 16, h)[ok] for i in range(2))
            o, l, A, X = ref.attend_rows(q[b, 0, 4 * h:4 * h + 4], k, v, [n] * 4, 0.1)
            to, tl = ref.tolerances(o, l, A, X, 128, n, F16, 11)
            ref.assert_close(out[b, 0, 4 * h:4 * h + 4], o, to, "out")
            ref.assert_close(z[b, 0, 4 * h:4 * h + 4], l, tl, "lse")
    full = torch.tensor([table.shape[1] * 16, 40, 0], dtype=torch.int32)
    want, _, st = run_attend(fmt, q.cuda(), dev(pools), dev(scales), table.clamp(min=0).cuda(), full.cuda(), 2, 16, 0.1)
    assert st == cg.CG_OK
    got, _, st = run_attend(fmt, q.cuda(), dev(pools), dev(scales), table.clamp(min=0).cuda(),
                            torch.tensor([2 ** 31 - 1, 40, -5], dtype=torch.int32).cuda(), 2, 16, 0.1)
    assert st == cg.CG_ERR_INVALID_ARG and torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(), want.nan_to_num())


def test_attend_values_far_apart():
    """Scores of hundreds, pages whose scales differ by 2^40, a page of zeros."""
    q, pools, scales, table, lens = _small("int8", lens=(300, 64), dt=BF16)
    q *= 40.0
    scales[1][int(table[0, 2])] *= 2.0 ** 20
    scales[1][int(table[0, 5])] *= 2.0 ** -20
    pools[1][int(table[0, 1])], scales[1][int(table[0, 1])] = 0, 0.0
    pools[0][int(table[1, 1])], scales[0][int(table[1, 1])] = 0, 0.0
    out, z, st = run_attend("int8", q.cuda(), dev(pools), dev(scales), table.cuda(), lens.cuda(), 2, 16, 128 ** -0.5)
    assert st == cg.CG_OK
    for b, n in enumerate(lens.tolist()):
        for h in range(2):
            k, v = (tokens_of(pools[i], scales[i], table[b], n, 16, h) for i in range(2))
            o, l, A, X = ref.attend_rows(q[b, 0, 4 * h:4 * h + 4], k, v, [n] * 4, 128 ** -0.5)
            to, tl = ref.tolerances(o, l, A, X, 128, n, BF16, 11)
            ref.assert_close(out[b, 0, 4 * h:4 * h + 4], o, to, "out")
            ref.assert_close(z[b, 0, 4 * h:4 * h + 4], l, tl, "lse")


def test_attend_a_row_of_nan_stays_alone():
    """An Inf or NaN in one query row reaches that row only; one in the cache reaches the rows that see it only."""
    q, pools, scales, table, lens = _small(T=4, lens=(100, 64))
    args = (dev(pools), dev(scales), table.cuda(), lens.cuda(), 2, 16, 0.1)
    clean, _, _ = run_attend("e4m3", q.cuda(), *args)
    bad = q.clone()
    bad[0, 1, 2, 5] = math.inf
    got, _, _ = run_attend("e4m3", bad.cuda(), *args)
    same = torch.ones(got.shape[:3], dtype=torch.bool)
    same[0, 1, 2] = False
    assert torch.equal(got.cpu()[same], clean.cpu()[same]) and got[0, 1, 2].isnan().any()
    # the last but one position of sequence 0, head 1: tokens 2 and 3 see it
    p = [t.clone() for t in pools]
    p[1].view(torch.uint8)[int(table[0, 98 // 16]), 1, 98 % 16, 7] = 0x7F
    got, _, _ = run_attend("e4m3", q.cuda(), dev(p), *args[1:])
    same = torch.ones(got.shape, dtype=torch.bool)
    same[0, 2:, 4:, 7] = False
    assert torch.equal(got.cpu()[same], clean.cpu()[same]) and got[0, 2:, 4:, 7].isnan().all()


def test_attend_offsets_past_32_bits():
    """Pages behind the first 2 GB of a pool."""
    H, d, bt, lens = 8, 128, 64, [150]
    n_blocks = (1 << 31) // (H * d * bt) + 8
    pools, scales, table = make_cache("e4m3", H, d, bt, lens, seed=5)
    q = torch.randn(1, 1, 8, d, generator=torch.Generator().manual_seed(4)).to(F16)
    want, zw, _ = run_attend("e4m3", q.cuda(), dev(pools), dev(scales), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), H, bt, 0.1)
    big = [torch.empty(n_blocks, H, bt, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    bigs = [torch.empty(n_blocks, H, device="cuda") for _ in range(2)]
    far = torch.full_like(table, -1)
    for j in range(table.shape[1]):
        far[0, j] = n_blocks - 1 - 2 * j
        for i in range(2):
            big[i][int(far[0, j])] = pools[i].view(torch.uint8)[int(table[0, j])].cuda()
            bigs[i][int(far[0, j])] = scales[i][int(table[0, j])].cuda()
    got, z, st = run_attend("e4m3", q.cuda(), big, bigs, far.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), H, bt, 0.1)
    assert st == cg.CG_OK and torch.equal(got, want) and torch.equal(z, zw)


# ---- writing ------------------------------------------------------------------
def run_write(fmt, k, v, cu, start, table, pools, scales, bt, max_new=None):
    H, d = k.shape[1:]
    cache = cg.Cache(1, H, d, bt, pools[0].shape[0], FMT[fmt])
    most = max([b - a for a, b in zip(cu, cu[1:])]) if max_new is None else max_new
    rows = cg.Rows(len(start), k.shape[0], most, DT[k.dtype], table.shape[1], k.stride(0), k.stride(1))
    ws = cg.empty_u8(256)
    ws.fill_(0xA5)
    i32 = dict(dtype=torch.int32, device="cuda")
    rc = cg.cg_cache_write(cache, rows, k, v, torch.tensor(cu, **i32), torch.tensor(start, **i32), table, pools[0], pools[1],
                           scales[0], scales[1], ws)
    assert rc == cg.CG_OK
    torch.cuda.synchronize()
    return cg.cg_read_status(ws)


WRITES = {
    # name: (format, dtype, H, d, block tokens, [(start, new)], token-major?)
    "one_token": ("e4m3", BF16, 8, 128, 64, [(0, 1), (63, 1), (64, 1), (100, 1)], True),
    "context": ("int8", F16, 2, 128, 64, [(0, 700)], False),
    "ragged": ("e4m3", F16, 3, 40, 24, [(5, 100), (0, 0), (24, 24), (47, 2), (1000, 30)], True),
    "page_1": ("int8", BF16, 1, 8, 1, [(3, 9), (0, 1)], True),
    "page_7": ("int8", F16, 5, 16, 7, [(6, 1), (6, 2), (0, 50)], True),
    "page_512": ("e4m3", BF16, 2, 128, 512, [(3, 900), (500, 600)], True),
    "one_sequence_in_codec_layout": ("e4m3", F16, 4, 96, 16, [(16, 333)], False),
}


@pytest.mark.parametrize("name", list(WRITES))
def test_write(name):
    fmt, dt, H, d, bt, seqs, packed = WRITES[name]
    pools, scales, table = make_cache(fmt, H, d, bt, [a + n for a, n in seqs], seed=11)
    pools = [torch.where(p.float().isnan(), 1.0, p.float()).to(p.dtype) for p in pools]  # kept rows are real ones
    g = torch.Generator().manual_seed(12)
    cu = [0]
    for _, n in seqs:
        cu.append(cu[-1] + n)
    x = torch.randn(2, cu[-1], H, d, generator=g) * torch.exp(2 * torch.randn(2, cu[-1], 1, 1, generator=g))
    x = x.to(dt)
    if packed:
        rows = torch.cat([x[0], x[1]], 1).cuda()
        k, v = rows[:, :H], rows[:, H:]
    else:
        k, v = (x[i].transpose(0, 1).contiguous().cuda().transpose(0, 1) for i in range(2))
    want = [p.clone() for p in pools], [s.clone() for s in scales]
    for b, (a, n) in enumerate(seqs):
        at = 0
        while at < n:
            pos = a + at
            m = min(n - at, bt - pos % bt)
            for i in range(2):
                ref.page_write(want[0][i], want[1][i], fmt, int(table[b, pos // bt]), pos % bt, x[i, cu[b] + at:cu[b] + at + m].float())
            at += m
    p, s = dev(pools), dev(scales)
    assert run_write(fmt, k, v, cu, [a for a, _ in seqs], table.cuda(), p, s, bt) == cg.CG_OK
    for i in range(2):  # fp32 steps in a fixed order: the same bits
        assert torch.equal(s[i].cpu().view(torch.int32), want[1][i].view(torch.int32)), "scales"
        assert torch.equal(p[i].cpu().view(torch.uint8), want[0][i].view(torch.uint8)), "codes"


def test_write_nonfinite_zero_and_tiny():
    pools, scales, table = make_cache("e4m3", 2, 16, 8, [24], seed=1)
    x = torch.randn(24, 2, 16, generator=torch.Generator().manual_seed(2)).to(BF16)
    x[3, 0, 5], x[4, 1, 0] = math.inf, math.nan
    x[8:16] = 0.0
    x[16:24] = 1e-38
    want = [pools[0].clone(), scales[0].clone()]
    clean = torch.where(x.float().isfinite(), x.float(), 0.0)
    for j in range(3):
        ref.page_write(want[0], want[1], "e4m3", int(table[0, j]), 0, clean[8 * j:8 * j + 8])
    p, s = dev(pools), dev(scales)
    assert run_write("e4m3", x.cuda(), x.cuda(), [0, 24], [0], table.cuda(), p, s, 8) == cg.CG_ERR_NONFINITE
    assert torch.equal(p[0].cpu().view(torch.uint8), want[0].view(torch.uint8))
    assert torch.equal(s[0].cpu().view(torch.int32), want[1].view(torch.int32))
    assert float(s[0][int(table[0, 1])].abs().max()) == 0.0 and float(s[0][int(table[0, 2])].abs().max()) == 0.0


def test_write_nothing():
    pools, scales, table = make_cache("int8", 1, 16, 8, [16, 16], seed=1)
    x = torch.empty(0, 1, 16, dtype=F16, device="cuda")
    p, s = dev(pools), dev(scales)
    for most in (0, 3):
        assert run_write("int8", x, x, [0, 0, 0], [5, 16], table.cuda(), p, s, 8, max_new=most) == cg.CG_OK
    assert torch.equal(p[0].cpu(), pools[0]) and torch.equal(p[1].cpu(), pools[1])


def test_write_refuses_on_the_device():
    """A bad page, offsets that fall or pass the rows, a position outside the table: reported, that much left out."""
    for what in ("page", "offsets", "rows", "many", "position", "negative"):
        pools, scales, table = make_cache("int8", 1, 16, 8, [16, 16], seed=1, width=2)
        x = torch.randn(20, 1, 16, generator=torch.Generator().manual_seed(2)).to(F16).cuda()
        cu, start, most, good = [0, 8, 16], [0, 0], 8, 1
        if what == "page":
            table[0, 0] = pools[0].shape[0]
        elif what == "offsets":
            cu, good = [0, -4, 8], None
        elif what == "rows":
            cu, good = [0, 8, 21], 0
            most = 13
        elif what == "many":
            cu, good = [0, 8, 17], 0
        elif what == "position":
            start, good = [0, 9], 0
        else:
            start, good = [-1, 0], 1
        p, s = dev(pools), dev(scales)
        assert run_write("int8", x, x, cu, start, table.cuda(), p, s, 8, max_new=most) == cg.CG_ERR_INVALID_ARG, what
        want, wants = pools[0].clone(), scales[0].clone()
        if good is not None:
            ref.page_write(want, wants, "int8", int(table[good, 0]), 0, x[8 * good:8 * good + 8].cpu().float())
        assert torch.equal(p[0].cpu(), want), what


def test_write_then_attend_token_by_token():
    """A context grown one token at a time, attended at every step, stays within the codes' own error."""
    H, d, bt = 2, 64, 16
    n = 40
    x = torch.randn(2, n, H, d, generator=torch.Generator().manual_seed(8)).to(F16)
    pools = [torch.zeros(4, H, bt, d, dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(4, H, device="cuda") for _ in range(2)]
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32).cuda()
    want = [torch.zeros(4, H, bt, d, dtype=torch.int8) for _ in range(2)], [torch.zeros(4, H) for _ in range(2)]
    for t in range(n):
        k, v = x[0, t:t + 1].cuda(), x[1, t:t + 1].cuda()
        assert run_write("int8", k, v, [0, 1], [t], table, pools, scales, bt) == cg.CG_OK
        for i in range(2):
            ref.page_write(want[0][i], want[1][i], "int8", int(table[0, t // bt]), t % bt, x[i, t:t + 1].float())
    for i in range(2):
        assert torch.equal(pools[i].cpu(), want[0][i]) and torch.equal(scales[i].cpu(), want[1][i])


def test_write_of_no_rows_looks_at_the_offsets():
    """With max_new = 0 a sequence that brings rows, an offset that falls or a position outside the table is reported as
    it is with any other limit, and nothing is written."""
    pools, scales, table = make_cache("int8", 1, 16, 8, [16, 16], seed=1)
    x = torch.randn(4, 1, 16, generator=torch.Generator().manual_seed(2)).to(F16).cuda()
    for bt_pages, cu, start, want in ((8, [0, 0, 0], [5, 16], cg.CG_OK), (8, [2, 2, 2], [0, 0], cg.CG_OK), (8, [0, 2, 2], [0, 0], cg.CG_ERR_INVALID_ARG),
                                      (8, [0, 0, 4], [0, 0], cg.CG_ERR_INVALID_ARG), (8, [2, 0, 0], [0, 0], cg.CG_ERR_INVALID_ARG),
                                      (8, [0, 0, 0], [-1, 0], cg.CG_ERR_INVALID_ARG), (8, [0, 0, 0], [0, 17], cg.CG_ERR_INVALID_ARG),
                                      (8, [5, 5, 5], [0, 0], cg.CG_ERR_INVALID_ARG), (1, [0, 0, 1], [0, 0], cg.CG_ERR_INVALID_ARG)):
        p, s = dev(pools), dev(scales)
        if bt_pages == 1:  # pages of one token: a run of none touches no page at all
            p, s = [t.reshape(-1, 1, 1, 16).contiguous() for t in p], [t.repeat_interleave(8, 0) for t in s]
        kept = [t.clone() for t in p], [t.clone() for t in s]
        assert run_write("int8", x, x, cu, start, table.cuda(), p, s, bt_pages, max_new=0) == want, (cu, start)
        for a, b in zip(kept, (p, s)):
            assert all(torch.equal(c.view(torch.uint8), e.view(torch.uint8)) for c, e in zip(a, b))


def cancelling(fmt, dt, T, d, bt, seed):
    """A sequence of eight pages whose values cancel in pairs, so that outputs are small against the weights they are made
    of and show how exactly the weights went into the second product.  Page i alone has values in the i-th eighth of
    the channels; every other page has a V scale 2^-8, 2^-16, 2^-24 and 2^-30 of its neighbour's.  A query row has two
    channels, powers of two, so that its products and their sums are exact."""
    g = torch.Generator().manual_seed(seed)
    H, G, n = 2, 4, 8 * bt
    k = (torch.randn(8, H, bt, d, generator=g) * 40).clamp(-100, 100)
    k = ref.codes(k, fmt).float()
    k[:, :, 1::2, :d // 2] = k[:, :, ::2, :d // 2]
    v = torch.zeros(8, H, bt, d)
    for i in range(8):
        c = slice(i * (d // 8), (i + 1) * (d // 8))
        v[i, :, ::2, c] = ref.codes((torch.randn(H, bt // 2, d // 8, generator=g) * 40).clamp(-100, 100), fmt).float()
        v[i, :, 1::2, c] = -v[i, :, ::2, c]
    scales = [torch.full((8, H), 2.0 ** -5), torch.ones(8, H)]
    scales[1][1::2] = 2.0 ** -torch.tensor([8.0, 16.0, 24.0, 30.0])[:, None]
    q = torch.zeros(1, T, G * H, d)
    for t in range(T):
        for h in range(G * H):
            q[0, t, h, (3 * h + t) % (d // 2)], q[0, t, h, d // 2 + (5 * h + t) % (d // 2)] = 1.0, 2.0 ** -6
    return q.to(dt), [ref.codes(x, fmt) for x in (k, v)], scales, torch.arange(8, dtype=torch.int32)[None], n


def weight_tolerance(q, k, v_codes, v_scale, last, dtype):
    """out and its tolerance where weights w_j = exp(s_j - lse) * (V scale of j) are off by at most 2^-23 of themselves or
    2^-36 of the largest probability times the largest scale, whichever is more, and by 2^-11 of themselves at most.
    Products and their sums are exact; a score is rounded four times; eight lanes share a row's sum; exp2, log2, the
    joins and the final product take 2^-20 together; the second product sums the n / 8 positions of a page sixteen at a
    time, each off by 2^-24 of the largest."""
    n = k.shape[0]
    s = q.double() @ k.double().T
    s.masked_fill_(torch.arange(n) > last[:, None], -math.inf)
    p = torch.softmax(s, 1)
    w = p * v_scale.double()
    most = p.max(1, keepdim=True).values * v_scale.max()
    off = torch.minimum(2.0 ** -11 * w, torch.maximum(2.0 ** -23 * w, 2.0 ** -36 * most))
    ds = 4 * 2.0 ** -24 * float(s[s.isfinite()].abs().max()) + (n / 8 + 8) * 2.0 ** -24 + 2.0 ** -20
    out, raw = w @ v_codes.double(), (off + (2 * ds + (n / 8 + 16) * 2.0 ** -24) * w) @ v_codes.double().abs()
    half = torch.finfo(dtype).eps / 2
    return out, raw + half * (out.abs() + raw) + torch.finfo(dtype).smallest_normal * half, w


@pytest.mark.parametrize("fmt,dt,T,d,bt", [("int8", BF16, 1, 128, 16), ("e4m3", BF16, 1, 64, 16), ("int8", BF16, 3, 128, 32), ("e4m3", BF16, 2, 80, 24),
                                           ("int8", F16, 1, 64, 48)])
def test_attend_weights_carry_their_low_part(fmt, dt, T, d, bt):
    """Values that cancel: weights of 11 bits would be off by many times the tolerance (which is checked, too)."""
    q, pools, scales, table, n = cancelling(fmt, dt, T, d, bt, seed=d + bt)
    out, _, st = run_attend(fmt, q.cuda(), dev(pools), dev(scales), table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), 2, bt, 1.0)
    assert st == cg.CG_OK
    for h in range(2):
        k = torch.cat([pools[0][i, h].double() * float(scales[0][i, h]) for i in range(8)])
        v = torch.cat([pools[1][i, h].double() for i in range(8)])
        rows = q[0, :, 4 * h:4 * h + 4].reshape(4 * T, d)
        last = (torch.arange(T) + n - T).repeat_interleave(4)
        want, tol, w = weight_tolerance(rows, k, v, scales[1][:, h].repeat_interleave(bt), last, dt)
        ref.assert_close(out[0, :, 4 * h:4 * h + 4].reshape(4 * T, d), want, tol, f"head {h}")
        coarse = torch.ldexp((torch.frexp(w)[0] * 2 ** 11).round(), torch.frexp(w)[1] - 11)  # weights of 11 bits
        assert float((((coarse - w) @ v).abs() / tol).max()) > 4
