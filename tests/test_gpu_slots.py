"""cg_pages_slots and cg_pages_groups on the GPU against plain lists."""
import random

import pytest
import torch

from kv_cache_compression_02_gb300 import cachegen as cg
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    gu.ready()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def book(table, lens, n_blocks, bt):
    cache = cg.Cache(1, 2, 16, bt, n_blocks, cg.CG_CACHE_INT8)
    pages = cg.Pages(torch.zeros(n_blocks, dtype=torch.int32, device="cuda"), i32(table), i32(lens))
    ws = cg.empty_u8(cg.cg_pages_workspace_bytes(cache, pages, len(lens)))
    ws.fill_(0xFF)
    return cache, pages, ws


def slots(table, lens, new, n_blocks, bt, n_rows, skip=()):
    cache, pages, ws = book(table, lens, n_blocks, bt)
    got = dict(cu=i32([-9] * (len(lens) + 1)), start=i32([-9] * len(lens)), seq=i32([-9] * n_rows), pos=i32([-9] * n_rows),
               slot=torch.full((n_rows,), -9, dtype=torch.int64, device="cuda"))
    args = [None if k in skip else got[k] for k in ("seq", "pos", "slot")]
    assert cg.cg_pages_slots(cache, pages, n_rows, i32(new), got["cu"], got["start"], *args, ws) == cg.CG_OK
    torch.cuda.synchronize()
    return {k: t.tolist() for k, t in got.items()}, cg.cg_read_status(ws)


def want_slots(table, lens, new, n_blocks, bt, n_rows):
    cu, start, rows = [0], [], []
    for s, (n, m) in enumerate(zip(lens, new)):
        if not (0 <= n <= len(table[s]) * bt and 0 <= m <= n):
            n = m = 0
        start.append(n - m)
        cu.append(cu[-1] + m)
        for p in range(n - m, n):
            page = table[s][p // bt]
            rows.append((s, p, page * bt + p % bt if 0 <= page < n_blocks else -1))
    rows = rows[:n_rows] + [(-1, -1, -1)] * (n_rows - len(rows))
    return dict(cu=[min(c, n_rows) for c in cu], start=start, seq=[r[0] for r in rows], pos=[r[1] for r in rows], slot=[r[2] for r in rows])


def pages_table(lens, bt, width, n_blocks, rng):
    order = list(range(n_blocks))
    rng.shuffle(order)
    return [[order.pop() if j < -(-n // bt) else -1 for j in range(width)] for n in lens]


@pytest.mark.parametrize("bt", [1, 7, 16, 64])
@pytest.mark.parametrize("n_seqs", [1, 2, 31, 700, 2500])
def test_slots(bt, n_seqs):
    rng = random.Random(n_seqs * bt)
    lens = [rng.choice([0, 1, bt, bt + 1, rng.randint(0, 3 * bt + 5)]) for _ in range(n_seqs)]
    new = [rng.choice([0, 1, n, rng.randint(0, n)]) if n else 0 for n in lens]
    table = pages_table(lens, bt, 9 if bt > 1 else 10, 10 * n_seqs + 3, rng)
    for spare in (0, 1, 300):
        n_rows = sum(new) + spare
        got, st = slots(table, lens, new, 10 * n_seqs + 3, bt, n_rows)
        assert st == cg.CG_OK and got == want_slots(table, lens, new, 10 * n_seqs + 3, bt, n_rows)


def test_slots_errors_and_outputs_that_are_not_wanted():
    bt, n_blocks = 4, 30
    table = [[3, 4, -1], [5, 99, 6], [7, -5, -1], [8, 9, 10], [11, -1, -1], [12, 13, 14]]
    lens, new = [8, 12, 5, 13, 4, 12], [3, 9, 5, 1, 5, -1]
    got, st = slots(table, lens, new, n_blocks, bt, 40)
    assert st == cg.CG_ERR_INVALID_ARG and got == want_slots(table, lens, new, n_blocks, bt, 40)
    assert got["slot"].count(-1) == 40 - 12  # 17 rows, of which five lie in bad pages
    table[1][1], table[2][1] = 20, 21
    lens, new = [8, 12, 5, 12, 4, -1], [3, 9, 5, 1, 4, 0]
    got, st = slots(table, lens, new, n_blocks, bt, 40)
    assert st == cg.CG_ERR_INVALID_ARG and got == want_slots(table, lens, new, n_blocks, bt, 40)
    lens[5] = 12
    for n_rows in (22, 21, 5, 1, 0):
        got, st = slots(table, lens, new, n_blocks, bt, n_rows)
        assert st == (cg.CG_OK if n_rows == 22 else cg.CG_ERR_CAPACITY) and got == want_slots(table, lens, new, n_blocks, bt, n_rows)
    full = want_slots(table, lens, new, n_blocks, bt, 22)
    for skip in (("seq",), ("pos", "slot"), ("seq", "pos", "slot")):
        got, st = slots(table, lens, new, n_blocks, bt, 22, skip)
        assert st == cg.CG_OK
        for k in got:
            assert got[k] == ([-9] * 22 if k in skip else full[k])


def test_slots_pass_32_bits():
    """Places in pages whose rows pass 2^32 (the pages themselves are not touched)."""
    bt, n_blocks = 1 << 20, 1 << 20
    got, st = slots([[n_blocks - 1, 5]], [bt + 3], [bt // 512 + 3], n_blocks, bt, 3000)
    assert st == cg.CG_OK and got == want_slots([[n_blocks - 1, 5]], [bt + 3], [bt // 512 + 3], n_blocks, bt, 3000)
    assert got["slot"][0] == (n_blocks - 1) * bt + bt - bt // 512


def groups(table, lens, n_blocks, bt, min_pages):
    cache, pages, ws = book(table, lens, n_blocks, bt)
    n = len(lens)
    got = dict(cu=i32([-9] * (n // 2 + 1)), member=i32([-9] * n), shared=i32([-9] * (n // 2)))
    assert cg.cg_pages_groups(cache, pages, min_pages, got["cu"], got["member"], got["shared"], ws) == cg.CG_OK
    torch.cuda.synchronize()
    return {k: t.tolist() for k, t in got.items()}, cg.cg_read_status(ws)


def want_groups(table, lens, n_blocks, bt, m):
    n, sets = len(lens), {}
    for s, row in enumerate(table):
        if 0 <= lens[s] <= len(row) * bt and lens[s] // bt >= m and 0 <= row[m - 1] < n_blocks:
            sets.setdefault(row[m - 1], []).append(s)
    found = [g for g in sets.values() if len(g) > 1]
    cu, member, shared = [0], [], []
    for g in found:
        member += g
        cu.append(len(member))
        k = 0
        while k < min(lens[s] for s in g) // bt and len({table[s][k] for s in g}) == 1 and 0 <= table[g[0]][k] < n_blocks:
            k += 1
        shared.append(k)
    cu += [cu[-1]] * (n // 2 + 1 - len(cu))
    return dict(cu=cu, member=member + [-1] * (n - len(member)), shared=shared + [0] * (n // 2 - len(shared)))


@pytest.mark.parametrize("bt", [1, 16, 24])
@pytest.mark.parametrize("n_seqs", [1, 2, 3, 40, 1500])
def test_groups(bt, n_seqs):
    rng = random.Random(n_seqs + bt)
    width, n_blocks = 37, 37 * 8 + 6 * n_seqs
    stems = [[g * 37 + j for j in range(rng.choice([3, 9, 30]))] for g in range(8)]
    at, table, lens = 37 * 8, [], []
    for _ in range(n_seqs):
        stem = rng.choice(stems + [[]])
        stem = stem[:rng.choice([len(stem), len(stem), rng.randint(0, len(stem))])]
        n = len(stem) * bt + rng.choice([0, 0, 1, 3 * bt, 5 * bt + 1 if bt > 1 else 5])
        more = -(-n // bt) - len(stem)
        table.append(stem + list(range(at, at + more)) + [-1] * (width - len(stem) - more))
        lens.append(n)
        at += more
    for m in (1, 2, 5, 9, 37, 38):
        got, st = groups(table, lens, n_blocks, bt, m)
        assert st == cg.CG_OK and got == want_groups(table, lens, n_blocks, bt, m), m


def test_groups_of_long_rows():
    """Rows of 9000 pages that part late."""
    rng = random.Random(1)
    stem = list(range(9000))
    rng.shuffle(stem)
    table = [stem[:n] + [9000 + 40 * i + j for j in range(9030 - n)] for i, n in enumerate([9000, 8999, 8700, 9000, 8999])]
    table = [r[:9030] for r in table]
    lens = [16 * 9000 + 7, 16 * 8999 + 1, 16 * 8900, 16 * 9000, 16 * 9001]
    for m in (1, 8000, 8901):
        got, st = groups(table, lens, 20000, 16, m)
        assert st == cg.CG_OK and got == want_groups(table, lens, 20000, 16, m)


def test_groups_errors():
    table = [[0, 1, 2, 3], [0, 1, 2, 4], [0, 99, 5, -1], [0, 99, 6, -1], [0, 1, -7, 8], [0, 1, -7, 9], [7, 1, 2, 3]]
    for lens, m in (([64] * 7, 1), ([64] * 7, 2), ([64] * 7, 3), ([64, 65, 64, -1, 64, 64, 64], 1), ([64, 64, 48, 48, 64, 64, 30], 1)):
        got, st = groups(table, lens, 30, 16, m)
        assert st == cg.CG_ERR_INVALID_ARG and got == want_groups(table, lens, 30, 16, m)
    got, st = groups([table[0], table[6], table[1]], [64] * 3, 30, 16, 2)  # alike at the second page, but not at the first
    assert st == cg.CG_OK and got == dict(cu=[0, 3], member=[0, 1, 2], shared=[0])


def test_on_another_stream_and_in_a_graph():
    bt, n = 16, 12
    table = [[0, 1, 2, 3 + s] for s in range(n)]
    lens = [49 + s % 4 for s in range(n)]
    cache, pages, ws = book(table, lens, 40, bt)
    ws2 = cg.empty_u8(256)
    new, cu, start = i32([1] * n), i32([0] * (n + 1)), i32([0] * n)
    seq, pos, slot = i32([0] * n), i32([0] * n), torch.zeros(n, dtype=torch.int64, device="cuda")
    g = [i32([0] * k) for k in (n // 2 + 1, n, n // 2)]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        cg.check(cg.cg_pages_slots(cache, pages, n, new, cu, start, seq, pos, slot, ws2), "slots")
        cg.check(cg.cg_pages_groups(cache, pages, 2, *g, ws), "groups")
    for lens in ([49 + s % 4 for s in range(n)], [33 + s for s in range(n)]):
        pages.tensors[2].copy_(i32(lens))
        graph.replay()
        torch.cuda.synchronize()
        want = want_slots(table, lens, [1] * n, 40, bt, n)
        assert dict(cu=cu.tolist(), start=start.tolist(), seq=seq.tolist(), pos=pos.tolist(), slot=slot.tolist()) == want
        assert dict(zip(("cu", "member", "shared"), (t.tolist() for t in g))) == want_groups(table, lens, 40, bt, 2)
        assert cg.cg_read_status(ws) == cg.cg_read_status(ws2) == cg.CG_OK
