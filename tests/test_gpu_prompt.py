"""cg_prompt_attend on the GPU against its 64-bit definition (tests/serve_ref.py)."""
import math

import pytest
import torch

from kv_cache_compression_02_gb300 import cachegen as cg
from tests import gpu_util as gu
from tests import serve_ref as ref

pytestmark = pytest.mark.gpu

DT = {torch.float16: cg.CG_F16, torch.bfloat16: cg.CG_BF16}
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    gu.ready()


def run(q, k, v, cu_q, cu_k, scale, max_q=None, max_k=None, lse=True, stream=None):
    n_q, Hq, d = q.shape
    n_k, H = k.shape[:2]
    most = lambda c: max([b - a for a, b in zip(c, c[1:])] + [0])  # noqa: E731
    p = cg.Prompt(len(cu_q) - 1, Hq, H, d, DT[q.dtype], n_q, n_k, most(cu_q) if max_q is None else max_q,
                  most(cu_k) if max_k is None else max_k, scale, q.stride()[:2], k.stride()[:2], v.stride()[:2])
    ws = cg.empty_u8(cg.cg_prompt_workspace_bytes(p))
    ws.fill_(0xA5)  # a workspace may hold anything
    out = torch.full((n_q, Hq, d), math.nan, dtype=q.dtype, device="cuda")
    z = torch.full((n_q, Hq), math.nan, device="cuda") if lse else None
    cq, ck = (torch.tensor(c, dtype=torch.int32, device="cuda") for c in (cu_q, cu_k))
    torch.cuda.synchronize()
    assert cg.cg_prompt_attend(p, q, k, v, cq, ck, out, z, ws, stream) == cg.CG_OK
    torch.cuda.synchronize()
    return out, z, cg.cg_read_status(ws)


def rows(n, H, d, dt, seed, key=False):
    x = torch.randn(n, H, d, generator=torch.Generator().manual_seed(seed))
    if key:
        x[..., 3::32] *= 8.0
    return x.to(dt)


def check(out, z, q, k, v, cu_q, cu_k, scale, heads=None, pick=None):
    G, d = q.shape[1] // k.shape[1], q.shape[2]
    for b in range(len(cu_q) - 1):
        nq, nk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        i = torch.arange(nq) if pick is None else torch.tensor([x for x in pick if x < nq], dtype=torch.long)
        for h in range(q.shape[1]) if heads is None else heads:
            o, l, A, X = ref.attend_rows(q[cu_q[b] + i, h].cpu(), k[cu_k[b]:cu_k[b + 1], h // G].cpu(),
                                         v[cu_k[b]:cu_k[b + 1], h // G].cpu(), i + nk - nq, scale)
            to, tl = ref.tolerances(o, l, A, X, d, nk, q.dtype, ref.WEIGHT_BITS[q.dtype])
            ref.assert_close(out[cu_q[b] + i, h], o, to, f"out of sequence {b}, head {h}")
            ref.assert_close(z[cu_q[b] + i, h], l, tl, f"lse of sequence {b}, head {h}")


CASES = {
    # name: (dtype, Hq, H, d, [(queries, keys)])
    "one_of_one": (F16, 1, 1, 128, [(1, 1)]),
    "one_tile": (BF16, 2, 1, 128, [(128, 128)]),
    "whole": (BF16, 4, 2, 128, [(300, 300)]),
    "mha": (F16, 3, 3, 128, [(200, 200)]),
    "question": (F16, 16, 2, 128, [(13, 1500)]),
    "one_token": (BF16, 8, 1, 128, [(1, 700)]),
    "ragged": (BF16, 8, 2, 128, [(1, 1), (129, 129), (0, 0), (64, 200), (17, 17), (255, 300), (0, 50), (3, 130)]),
    "more_queries_than_keys": (F16, 4, 1, 64, [(100, 40), (5, 0), (33, 33)]),
    "group_7": (F16, 7, 1, 128, [(90, 400), (20, 20)]),
    "group_3_d96": (BF16, 6, 2, 96, [(150, 170)]),
    "group_128": (F16, 128, 1, 128, [(5, 300)]),
    "group_71_d64": (BF16, 71, 1, 64, [(9, 140), (1, 1)]),
    "d8": (F16, 4, 2, 8, [(70, 90), (1, 2)]),
    "d16": (BF16, 5, 5, 16, [(140, 140)]),
    "d40": (F16, 2, 2, 40, [(257, 513)]),
    "d80": (BF16, 4, 4, 80, [(65, 66)]),
    "d120": (F16, 4, 1, 120, [(33, 260)]),
    "long_context": (F16, 2, 1, 128, [(40, 6000)]),
    "many_sequences": (BF16, 2, 1, 16, [((5 * i) % 7, (5 * i) % 7 + (3 * i) % 11) for i in range(900)]),
    "many_queries_few_keys": (F16, 4, 2, 64, [(700, 9), (600, 300)]),
}


@pytest.mark.parametrize("name", list(CASES))
def test_prompt(name):
    dt, Hq, H, d, seqs = CASES[name]
    cu_q, cu_k = [0], [0]
    for a, b in seqs:
        cu_q.append(cu_q[-1] + a)
        cu_k.append(cu_k[-1] + b)
    q, k, v = rows(cu_q[-1], Hq, d, dt, 1).cuda(), rows(cu_k[-1], H, d, dt, 2, True).cuda(), rows(cu_k[-1], H, d, dt, 3).cuda()
    out, z, st = run(q, k, v, cu_q, cu_k, d ** -0.5)
    assert st == cg.CG_OK
    check(out, z, q, k, v, cu_q, cu_k, d ** -0.5)


@pytest.mark.parametrize("dt", [F16, BF16])
def test_prompt_long_whole(dt):
    """2500 tokens, rows of every kind of tile checked."""
    n = 2500
    q, k, v = rows(n, 8, 128, dt, 1).cuda(), rows(n, 1, 128, dt, 2, True).cuda(), rows(n, 1, 128, dt, 3).cuda()
    out, z, st = run(q, k, v, [0, n], [0, n], 128 ** -0.5)
    assert st == cg.CG_OK and bool(out.isfinite().all())
    check(out, z, q, k, v, [0, n], [0, n], 128 ** -0.5, heads=[0, 3, 7],
          pick=list(range(0, n, 37)) + list(range(120, 136)) + list(range(250, 262)) + list(range(2490, 2500)))


def test_prompt_layouts():
    """A fused projection's rows, and one layer of the codec's [L, 2, H, S, d], give the bits of the packed rows."""
    n, Hq, H, d = 200, 8, 2, 128
    q, k, v = rows(n, Hq, d, F16, 1), rows(n, H, d, F16, 2), rows(n, H, d, F16, 3)
    want, zw, _ = run(q.cuda(), k.cuda(), v.cuda(), [0, n], [0, n], 0.09)
    fused = torch.cat([q, k, v], 1).cuda()
    got, z, st = run(fused[:, :Hq], fused[:, Hq:Hq + H], fused[:, Hq + H:], [0, n], [0, n], 0.09)
    assert st == cg.CG_OK and torch.equal(got, want) and torch.equal(z, zw)
    kv = torch.full((2, H, n + 30, d), math.nan, dtype=F16)  # a buffer with room behind the context
    kv[0, :, :n], kv[1, :, :n] = k.transpose(0, 1), v.transpose(0, 1)
    kv = kv.cuda()
    got, z, st = run(q.cuda(), kv[0].transpose(0, 1), kv[1].transpose(0, 1), [0, n], [0, n], 0.09, lse=False)
    assert st == cg.CG_OK and torch.equal(got, want)


def test_prompt_neighbours_do_not_matter():
    """Inf and NaN in the rows before, behind and between the sequences."""
    d, H = 128, 2
    for nan in (math.nan, math.inf):
        seqs_q, seqs_k = [(10, 47), (60, 130)], [(20, 75), (90, 301)]
        q, k, v = rows(140, 4, d, BF16, 1), rows(320, H, d, BF16, 2), rows(320, H, d, BF16, 3)
        cu_q, cu_k = [10, 47, 60, 130], [20, 75, 90, 301]
        # three sequences: the middle one (13 queries, 15 keys) is the neighbour full of NaN
        for x, (a, b) in ((q, (47, 60)), (k, (75, 90)), (v, (75, 90))):
            x[:10], x[a:b] = nan, nan
        k[301:], v[301:], k[:20], v[:20] = nan, nan, nan, nan
        q, k, v = q.cuda(), k.cuda(), v.cuda()
        out, z, st = run(q, k, v, cu_q, cu_k, 0.1)
        assert st == cg.CG_OK
        for (qa, qb), (ka, kb) in zip(seqs_q, seqs_k):
            check(out[qa:qb], z[qa:qb], q[qa:qb], k[ka:kb], v[ka:kb], [0, qb - qa], [0, kb - ka], 0.1)
        assert bool(out[47:60].isnan().all())
        assert bool(out[:10].isnan().all()) and bool(z[130:].isnan().all()), "rows outside every sequence are not written"


def test_prompt_a_key_of_nan_is_not_seen_before_it():
    """A NaN key row, or a NaN query row, stays with the rows that see it."""
    n, d = 300, 128
    q, k, v = rows(n, 4, d, F16, 1), rows(n, 2, d, F16, 2), rows(n, 2, d, F16, 3)
    want, _, _ = run(q.cuda(), k.cuda(), v.cuda(), [0, n], [0, n], 0.1)
    k2, q2 = k.clone(), q.clone()
    k2[200, 1] = math.nan
    got, _, _ = run(q.cuda(), k2.cuda(), v.cuda(), [0, n], [0, n], 0.1)
    assert torch.equal(got[:200], want[:200]) and torch.equal(got[:, :2], want[:, :2]) and bool(got[200:, 2:].isnan().all())
    q2[150, 1] = math.inf
    got, _, _ = run(q2.cuda(), k.cuda(), v.cuda(), [0, n], [0, n], 0.1)
    same = torch.ones(n, 4, dtype=torch.bool)
    same[150, 1] = False
    assert torch.equal(got.cpu()[same], want.cpu()[same])


@pytest.mark.parametrize("d,G,dt", [(128, 4, F16), (64, 1, BF16), (80, 3, BF16)])
def test_prompt_a_value_of_nan_is_not_seen_before_it(d, G, dt):
    """NaN, inf and -inf in V reach the rows that see their keys, in their channels, and no others."""
    n, ctx = 290, 150
    q, k, v = rows(n, 2 * G, d, dt, 1), rows(n + ctx, 2, d, dt, 2), rows(n + ctx, 2, d, dt, 3)
    args = ([0, n], [0, n + ctx], 0.1)
    want, zw, _ = run(q.cuda(), k.cuda(), v.cuda(), *args)
    odd = {(ctx + 100, 0, 3): math.nan, (ctx + 101, 0, 5): math.inf, (ctx + 260, 0, 5): -math.inf, (ctx + 129, 1, 0): -math.inf,
           (ctx + n - 1, 1, d - 1): math.nan, (ctx + 280, 1, 7): math.inf, (40, 1, 1): math.nan}
    bad, expect = v.clone(), want.cpu().double()
    for (j, h, c), x in odd.items():
        bad[j, h, c] = x
        seen = torch.arange(n) >= j - ctx
        expect[seen, h * G:(h + 1) * G, c] += x  # inf - inf is NaN
    got, z, st = run(q.cuda(), k.cuda(), bad.cuda(), *args)
    assert st == cg.CG_OK and torch.equal(z, zw)
    got = got.cpu().double()
    assert torch.equal(got.isnan(), expect.isnan()) and torch.equal(got.isinf(), expect.isinf())
    assert torch.equal(got[got.isinf()], expect[expect.isinf()])
    # other channels, and rows before, keep their bits; a key's channel that became 0 or odd changes rows that see it only
    fine = expect.isfinite()
    assert torch.equal(got[fine], want.cpu().double()[fine])


def test_prompt_scores_far_apart():
    """Scores of hundreds whose maximum keeps growing along the keys, and falling."""
    n, d = 700, 64
    q, k, v = rows(n, 2, d, BF16, 1), rows(n, 1, d, BF16, 2), rows(n, 1, d, BF16, 3)
    for ramp in (torch.linspace(0.1, 30.0, n), torch.linspace(30.0, 0.1, n)):
        kk = (k.float() * ramp[:, None, None]).to(BF16)
        out, z, st = run(q.cuda(), kk.cuda(), v.cuda(), [0, n], [0, n], 1.0)
        assert st == cg.CG_OK
        check(out, z, q, kk, v, [0, n], [0, n], 1.0)


def test_prompt_without_keys_or_queries():
    """Empty tensors: every row sees nothing; no rows at all is no error."""
    q = rows(9, 4, 64, F16, 1).cuda()
    none = torch.empty(0, 2, 64, dtype=F16, device="cuda")
    out, z, st = run(q, none, none, [0, 4, 9], [0, 0, 0], 0.1)
    assert st == cg.CG_OK and not out.any() and bool((z == -math.inf).all())
    k = rows(5, 2, 64, F16, 2).cuda()
    _, _, st = run(q[:0], k, k, [0, 0], [0, 5], 0.1)
    assert st == cg.CG_OK
    out, z, st = run(q, none, none, [0, 4, 9], [0, 0, 1], 0.1, max_k=1)
    assert st == cg.CG_ERR_INVALID_ARG and not out[:4].any() and bool(out[4:].isnan().all())


def test_prompt_refuses_on_the_device():
    """Offsets that fall or pass the rows, and a sequence longer than said, are reported; other sequences are right."""
    d = 64
    q, k, v = rows(100, 2, d, F16, 1).cuda(), rows(100, 1, d, F16, 2).cuda(), rows(100, 1, d, F16, 3).cuda()
    for cu_q, cu_k, mq, mk in (([0, 40, 101], [0, 40, 100], 61, 60), ([0, 40, 100], [0, 40, 101], 60, 61),
                               ([0, 40, 30], [0, 40, 100], 60, 60), ([0, 40, 100], [0, 40, 39], 60, 60),
                               ([0, 40, 100], [0, 40, 100], 59, 60), ([0, 40, 100], [0, 40, 100], 60, 59)):
        out, z, st = run(q, k, v, cu_q, cu_k, 0.1, mq, mk)
        assert st == cg.CG_ERR_INVALID_ARG, (cu_q, cu_k, mq, mk)
        check(out[:40], z[:40], q[:40], k[:40], v[:40], [0, 40], [0, 40], 0.1)
        assert bool(out[40:].isnan().all())


def test_prompt_repeats_other_stream_and_graph():
    q, k, v = rows(50, 8, 128, BF16, 1).cuda(), rows(4000, 2, 128, BF16, 2).cuda(), rows(4000, 2, 128, BF16, 3).cuda()
    args = (q, k, v, [0, 20, 50], [0, 3000, 4000], 0.1)
    want, zw, _ = run(*args)
    for s in (None, None, torch.cuda.Stream()):
        got, z, _ = run(*args, stream=s)
        assert torch.equal(got, want) and torch.equal(z, zw)
    p = cg.Prompt(2, 8, 2, 128, cg.CG_BF16, 50, 4000, 30, 3000, 0.1, q.stride()[:2], k.stride()[:2], v.stride()[:2])
    ws, out = cg.empty_u8(cg.cg_prompt_workspace_bytes(p)), torch.zeros_like(q)
    cq, ck = torch.tensor(args[3], dtype=torch.int32).cuda(), torch.tensor(args[4], dtype=torch.int32).cuda()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert cg.cg_prompt_attend(p, q, k, v, cq, ck, out, None, ws) == cg.CG_OK
    for mid in (3000, 2000):  # a captured call follows the offsets in memory
        ck[1] = mid
        ck[2] = mid + 1000
        graph.replay()
        torch.cuda.synchronize()
        again, _, _ = run(q, k, v, [0, 20, 50], [0, mid, mid + 1000], 0.1)
        assert torch.equal(out, again)


def test_prompt_of_no_queries_looks_at_the_offsets():
    """Without query rows, or with max_q = 0, offsets are checked as they are in any other call, and nothing is written."""
    q, k = rows(6, 4, 64, F16, 1).cuda(), rows(9, 2, 64, F16, 2).cuda()
    bad, ok = cg.CG_ERR_INVALID_ARG, cg.CG_OK
    for n_q, cu_q, cu_k, max_k, want in ((6, [0, 0, 0], [0, 4, 9], 5, ok), (6, [3, 3, 3], [0, 0, 0], 0, ok), (0, [0, 0, 0], [2, 4, 9], 5, ok),
                                         (6, [0, 2, 2], [0, 4, 9], 5, bad), (6, [2, 0, 0], [0, 4, 9], 5, bad), (6, [7, 7, 7], [0, 4, 9], 5, bad),
                                         (6, [0, 0, 0], [0, 4, 10], 6, bad), (6, [0, 0, 0], [0, 4, 9], 4, bad), (6, [0, 0, 0], [4, 0, 5], 5, bad),
                                         (0, [0, 0, 1], [0, 4, 9], 5, bad), (0, [-1, 0, 0], [0, 4, 9], 5, bad)):
        out, z, st = run(q[:n_q], k, k, cu_q, cu_k, 0.1, max_q=0 if n_q else 1, max_k=max_k)
        assert st == want, (n_q, cu_q, cu_k)
        assert bool(out.isnan().all()) and bool(z.isnan().all())
    many = [0] * 2001  # more sequences than threads
    assert run(q, k, k, many, many, 0.1, max_q=0)[2] == ok
    many[-1] = 1
    assert run(q, k, k, many, [0] * 2001, 0.1, max_q=0)[2] == bad
