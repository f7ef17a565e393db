"""cg_cross_attend on the GPU against its 64-bit definition (tests/serve_ref.py)."""
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


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(q, k, v, cu_q, begin, count, scale, max_q=None, max_k=None, lse=True, stream=None):
    n_q, Hq, d = q.shape
    n_k, H = k.shape[:2]
    p = cg.Prompt(len(cu_q) - 1, Hq, H, d, DT[q.dtype], n_q, n_k, max([b - a for a, b in zip(cu_q, cu_q[1:])]) if max_q is None else max_q,
                  max(count) if max_k is None else max_k, scale, q.stride()[:2], k.stride()[:2], v.stride()[:2])
    ws = cg.empty_u8(cg.cg_prompt_workspace_bytes(p))
    ws.fill_(0xFF)  # a workspace may hold anything, NaN among it
    out = torch.full((n_q, Hq, d), math.nan, dtype=q.dtype, device="cuda")
    z = torch.full((n_q, Hq), math.nan, device="cuda") if lse else None
    args = i32(cu_q), i32(begin), i32(count)
    torch.cuda.synchronize()
    assert cg.cg_cross_attend(p, q, k, v, *args, out, z, ws, stream) == cg.CG_OK
    torch.cuda.synchronize()
    return out, z, cg.cg_read_status(ws)


def rows(n, H, d, dt, seed, key=False):
    x = torch.randn(n, H, d, generator=torch.Generator().manual_seed(seed))
    if key:
        x[..., 3::32] *= 8.0
    return x.to(dt)


def check(out, z, q, k, v, cu_q, begin, count, scale, only=None):
    G, d = q.shape[1] // k.shape[1], q.shape[2]
    for b in range(len(count)) if only is None else only:
        i = torch.arange(cu_q[b], cu_q[b + 1])
        last = torch.full((i.numel(),), count[b] - 1)
        keys = slice(begin[b], begin[b] + count[b])
        for h in range(q.shape[1]):
            o, l, A, X = ref.attend_rows(q[i, h].cpu(), k[keys, h // G].cpu(), v[keys, h // G].cpu(), last, scale)
            to, tl = ref.tolerances(o, l, A, X, d, count[b], q.dtype, ref.WEIGHT_BITS[q.dtype])
            ref.assert_close(out[i, h], o, to, f"out of sequence {b}, head {h}")
            ref.assert_close(z[i, h], l, tl, f"lse of sequence {b}, head {h}")


CASES = {
    # name: (dtype, Hq, H, d, queries of each sequence, first keys, keys)
    "one_of_one": (F16, 1, 1, 128, [1], [0], [1]),
    "one_tile": (BF16, 2, 1, 128, [128], [0], [128]),
    "one_token_of_many": (BF16, 4, 4, 64, [1] * 40, [150 * i for i in range(40)], [1 + (37 * i) % 150 for i in range(40)]),
    "more_queries_than_keys": (F16, 4, 1, 64, [300, 5, 33], [0, 7, 0], [40, 0, 33]),
    "none_has_keys": (BF16, 4, 2, 128, [5, 0, 200], [0, 3, 9], [0, 0, 0]),
    "ragged": (BF16, 8, 2, 128, [1, 129, 0, 64, 17, 255, 0, 3], [0, 1, 130, 130, 330, 347, 647, 650], [1, 129, 0, 200, 17, 300, 50, 130]),
    "shared_and_overlapping": (F16, 6, 2, 96, [3, 4, 1, 70, 2], [0, 0, 100, 57, 0], [300, 300, 129, 243, 1]),
    "group_7": (F16, 7, 1, 128, [90, 20], [20, 0], [400, 20]),
    "group_128": (F16, 128, 1, 128, [5], [0], [300]),
    "d8": (F16, 4, 2, 8, [70, 1], [0, 2], [90, 2]),
    "d40": (BF16, 2, 2, 40, [257], [0], [513]),
    "d120": (F16, 4, 1, 120, [33], [0], [260]),
    "long_states": (F16, 2, 1, 128, [40], [3], [6000]),
    "many_sequences": (BF16, 2, 1, 16, [(5 * i) % 7 for i in range(900)], [i for i in range(900)], [(3 * i) % 11 for i in range(900)]),
    "whole_tiles": (BF16, 4, 2, 64, [64, 130], [128, 0], [256, 384]),
    # up to 16 rows of a KV head: another kernel
    "few_one_key": (F16, 1, 1, 128, [1], [5], [1]),
    "few_one_tile": (BF16, 2, 2, 128, [1, 2], [0, 32], [32, 32]),
    "few_8_rows": (F16, 16, 2, 128, [1, 1, 1], [0, 40, 3], [333, 31, 1000]),
    "few_9_rows": (BF16, 9, 1, 128, [1], [7], [700]),
    "few_16_rows": (F16, 8, 2, 128, [4, 1, 0, 3], [0, 100, 5, 2], [901, 33, 600, 0]),
    "few_d64_5_beams": (BF16, 6, 2, 64, [5, 4, 5, 1, 0], [0, 0, 0, 77, 77], [500, 500, 500, 64, 65]),
    "few_d8": (F16, 3, 3, 8, [2, 1], [1, 0], [70, 33]),
    "few_d16": (BF16, 8, 1, 16, [2, 1], [1, 0], [70, 33]),
    "few_d40": (F16, 4, 2, 40, [3, 1, 2], [0, 9, 100], [257, 0, 31]),
    "few_d72": (BF16, 5, 5, 72, [7], [0], [300]),
    "few_d120": (BF16, 12, 4, 120, [3, 5], [4, 0], [260, 95]),
    "few_long": (F16, 8, 1, 128, [2], [1], [30000]),
    "few_long_d64": (BF16, 4, 2, 64, [1], [0], [40001]),
    "few_many": (F16, 4, 4, 64, [1 + i % 3 for i in range(1500)], [3 * i for i in range(1500)], [(7 * i) % 100 for i in range(1500)]),
    "few_without_keys": (F16, 4, 2, 64, [1, 2, 1], [0, 0, 4], [0, 0, 0]),
}


@pytest.mark.parametrize("name", list(CASES))
def test_cross(name):
    dt, Hq, H, d, nq, begin, count = CASES[name]
    n_k = max(b + n for b, n in zip(begin, count))
    cu = [sum(nq[:i]) for i in range(len(nq) + 1)]
    q, k, v = rows(cu[-1], Hq, d, dt, 1), rows(max(1, n_k), H, d, dt, 2, True), rows(max(1, n_k), H, d, dt, 3)
    out, z, st = run(q.cuda(), k.cuda(), v.cuda(), cu, begin, count, d ** -0.5)
    assert st == cg.CG_OK
    some = list(range(0, len(nq), 23)) + [len(nq) - 1] if len(nq) > 100 else None
    check(out, z, q, k, v, cu, begin, count, d ** -0.5, some)
    assert torch.isfinite(out).all() and not torch.isnan(z).any()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cu", [[0, 3, 5, 70, 71, 200], [0, 3, 5, 6, 13, 20]])
@pytest.mark.parametrize("dt", [F16, BF16])
def test_what_a_sequence_does_not_see_does_not_matter(dt, cu, d):
    """NaN and infinities behind a sequence's last key, of padded and of other sequences' keys."""
    H, width, count = 2, 200, [130, 0, 200, 1, 128]
    begin = [width * i for i in range(5)]
    q, k, v = rows(cu[-1], 4, d, dt, 4), rows(5 * width, H, d, dt, 5, True), rows(5 * width, H, d, dt, 6)
    for b, n in enumerate(count):
        for x, bad in ((k, math.nan), (v, math.inf)):
            x[begin[b] + n:begin[b] + width] = bad
            x[begin[b] + n + 1:begin[b] + width:3] = math.nan
    out, z, st = run(q.cuda(), k.cuda(), v.cuda(), cu, begin, count, 0.2)
    assert st == cg.CG_OK
    check(out, z, q, k, v, cu, begin, count, 0.2)


@pytest.mark.parametrize("n", [2, 40])
def test_values_that_are_seen_count(n):
    """An Inf or NaN among the keys' values that a row does see reaches the row, in its channel."""
    q, k, v = rows(n + 1, 2, 64, F16, 7), rows(150, 1, 64, F16, 8), rows(150, 1, 64, F16, 9)
    v[140, 0, 5], v[3, 0, 9], v[149, 0, 11] = math.inf, math.nan, -math.inf
    out, _, st = run(q.cuda(), k.cuda(), v.cuda(), [0, n, n + 1], [0, 0], [150, 140], 0.1)
    out = out.cpu()
    assert st == cg.CG_OK
    assert (out[:n, :, 5] == math.inf).all() and (out[:n, :, 11] == -math.inf).all() and torch.isnan(out[:, :, 9]).all()
    assert torch.isfinite(out[n, :, 5]).all() and torch.isfinite(out[n, :, 11]).all()


@pytest.mark.parametrize("cu", [[2, 9, 17], [2, 9, 40]])
def test_strided_rows_no_lse_and_rows_of_no_sequence(cu):
    """The codec's layout [H][S][d], queries between other heads, queries before and behind those of the sequences."""
    H, d, n, last = 2, 64, 333, cu[-1]
    kv = torch.randn(2, H, n, d, generator=torch.Generator().manual_seed(1)).half()
    k, v = kv[0].transpose(0, 1), kv[1].transpose(0, 1)
    wide = torch.full((50, 7, d), math.nan, dtype=F16)
    wide[:, 1:5] = rows(50, 4, d, F16, 2)
    w, kvd = wide.cuda(), kv.cuda()
    out, _, st = run(w[:, 1:5], kvd[0].transpose(0, 1), kvd[1].transpose(0, 1), cu, [5, 0], [300, 333], 0.1, lse=False)
    assert st == cg.CG_OK and torch.isnan(out[:2]).all() and torch.isnan(out[last:]).all()
    want, z, _ = run(wide[:, 1:5].contiguous().cuda(), k.contiguous().cuda(), v.contiguous().cuda(), cu, [5, 0], [300, 333], 0.1)
    assert torch.equal(out[2:last], want[2:last])
    check(want, z, wide[:, 1:5], k, v, cu, [5, 0], [300, 333], 0.1)


@pytest.mark.parametrize("most", [None, 12])
def test_bad_sequences_are_left_out(most):
    """(more than 16 rows of a KV head might come where `most` says so)"""
    q, k, v = rows(12, 2, 64, F16, 1), rows(100, 1, 64, F16, 2), rows(100, 1, 64, F16, 3)
    d = (q.cuda(), k.cuda(), v.cuda())
    cu = [0, 2, 4, 6, 8, 10, 12]
    big = 2 ** 31 - 1
    for begin, count, bad in (([0, -1, 0, 0, 0, 50], [100, 5, -1, 101, 90, 51], [1, 2, 3, 5]), ([0, big, 0, 99, 100, 5], [1, 1, big, 1, 0, big], [1, 2, 5])):
        out, z, st = run(*d, cu, begin, count, 0.1, max_q=most, max_k=100)
        assert st == cg.CG_ERR_INVALID_ARG
        for b in range(6):
            if b in bad:
                assert torch.isnan(out[2 * b:2 * b + 2]).all() and torch.isnan(z[2 * b:2 * b + 2]).all()
        check(out, z, q, k, v, cu, begin, count, 0.1, [b for b in range(6) if b not in bad])
    out, z, st = run(*d, cu, [0] * 6, [10, 20, 30, 31, 30, 1], 0.1, max_q=most, max_k=30)
    assert st == cg.CG_ERR_INVALID_ARG and torch.isnan(out[6:8]).all()
    for bad_cu in ([0, 2, 1, 6, 8, 10, 12], [0, 2, 4, 6, 8, 10, 13], [-1, 2, 4, 6, 8, 10, 12]):
        assert run(*d, bad_cu, [0] * 6, [9] * 6, 0.1, max_q=20 if most else 8)[2] == cg.CG_ERR_INVALID_ARG
    assert run(*d, [0, 5, 5, 5, 5, 5, 12], [0] * 6, [9] * 6, 0.1, max_q=6)[2] == cg.CG_ERR_INVALID_ARG


def test_no_queries_and_no_keys():
    p = cg.Prompt(2, 2, 1, 64, cg.CG_F16, 0, 0, 0, 0, 0.1, (128, 64), (64, 64), (64, 64))
    ws = cg.empty_u8(cg.cg_prompt_workspace_bytes(p))
    assert cg.cg_cross_attend(p, None, None, None, i32([0, 0, 0]), i32([0, 0]), i32([0, 0]), None, None, ws) == cg.CG_OK
    assert cg.cg_read_status(ws) == cg.CG_OK
    assert cg.cg_cross_attend(p, None, None, None, i32([0, 0, 0]), i32([0, 0]), i32([0, 1]), None, None, ws) == cg.CG_OK
    assert cg.cg_read_status(ws) == cg.CG_ERR_INVALID_ARG
    p = cg.Prompt(1, 2, 1, 64, cg.CG_F16, 3, 0, 3, 0, 0.1, (128, 64), (64, 64), (64, 64))
    ws = cg.empty_u8(cg.cg_prompt_workspace_bytes(p))
    q, out, z = rows(3, 2, 64, F16, 1).cuda(), torch.full((3, 2, 64), 7.0, dtype=F16, device="cuda"), torch.zeros(3, 2, device="cuda")
    assert cg.cg_cross_attend(p, q, None, None, i32([0, 3]), i32([0]), i32([0]), out, z, ws) == cg.CG_OK
    assert cg.cg_read_status(ws) == cg.CG_OK and (out == 0).all() and (z == -math.inf).all()


@pytest.mark.parametrize("nq", [[77, 13], [3, 4]])
def test_repeats_other_stream_graph_and_two_calls_at_once(nq):
    n = sum(nq)
    q, k, v = (x.cuda() for x in (rows(n, 8, 128, BF16, 1), rows(3000, 2, 128, BF16, 2, True), rows(3000, 2, 128, BF16, 3)))
    args = ([0, nq[0], n], [0, 100], [3000, 2000], 0.1)
    want, zw, _ = run(q, k, v, *args)
    side = torch.cuda.Stream()
    got, z, st = run(q, k, v, *args, stream=side)
    assert st == cg.CG_OK and torch.equal(got, want) and torch.equal(z, zw)
    p = cg.Prompt(2, 8, 2, 128, cg.CG_BF16, n, 3000, max(nq), 3000, 0.1, q.stride()[:2], k.stride()[:2], v.stride()[:2])
    ws = [cg.empty_u8(cg.cg_prompt_workspace_bytes(p)) for _ in range(2)]
    outs = [torch.zeros_like(q) for _ in range(2)]
    cu, begin, count = i32(args[0]), i32(args[1]), i32(args[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cg.check(cg.cg_cross_attend(p, q, k, v, cu, begin, count, outs[0], None, ws[0]), "cross")
    for _ in range(3):
        outs[0].zero_(), outs[1].zero_()
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            cg.check(cg.cg_cross_attend(p, q, k, v, cu, begin, count, outs[1], None, ws[1]), "cross")
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    # other lengths in the captured call
    count.copy_(i32([1, 7]))
    graph.replay()
    torch.cuda.synchronize()
    again, _, _ = run(q, k, v, args[0], args[1], [1, 7], 0.1, max_k=3000)
    assert torch.equal(outs[0], again)


def test_parts_join_to_the_whole():
    """A loaded context by cg_cross_attend and a question's own keys by cg_prompt_attend, joined by their lse, are the causal attention over both."""
    n, c, H, Hq, d = 50, 700, 2, 8, 64
    q, k, v = rows(n, Hq, d, F16, 1).cuda(), rows(c + n, H, d, F16, 2, True).cuda(), rows(c + n, H, d, F16, 3).cuda()
    a, za, _ = run(q, k, v, [0, n], [0], [c], 0.1)

    def prompt(kk, vv, nk):
        p = cg.Prompt(1, Hq, H, d, cg.CG_F16, n, nk, n, nk, 0.1, q.stride()[:2], kk.stride()[:2], vv.stride()[:2])
        ws, out, z = cg.empty_u8(cg.cg_prompt_workspace_bytes(p)), torch.empty_like(q), torch.empty(n, Hq, device="cuda")
        cg.check(cg.cg_prompt_attend(p, q, kk, vv, i32([0, n]), i32([0, nk]), out, z, ws), "prompt")
        return out, z

    b, zb = prompt(k[c:], v[c:], n)
    want, zw = prompt(k, v, c + n)
    z = torch.logaddexp(za.double(), zb.double())
    out = torch.exp(za.double() - z)[..., None] * a.double() + torch.exp(zb.double() - z)[..., None] * b.double()
    # three outputs, each rounded once to f16 (2^-11 of the largest value), with weights rounded to 11 bits before it
    assert (out - want.double()).abs().max() <= 6 * 2.0 ** -11 * v.abs().max().item()
    assert (z - zw.double()).abs().max() <= 1e-4
