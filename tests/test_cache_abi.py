"""The serving calls refuse bad arguments at once, before any CUDA call (no GPU), and their sizes add up."""
import ctypes

import pytest

from kv_cache_compression_02_gb300 import build, cachegen as cg

FAKE = 1 << 20  # an aligned non-null address that is never dereferenced
BIG = 1 << 34


@pytest.fixture(scope="module")
def lib():
    build.build()
    return cg.lib()


def cache(**kw):
    a = dict(L=2, H=4, d=128, block_tokens=16, n_blocks=100, format=cg.CG_CACHE_E4M3)
    a.update(kw)
    return cg.Cache(**a)


def refused(rc):
    return rc == cg.CG_ERR_INVALID_ARG


BAD_CACHES = [dict(L=0), dict(H=0), dict(d=4), dict(d=12), dict(d=136), dict(block_tokens=0), dict(n_blocks=0), dict(format=3), dict(format=-1)]


def write_args(lib, c, rows, **kw):
    a = dict(k=FAKE, v=FAKE, cu=FAKE, start=FAKE, table=FAKE, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, ws=FAKE, nb=256)
    a.update(kw)
    return lib.cg_cache_write(c if c is None else c.ref, rows if rows is None else rows.ref, a["k"], a["v"], a["cu"], a["start"], a["table"], a["kp"],
                              a["vp"], a["ks"], a["vs"], a["ws"], a["nb"], None)


def test_write_refuses(lib):
    rows = lambda **kw: cg.Rows(**{**dict(n_seq=1, n_rows=8, max_new=8, dtype=0, table_stride=4, stride_token=512, stride_head=128), **kw})  # noqa: E731
    assert refused(write_args(lib, None, rows())) and refused(write_args(lib, cache(), None))
    for kw in BAD_CACHES + [dict(format=cg.CG_CACHE_F16)]:
        assert refused(write_args(lib, cache(**kw), rows())), kw
    for kw in (dict(n_seq=0), dict(n_rows=-1), dict(max_new=-1), dict(dtype=2), dict(table_stride=0), dict(stride_token=4), dict(stride_head=3)):
        assert refused(write_args(lib, cache(), rows(**kw))), kw
    for name in ("k", "v", "cu", "start", "table", "kp", "vp", "ks", "vs", "ws"):
        assert refused(write_args(lib, cache(), rows(), **{name: None})), name
        assert refused(write_args(lib, cache(), rows(), **{name: FAKE + 2})), name
    assert refused(write_args(lib, cache(), rows(), nb=255)) and refused(write_args(lib, cache(), rows(), ws=FAKE + 128))
    r = rows()
    r.c.reserved = 1
    assert refused(write_args(lib, cache(), r))


def test_attend_refuses(lib):
    att = lambda **kw: cg.Attend(**{**dict(n_seq=2, q_tokens=1, Hq=8, dtype=0, table_stride=4, scale=0.1), **kw})  # noqa: E731

    def call(c, t, **kw):
        a = dict(q=FAKE, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, table=FAKE, len=FAKE, out=FAKE, lse=FAKE, ws=FAKE, nb=BIG)
        a.update(kw)
        return lib.cg_cache_attend(c.ref, t if t is None else t.for_cache(c), a["q"], a["kp"], a["vp"], a["ks"], a["vs"], a["table"], a["len"], a["out"],
                                   a["lse"], a["ws"], a["nb"], None)

    nan, inf = float("nan"), float("inf")
    assert refused(call(cache(), None)) and lib.cg_cache_workspace_bytes(None, None) == 0
    for kw in BAD_CACHES + [dict(format=cg.CG_CACHE_F16)]:
        assert refused(call(cache(**kw), att())), kw
        assert cg.cg_cache_workspace_bytes(cache(**kw), att()) == 0
    for kw in (dict(n_seq=0), dict(q_tokens=0), dict(Hq=0), dict(Hq=6), dict(dtype=-1), dict(table_stride=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=nan),
               dict(scale=inf), dict(q_stride=(1024, 1024, 100)), dict(q_stride=(1, 1024, 128)),
               dict(table_stride=(1 << 26) + 1)):
        assert refused(call(cache(), att(**kw))), kw
        assert cg.cg_cache_workspace_bytes(cache(), att(**kw)) == 0
    for name in ("q", "kp", "vp", "ks", "vs", "table", "len", "out", "ws"):
        assert refused(call(cache(), att(), **{name: None})), name
        assert refused(call(cache(), att(), **{name: FAKE + 2})), name
    assert refused(call(cache(), att(), lse=FAKE + 1))
    assert refused(call(cache(), att(), nb=cg.cg_cache_workspace_bytes(cache(), att()) - 1))
    assert 256 <= cg.cg_cache_workspace_bytes(cache(), att()) < 1 << 26


def test_prompt_refuses(lib):
    ok = dict(n_seq=1, Hq=8, H=4, d=128, dtype=1, n_q=10, n_k=10, max_q=10, max_k=10, scale=0.1, q_stride=(1024, 128), k_stride=(512, 128),
              v_stride=(512, 128))
    prompt = lambda **kw: cg.Prompt(**{**ok, **kw})  # noqa: E731

    def call(p, **kw):
        a = dict(q=FAKE, k=FAKE, v=FAKE, cq=FAKE, ck=FAKE, out=FAKE, lse=FAKE, ws=FAKE, nb=BIG)
        a.update(kw)
        return lib.cg_prompt_attend(p if p is None else p.ref, a["q"], a["k"], a["v"], a["cq"], a["ck"], a["out"], a["lse"], a["ws"], a["nb"], None)

    assert refused(call(None)) and lib.cg_prompt_workspace_bytes(None) == 0
    for kw in (dict(n_seq=0), dict(Hq=0), dict(H=0), dict(Hq=6), dict(Hq=4 * 129), dict(d=4), dict(d=20), dict(d=136), dict(dtype=2), dict(n_q=-1), dict(n_k=-1), dict(n_k=(1 << 30) + 1),
               dict(max_q=-1), dict(max_k=-1), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q_stride=(1023, 128)),
               dict(k_stride=(512, 4)), dict(v_stride=(2, 128))):
        assert refused(call(prompt(**kw))), kw
        assert cg.cg_prompt_workspace_bytes(prompt(**kw)) == 0, kw
    for name in ("q", "k", "v", "cq", "ck", "out", "ws"):
        assert refused(call(prompt(), **{name: None})), name
        assert refused(call(prompt(), **{name: FAKE + 2})), name
    assert refused(call(prompt(), lse=FAKE + 1))
    assert refused(call(prompt(), nb=cg.cg_prompt_workspace_bytes(prompt()) - 1))
    assert 256 <= cg.cg_prompt_workspace_bytes(prompt()) < 1 << 30


def test_page_calls_refuse(lib):
    c = cache()
    ok = cg.cg_pages(4, 8, FAKE, FAKE, FAKE)
    ref = lambda p: None if p is None else ctypes.addressof(p)  # noqa: E731
    size = lib.cg_pages_workspace_bytes(c.ref, ref(ok), 10)
    assert size >= 256 + 4 * 4 + 3 * 4 * 100 and lib.cg_pages_workspace_bytes(c.ref, None, 10) > 0
    extend = lambda c, p, n=3, s=FAKE, t=FAKE, ws=FAKE, nb=BIG: lib.cg_pages_extend(c.ref, ref(p), n, s, t, ws, nb, None)  # noqa: E731
    fork = lambda c, p, n=3, po=FAKE, sc=FAKE, s=FAKE, t=FAKE, ws=FAKE, nb=BIG: lib.cg_pages_fork(  # noqa: E731
        c.ref, ref(p), po, sc, n, s, t, ws, nb, None)
    free = lambda c, p, n=3, s=FAKE, ws=FAKE, nb=BIG: lib.cg_pages_free(c.ref, ref(p), n, s, ws, nb, None)  # noqa: E731
    compact = lambda c, p, po=FAKE, sc=FAKE, s=FAKE, t=FAKE, nl=FAKE, ws=FAKE, nb=BIG: lib.cg_pages_compact(  # noqa: E731
        c.ref, ref(p), po, sc, s, t, nl, ws, nb, None)
    copy = lambda c, n=3, po=FAKE, sc=FAKE, s=FAKE, t=FAKE, ws=FAKE, nb=BIG: lib.cg_pages_copy(c.ref, po, sc, n, s, t, ws, nb, None)  # noqa: E731
    bad_books = [None, cg.cg_pages(0, 8, FAKE, FAKE, FAKE), cg.cg_pages(4, 0, FAKE, FAKE, FAKE), cg.cg_pages(4, 8, None, FAKE, FAKE),
                 cg.cg_pages(4, 8, FAKE, None, FAKE), cg.cg_pages(4, 8, FAKE, FAKE, None), cg.cg_pages(4, 8, FAKE + 2, FAKE, FAKE)]
    for call in (extend, fork, free, compact):
        for p in bad_books:
            assert refused(call(c, p))
        for kw in BAD_CACHES:
            assert refused(call(cache(**kw), ok)), kw
        assert refused(call(c, ok, ws=None)) and refused(call(c, ok, ws=FAKE + 16)) and refused(call(c, ok, nb=300))
        assert refused(call(c, ok, s=None)) and refused(call(c, ok, s=FAKE + 2))
    for kw in BAD_CACHES:
        assert refused(copy(cache(**kw))), kw
        assert lib.cg_pages_workspace_bytes(cache(**kw).ref, ref(ok), 3) == 0
    for call in (extend, fork, free):
        assert refused(call(c, ok, n=-1))
    for call in (lambda **kw: fork(c, ok, **kw), lambda **kw: compact(c, ok, **kw), lambda **kw: copy(c, **kw)):
        assert refused(call(po=None)) and refused(call(po=FAKE + 4)) and refused(call(sc=FAKE + 4))
        assert refused(call(sc=None)), "8-bit pages have scales"
        assert refused(call(s=None)) and refused(call(t=None)) and refused(call(t=FAKE + 1))
    assert refused(copy(c, n=-1)) and refused(copy(c, ws=None)) and refused(copy(c, nb=255))
    assert refused(extend(c, ok, t=None)) and refused(compact(c, ok, nl=None)) and refused(compact(c, ok, nl=FAKE + 2))
    assert lib.cg_pages_workspace_bytes(c.ref, ref(ok), -1) == 0


def test_write_refuses_pages_that_its_counts_cannot_hold(lib):
    """block_tokens * d over 2^32 (a head's codes of one page over 4 GB), which cg_cache_attend and the page calls may have."""
    for d, bt in ((128, (1 << 25) + 1), (128, 1 << 27), (128, 1 << 30), (8, (1 << 29) + 1), (72, 1 << 29)):
        big = cache(L=1, H=1, d=d, block_tokens=bt, n_blocks=2)
        rows = cg.Rows(1, 8, 8, cg.CG_F16, 1, d, d)
        assert refused(write_args(lib, big, rows)), (d, bt)
        assert cg.cg_pages_workspace_bytes(big, None, 1) > 0
