"""Slots, groups, shared prefixes and cross attention refuse bad arguments at once, before any CUDA call (no GPU)."""
import ctypes

import pytest

from kv_cache_compression_02_gb300 import build, cachegen as cg

FAKE = 1 << 20  # an aligned non-null address that is never dereferenced
BIG = 1 << 34
BAD_CACHES = [dict(L=0), dict(H=0), dict(d=4), dict(d=12), dict(d=136), dict(block_tokens=0), dict(n_blocks=0), dict(format=3), dict(format=-1)]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return cg.lib()


def cache(**kw):
    return cg.Cache(**{**dict(L=2, H=4, d=128, block_tokens=16, n_blocks=100, format=cg.CG_CACHE_E4M3), **kw})


def refused(rc):
    return rc == cg.CG_ERR_INVALID_ARG


def ref(p):
    return None if p is None else ctypes.addressof(p)


BAD_BOOKS = [None, cg.cg_pages(0, 8, FAKE, FAKE, FAKE), cg.cg_pages(4, 0, FAKE, FAKE, FAKE), cg.cg_pages(4, 8, None, FAKE, FAKE),
             cg.cg_pages(4, 8, FAKE, None, FAKE), cg.cg_pages(4, 8, FAKE, FAKE, None), cg.cg_pages(4, 8, FAKE + 2, FAKE, FAKE)]


def test_slots_refuses(lib):
    def call(c=cache(), p=cg.cg_pages(4, 8, FAKE, FAKE, FAKE), n=5, **kw):
        a = {**dict(new=FAKE, cu=FAKE, start=FAKE, seq=FAKE, pos=FAKE, slot=FAKE, ws=FAKE, nb=256), **kw}
        return lib.cg_pages_slots(c.ref, ref(p), n, a["new"], a["cu"], a["start"], a["seq"], a["pos"], a["slot"], a["ws"], a["nb"], None)

    for p in BAD_BOOKS:
        assert refused(call(p=p))
    for kw in BAD_CACHES:
        assert refused(call(c=cache(**kw))), kw
    assert refused(call(n=-1))
    for name in ("new", "cu", "start", "ws"):
        assert refused(call(**{name: None})), name
    for name in ("new", "cu", "start", "seq", "pos", "ws"):
        assert refused(call(**{name: FAKE + 2})), name
    assert refused(call(slot=FAKE + 4)) and refused(call(nb=255)) and refused(call(ws=FAKE + 128))


def test_groups_refuses(lib):
    book = cg.cg_pages(4, 8, FAKE, FAKE, FAKE)
    some = cache()
    need = lib.cg_pages_workspace_bytes(some.ref, ref(book), 4)
    assert need > 256

    def call(c=cache(), p=book, m=1, **kw):
        a = {**dict(cu=FAKE, member=FAKE, shared=FAKE, ws=FAKE, nb=BIG), **kw}
        return lib.cg_pages_groups(c.ref, ref(p), m, a["cu"], a["member"], a["shared"], a["ws"], a["nb"], None)

    for p in BAD_BOOKS:
        assert refused(call(p=p))
    for kw in BAD_CACHES:
        assert refused(call(c=cache(**kw))), kw
    assert refused(call(m=0)) and refused(call(m=-3))
    for name in ("cu", "member", "shared", "ws"):
        assert refused(call(**{name: None})) and refused(call(**{name: FAKE + 2})), name
    assert refused(call(nb=need - 1)) and refused(call(ws=FAKE + 128))


def test_cross_refuses(lib):
    ok = dict(n_seq=1, Hq=8, H=4, d=128, dtype=1, n_q=10, n_k=10, max_q=10, max_k=10, scale=0.1, q_stride=(1024, 128), k_stride=(512, 128),
              v_stride=(512, 128))
    prompt = lambda **kw: cg.Prompt(**{**ok, **kw})  # noqa: E731

    def call(p, **kw):
        a = {**dict(q=FAKE, k=FAKE, v=FAKE, cq=FAKE, kb=FAKE, kl=FAKE, out=FAKE, lse=FAKE, ws=FAKE, nb=BIG), **kw}
        return lib.cg_cross_attend(p if p is None else p.ref, a["q"], a["k"], a["v"], a["cq"], a["kb"], a["kl"], a["out"], a["lse"], a["ws"], a["nb"], None)

    assert refused(call(None))
    for kw in (dict(n_seq=0), dict(Hq=0), dict(H=0), dict(Hq=6), dict(Hq=4 * 129), dict(d=4), dict(d=20), dict(d=136), dict(dtype=2), dict(n_q=-1),
               dict(n_k=-1), dict(n_k=(1 << 30) + 1), dict(max_q=-1), dict(max_k=-1), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(q_stride=(1023, 128)), dict(k_stride=(512, 4)), dict(v_stride=(2, 128))):
        assert refused(call(prompt(**kw))), kw
    for name in ("q", "k", "v", "cq", "kb", "kl", "out", "ws"):
        assert refused(call(prompt(), **{name: None})), name
        assert refused(call(prompt(), **{name: FAKE + 2})), name
    assert refused(call(prompt(), lse=FAKE + 1))
    assert refused(call(prompt(), nb=cg.cg_prompt_workspace_bytes(prompt()) - 1))


def test_shared_refuses(lib):
    att = lambda **kw: cg.Attend(**{**dict(n_seq=6, q_tokens=1, Hq=8, dtype=0, table_stride=4, scale=0.1), **kw})  # noqa: E731
    ok = cg.cg_groups(2, 6, FAKE, FAKE, FAKE)

    def call(c=cache(), t=None, g=ok, **kw):
        t = att() if t is None else t
        a = {**dict(q=FAKE, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, table=FAKE, len=FAKE, out=FAKE, lse=FAKE, ws=FAKE, nb=BIG), **kw}
        return lib.cg_shared_attend(c.ref, t.for_cache(c), ref(g), a["q"], a["kp"], a["vp"], a["ks"], a["vs"], a["table"], a["len"], a["out"], a["lse"],
                                    a["ws"], a["nb"], None)

    size = lambda c, t, g: lib.cg_shared_workspace_bytes(c.ref, t.for_cache(c), ref(g))  # noqa: E731
    nan, inf = float("nan"), float("inf")
    assert lib.cg_shared_workspace_bytes(None, None, None) == 0
    for kw in BAD_CACHES + [dict(format=cg.CG_CACHE_F16)]:
        assert refused(call(c=cache(**kw))) and size(cache(**kw), att(), ok) == 0, kw
    for kw in (dict(n_seq=0), dict(q_tokens=0), dict(Hq=0), dict(Hq=6), dict(dtype=-1), dict(table_stride=0), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=nan), dict(scale=inf), dict(q_stride=(1024, 1024, 100)), dict(q_stride=(1, 1024, 128)), dict(table_stride=(1 << 26) + 1)):
        assert refused(call(t=att(**kw))) and size(cache(), att(**kw), ok) == 0, kw
    for g in (None, cg.cg_groups(-1, 6, FAKE, FAKE, FAKE), cg.cg_groups(2, -1, FAKE, FAKE, FAKE), cg.cg_groups((1 << 20) + 1, 6, FAKE, FAKE, FAKE),
              cg.cg_groups(2, (1 << 20) + 1, FAKE, FAKE, FAKE)):
        assert refused(call(g=g)) and size(cache(), att(), g) == 0
    assert refused(call(t=att(n_seq=1, q_tokens=1 << 14), g=cg.cg_groups(1, 1 << 17, FAKE, FAKE, FAKE))), "more rows than are counted"
    for bad in (None, FAKE + 2):
        for i in range(3):
            p = [FAKE] * 3
            p[i] = bad
            assert refused(call(g=cg.cg_groups(2, 6, *p)))
    for name in ("q", "kp", "vp", "ks", "vs", "table", "len", "out", "ws"):
        assert refused(call(**{name: None})) and refused(call(**{name: FAKE + 2})), name
    assert refused(call(lse=FAKE + 1))
    some, t = cache(), att()
    need = size(some, t, ok)
    assert lib.cg_cache_workspace_bytes(some.ref, t.for_cache(some)) < need < 1 << 28
    assert refused(call(c=some, t=t, nb=need - 1)) and refused(call(c=some, t=t, ws=FAKE + 128))


def test_offsets_and_groups_have_their_lengths():
    import torch
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    for n, m in ((3, 3), (3, 1), (1, 1), (2, 0)):
        with pytest.raises(ValueError, match="offsets"):
            cg.Groups(i32(n), i32(4), i32(m))
