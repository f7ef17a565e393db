"""Serving a context that came out of the codec: what is measured, in plain torch and through the library.

Four operators of a server that keeps decoded contexts in pages:

  attend   attention of a few new tokens over a cache held in 8 bits (e4m3 or int8 codes, one scale for each page and KV head)
  write    new keys and values into those pages
  prompt   causal attention of packed prompts with grouped heads, each prompt at the end of its own keys
  branch, compact, copy   the pages themselves: dropping and forking sequences that share pages, closing the gaps, copying pages

Each is reached through `run`, which computes it from elementary torch operations where `own` is false and makes the library's calls
where it is true. `exact` restates attend, write and prompt in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

QMAX = {"e4m3": 448.0, "int8": 127.0}
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TINY_SCALE = 2.0 ** -100  # a page whose scale would be under this is held as zeros


# ---- cases --------------------------------------------------------------------
def listed():
    return [
        # one reader's next token on a short context of an 8-KV-head, 32-head model: the latency of a single call
        dict(name="attend_one_short", op="attend", format="e4m3", dtype="float16", batch=1, tokens=1, heads=32, kv_heads=8, d=128, page=16,
             longest=500, shortest=500, lens=1),
        # a full batch of readers, 64 heads on 8 KV heads, contexts from a few tokens to 8K
        dict(name="attend_batch_ragged", op="attend", format="e4m3", dtype="bfloat16", batch=64, tokens=1, heads=64, kv_heads=8, d=128, page=64,
             longest=8192, shortest=20, lens=2),
        # the longest contexts of the workloads (131072 tokens), int8 codes
        dict(name="attend_long_context", op="attend", format="int8", dtype="float16", batch=4, tokens=1, heads=64, kv_heads=8, d=128, page=64,
             longest=131072, shortest=120000, lens=3),
        # a batch that verifies five drafted tokens each, three heads to a KV head, d = 80, pages of 24, empty sequences among them
        dict(name="attend_drafts_odd", op="attend", format="int8", dtype="bfloat16", batch=17, tokens=5, heads=12, kv_heads=4, d=80, page=24,
             longest=3001, shortest=0, lens=4),
        # the step's new token of 64 readers goes into their last pages
        dict(name="write_one_token", op="write", format="e4m3", dtype="bfloat16", batch=64, kv_heads=8, d=128, page=64, new=1, ragged=False,
             start=8000, layout="packed", lens=5),
        # a decoded context of 32768 tokens, in the codec's layout, goes into pages
        dict(name="write_context", op="write", format="int8", dtype="float16", batch=1, kv_heads=8, d=128, page=64, new=32768, ragged=False,
             start=0, layout="codec", lens=6),
        # a question of 77 tokens on a loaded context of 32768, 64 heads on 8: the time to the first token
        dict(name="prompt_question", op="prompt", dtype="float16", batch=1, heads=64, kv_heads=8, d=128, longest=77, shortest=77, context=32768,
             layout="codec", lens=7),
        # a batch of ragged prompts in one pack, some of them behind a context
        dict(name="prompt_packed_ragged", op="prompt", dtype="bfloat16", batch=13, heads=32, kv_heads=8, d=128, longest=2000, shortest=1, context=700,
             layout="fused", lens=8),
        # one whole prompt of 8192 tokens
        dict(name="prompt_long", op="prompt", dtype="bfloat16", batch=1, heads=32, kv_heads=8, d=128, longest=8192, shortest=8192, context=0,
             layout="fused", lens=9),
        # four readers branch off one short context of a two-layer cache
        dict(name="branch_small", op="branch", format="e4m3", layers=2, kv_heads=2, d=64, page=16, parents=1, fan=4, longest=250, grow=9, spare=40,
             lens=10),
        # 64 branches off eight contexts of a 32-layer cache with 8 KV heads
        dict(name="branch_wide", op="branch", format="int8", layers=32, kv_heads=8, d=128, page=64, parents=8, fan=8, longest=1024, grow=40, spare=200,
             lens=11),
        # a third of that cache's pages are left, all over the pool: they move to its front
        dict(name="compact_layers", op="compact", format="int8", layers=32, kv_heads=8, d=128, page=64, n_blocks=260, seqs=12, longest=512, lens=12),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "write", "prompt", "prompt", "branch", "compact", "copy"])
    seed = rng.randrange(1 << 30)
    fmt, dt = rng.choice(["e4m3", "int8"]), rng.choice(["float16", "bfloat16"])
    d, page = rng.choice([128, 128, 64, 96, 80, 40, 16, 8]), rng.choice([16, 32, 64, 128, 24, 7, 1])
    kv, group = rng.choice([1, 2, 4, 8, 8, 5]), rng.choice([1, 2, 3, 4, 8, 8, 16, 7])
    if op == "attend":
        batch, tokens = _log(rng, 1, 128), rng.choice([1, 1, 1, 2, 3, 5, 8])
        room = 500_000_000 // (batch * kv * d * 2)
        longest = _log(rng, 1, max(2, min(131072, room)))
        if page == 1:
            longest = min(longest, 4096)
        return dict(op=op, format=fmt, dtype=dt, batch=batch, tokens=tokens, heads=kv * group, kv_heads=kv, d=d, page=page, longest=longest,
                    shortest=rng.choice([0, 1, longest]), lens=seed)
    if op == "write":
        batch = _log(rng, 1, 128)
        new = rng.choice([1, 1, _log(rng, 1, max(2, min(32768, 60000 // batch)))])
        layout = "packed" if batch > 1 else rng.choice(["packed", "codec"])
        return dict(op=op, format=fmt, dtype=dt, batch=batch, kv_heads=kv, d=d, page=page, new=new, ragged=rng.random() < 0.5,
                    start=rng.choice([0, 5, 1000]), layout=layout, lens=seed)
    if op == "prompt":
        batch, heads = rng.choice([1, 1, 2, 5, 13, 40]), kv * group
        longest = _log(rng, 1, 4096)
        context = rng.choice([0, 0, _log(rng, 1, 32768)])
        while batch * heads * longest * (longest + context) > 1_000_000_000:
            longest, context, batch = max(1, longest * 2 // 3), context * 2 // 3, max(1, batch * 3 // 4)
        layout = rng.choice(["fused", "codec"]) if batch == 1 else "fused"
        return dict(op=op, dtype=dt, batch=batch, heads=heads, kv_heads=kv, d=d, longest=longest, shortest=rng.choice([1, longest]), context=context,
                    layout=layout, lens=seed)
    layers = rng.choice([1, 2, 8, 32])
    page = max(page, 7)
    pages = max(30, min(3000, 1_000_000_000 // (2 * layers * kv * d * page)))
    if op == "branch":
        parents, fan = rng.choice([1, 2, 5]), rng.choice([1, 2, 4, 8])
        longest = max(1, min(_log(rng, 1, 4000), pages // (2 * parents) * page))
        return dict(op=op, format=fmt, layers=layers, kv_heads=kv, d=d, page=page, parents=parents, fan=fan, longest=longest, grow=rng.choice([0, 1, 30]),
                    spare=min(pages, 300), lens=seed)
    if op == "compact":
        seqs = rng.choice([1, 3, 12])
        return dict(op=op, format=fmt, layers=layers, kv_heads=kv, d=d, page=page, n_blocks=pages, seqs=seqs,
                    longest=max(1, min(2000, pages // (2 * seqs) * page)), lens=seed)
    return dict(op=op, format=fmt, layers=layers, kv_heads=kv, d=d, page=page, n_blocks=min(pages, 600), copies=_log(rng, 1, min(pages, 600) // 3),
                lens=seed)


def _lengths(case, count, shortest, longest):
    """Lengths spread over their logarithm, the longest first; where `shortest` is 0 some are empty."""
    rng = random.Random(case["lens"])
    got = [longest] + [_log(rng, max(1, shortest), longest) if longest else 0 for _ in range(count - 1)]
    if shortest == 0:
        got = [0 if i % 5 == 3 else n for i, n in enumerate(got)]
    return got


def _write_lengths(case):
    rng = random.Random(case["lens"])
    new = [case["new"] if i == 0 or not case["ragged"] else rng.randint(0, case["new"]) for i in range(case["batch"])]
    start = [rng.randint(0, case["start"]) for _ in range(case["batch"])]
    return new, start


def _prompt_lengths(case):
    nq = _lengths(case, case["batch"], case["shortest"], case["longest"])
    rng = random.Random(case["lens"] + 1)
    if case["batch"] == 1:
        return nq, [nq[0] + case["context"]]
    return nq, [n + (rng.randint(0, case["context"]) if rng.random() < 0.5 else 0) for n in nq]


def _branch_lengths(case):
    return _lengths(case, case["parents"], 1, case["longest"])


# ---- what a program has in hand ---------------------------------------------------
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _keys(shape, g):
    """Normal values with a few channels that are ten times as large, as keys have."""
    x = torch.randn(shape, generator=g, device="cuda")
    x[..., 3::64] *= 10.0
    return x


def _codes_of(x, fmt):
    q = QMAX[fmt]
    return x.clamp(-q, q).to(CODE[fmt]) if fmt == "e4m3" else x.round().clamp(-q, q).to(CODE[fmt])


def _page_pool(x, fmt):
    """x [n_blocks, H, page, d] -> codes of the same shape, scales [n_blocks, H]."""
    s = x.abs().amax((2, 3)) / QMAX[fmt]
    return _codes_of(x / s[:, :, None, None], fmt), s


def _shuffled(n, g):
    return torch.randperm(n, generator=g, device="cuda").to(torch.int32)


def _table(lengths, page, order, width=None):
    """A table [n, width] whose rows take the pages of `order` in turn; -1 where a row has none."""
    counts = torch.tensor([-(-n // page) for n in lengths], device="cuda")
    width = max(1, int(counts.max())) if width is None else width
    at = torch.arange(width, device="cuda")
    took = (counts.cumsum(0) - counts)[:, None] + at
    return torch.where(at < counts[:, None], order[took.clamp(max=order.numel() - 1)], -1).to(torch.int32)


def prepare(case, seed):
    s = dict(case=case)
    {"attend": _prepare_attend, "write": _prepare_write, "prompt": _prepare_prompt, "branch": _prepare_branch, "compact": _prepare_compact,
     "copy": _prepare_copy}[case["op"]](s, case, _generator(seed))
    return s


def _prepare_attend(s, case, g):
    B, T, Hq, H, d, bt = (case[k] for k in ("batch", "tokens", "heads", "kv_heads", "d", "page"))
    lens = _lengths(case, B, case["shortest"], case["longest"])
    need = sum(-(-n // bt) for n in lens)
    n_blocks = need + need // 8 + 2
    s["table"] = _table(lens, bt, _shuffled(n_blocks, g))
    s["lens"] = _ints(lens)
    s["q"] = torch.randn((B, T, Hq, d), generator=g, device="cuda").to(getattr(torch, case["dtype"]))
    s["scale"] = d ** -0.5
    s["k"], s["k_scale"] = _page_pool(_keys((n_blocks, H, bt, d), g), case["format"])
    s["v"], s["v_scale"] = _page_pool(torch.randn((n_blocks, H, bt, d), generator=g, device="cuda"), case["format"])
    # what an earlier owner left: in pages that no sequence has, and behind each sequence's last token
    stale = torch.ones((n_blocks, bt), dtype=torch.bool, device="cuda")
    at = torch.arange(s["table"].shape[1] * bt, device="cuda")
    live = at < s["lens"][:, None]
    page = s["table"].long().repeat_interleave(bt, 1)
    stale[page[live], (at % bt).expand_as(page)[live]] = False
    for pool in (s["k"], s["v"]):
        pool.view(torch.uint8).masked_fill_(stale[:, None, :, None], 0x7F)  # e4m3's NaN
    unused = stale.all(1)
    s["k_scale"][unused] = float("nan")
    s["v_scale"][unused] = float("nan")


def _prepare_write(s, case, g):
    B, H, d, bt = (case[k] for k in ("batch", "kv_heads", "d", "page"))
    dt = getattr(torch, case["dtype"])
    new, start = _write_lengths(case)
    total = [a + n for a, n in zip(start, new)]
    need = sum(-(-n // bt) for n in total)
    n_blocks = need + need // 8 + 2
    s["table"] = _table(total, bt, _shuffled(n_blocks, g))
    s["start"], s["cu"] = _ints(start), _ints(np.concatenate([[0], np.cumsum(new)]))
    s["k"], s["k_scale"] = _page_pool(_keys((n_blocks, H, bt, d), g), case["format"])
    s["v"], s["v_scale"] = _page_pool(torch.randn((n_blocks, H, bt, d), generator=g, device="cuda"), case["format"])
    n = sum(new)
    if case["layout"] == "codec":  # one layer of the codec's [L, 2, H, S, d]
        kv = torch.stack([_keys((H, n, d), g), torch.randn((H, n, d), generator=g, device="cuda")]).to(dt)
        s["new_k"], s["new_v"] = kv[0].transpose(0, 1), kv[1].transpose(0, 1)
    else:  # one projection's rows, keys and values side by side
        kv = torch.cat([_keys((n, H, d), g), torch.randn((n, H, d), generator=g, device="cuda")], 1).to(dt)
        s["new_k"], s["new_v"] = kv[:, :H], kv[:, H:]


def _prepare_prompt(s, case, g):
    Hq, H, d = (case[k] for k in ("heads", "kv_heads", "d"))
    dt = getattr(torch, case["dtype"])
    nq, nk = _prompt_lengths(case)
    s["cu_q"], s["cu_k"] = (_ints(np.concatenate([[0], np.cumsum(n)])) for n in (nq, nk))
    s["scale"] = d ** -0.5
    if case["layout"] == "codec":
        s["q"] = torch.randn((sum(nq), Hq, d), generator=g, device="cuda").to(dt)
        kv = torch.stack([_keys((H, sum(nk), d), g), torch.randn((H, sum(nk), d), generator=g, device="cuda")]).to(dt)
        s["k"], s["v"] = kv[0].transpose(0, 1), kv[1].transpose(0, 1)
    else:  # one projection's rows; the keys' rows are more where prompts have a context
        s["q"] = torch.randn((sum(nq), Hq + 2 * H, d), generator=g, device="cuda").to(dt)[:, :Hq]
        kv = torch.cat([_keys((sum(nk), H, d), g), torch.randn((sum(nk), H, d), generator=g, device="cuda")], 1).to(dt)
        s["k"], s["v"] = kv[:, :H], kv[:, H:]


def _random_pools(s, case, n_blocks, g):
    L, H, d, bt = (case[k] for k in ("layers", "kv_heads", "d", "page"))
    s["pools"] = torch.randint(0, 120, (2 * L, n_blocks, H, bt, d), generator=g, device="cuda", dtype=torch.uint8)
    s["scales"] = torch.rand((2 * L, n_blocks, H), generator=g, device="cuda")


def _prepare_branch(s, case, g):
    lens = _branch_lengths(case)
    P, fan, bt = case["parents"], case["fan"], case["page"]
    need = sum(-(-n // bt) for n in lens)
    grown = sum(fan * (-(-(n + case["grow"]) // bt) - n // bt) for n in lens)
    n_blocks = need + grown + case["spare"]
    width = -(-(max(lens) + case["grow"]) // bt)
    order = _shuffled(n_blocks, g)
    s["refs"] = torch.zeros(n_blocks, dtype=torch.int32, device="cuda")
    s["refs"][order[:need].long()] = 1
    s["table"] = torch.cat([_table(lens, bt, order, width), torch.full((P * fan, width), -1, dtype=torch.int32, device="cuda")])
    s["lens"] = _ints(lens + [0] * (P * fan))
    s["parents"] = _ints([p for p in range(P) for _ in range(fan)])
    s["children"] = _ints(range(P, P + P * fan))
    s["new_len"] = _ints([lens[p] + case["grow"] for p in range(P) for _ in range(fan)])
    _random_pools(s, case, n_blocks, g)


def _prepare_compact(s, case, g):
    lens = _lengths(case, case["seqs"], 1, case["longest"])
    order = _shuffled(case["n_blocks"], g)
    need = sum(-(-n // case["page"]) for n in lens)
    s["table"] = _table(lens, case["page"], order)
    s["table"] = torch.cat([s["table"], s["table"][:1]])  # the last sequence shares the first one's pages
    s["refs"] = torch.zeros(case["n_blocks"], dtype=torch.int32, device="cuda")
    s["refs"][order[:need].long()] = 1
    s["refs"][s["table"][-1][s["table"][-1] >= 0].long()] += 1
    s["lens"] = _ints(lens + lens[:1])
    _random_pools(s, case, case["n_blocks"], g)


def _prepare_copy(s, case, g):
    order = _shuffled(case["n_blocks"], g)
    s["src"], s["dst"] = order[:case["copies"]].clone(), order[case["copies"]:2 * case["copies"]].clone()
    _random_pools(s, case, case["n_blocks"], g)


# ---- one pass -------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    return (_OWN if own else _PLAIN)[op](state)


def _softmax_product(scores, seen, v):
    """scores [..., n, S] with `seen` of their shape, v [..., S, d] -> outputs, natural log-sum-exp; 0 and -inf for rows that see nothing."""
    scores = torch.where(seen, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total == 0.0, 1.0, total)
    return out, (torch.log(total) + top).squeeze(-1)


def _plain_attend(s):
    c, q = s["case"], s["q"]
    B, T, Hq, d = q.shape
    H, bt = c["kv_heads"], c["page"]
    table = s["table"].clamp(min=0).long()
    at = torch.arange(table.shape[1] * bt, device="cuda")
    live = (at < s["lens"][:, None])[:, None, :, None]

    def rows(codes, scale):
        x = codes[table].float() * scale[table][..., None, None]
        return torch.where(live, x.transpose(1, 2).reshape(B, H, -1, d), 0.0)

    qh = q.float().view(B, T, H, Hq // H, d).permute(0, 2, 1, 3, 4).reshape(B, H, -1, d)
    scores = (qh @ rows(s["k"], s["k_scale"]).transpose(2, 3)) * s["scale"]
    last = s["lens"][:, None] - T + torch.arange(T, device="cuda").repeat_interleave(Hq // H)
    out, lse = _softmax_product(scores, (at <= last[..., None])[:, None], rows(s["v"], s["v_scale"]))
    out = out.view(B, H, T, Hq // H, d).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, d)
    return dict(out=out.to(q.dtype), lse=lse.view(B, H, T, Hq // H).permute(0, 2, 1, 3).reshape(B, T, Hq))


def _plain_write(s):
    c = s["case"]
    bt, fmt = c["page"], c["format"]
    n = s["new_k"].shape[0]
    row = torch.arange(n, device="cuda")
    seq = torch.searchsorted(s["cu"][1:].contiguous(), row.to(torch.int32), right=True)
    pos = s["start"][seq] + row - s["cu"][seq]
    page, slot = s["table"][seq, pos // bt].long(), (pos % bt).long()

    def write(x, codes, scale):
        x = x.float()
        top = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(2), "amax")
        first = torch.full((scale.shape[0],), bt, device="cuda").index_reduce_(0, page, slot, "amin")
        touched, kept = (first < bt)[:, None], ((first > 0) & (first < bt))[:, None]
        fresh = top / QMAX[fmt]
        fresh = torch.where(fresh < TINY_SCALE, 0.0, fresh)
        now = torch.where(kept, torch.maximum(scale, fresh), fresh)
        ratio = torch.where(kept & (now > scale), scale / now, 1.0)
        old = (torch.arange(bt, device="cuda") < first[:, None])[:, None, :, None] & (ratio != 1.0)[..., None, None]
        again = _codes_of(codes.float() * ratio[..., None, None], fmt)
        codes.view(torch.uint8).copy_(torch.where(old, again.view(torch.uint8), codes.view(torch.uint8)))
        scale.copy_(torch.where(touched, now, scale))
        turn = torch.where(now > 0, 1.0 / now, 0.0)
        codes.view(torch.uint8)[page, :, slot] = _codes_of(x * turn[page][..., None], fmt).view(torch.uint8)

    write(s["new_k"], s["k"], s["k_scale"])
    write(s["new_v"], s["v"], s["v_scale"])
    return dict(k=s["k"], v=s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"])


def _plain_prompt(s):
    c, q = s["case"], s["q"]
    H, G, d, mq = c["kv_heads"], c["heads"] // c["kv_heads"], c["d"], c["longest"]
    nq, nk = s["cu_q"].diff(), s["cu_k"].diff()
    mk = c["longest"] + c["context"]
    iq, ik = torch.arange(mq, device="cuda"), torch.arange(mk, device="cuda")
    rq = (s["cu_q"][:-1, None] + iq).clamp(max=q.shape[0] - 1)
    rk = (s["cu_k"][:-1, None] + ik).clamp(max=s["k"].shape[0] - 1)
    B = nq.numel()

    def rows(x):
        return torch.where((ik < nk[:, None])[..., None, None], x[rk].float(), 0.0).permute(0, 2, 1, 3)

    qh = q[rq].float().view(B, mq, H, G, d).permute(0, 2, 3, 1, 4).reshape(B, H, G * mq, d)
    scores = (qh @ rows(s["k"]).transpose(2, 3)) * s["scale"]
    last = (nk - nq)[:, None] + iq
    seen = (ik <= last[..., None]).repeat(1, G, 1)[:, None]
    out, lse = _softmax_product(scores, seen, rows(s["v"]))
    out = out.view(B, H * G, mq, d).transpose(1, 2)
    lse = lse.view(B, H * G, mq).transpose(1, 2)
    real = iq < nq[:, None]
    return dict(out=out[real].to(q.dtype), lse=lse[real])


def _share(refs, rows, by):
    """refs + by for each entry >= 0 of rows."""
    flat = rows.flatten().long()
    return refs.index_add_(0, flat.clamp(min=0), torch.where(flat >= 0, by, 0).to(refs.dtype))


def _plain_branch(s):
    refs, table, lens, bt = s["refs"], s["table"], s["lens"], s["case"]["page"]
    parents, children = s["parents"].long(), s["children"].long()
    # the last step's branches are dropped
    _share(refs, table[children], -1)
    table[children] = -1
    lens[children] = 0
    # new ones share the parents' whole pages and have a copy of the part of a page
    free = torch.sort((refs > 0).to(torch.int8), stable=True).indices
    part = lens[parents] % bt != 0
    fresh = free[(part.cumsum(0) - 1).clamp(min=0)]
    rows, last = table[parents], (lens[parents] // bt).long()[:, None].clamp(max=table.shape[1] - 1)
    old = rows.gather(1, last)[:, 0].long()
    _share(refs, rows, 1)
    refs.index_add_(0, torch.where(part, old, 0), -part.to(refs.dtype))
    refs.index_add_(0, torch.where(part, fresh, 0), part.to(refs.dtype))
    table[children] = rows.scatter(1, last, torch.where(part, fresh, old).to(rows.dtype)[:, None])
    lens[children] = lens[parents]
    s["pools"][:, fresh[part]] = s["pools"][:, old[part]]
    s["scales"][:, fresh[part]] = s["scales"][:, old[part]]
    # and grow by the step's tokens
    at = torch.arange(table.shape[1], device="cuda")
    have, want = -(-lens[children] // bt), -(-s["new_len"] // bt)
    lacks = (at >= have[:, None]) & (at < want[:, None])
    free = torch.sort((refs > 0).to(torch.int8), stable=True).indices
    took = free[(lacks.flatten().cumsum(0) - 1).clamp(min=0)].view_as(lacks)
    table[children] = torch.where(lacks, took.to(table.dtype), table[children])
    refs.index_add_(0, torch.where(lacks, took, 0).flatten(), lacks.flatten().to(refs.dtype))
    lens[children] = s["new_len"]
    return dict(refs=refs, table=table, lens=lens, pools=s["pools"], scales=s["scales"])


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    live = refs > 0
    n_live = live.sum()
    at = torch.arange(refs.numel(), device="cuda")
    holes, movers = torch.nonzero(~live & (at < n_live))[:, 0], torch.nonzero(live & (at >= n_live))[:, 0]
    place = at.clone()
    place[movers] = holes
    refs_out = torch.where(live & (at < n_live), refs, 0)
    refs_out[holes] = refs[movers]
    table_out = torch.where(table >= 0, place[table.clamp(min=0).long()].to(table.dtype), table)
    s["pools"][:, holes] = s["pools"][:, movers]
    s["scales"][:, holes] = s["scales"][:, movers]
    return dict(n_live=n_live.to(torch.int32).view(1), refs=refs_out, table=table_out, pools=s["pools"], scales=s["scales"])


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    s["pools"][:, dst] = s["pools"][:, src]
    s["scales"][:, dst] = s["scales"][:, src]
    return dict(pools=s["pools"], scales=s["scales"])


_PLAIN = dict(attend=_plain_attend, write=_plain_write, prompt=_plain_prompt, branch=_plain_branch, compact=_plain_compact, copy=_plain_copy)


# ---- the same pass through the library --------------------------------------------
def _kept(s, make):
    """The descriptions, workspace and output buffers that a server keeps from call to call."""
    if "kept" not in s:
        from kv_cache_compression_02_gb300 import cachegen as cg
        s["kept"] = make(cg, s, s["case"])
    return s["kept"]


def _format(cg, c):
    return {"e4m3": cg.CG_CACHE_E4M3, "int8": cg.CG_CACHE_INT8}[c["format"]]


def _dtype(cg, c):
    return {"float16": cg.CG_F16, "bfloat16": cg.CG_BF16}[c["dtype"]]


def _own_attend(s):
    def make(cg, s, c):
        cache = cg.Cache(1, c["kv_heads"], c["d"], c["page"], s["k"].shape[0], _format(cg, c))
        att = cg.Attend(c["batch"], c["tokens"], c["heads"], _dtype(cg, c), s["table"].shape[1], s["scale"])
        return cg, cache, att, torch.empty_like(s["q"]), torch.empty(s["q"].shape[:3], device="cuda"), cg.empty_u8(cg.cg_cache_workspace_bytes(cache, att))

    cg, cache, att, out, lse, ws = _kept(s, make)
    cg.check(cg.cg_cache_attend(cache, att, s["q"], s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"], s["lens"], out, lse, ws), "attend")
    return dict(out=out, lse=lse)


def _own_write(s):
    def make(cg, s, c):
        cache = cg.Cache(1, c["kv_heads"], c["d"], c["page"], s["k"].shape[0], _format(cg, c))
        k = s["new_k"]
        return cg, cache, cg.Rows(c["batch"], k.shape[0], c["new"], _dtype(cg, c), s["table"].shape[1], k.stride(0), k.stride(1)), cg.empty_u8(256)

    cg, cache, rows, ws = _kept(s, make)
    cg.check(cg.cg_cache_write(cache, rows, s["new_k"], s["new_v"], s["cu"], s["start"], s["table"], s["k"], s["v"], s["k_scale"], s["v_scale"], ws),
             "write")
    return dict(k=s["k"], v=s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"])


def _own_prompt(s):
    def make(cg, s, c):
        q, k, v = s["q"], s["k"], s["v"]
        p = cg.Prompt(c["batch"], c["heads"], c["kv_heads"], c["d"], _dtype(cg, c), q.shape[0], k.shape[0], c["longest"], c["longest"] + c["context"],
                      s["scale"], q.stride()[:2], k.stride()[:2], v.stride()[:2])
        return cg, p, torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(q.shape[:2], device="cuda"), cg.empty_u8(cg.cg_prompt_workspace_bytes(p))

    cg, p, out, lse, ws = _kept(s, make)
    cg.check(cg.cg_prompt_attend(p, s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], out, lse, ws), "prompt")
    return dict(out=out, lse=lse)


def _make_pages(cg, s, c):
    pools, scales = s["pools"], s["scales"]
    cache = cg.Cache(c["layers"], c["kv_heads"], c["d"], c["page"], pools.shape[1], _format(cg, c))
    addr = [torch.tensor([t[i].data_ptr() for i in range(t.shape[0])], dtype=torch.int64, device="cuda") for t in (pools, scales)]
    pages = cg.Pages(s["refs"], s["table"], s["lens"]) if "refs" in s else None
    ws = cg.empty_u8(cg.cg_pages_workspace_bytes(cache, pages, s["children"].numel() if "children" in s else 0))
    more = [torch.empty_like(s["refs"]), torch.empty_like(s["table"]), _ints([0])] if c["op"] == "compact" else []
    return cg, cache, pages, addr, ws, more


def _own_branch(s):
    cg, cache, pages, (pools, scales), ws, _ = _kept(s, _make_pages)
    cg.check(cg.cg_pages_free(cache, pages, s["children"], ws), "free")
    cg.check(cg.cg_pages_fork(cache, pages, pools, scales, s["parents"], s["children"], ws), "fork")
    cg.check(cg.cg_pages_extend(cache, pages, s["children"], s["new_len"], ws), "extend")
    return dict(refs=s["refs"], table=s["table"], lens=s["lens"], pools=s["pools"], scales=s["scales"])


def _own_compact(s):
    cg, cache, pages, (pools, scales), ws, (refs, table, n_live) = _kept(s, _make_pages)
    cg.check(cg.cg_pages_compact(cache, pages, pools, scales, refs, table, n_live, ws), "compact")
    return dict(n_live=n_live, refs=refs, table=table, pools=s["pools"], scales=s["scales"])


def _own_copy(s):
    cg, cache, _, (pools, scales), ws, _ = _kept(s, _make_pages)
    cg.check(cg.cg_pages_copy(cache, pools, scales, s["src"], s["dst"], ws), "copy")
    return dict(pools=s["pools"], scales=s["scales"])


_OWN = dict(attend=_own_attend, write=_own_write, prompt=_own_prompt, branch=_own_branch, compact=_own_compact, copy=_own_copy)


# ---- what a pass cannot do without ---------------------------------------------------
def work(case):
    op = case["op"]
    if op == "attend":
        T, Hq, H, d, bt = (case[k] for k in ("tokens", "heads", "kv_heads", "d", "page"))
        lens = _lengths(case, case["batch"], case["shortest"], case["longest"])
        pages = sum(-(-n // bt) for n in lens)
        seen = sum(max(0, n - T + 1 + t) for n in lens for t in range(T))
        return dict(bytes=2 * sum(lens) * H * d + pages * (4 + 8 * H) + case["batch"] * (4 + T * Hq * (4 * d + 4)), flops=4.0 * seen * Hq * d)
    if op == "write":
        new, start = _write_lengths(case)
        rows, H, d, bt = sum(new), case["kv_heads"], case["d"], case["page"]
        pages = sum(-(-(a + n) // bt) - a // bt for a, n in zip(start, new) if n)
        return dict(bytes=2 * rows * H * d * 3 + pages * (4 + 2 * H * 4) + case["batch"] * 8, flops=2.0 * 2 * rows * H * d)
    if op == "prompt":
        nq, nk = _prompt_lengths(case)
        Hq, H, d = case["heads"], case["kv_heads"], case["d"]
        seen = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(nq, nk))
        return dict(bytes=4 * sum(nq) * Hq * d + 4 * sum(nq) * Hq + 4 * sum(nk) * H * d + 8 * (case["batch"] + 1), flops=4.0 * seen * Hq * d)
    one = 2 * 2 * case["layers"] * case["kv_heads"] * (case["page"] * case["d"] + 4)  # a page read and written, with its scales
    if op == "branch":
        bt, fan, lens = case["page"], case["fan"], _branch_lengths(case)
        width = -(-(max(lens) + case["grow"]) // bt)
        n_blocks = case["spare"] + sum(-(-n // bt) + fan * (-(-(n + case["grow"]) // bt) - n // bt) for n in lens)
        return dict(bytes=one * fan * sum(n % bt != 0 for n in lens) + 4 * (2 * n_blocks + 4 * len(lens) * fan * width), flops=0)
    if op == "compact":
        lens = _lengths(case, case["seqs"], 1, case["longest"])
        live, n = sum(-(-m // case["page"]) for m in lens), case["n_blocks"]
        # pages lie all over the pool: (n - live) / n of the live ones are behind the first `live` places
        return dict(bytes=one * live * (n - live) / n + 8 * n + 8 * (len(lens) + 1) * -(-max(lens) // case["page"]), flops=0)
    return dict(bytes=one * case["copies"] + 8 * case["copies"], flops=0)


# ---- the definitions in 64 bits ------------------------------------------------------
def exact(case, seed):
    op = case["op"]
    if op not in ("attend", "write", "prompt"):
        return None  # pages are moved as they are
    s = prepare(case, seed)
    return {"attend": _exact_attend, "write": _exact_write, "prompt": _exact_prompt}[op](s, case)


def _exact_rows(q, k, v, last, scale):
    """q [n, d], k and v [S, d]; row i sees keys 0 .. last[i]."""
    out = torch.zeros((q.shape[0], v.shape[1]), dtype=torch.float64, device="cuda")
    lse = torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device="cuda")
    if k.shape[0]:
        step = max(1, (1 << 28) // k.shape[0])
        for a in range(0, q.shape[0], step):
            x = torch.einsum("nd,sd->ns", q[a:a + step], k) * scale
            x.masked_fill_(torch.arange(k.shape[0], device="cuda") > last[a:a + step, None], -math.inf)
            z = torch.logsumexp(x, 1)
            w = torch.exp(x - z[:, None]).nan_to_num_(0.0)
            lse[a:a + step], out[a:a + step] = z, torch.einsum("ns,sd->nd", w, v)
    return out, lse


def _exact_attend(s, c):
    B, T, Hq, d = s["q"].shape
    H, bt = c["kv_heads"], c["page"]
    G = Hq // H
    out = torch.zeros((B, T, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        j = torch.arange(n, device="cuda")
        page = s["table"][b][j // bt].long()
        last = (torch.arange(T, device="cuda") + n - T).repeat_interleave(G)
        for h in range(H):
            k = s["k"][page, h, j % bt].to(torch.float64) * s["k_scale"][page, h].double()[:, None]
            v = s["v"][page, h, j % bt].to(torch.float64) * s["v_scale"][page, h].double()[:, None]
            o, z = _exact_rows(s["q"][b, :, h * G:(h + 1) * G].double().reshape(T * G, d), k, v, last, s["scale"])
            out[b, :, h * G:(h + 1) * G], lse[b, :, h * G:(h + 1) * G] = o.view(T, G, d), z.view(T, G)
    return dict(out=out, lse=lse)


def _exact_prompt(s, c):
    n_q, Hq, d = s["q"].shape
    G = Hq // c["kv_heads"]
    out = torch.zeros((n_q, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((n_q, Hq), -math.inf, dtype=torch.float64, device="cuda")
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    for b in range(len(cq) - 1):
        q0, q1, k0, k1 = cq[b], cq[b + 1], ck[b], ck[b + 1]
        last = torch.arange(q1 - q0, device="cuda") + (k1 - k0) - (q1 - q0)
        for h in range(Hq):
            out[q0:q1, h], lse[q0:q1, h] = _exact_rows(s["q"][q0:q1, h].double(), s["k"][k0:k1, h // G].double(), s["v"][k0:k1, h // G].double(), last,
                                                       s["scale"])
    return dict(out=out, lse=lse)


def _nearest_e4m3(x):
    """Doubles rounded to the nearest value of e4m3, halves to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_write(s, c):
    bt, fmt = c["page"], c["format"]
    cu, start = s["cu"].tolist(), s["start"].tolist()
    table = s["table"].tolist()
    pages, kept, parts = [], [], []
    for b in range(len(cu) - 1):
        at = cu[b]
        while at < cu[b + 1]:
            pos = start[b] + at - cu[b]
            n = min(cu[b + 1] - at, bt - pos % bt)
            pages.append(table[b][pos // bt])
            kept.append(pos % bt)
            parts.append((at, n))
            at += n
    got = {}
    for name in ("k", "v"):
        codes, scale = s[name].to(torch.float64), s[name + "_scale"].double()
        x = s["new_" + name].double()
        for p, s0, (at, n) in zip(pages, kept, parts):
            rows = x[at:at + n].transpose(0, 1)
            new = rows.abs().amax((1, 2)) / QMAX[fmt]
            now = torch.maximum(new, scale[p]) if s0 else new
            if s0:
                codes[p, :, :s0] = _nearest_e4m3(codes[p, :, :s0] * (scale[p] / now)[:, None, None])
            codes[p, :, s0:s0 + n] = _nearest_e4m3(rows / now[:, None, None])
            scale[p] = now
        got[name] = codes if fmt == "e4m3" else None  # int8 codes are whole numbers
        got[name + "_scale"] = scale
    return got
