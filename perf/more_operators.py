"""Many readers of one context: what is measured, in plain torch and through the library.

Four operators of a server whose sequences branch off decoded contexts:

  shared   attention of a few new tokens over an 8-bit paged cache, for sequences that share the pages of a long prefix: the prefix is gone over once
           for all of its readers, what each of them has of its own beside it
  groups   which sequences of a block table share a prefix, and how many pages of it
  slots    the rows of a step from the sequences' lengths: offsets, positions and places in the pages
  cross    attention of packed queries to the states of an encoder, or of a loaded context, of other lengths, which several sequences may share

Each is reached through `run`, which computes it from elementary torch operations where `own` is false and makes the library's calls
where it is true. `exact` restates shared and cross in 64 bits; the other two give whole numbers.
"""
import math
import random

import torch

own = False

QMAX = {"e4m3": 448.0, "int8": 127.0}
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


# ---- cases --------------------------------------------------------------------
def listed():
    return [
        # three readers that have just branched off a short context: the latency of a step's call
        dict(name="shared_few_short", op="shared", format="e4m3", dtype="float16", groups=1, readers=3, loose=0, tokens=1, heads=8, kv_heads=2, d=128,
             page=16, prefix=1536, own=9, least=1, lens=1),
        # a full batch of readers of one context of 32768 tokens, 64 heads on 8 KV heads, with 20 to 2000 tokens of their own
        dict(name="shared_batch", op="shared", format="e4m3", dtype="bfloat16", groups=1, readers=64, loose=0, tokens=1, heads=64, kv_heads=8, d=128,
             page=64, prefix=32768, own=2000, least=20, lens=2),
        # the longest context of the workloads (131072 tokens) and 16 readers of it, int8 codes: the read of the codes counts
        dict(name="shared_long", op="shared", format="int8", dtype="float16", groups=1, readers=16, loose=0, tokens=1, heads=64, kv_heads=8, d=128,
             page=64, prefix=131072, own=300, least=1, lens=3),
        # three contexts in one batch, five drafted tokens each, three heads to a KV head, d = 80, pages of 24, readers without a prefix among them
        dict(name="shared_drafts_odd", op="shared", format="int8", dtype="bfloat16", groups=3, readers=9, loose=4, tokens=5, heads=12, kv_heads=4, d=80,
             page=24, prefix=9001, own=333, least=0, lens=4),
        # 64 readers of eight contexts of 32768 tokens: who reads what, before a step
        dict(name="groups_step", op="groups", groups=8, readers=8, loose=3, kv_heads=8, d=128, page=64, prefix=32768, own=2000, least=0, min_pages=8, lens=5),
        # 256 readers of one context of 131072 tokens in pages of 16, nine others among them: the longest rows of the table
        dict(name="groups_long", op="groups", groups=1, readers=256, loose=9, kv_heads=8, d=128, page=16, prefix=131072, own=500, least=1, min_pages=64, lens=6),
        # the step's new token of 64 readers
        dict(name="slots_step", op="slots", batch=64, new=1, ragged=False, spare=0, start=8000, kv_heads=8, d=128, page=64, lens=7),
        # 40 ragged prompts of up to 8192 tokens, some behind a context, in a buffer of fixed size
        dict(name="slots_prompts", op="slots", batch=40, new=8192, ragged=True, spare=777, start=3000, kv_heads=8, d=128, page=16, lens=8),
        # a question of 77 tokens, 64 heads, on the 32768 keys of a context as the codec leaves them
        dict(name="cross_question", op="cross", dtype="float16", batch=1, heads=64, kv_heads=8, d=128, longest=77, shortest=77, keys=32768, fewest=32768,
             layout="codec", lens=9),
        # a decoder's step: one token of each of 64 sequences on padded states of up to 1500, heads of 64 channels that share nothing
        dict(name="cross_step_padded", op="cross", dtype="bfloat16", batch=64, heads=16, kv_heads=16, d=64, longest=1, shortest=1, keys=1500, fewest=100,
             layout="padded", lens=10),
        # ragged queries on ragged states, packed, some of them without any
        dict(name="cross_packed_ragged", op="cross", dtype="bfloat16", batch=13, heads=32, kv_heads=8, d=128, longest=2000, shortest=1, keys=2500,
             fewest=0, layout="packed", lens=11),
        # five beams of each of eight sources, a few tokens each: beams share their source's states
        dict(name="cross_beams_shared", op="cross", dtype="float16", batch=40, heads=12, kv_heads=4, d=96, longest=4, shortest=1, keys=901, fewest=333,
             layout="shared", lens=12),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "shared", "cross", "cross", "cross", "groups", "slots"])
    seed = rng.randrange(1 << 30)
    fmt, dt = rng.choice(["e4m3", "int8"]), rng.choice(["float16", "bfloat16"])
    d, page = rng.choice([128, 128, 64, 96, 80, 40, 16, 8]), rng.choice([16, 32, 64, 128, 24, 7, 1])
    kv, group = rng.choice([1, 2, 4, 8, 8, 5]), rng.choice([1, 2, 3, 4, 8, 8, 16, 7])
    if op == "shared":
        groups, readers, loose, tokens = rng.choice([1, 1, 2, 5]), _log(rng, 1, 64), rng.choice([0, 0, 1, 4]), rng.choice([1, 1, 1, 2, 3, 5, 8])
        prefix, more = _log(rng, 1, 131072), _log(rng, 1, 2000)
        if page == 1:
            prefix, more = min(prefix, 4096), min(more, 500)
        while (groups * readers + loose) * tokens * kv * group * (prefix + more) > 130_000_000:
            readers, prefix, more, loose = max(1, readers * 3 // 4), max(1, prefix * 3 // 4), max(1, more * 3 // 4), loose // 2
        return dict(op=op, format=fmt, dtype=dt, groups=groups, readers=readers, loose=loose, tokens=tokens, heads=kv * group, kv_heads=kv, d=d, page=page,
                    prefix=prefix, own=more, least=rng.choice([0, 1, more]), lens=seed)
    if op == "groups":
        groups = rng.choice([1, 1, 2, 8])
        return dict(op=op, groups=groups, readers=_log(rng, 1, 200 // groups), loose=rng.choice([0, 1, 5]), kv_heads=kv, d=d, page=page,
                    prefix=_log(rng, 1, min(131072, 8000 * page)), own=_log(rng, 1, 2000), least=rng.choice([0, 1]), min_pages=_log(rng, 1, 64),
                    lens=seed)
    if op == "slots":
        batch = _log(rng, 1, 300)
        return dict(op=op, batch=batch, new=rng.choice([1, 4, _log(rng, 1, max(2, min(32768, 60000 // batch)))]), ragged=rng.random() < 0.5,
                    spare=rng.choice([0, 1, 500]), start=rng.choice([0, 5, 3000]), kv_heads=kv, d=d, page=page, lens=seed)
    batch = rng.choice([1, 1, 2, 5, 13, 40])
    longest, keys = rng.choice([1, _log(rng, 1, 4096)]), _log(rng, 1, 32768)
    while batch * kv * group * (longest + 8) * (keys + 64) > 1_200_000_000 or batch * kv * keys * d > 500_000_000:
        longest, keys = max(1, longest * 2 // 3), max(1, keys * 2 // 3)
    return dict(op=op, dtype=dt, batch=batch, heads=kv * group, kv_heads=kv, d=d, longest=longest, shortest=rng.choice([1, longest]), keys=keys,
                fewest=rng.choice([0, 1, keys]), layout=rng.choice(["packed", "padded", "shared"] if batch > 1 else ["packed", "codec"]), lens=seed)


def _spread(rng, count, shortest, longest):
    """Lengths spread over their logarithm, the longest first; where `shortest` is 0 some are 0."""
    got = [longest] + [_log(rng, max(1, shortest), longest) if longest else 0 for _ in range(count - 1)]
    return [0 if shortest == 0 and i % 5 == 3 else n for i, n in enumerate(got)]


def _readers(case):
    """-> pages of each group's prefix; of each sequence its group (-1: none) and its own tokens. Groups lie mixed in the batch."""
    rng = random.Random(case["lens"])
    pages = [max(1, n // case["page"]) for n in _spread(rng, case["groups"], max(1, case["prefix"] // 20), case["prefix"])]
    group = [g for g in range(case["groups"]) for _ in range(case["readers"])] + [-1] * case["loose"]
    rng.shuffle(group)
    return pages, group, _spread(rng, len(group), case["least"], case["own"])


def _new_rows(case):
    rng = random.Random(case["lens"])
    new = [case["new"] if i == 0 or not case["ragged"] else rng.choice([0, _log(rng, 1, case["new"]), _log(rng, 1, case["new"])])
           for i in range(case["batch"])]
    return new, [rng.randint(0, case["start"]) for _ in new]


def _cross_lengths(case):
    """-> queries and keys of each sequence, the keys' first rows, rows of the keys."""
    rng = random.Random(case["lens"])
    nq, B = _spread(rng, case["batch"], case["shortest"], case["longest"]), case["batch"]
    sources = -(-B // 5) if case["layout"] == "shared" else B
    nk = _spread(rng, sources, case["fewest"], case["keys"])
    width = [case["keys"]] * sources if case["layout"] == "padded" else nk
    first = [sum(width[:i]) for i in range(sources)]
    if case["layout"] == "shared":
        nk, first = [nk[b // 5] for b in range(B)], [first[b // 5] for b in range(B)]
    return nq, nk, first, sum(width)


# ---- what a program has in hand ---------------------------------------------------
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 23)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _keys(shape, g):
    """Normal values with a few channels that are ten times as large, as keys have."""
    x = torch.randn(shape, generator=g, device="cuda")
    x[..., 3::64] *= 10.0
    return x


def _page_pool(x, fmt):
    """x [n_blocks, H, page, d] -> codes of the same shape, scales [n_blocks, H]."""
    q = QMAX[fmt]
    s = x.abs().amax((2, 3)) / q
    x = x / s[:, :, None, None]
    return (x.clamp(-q, q).to(CODE[fmt]) if fmt == "e4m3" else x.round().clamp(-q, q).to(CODE[fmt])), s


def _branched_table(case, g, spare):
    """A table whose readers' rows begin with their group's pages; -> table, lengths (a list), pages in the pool."""
    bt = case["page"]
    pages, group, more = _readers(case)
    lens = [(pages[k] * bt if k >= 0 else 0) + n for k, n in zip(group, more)]
    need = sum(pages) + sum(-(-n // bt) for n in more)
    n_blocks = need + spare
    order = torch.randperm(n_blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(group), max(1, max(-(-n // bt) for n in lens))), -1, dtype=torch.int32, device="cuda")
    prefix, at = [], 0
    for n in pages:
        prefix.append(order[at:at + n])
        at += n
    for b, (k, n) in enumerate(zip(group, more)):
        n, first = -(-n // bt), pages[k] if k >= 0 else 0
        if k >= 0:
            table[b, :first] = prefix[k]
        table[b, first:first + n] = order[at:at + n]
        at += n
    return table, lens, n_blocks


def prepare(case, seed):
    s = dict(case=case)
    {"shared": _prepare_shared, "groups": _prepare_groups, "slots": _prepare_slots, "cross": _prepare_cross}[case["op"]](s, case, _generator(seed))
    return s


def _prepare_shared(s, case, g):
    T, Hq, H, d, bt = (case[k] for k in ("tokens", "heads", "kv_heads", "d", "page"))
    pages, group, _ = _readers(case)
    s["table"], lens, n_blocks = _branched_table(case, g, 5)
    s["lens"] = _ints(lens)
    s["pages"], s["members"] = pages, [[b for b, k in enumerate(group) if k == i] for i in range(len(pages))]
    cu = [0]
    for m in s["members"]:
        cu.append(cu[-1] + len(m))
    s["offsets"], s["cu_group"], s["member"], s["shared"] = cu, _ints(cu), _ints([b for m in s["members"] for b in m]), _ints(pages)
    s["q"] = torch.randn((len(group), T, Hq, d), generator=g, device="cuda").to(getattr(torch, case["dtype"]))
    s["scale"] = d ** -0.5
    s["k"], s["k_scale"] = _page_pool(_keys((n_blocks, H, bt, d), g), case["format"])
    s["v"], s["v_scale"] = _page_pool(torch.randn((n_blocks, H, bt, d), generator=g, device="cuda"), case["format"])
    # what an earlier owner left: in pages that no sequence has, and behind each sequence's last token
    stale = torch.ones((n_blocks, bt), dtype=torch.bool, device="cuda")
    at = torch.arange(s["table"].shape[1] * bt, device="cuda")
    for b, n in enumerate(lens):
        stale[s["table"][b].long().repeat_interleave(bt)[:n], at[:n] % bt] = False
    for pool in (s["k"], s["v"]):
        pool.view(torch.uint8).masked_fill_(stale[:, None, :, None], 0x7F)  # e4m3's NaN
    unused = stale.all(1)
    s["k_scale"][unused] = float("nan")
    s["v_scale"][unused] = float("nan")


def _prepare_groups(s, case, g):
    table, lens, s["n_blocks"] = _branched_table(case, g, 40)
    turn = torch.randperm(len(lens), generator=g, device="cuda")
    s["table"], s["lens"] = table[turn], _ints(lens)[turn]
    s["refs"] = torch.zeros(s["n_blocks"], dtype=torch.int32, device="cuda")
    used = s["table"][s["table"] >= 0].long()
    s["refs"].index_add_(0, used, torch.ones_like(used, dtype=torch.int32))


def _prepare_slots(s, case, g):
    new, start = _new_rows(case)
    bt = case["page"]
    lens = [a + n for a, n in zip(start, new)]
    counts = torch.tensor([-(-n // bt) for n in lens], device="cuda")
    s["n_blocks"] = int(counts.sum()) + 10
    order = torch.randperm(s["n_blocks"], generator=g, device="cuda").to(torch.int32)
    at = torch.arange(max(1, int(counts.max())), device="cuda")
    took = ((counts.cumsum(0) - counts)[:, None] + at).clamp(max=s["n_blocks"] - 1)
    s["table"] = torch.where(at < counts[:, None], order[took], -1).to(torch.int32)
    s["refs"] = torch.zeros(s["n_blocks"], dtype=torch.int32, device="cuda")
    s["refs"][order[:int(counts.sum())].long()] = 1
    s["lens"], s["new"] = _ints(lens), _ints(new)
    s["n_rows"] = sum(new) + case["spare"]


def _prepare_cross(s, case, g):
    Hq, H, d = (case[k] for k in ("heads", "kv_heads", "d"))
    dt = getattr(torch, case["dtype"])
    nq, nk, first, n_k = _cross_lengths(case)
    s["cu_q"] = _ints([sum(nq[:i]) for i in range(len(nq) + 1)])
    s["k_begin"], s["k_len"] = _ints(first), _ints(nk)
    s["scale"] = d ** -0.5
    s["q"] = torch.randn((sum(nq), Hq, d), generator=g, device="cuda").to(dt)
    if case["layout"] == "codec":  # one layer of the codec's [L, 2, H, S, d]
        kv = torch.stack([_keys((H, n_k, d), g), torch.randn((H, n_k, d), generator=g, device="cuda")]).to(dt)
        s["k"], s["v"] = kv[0].transpose(0, 1), kv[1].transpose(0, 1)
    else:  # one projection's rows, keys and values side by side
        kv = torch.cat([_keys((n_k, H, d), g), torch.randn((n_k, H, d), generator=g, device="cuda")], 1).to(dt)
        s["k"], s["v"] = kv[:, :H], kv[:, H:]
    if case["layout"] == "padded":  # behind a source's last state is what an earlier one left
        at = torch.arange(case["keys"], device="cuda")
        kv.view(case["batch"], case["keys"], 2 * H, d).masked_fill_((at >= s["k_len"][:, None])[..., None, None], float("nan"))


# ---- one pass -------------------------------------------------------------------
def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


def _part(scores, seen, v):
    """scores [..., n, S] with `seen` of their shape, v [..., S, d] -> the row's maximum, sum of exp(score - maximum) and sum of that times v."""
    scores = torch.where(seen, scores, -math.inf)
    top = scores.amax(-1, keepdim=True) if scores.shape[-1] else torch.full_like(scores[..., :0].sum(-1, keepdim=True), -math.inf)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    return top, p.sum(-1, keepdim=True), p @ v


def _finish(total, top, acc):
    return acc / torch.where(total == 0.0, 1.0, total), (torch.log(total) + top).squeeze(-1)


def _plain_shared(s):
    c, q = s["case"], s["q"]
    B, T, Hq, d = q.shape
    H, bt = c["kv_heads"], c["page"]
    G = Hq // H
    table = s["table"].clamp(min=0).long()

    def rows(codes, scale, entries, live):  # entries [..., n] -> [..., H, n * bt, d]
        x = codes[entries].float() * scale[entries][..., None, None]
        x = x.transpose(-4, -3).flatten(-3, -2)
        return torch.where(live[..., None, :, None], x, 0.0)

    qh = q.float().view(B, T, H, G, d).permute(0, 2, 1, 3, 4).reshape(B, H, T * G, d)
    last = (s["lens"][:, None] - T + torch.arange(T, device="cuda").repeat_interleave(G))  # [B, T * G]
    top = torch.full((B, H, T * G, 1), -math.inf, device="cuda")
    total, acc = torch.zeros((B, H, T * G, 1), device="cuda"), torch.zeros((B, H, T * G, d), device="cuda")
    begin = torch.zeros(B, dtype=torch.long, device="cuda")
    for i, n in enumerate(s["pages"]):  # a prefix once, for the rows of all of its readers
        who = s["member"][s["offsets"][i]:s["offsets"][i + 1]].long()
        entries, at = table[who[0], :n], torch.arange(n * bt, device="cuda")
        live = torch.ones(n * bt, dtype=torch.bool, device="cuda")
        x = qh[who].transpose(0, 1).reshape(H, -1, d)
        scores = (x @ rows(s["k"], s["k_scale"], entries, live).transpose(1, 2)) * s["scale"]
        seen = (at <= last[who].reshape(-1, 1))[None]
        m, t, a = (y.view(H, who.numel(), T * G, -1).transpose(0, 1) for y in _part(scores, seen, rows(s["v"], s["v_scale"], entries, live)))
        top[who], total[who], acc[who] = m, t, a
        begin[who] = n
    # what each sequence has behind its prefix
    width = -(-c["own"] // bt)
    entries = table.gather(1, (begin[:, None] + torch.arange(width, device="cuda")).clamp(max=table.shape[1] - 1))
    at = begin[:, None] * bt + torch.arange(width * bt, device="cuda")
    live = at < s["lens"][:, None]
    scores = (qh @ rows(s["k"], s["k_scale"], entries, live).transpose(2, 3)) * s["scale"]
    m, t, a = _part(scores, (at[:, None] <= last[..., None])[:, None], rows(s["v"], s["v_scale"], entries, live))
    both = torch.maximum(top, m)
    safe = torch.where(both == -math.inf, 0.0, both)
    f, h = torch.exp(top - safe), torch.exp(m - safe)
    out, lse = _finish(f * total + h * t, both, f * acc + h * a)
    out = out.view(B, H, T, G, d).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, d)
    return dict(out=out.to(q.dtype), lse=lse.view(B, H, T, G).permute(0, 2, 1, 3).reshape(B, T, Hq))


def _plain_groups(s):
    table, bt, m = s["table"], s["case"]["page"], s["case"]["min_pages"]
    n, width = table.shape
    i = torch.arange(n, device="cuda")
    whole = s["lens"] // bt
    able = whole >= m
    key = torch.where(able, table[:, min(m, width) - 1], -1 - i.to(torch.int32))
    same = key[:, None] == key
    lead = torch.where(same, i, n).amin(1)
    grouped = able & (same.sum(1) > 1)
    place, who = torch.sort(torch.where(grouped, lead, n), stable=True)
    head = grouped & (lead == i)
    number = head.cumsum(0) - 1
    at = torch.arange(width, device="cuda")
    alike = (table == table[lead]) & (at < torch.minimum(whole, whole[lead])[:, None])
    common = alike.to(torch.int32).cumprod(1).sum(1)
    g = torch.where(grouped, number[lead], n // 2)
    sizes = torch.zeros(n // 2 + 1, dtype=torch.long, device="cuda").index_add_(0, g, grouped.long())
    shared = torch.full((n // 2 + 1,), width, device="cuda").index_reduce_(0, g, common, "amin")
    shared = torch.where(sizes > 0, shared, 0)[:n // 2]
    cu = torch.cat([torch.zeros_like(sizes[:1]), sizes[:n // 2].cumsum(0)])
    return dict(cu=cu.to(torch.int32), member=torch.where(place < n, who, -1).to(torch.int32), shared=shared.to(torch.int32))


def _plain_slots(s):
    new, table, bt = s["new"].long(), s["table"], s["case"]["page"]
    cu = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    start = s["lens"].long() - new
    row = torch.arange(s["n_rows"], device="cuda")
    seq = torch.searchsorted(cu[1:], row, right=True)
    real = seq < new.numel()
    b = seq.clamp(max=new.numel() - 1)
    pos = start[b] + row - cu[b]
    page = table[b, (pos // bt).clamp(0, table.shape[1] - 1)].long()
    return dict(cu=cu.to(torch.int32), start=start.to(torch.int32), seq=torch.where(real, seq, -1).to(torch.int32),
                pos=torch.where(real, pos, -1).to(torch.int32), slot=torch.where(real, page * bt + pos % bt, -1))


def _plain_cross(s):
    c, q = s["case"], s["q"]
    H, G, d, mq, mk = c["kv_heads"], c["heads"] // c["kv_heads"], c["d"], c["longest"], c["keys"]
    nq = s["cu_q"].diff()
    iq, ik = torch.arange(mq, device="cuda"), torch.arange(mk, device="cuda")
    rq = (s["cu_q"][:-1, None] + iq).clamp(max=q.shape[0] - 1)
    rk = (s["k_begin"][:, None] + ik).clamp(max=s["k"].shape[0] - 1)
    live = ik < s["k_len"][:, None]
    B = nq.numel()

    def rows(x):
        return torch.where(live[..., None, None], x[rk].float(), 0.0).permute(0, 2, 1, 3)

    qh = q[rq].float().view(B, mq, H, G, d).permute(0, 2, 3, 1, 4).reshape(B, H, G * mq, d)
    scores = (qh @ rows(s["k"]).transpose(2, 3)) * s["scale"]
    top, total, acc = _part(scores, live[:, None, None], rows(s["v"]))
    out, lse = _finish(total, top, acc)
    out = out.view(B, H * G, mq, d).transpose(1, 2)
    lse = lse.view(B, H * G, mq).transpose(1, 2)
    real = iq < nq[:, None]
    return dict(out=out[real].to(q.dtype), lse=lse[real])


_PLAIN = dict(shared=_plain_shared, groups=_plain_groups, slots=_plain_slots, cross=_plain_cross)


# ---- the same pass through the library --------------------------------------------
def _kept(s, make):
    """The descriptions, workspace and output buffers that a server keeps from call to call."""
    if "kept" not in s:
        from kv_cache_compression_02_gb300 import cachegen as cg
        s["kept"] = make(cg, s, s["case"])
    return s["kept"]


def _dtype(cg, c):
    return {"float16": cg.CG_F16, "bfloat16": cg.CG_BF16}[c["dtype"]]


def _own_shared(s):
    def make(cg, s, c):
        fmt = {"e4m3": cg.CG_CACHE_E4M3, "int8": cg.CG_CACHE_INT8}[c["format"]]
        cache = cg.Cache(1, c["kv_heads"], c["d"], c["page"], s["k"].shape[0], fmt)
        att = cg.Attend(s["q"].shape[0], c["tokens"], c["heads"], _dtype(cg, c), s["table"].shape[1], s["scale"])
        groups = cg.Groups(s["cu_group"], s["member"], s["shared"])
        ws = cg.empty_u8(cg.cg_shared_workspace_bytes(cache, att, groups))
        return cg, cache, att, groups, torch.empty_like(s["q"]), torch.empty(s["q"].shape[:3], device="cuda"), ws

    cg, cache, att, groups, out, lse, ws = _kept(s, make)
    cg.check(cg.cg_shared_attend(cache, att, groups, s["q"], s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"], s["lens"], out, lse, ws), "shared")
    return dict(out=out, lse=lse)


def _make_pages(cg, s, c):
    cache = cg.Cache(1, c["kv_heads"], c["d"], c["page"], s["n_blocks"], cg.CG_CACHE_E4M3)
    pages = cg.Pages(s["refs"], s["table"], s["lens"])
    n = s["table"].shape[0]
    if c["op"] == "groups":
        got = [_ints([0] * k) for k in (n // 2 + 1, n, n // 2)]
    else:
        got = [_ints([0] * k) for k in (n + 1, n, s["n_rows"], s["n_rows"])] + [torch.zeros(s["n_rows"], dtype=torch.int64, device="cuda")]
    return cg, cache, pages, got, cg.empty_u8(cg.cg_pages_workspace_bytes(cache, pages, n))


def _own_groups(s):
    cg, cache, pages, (cu, member, shared), ws = _kept(s, _make_pages)
    cg.check(cg.cg_pages_groups(cache, pages, s["case"]["min_pages"], cu, member, shared, ws), "groups")
    return dict(cu=cu, member=member, shared=shared)


def _own_slots(s):
    cg, cache, pages, (cu, start, seq, pos, slot), ws = _kept(s, _make_pages)
    cg.check(cg.cg_pages_slots(cache, pages, s["n_rows"], s["new"], cu, start, seq, pos, slot, ws), "slots")
    return dict(cu=cu, start=start, seq=seq, pos=pos, slot=slot)


def _own_cross(s):
    def make(cg, s, c):
        q, k, v = s["q"], s["k"], s["v"]
        p = cg.Prompt(c["batch"], c["heads"], c["kv_heads"], c["d"], _dtype(cg, c), q.shape[0], k.shape[0], c["longest"], c["keys"], s["scale"],
                      q.stride()[:2], k.stride()[:2], v.stride()[:2])
        return cg, p, torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(q.shape[:2], device="cuda"), cg.empty_u8(cg.cg_prompt_workspace_bytes(p))

    cg, p, out, lse, ws = _kept(s, make)
    cg.check(cg.cg_cross_attend(p, s["q"], s["k"], s["v"], s["cu_q"], s["k_begin"], s["k_len"], out, lse, ws), "cross")
    return dict(out=out, lse=lse)


_OWN = dict(shared=_own_shared, groups=_own_groups, slots=_own_slots, cross=_own_cross)


# ---- what a pass cannot do without ---------------------------------------------------
def work(case):
    op = case["op"]
    if op == "cross":
        nq, nk, _, _ = _cross_lengths(case)
        Hq, H, d = case["heads"], case["kv_heads"], case["d"]
        distinct = nk[::5] if case["layout"] == "shared" else nk
        return dict(bytes=4 * sum(nq) * Hq * (d + 1) + 4 * sum(distinct) * H * d + 12 * len(nq), flops=4.0 * sum(a * b for a, b in zip(nq, nk)) * Hq * d)
    bt = case["page"]
    if op == "slots":
        new, start = _new_rows(case)
        pages = sum(-(-(a + n) // bt) - a // bt for a, n in zip(start, new) if n)
        return dict(bytes=16 * len(new) + 4 * pages + 16 * (sum(new) + case["spare"]), flops=0)
    pages, group, more = _readers(case)
    if op == "groups":
        # the shared part of each reader's row has to be compared
        compared = sum(pages[k] for k in group if k >= 0)
        return dict(bytes=4 * compared + 4 * len(group) + 4 * (2 * len(group) + 1), flops=0)
    T, Hq, H, d = (case[k] for k in ("tokens", "heads", "kv_heads", "d"))
    tokens = sum(n * bt for n in pages) + sum(more)
    held = sum(pages) + sum(-(-n // bt) for n in more)
    seen = sum(max(0, (pages[k] * bt if k >= 0 else 0) + n - T + 1 + t) for k, n in zip(group, more) for t in range(T))
    return dict(bytes=2 * tokens * H * d + held * (4 + 8 * H) + len(group) * (12 + T * Hq * (4 * d + 4)), flops=4.0 * seen * Hq * d)


# ---- the definitions in 64 bits ------------------------------------------------------
def exact(case, seed):
    if case["op"] not in ("shared", "cross"):
        return None  # whole numbers
    s = prepare(case, seed)
    return {"shared": _exact_shared, "cross": _exact_cross}[case["op"]](s, case)


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


def _exact_shared(s, c):
    # each sequence by itself, over its own row of the table from the first entry to the last
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


def _exact_cross(s, c):
    n_q, Hq, d = s["q"].shape
    G = Hq // c["kv_heads"]
    out = torch.zeros((n_q, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((n_q, Hq), -math.inf, dtype=torch.float64, device="cuda")
    cq, first, count = s["cu_q"].tolist(), s["k_begin"].tolist(), s["k_len"].tolist()
    for b, (k0, n) in enumerate(zip(first, count)):
        q0, q1 = cq[b], cq[b + 1]
        last = torch.full((q1 - q0,), n, device="cuda")
        for h in range(Hq):
            out[q0:q1, h], lse[q0:q1, h] = _exact_rows(s["q"][q0:q1, h].double(), s["k"][k0:k0 + n, h // G].double(), s["v"][k0:k0 + n, h // G].double(),
                                                       last, s["scale"])
    return dict(out=out, lse=lse)
