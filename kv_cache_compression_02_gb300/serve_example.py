"""Serving a decoded context, end to end: ``python -m kv_cache_compression_02_gb300.serve_example``.

A context's KV (synthetic, from :mod:`.synth`) is fitted, encoded and decoded by the codec into a buffer with room for
a question.  Each layer of the decoded context goes into 8-bit pages (cg_pages_extend, cg_cache_write); a question is
run against the decoded fp16 keys (cg_prompt_attend) and its own keys join the pages; three readers branch off it
(cg_pages_fork, cg_pages_groups) and generate a few tokens each (cg_pages_extend, cg_pages_slots, cg_cache_write and, where
the context that they share is long enough, cg_shared_attend, which reads it once for all of them, else cg_cache_attend);
another look at the context alone is taken by rows that are no part of it (cg_cross_attend); two readers are dropped
(cg_pages_free), the cache is compacted (cg_pages_compact) and the last one attends by itself (cg_cache_attend).  Queries,
keys and values of the new tokens are random rows: there is no model here, only what a server does around one.
"""
from __future__ import annotations

import math

import numpy as np


SHARING_PAYS = 500_000  # positions of KV heads that are not read again, from which cg_shared_attend is faster than cg_cache_attend


def run(L=2, H=2, G=4, S=1500, question=37, steps=5, block_tokens=16, fmt=None, seed=0, verbose=True, share=None):
    """-> a dict with what the calls produced, for a caller that wants to check it.  share: whether the readers attend by
    cg_shared_attend (None: where it pays)."""
    import torch

    from . import cachegen as cg, synth

    fmt = cg.CG_CACHE_E4M3 if fmt is None else fmt
    d, Hq, readers = 128, G * H, 3
    dev = dict(device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(seed)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, **dev)  # noqa: E731
    rows = lambda *shape: torch.randn(shape, generator=gen, **dev).half()  # noqa: E731

    def done(rc, what, ws):
        cg.check(rc, what)
        torch.cuda.synchronize()
        cg.check(cg.cg_read_status(ws), what)

    # the codec: the context as its receiver gets it, with room for the question behind each head's tokens
    cfg = cg.Config(L, H, d, S, 512)
    kv = torch.from_numpy(synth.generate(synth.GenSpec(L=L, H=H, d=d, S=S, seed=seed)).view(np.int16).reshape(-1)).cuda()
    tables = cg.empty_u8(cg.cg_tables_bytes(cfg))
    ws = cg.empty_u8(max(cg.cg_workspace_bytes(cfg, op) for op in (0, 1, 2)))
    done(cg.cg_fit_tables(cfg, kv, tables, ws), "fit", ws)
    out, nbytes = cg.empty_u8(cg.cg_encode_bound(cfg)), torch.zeros(1, dtype=torch.int64, **dev)
    done(cg.cg_encode(cfg, tables, kv, [0] * cfg.n_chunks, out, nbytes, ws), "encode", ws)
    decoded = torch.empty(L, 2, H, S, d, dtype=torch.float16, **dev)
    done(cg.cg_decode(cfg, tables, out, int(nbytes.item()), 0, -1, decoded, ws), "decode", ws)
    context = torch.zeros(L, 2, H, S + question, d, dtype=torch.float16, **dev)
    context[:, :, :, :S] = decoded
    context[:, :, :, S:] = rows(L, 2, H, question, d)  # what the layers' projections give for the question

    # the cache: one sequence for the context and question, one for each reader
    n_tok = S + question
    per = -(-(n_tok + steps) // block_tokens)
    n_blocks, n_seqs = 3 * per, 1 + readers
    pools = torch.zeros(L, 2, n_blocks, H, block_tokens, d, dtype=torch.uint8, **dev)
    scales = torch.zeros(L, 2, n_blocks, H, **dev)
    addr = [torch.tensor([t[l, i].data_ptr() for l in range(L) for i in range(2)], dtype=torch.int64, **dev) for t in (pools, scales)]
    cache = cg.Cache(L, H, d, block_tokens, n_blocks, fmt)
    pages = cg.Pages(torch.zeros(n_blocks, dtype=torch.int32, **dev), torch.full((n_seqs, per), -1, dtype=torch.int32, **dev), i32([0] * n_seqs))
    refs, table, lens = pages.tensors
    ws = cg.empty_u8(cg.cg_pages_workspace_bytes(cache, pages, n_seqs))
    done(cg.cg_pages_extend(cache, pages, i32([0]), i32([n_tok]), ws), "extend", ws)
    wsw = cg.empty_u8(256)
    shape = cg.Rows(1, n_tok, n_tok, cg.CG_F16, per, d, n_tok * d)  # a layer's [H][tokens][d], tokens first
    for l in range(L):
        done(cg.cg_cache_write(cache, shape, context[l, 0], context[l, 1], i32([0, n_tok]), i32([0]), table, pools[l, 0], pools[l, 1],
                               scales[l, 0], scales[l, 1], wsw), "write", wsw)

    # the question, against the decoded keys themselves
    q = rows(question, Hq, d)
    answer = torch.empty_like(q)
    prompt = cg.Prompt(1, Hq, H, d, cg.CG_F16, question, n_tok, question, n_tok, 1.0 / math.sqrt(d), (Hq * d, d), (d, n_tok * d), (d, n_tok * d))
    wsp = cg.empty_u8(cg.cg_prompt_workspace_bytes(prompt))
    last = context[L - 1]
    done(cg.cg_prompt_attend(prompt, q, last[0], last[1], i32([0, question]), i32([0, n_tok]), answer, None, wsp), "prompt", wsp)

    # what the context alone says to the question, without the question's own keys: one pass over it for two sequences of rows
    look, look_lse = torch.empty_like(q), torch.empty(question, Hq, **dev)
    half = question // 2
    cross = cg.Prompt(2, Hq, H, d, cg.CG_F16, question, n_tok, question - half, S, 1.0 / math.sqrt(d), (Hq * d, d), (d, n_tok * d), (d, n_tok * d))
    wsp = cg.empty_u8(cg.cg_prompt_workspace_bytes(cross))
    done(cg.cg_cross_attend(cross, q, last[0], last[1], i32([0, half, question]), i32([0, 0]), i32([S, S]), look, look_lse, wsp), "cross", wsp)

    # three readers branch off and generate: one batched call of each kind a step (the last layer here)
    ids = i32([1, 2, 3])
    done(cg.cg_pages_fork(cache, pages, addr[0], addr[1], i32([0] * readers), ids, ws), "fork", ws)
    att = cg.Attend(n_seqs, 1, Hq, cg.CG_F16, per, 1.0 / math.sqrt(d))
    one = cg.Rows(n_seqs, readers, 1, cg.CG_F16, per, H * d, d)
    new_q, new_k, new_v = rows(steps, n_seqs, 1, Hq, d), rows(steps, readers, H, d), rows(steps, readers, H, d)
    outs, lse = torch.empty(steps, n_seqs, 1, Hq, d, dtype=torch.float16, **dev), torch.empty(steps, n_seqs, 1, Hq, **dev)
    new, cu, start, wsr = i32([0, 1, 1, 1]), i32([0] * (n_seqs + 1)), i32([0] * n_seqs), cg.empty_u8(256)
    groups = cg.Groups(i32([0] * (n_seqs // 2 + 1)), i32([0] * n_seqs), i32([0] * (n_seqs // 2)))
    wsg = cg.empty_u8(cg.cg_pages_workspace_bytes(cache, pages, n_seqs))
    # who shares what stays as it is while they generate: it is found once and looked at once, to see whether sharing pays
    done(cg.cg_pages_groups(cache, pages, max(1, S // block_tokens // 2), *groups.tensors, wsg), "groups", wsg)
    cu_group, _, shared = (t.tolist() for t in groups.tensors)
    saved = sum((b - a - 1) * n for a, b, n in zip(cu_group, cu_group[1:], shared)) * block_tokens * H
    share = saved >= SHARING_PAYS if share is None else share
    wsa = cg.empty_u8(cg.cg_shared_workspace_bytes(cache, att, groups) if share else cg.cg_cache_workspace_bytes(cache, att))
    k_pool, v_pool, k_scale, v_scale = pools[L - 1, 0], pools[L - 1, 1], scales[L - 1, 0], scales[L - 1, 1]
    for s in range(steps):
        done(cg.cg_pages_extend(cache, pages, ids, lens[1:] + 1, ws), "extend", ws)
        done(cg.cg_pages_slots(cache, pages, readers, new, cu, start, None, None, None, wsr), "slots", wsr)
        done(cg.cg_cache_write(cache, one, new_k[s], new_v[s], cu, start, table, k_pool, v_pool, k_scale, v_scale, wsw), "write", wsw)
        what = (new_q[s], k_pool, v_pool, k_scale, v_scale, table, lens, outs[s], lse[s], wsa)
        done(cg.cg_shared_attend(cache, att, groups, *what) if share else cg.cg_cache_attend(cache, att, *what), "attend", wsa)

    # two readers leave; the pages that are left move to the front
    used = int((refs > 0).sum())
    done(cg.cg_pages_free(cache, pages, ids[:2], ws), "free", ws)
    n_live = i32([0])
    done(cg.cg_pages_compact(cache, pages, addr[0], addr[1], refs, table, n_live, ws), "compact", ws)
    again, z, wsa = torch.empty_like(outs[0]), torch.empty_like(lse[0]), cg.empty_u8(cg.cg_cache_workspace_bytes(cache, att))
    done(cg.cg_cache_attend(cache, att, new_q[-1], k_pool, v_pool, k_scale, v_scale, table, lens, again, z, wsa), "attend", wsa)
    if verbose:
        fp16 = context.numel() * 2
        print(f"context of {S} tokens: {int(nbytes.item())} bytes on the wire; {n_tok} tokens in {int(n_live.item())} of {n_blocks} pages after "
              f"compaction ({used} with three readers), {pools.element_size() * 8}-bit codes of {fp16} bytes of fp16")
    return dict(context=context, q=q, answer=answer, look=look, look_lse=look_lse, groups=groups, share=share, new_q=new_q, new_k=new_k, new_v=new_v, outs=outs,
                lse=lse, again=again, used=used, n_live=int(n_live.item()), refs=refs, table=table, lens=lens, pools=pools, scales=scales)


if __name__ == "__main__":
    from . import build
    build.build()
    run()
