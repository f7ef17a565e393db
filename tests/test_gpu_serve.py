"""The serving example end to end: what it attends over is the decoded context, within the error of 8-bit codes."""
import pytest
import torch

from kv_cache_compression_02_gb300 import cachegen as cg, serve_example, synth
from tests import gpu_util as gu
from tests import serve_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [cg.CG_CACHE_E4M3, cg.CG_CACHE_INT8])
def test_serve_example(fmt):
    gu.ready()
    synth.build()
    S, question, steps, bt, H, G = 700, 21, 4, 16, 2, 4
    r = serve_example.run(S=S, question=question, steps=steps, block_tokens=bt, fmt=fmt, verbose=False)
    n = S + question
    # the question's rows against the definition, over fp16 keys
    ctx, scale = r["context"][-1].cpu(), 128 ** -0.5
    for h in range(G * H):
        o, l, A, X = ref.attend_rows(r["q"][:, h].cpu(), ctx[0, h // G], ctx[1, h // G], torch.arange(question) + S, scale)
        to, _ = ref.tolerances(o, l, A, X, 128, n, torch.float16, 11)
        ref.assert_close(r["answer"][:, h], o, to, f"question, head {h}")
    # the remaining reader's last step, over the codes that its pages hold
    code = ref.CODE["e4m3" if fmt == cg.CG_CACHE_E4M3 else "int8"]
    pools, scales, table = r["pools"][-1].cpu().view(code).to(torch.float64), r["scales"][-1].cpu(), r["table"].cpu()
    assert r["lens"].tolist() == [n, 0, 0, n + steps]
    pos = torch.arange(n + steps)
    for h in range(G * H):
        page = table[3][pos // bt].long()
        k, v = (pools[i][page, h // G, pos % bt] * scales[i][page, h // G].double()[:, None] for i in range(2))
        o, l, A, X = ref.attend_rows(r["new_q"][-1, 3, :, h].cpu(), k, v, [n + steps - 1], scale)
        to, tl = ref.tolerances(o, l, A, X, 128, n + steps, torch.float16, 11)
        ref.assert_close(r["outs"][-1, 3, :, h], o, to, f"reader, head {h}")
        ref.assert_close(r["lse"][-1, 3, :, h], l, tl, f"reader's lse, head {h}")
        # a code is off by at most half its step: 2^-4 of itself (e4m3, normal ones; half a step of 2^-9 below) or half of the scale (int8)
        want = torch.cat([ctx[1, h // G].double(), r["new_v"][:, 2, h // G].cpu().double()])
        step = torch.maximum(want.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10)) if fmt == cg.CG_CACHE_E4M3 else torch.tensor(0.5)
        s = scales[1][page, h // G].double()[:, None]
        grown = (pos >= n - n % bt)[:, None]  # pages that were written more than once have been rounded as often
        assert bool(((v - want).abs() <= torch.where(grown, 1 + steps, 1) * (step * (s if fmt == cg.CG_CACHE_INT8 else 1.0)).clamp(min=s * 2.0 ** -10) * 1.001).all())
    # the same pages after compaction, elsewhere (how a row's positions are shared out goes by the whole batch, so the
    # bits may be others); the readers that left see nothing
    for b, m in ((0, n), (3, n + steps)):
        for h in range(G * H):
            page = table[b][pos[:m] // bt].long()
            k, v = (pools[i][page, h // G, pos[:m] % bt] * scales[i][page, h // G].double()[:, None] for i in range(2))
            o, l, A, X = ref.attend_rows(r["new_q"][-1, b, :, h].cpu(), k, v, [m - 1], scale)
            to, _ = ref.tolerances(o, l, A, X, 128, m, torch.float16, 11)
            ref.assert_close(r["again"][b, :, h], o, to, f"after compaction, sequence {b}, head {h}")
    assert not r["again"][1:3].any()
    shared = n // bt
    assert r["used"] == shared + 1 + 3 * (-(-(n + steps) // bt) - shared) and r["n_live"] == r["used"] - 2 * (-(-(n + steps) // bt) - shared)
    assert int((r["refs"] > 0).sum()) == r["n_live"] and bool((r["refs"][r["n_live"]:] == 0).all())
