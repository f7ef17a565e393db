"""The serving example's readers: who shares the context, and what the context alone says to the question's rows."""
import pytest
import torch

from kv_cache_compression_02_gb300 import cachegen as cg, serve_example, synth
from tests import gpu_util as gu
from tests import serve_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("question", [21, 6])
def test_readers_of_the_example(question):
    gu.ready()
    synth.build()
    S, bt, H, G = 700, 16, 2, 4
    r = serve_example.run(S=S, question=question, steps=3, block_tokens=bt, fmt=cg.CG_CACHE_INT8, verbose=False)
    cu, member, shared = (t.tolist() for t in r["groups"].tensors)
    # the context's own sequence and its three readers
    assert (cu, member, shared) == ([0, 4, 4], [0, 1, 2, 3], [(S + question) // bt, 0])
    ctx, scale = r["context"][-1].cpu(), 128 ** -0.5
    for h in range(G * H):
        o, l, A, X = ref.attend_rows(r["q"][:, h].cpu(), ctx[0, h // G, :S], ctx[1, h // G, :S], torch.full((question,), S - 1), scale)
        to, tl = ref.tolerances(o, l, A, X, 128, S, torch.float16, 11)
        ref.assert_close(r["look"][:, h], o, to, f"context alone, head {h}")
        ref.assert_close(r["look_lse"][:, h], l, tl, f"context alone, lse of head {h}")
