"""The serving example's two ways of attention: each by itself, and the shared context once for all."""
import pytest
import torch

from kv_cache_compression_02_gb300 import cachegen as cg, serve_example, synth
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    gu.ready()
    synth.build()


@pytest.mark.parametrize("fmt", [cg.CG_CACHE_E4M3, cg.CG_CACHE_INT8])
def test_both_ways_of_the_example_agree(fmt):
    one, all_ = (serve_example.run(S=700, question=21, steps=4, fmt=fmt, share=share, verbose=False) for share in (False, True))
    assert one["share"] is False and all_["share"] is True
    for name in ("table", "lens", "new_q", "pools"):
        assert torch.equal(one[name], all_[name])
    # both outputs are rounded once to f16, and weights of the second have 11 bits: 2 2^-11 + 2^-11 of the largest value, half as much for sums in fp32
    top = (one["scales"][-1, 1].max() * (448.0 if fmt == cg.CG_CACHE_E4M3 else 127.0)).item()
    assert (one["outs"].double() - all_["outs"].double()).abs().max() <= 4.5 * 2.0 ** -11 * top
    assert (one["lse"] - all_["lse"]).abs().max() <= 1e-4
    assert torch.isfinite(all_["outs"]).all()


@pytest.mark.parametrize("H,S,pays", [(2, 1500, False), (8, 21000, True)])
def test_the_example_shares_where_it_pays(H, S, pays):
    """A context and three readers: three more would read it where it is not shared, 9,000 and 503,808 positions of KV heads."""
    r = serve_example.run(L=1, H=H, S=S, question=5, steps=2, verbose=False)
    cu, _, shared = (t.tolist() for t in r["groups"].tensors)
    saved = (cu[1] - cu[0] - 1) * shared[0] * 16 * H
    assert (saved >= serve_example.SHARING_PAYS) is pays and r["share"] is pays
    assert torch.isfinite(r["outs"]).all()
