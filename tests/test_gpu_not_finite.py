"""Infinities and NaN that a row sees."""
import math

import pytest
import torch

from kv_cache_compression_02_gb300 import cachegen as cg
from tests import gpu_util as gu
from tests import test_gpu_cross as cross
from tests import test_gpu_prompt as prompt
from tests import test_gpu_shared as shared

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    gu.ready()


def few_that_count(dt, d):
    """2 d keys: one in two has a score from 9 nats under the others' on, and an infinite value in one channel -> keys, values, the outputs' signs."""
    below = torch.linspace(9.0, 20.5 if dt == F16 else 75.0, d)
    below = below[torch.randperm(d, generator=torch.Generator().manual_seed(d))].to(dt)  # (the scores are what the type holds)
    k, v = torch.zeros(2 * d, 1, d), torch.randn(2 * d, 1, d, generator=torch.Generator().manual_seed(1))
    k[1::2, 0, 0] = -below.float()
    c = torch.arange(d)
    sign = torch.where(c % 3 == 0, -math.inf, math.inf)
    v[2 * c + 1, 0, c] = sign
    return k.to(dt), v.to(dt), sign


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 5, 8, 40])
@pytest.mark.parametrize("dt", [F16, BF16])
def test_infinite_values_under_small_weights(dt, n, d):
    """A value of plus or minus infinity counts as long as its weight is at least 2^-30 (f16, 20.79 nats) or 2^-110 (bf16, 76.2 nats) of the row's
    largest: where a weight of f16 is normal, subnormal, or only just above nothing."""
    k, v, sign = few_that_count(dt, d)
    q = torch.zeros(n, 2, d, dtype=dt)
    q[..., 0] = 1.0
    out, z, st = cross.run(q.cuda(), k.cuda(), v.cuda(), [0, n], [0], [2 * d], 1.0)
    assert st == cg.CG_OK and torch.isfinite(z).all()
    assert torch.equal(out.float().cpu(), sign.expand(n, 2, d))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("dt", [F16, BF16])
def test_infinite_values_under_small_weights_of_a_prompt(dt, n, d):
    """The same with the questions' own keys behind them, which each row sees as far as itself."""
    k, v, sign = few_that_count(dt, d)
    k, v = torch.cat([k, torch.zeros(n, 1, d, dtype=dt)]), torch.cat([v, torch.ones(n, 1, d, dtype=dt)])
    q = torch.zeros(n, 2, d, dtype=dt)
    q[..., 0] = 1.0
    out, z, st = prompt.run(q.cuda(), k.cuda(), v.cuda(), [0, n], [0, 2 * d + n], 1.0)
    assert st == cg.CG_OK and torch.isfinite(z).all()
    assert torch.equal(out.float().cpu(), sign.expand(n, 2, d))


@pytest.mark.parametrize("bt", [16, 64, 8, 7])
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_a_scale_that_is_nan_reaches_the_readers_of_its_page(fmt, which, bt):
    """K's scale (0) makes outputs and lse of its head NaN, V's (1) the outputs, for those who read the page and for no others, whatever the page size."""
    s = shared.Setup(fmt, BF16, 1, 16, 2, 128, bt, [(300 // bt, [5, 20, 3]), (160 // bt, [1, 2])], [30], seed=11 + bt)
    s.scales[which][s.table[s.members[0][0], 1].long(), 1] = math.nan
    out, z, st = s.run(fill=0xFF)
    assert st == cg.CG_OK
    hit = torch.zeros(len(s.lens), dtype=torch.bool)
    hit[s.members[0]] = True
    assert torch.isnan(out[hit.cuda(), :, 8:]).all() and torch.isfinite(out[hit.cuda(), :, :8]).all() and torch.isfinite(out[~hit.cuda()]).all()
    assert torch.equal(torch.isnan(z).cpu(), (hit[:, None, None] & (torch.arange(16) >= 8)) if which == 0 else torch.zeros(z.shape, dtype=torch.bool))
    s.check(out, z)
