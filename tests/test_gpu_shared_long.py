"""cg_shared_attend at the lengths that it is for, and in pools beyond 2^31 bytes, against the 64-bit definition (on the GPU)."""
import math

import pytest
import torch

from kv_cache_compression_02_gb300 import cachegen as cg
from tests import gpu_util as gu
from tests import serve_ref as ref

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
FMT = {"e4m3": cg.CG_CACHE_E4M3, "int8": cg.CG_CACHE_INT8}
DT = {F16: cg.CG_F16, BF16: cg.CG_BF16}


@pytest.fixture(scope="module", autouse=True)
def built():
    gu.ready()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


CASES = {
    # name: (format, dtype, Hq, H, d, page, pages of the pool, tokens of the prefix, own tokens of each reader)
    "32768_40_readers": ("e4m3", BF16, 64, 8, 128, 64, 700, 32768, [1 + (17 * i) % 190 for i in range(40)]),
    "131072_pool_of_2_2_GB": ("int8", F16, 64, 8, 128, 64, 34000, 131072, [300, 1, 64]),
    "131072_pages_of_24": ("int8", BF16, 16, 2, 80, 24, 5600, 131072, [5, 77]),
    "65536_pages_of_7": ("e4m3", F16, 8, 1, 64, 7, 9500, 65533, [1, 30, 8]),
}


@pytest.mark.parametrize("name", list(CASES))
def test_long_prefix(name):
    fmt, dt, Hq, H, d, bt, n_blocks, prefix, own = CASES[name]
    g = torch.Generator(device="cuda").manual_seed(len(name))
    G, B, shared = Hq // H, len(own), prefix // bt
    prefix = shared * bt
    # codes and scales as they come: e4m3 without its NaN (the low seven bits all set)
    pools = [torch.randint(-127, 128, (n_blocks, H, bt, d), dtype=torch.int8, generator=g, device="cuda") for _ in range(2)]
    if fmt == "e4m3":
        for p in pools:
            p[(p & 127) == 127] = 8
    scales = [(0.5 + torch.rand(n_blocks, H, generator=g, device="cuda")) * (0.02 if fmt == "int8" else 0.01) for _ in range(2)]
    order = torch.randperm(n_blocks, generator=g, device="cuda").flip(0).to(torch.int32)
    order = torch.cat([torch.tensor([n_blocks - 1, 0], dtype=torch.int32, device="cuda"), order[(order != 0) & (order != n_blocks - 1)]])
    lens = [prefix + n for n in own]
    table = torch.full((B, -(-max(lens) // bt)), -1, dtype=torch.int32, device="cuda")
    at = shared
    for b, n in enumerate(own):
        table[b, :shared] = order[:shared]
        table[b, shared:shared - (-n // bt)] = order[at:at - (-n // bt)]
        at -= -n // bt
    assert at <= n_blocks and (name != "131072_pool_of_2_2_GB" or pools[0].numel() > 2 ** 31)
    q = torch.randn(B, 1, Hq, d, generator=g, device="cuda").to(dt)
    scale = 0.5 * d ** -0.5
    cache, att = cg.Cache(1, H, d, bt, n_blocks, FMT[fmt]), cg.Attend(B, 1, Hq, DT[dt], table.shape[1], scale)
    groups = cg.Groups(i32([0, B]), i32(list(range(B))), i32([shared]))
    ws = cg.empty_u8(cg.cg_shared_workspace_bytes(cache, att, groups))
    ws.fill_(0xFF)
    out, z = torch.full_like(q, math.nan), torch.full((B, 1, Hq), math.nan, device="cuda")
    cg.check(cg.cg_shared_attend(cache, att, groups, q, *pools, *scales, table, i32(lens), out, z, ws), "shared")
    torch.cuda.synchronize()
    assert cg.cg_read_status(ws) == cg.CG_OK
    code = ref.CODE[fmt]
    for b in sorted({0, 1, B - 1}):
        j = torch.arange(lens[b], device="cuda")
        page = table[b, j // bt].long()
        for h in range(H):
            k, v = (p[page, h, j % bt].view(code).double() * s[page, h].double()[:, None] for p, s in zip(pools, scales))
            rows = slice(h * G, (h + 1) * G)
            x = q[b, 0, rows].double()
            score = (x @ k.T) * scale
            l = torch.logsumexp(score, 1)
            w = torch.exp(score - l[:, None])
            o, A, X = w @ v, w @ v.abs(), (x.abs() @ k.abs().T).amax(1) * scale
            to, tl = ref.tolerances(o.cpu(), l.cpu(), A.cpu(), X.cpu(), d, lens[b], dt, 11)
            # a small weight's own tolerance: 2^-31 max(scale of V) sum|codes|, as test_gpu_shared.py derives it
            small = (pools[1][page, h, j % bt].view(code).double().abs().sum(0) * scales[1][page, h].double().amax()).cpu()
            ref.assert_close(out[b, 0, rows], o.cpu(), to + 2.0 ** -31 * small, f"out of sequence {b}, head {h}")
            ref.assert_close(z[b, 0, rows], l.cpu(), tl, f"lse of sequence {b}, head {h}")
