"""Plain 64-bit definitions of the serving calls (include/cachegen_cache.h) on the CPU, for the tests.

Tolerances are derived from the number formats, not from results.  With A = sum_j w_j |v_j| (what a relative error of
the weights w_j can move) and X = scale * max_j sum_c |q_c k_jc| (what a relative error of the products can move):
  a weight rounded to `p` bits is off by at most 2^-p of itself;
  a score is a sum in fp32 of d exact products, at least eight at a time: off by at most (d / 8 + 4) 2^-23 X, which
  moves a weight by that share, and the normalisation by as much again;
  the n weights are summed in fp32: at most n 2^-24, and exp2 / log2 / the final product 2^-20 together;
  the result is rounded once: eps / 2 of itself, or half the spacing of subnormals.
"""
import math

import torch

QMAX = {"e4m3": 448.0, "int8": 127.0}
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
WEIGHT_BITS = {torch.float16: 11, torch.bfloat16: 8}  # significant bits: a rounding is off by 2^-bits at most


def attend_rows(q, k, v, last, scale):
    """q [n, d], k and v [S, d] (any float type), row i sees keys 0 .. last[i] -> out, lse, A, X in float64."""
    q, k, v = q.double(), k.double(), v.double()
    n, S = q.shape[0], k.shape[0]
    out, A = torch.zeros(n, v.shape[1], dtype=torch.float64), torch.zeros(n, v.shape[1], dtype=torch.float64)
    lse, X = torch.full((n,), -math.inf, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
    for i in range(n):
        m = min(int(last[i]) + 1, S)
        if m <= 0:
            continue
        s = (k[:m] @ q[i]) * scale
        lse[i] = torch.logsumexp(s, 0)
        w = torch.exp(s - lse[i])
        out[i], A[i] = w @ v[:m], w @ v[:m].abs()
        X[i] = (k[:m].abs() @ q[i].abs()).max() * scale
    return out, lse, A, X


def tolerances(out, lse, A, X, d, S, dtype, weight_bits):
    """Absolute tolerances of out and lse."""
    ds = (d / 8 + 4) * 2.0 ** -23 * X + S * 2.0 ** -24 + 2.0 ** -20
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    raw = (2.0 ** -weight_bits + 2 * ds)[..., None] * A
    return raw + half * (out.abs() + raw) + tiny, ds + 2.0 ** -23 * torch.where(lse.isinf(), 0.0, lse).abs()


def assert_close(got, want, tol, what):
    got = got.double().cpu()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), f"{what}: infinities"
    off = (got - want).abs()[fine] / tol.expand_as(want)[fine]
    worst = float(off.max()) if off.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the tolerance"


def codes(x, fmt):
    """fp32 values -> codes: nearest, halves to even, saturating."""
    q = QMAX[fmt]
    x = x.clamp(-q, q)
    return x.to(CODE[fmt]) if fmt == "e4m3" else x.round().to(CODE[fmt])


def quantise(x, fmt):
    """x [n, H, bt, d] -> codes, fp32 scales [n, H]."""
    x = x.float()
    s = x.abs().amax((2, 3)) / QMAX[fmt]
    return codes(torch.where(s > 0, 1.0 / s, 0.0)[..., None, None] * x, fmt), s


def page_write(pool, scale, fmt, page, s0, rows):
    """The definition of cg_cache_write for one page: rows [n, H, d] (fp32, finite) at slots s0 .. s0+n-1, in place."""
    fresh = rows.abs().amax((0, 2)) * (torch.tensor(1.0) / torch.tensor(QMAX[fmt]))
    fresh = torch.where(fresh < 2.0 ** -100, 0.0, fresh)
    old = scale[page].clone()
    now = torch.maximum(old, fresh) if s0 else fresh
    if s0:
        grew = now > old
        ratio = torch.where(grew, old / now, 1.0)
        again = codes(pool[page, :, :s0].float() * ratio[:, None, None], fmt)
        keep = pool[page, :, :s0]
        pool[page, :, :s0] = torch.where(grew[:, None, None], again.float(), keep.float()).to(CODE[fmt])
    turn = torch.where(now > 0, 1.0 / now, 0.0)
    pool[page, :, s0:s0 + rows.shape[0]] = codes(rows.transpose(0, 1) * turn[:, None, None], fmt)
    scale[page] = now


class Book:
    """Reference counts, tables and lengths as plain lists, with the page calls' definitions."""

    def __init__(self, refs, table, lens, bt):
        self.refs, self.table, self.lens, self.bt = list(refs), [list(r) for r in table], list(lens), bt

    def pages(self, n):
        return -(-n // self.bt)

    def free_pages(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def extend(self, seqs, new_len):
        free, at = self.free_pages(), 0
        if sum(self.pages(n) - self.pages(self.lens[s]) for s, n in zip(seqs, new_len)) > len(free):
            return False
        for s, n in zip(seqs, new_len):
            for j in range(self.pages(self.lens[s]), self.pages(n)):
                self.table[s][j], self.refs[free[at]], at = free[at], 1, at + 1
            self.lens[s] = n
        return True

    def fork(self, parents, children):
        """-> [(src, dst)] pages to copy, or None where the free pages are too few."""
        free, moves = self.free_pages(), []
        if sum(self.lens[p] % self.bt != 0 for p in parents) > len(free):
            return None
        for p, c in zip(parents, children):
            used = self.pages(self.lens[p])
            row = self.table[p][:used] + [-1] * (len(self.table[p]) - used)
            if self.lens[p] % self.bt:
                moves.append((row[used - 1], free[len(moves)]))
                row[used - 1] = moves[-1][1]
            for e in row[:used]:
                self.refs[e] += 1
            self.table[c], self.lens[c] = row, self.lens[p]
        return moves

    def free(self, seqs):
        for s in seqs:
            for e in self.table[s][:self.pages(self.lens[s])]:
                self.refs[e] -= 1
            self.table[s], self.lens[s] = [-1] * len(self.table[s]), 0

    def compact(self):
        """-> n_live, [(src, dst)]"""
        n_live = sum(r > 0 for r in self.refs)
        holes = [p for p in range(n_live) if self.refs[p] == 0]
        movers = [p for p in range(n_live, len(self.refs)) if self.refs[p] > 0]
        to = dict(zip(movers, holes))
        for s, t in to.items():
            self.refs[t], self.refs[s] = self.refs[s], 0
        self.table = [[to.get(e, e) for e in row] for row in self.table]
        return n_live, list(to.items())
