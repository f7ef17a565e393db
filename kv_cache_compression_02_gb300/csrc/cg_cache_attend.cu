// cg_cache_attend.cu -- cg_cache_attend: new tokens attend over 8-bit pages.
//
// For one KV head of one sequence the G = Hq / H query heads of the T new
// tokens are T * G rows that read the same keys and values: rows of one matrix
// product, in items of 8 or 16.  Both products are taken transposed, S^T = K Q^T
// and O^T = V^T P^T, with mma.sync m16n8k16 (f16 operands, fp32 sums): keys
// and channels fill the side of 16, query rows the side of 8.  Codes of either
// format are exact in f16; page scales are applied outside the products, on
// the scores (K) and on the probabilities (V).
//
// What bounds it is the read of the codes, 2 d bytes per token and head
// against 4 T G d operations, and, close behind it, the instructions that turn
// codes into operands.  The tensor cores of tcgen05 take their operands from
// shared memory in one format, which would add a pass that writes converted
// codes there.  Here codes go from shared memory to registers once, each
// thread 16 bytes of a row at a time, and become operands as they are: both
// products leave the order of their summed index free, so a thread takes 16
// consecutive channels of a token (K), or of two tokens (V), for the fragments
// of four or eight products.
//
// Work is cut into units of 128 positions of one item, and the units of the
// whole call are dealt in equal runs to as many CTAs as fit on the GPU: a long
// context is shared by all SMs, short ones are packed.  A CTA that covers only
// a part of an item leaves its running maximum, sum and output in the
// workspace, and a second kernel, already waiting when the first one ends,
// joins the parts in their order: the result does not depend on timing.
//
// Measured, ten calls in a graph: four readers of 131072 tokens, 8 KV heads, d =
// 128, 64 query heads, int8: 186 us or 5.5 TB/s (without any arithmetic the
// copies take 161 us; called back to back 195 us or 5.3 TB/s); one short reader, 500 tokens: 10 us, the latency of five dependent loads, one
// tile and two joins.
#include <type_traits>

#include "cg_cache.cuh"
#include "cg_tma.cuh"

namespace cg {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTok = 32;              // positions of a warp's tile
constexpr int kUnit = kTok * kWarps;  // positions of a unit
constexpr int kShort = 2;             // units of an item that one CTA takes where items are few (with 8: 12.5, not 9.9 us for 500 tokens)
constexpr int kIn = 2;                // what an item's way in and out costs, in units (measured: 2.6 and 1.4 us)
constexpr int kLens = 512;            // sequences whose lengths are kept in shared memory

// NB blocks of eight query rows make an item.  One block leaves room for three
// CTAs on an SM, two for two.  Up to eight rows take one block (131072 tokens
// of 8 heads: 61 us; with an empty second block 74 us), more take two (16 rows:
// 79 us).
template <int NB>
struct Shape {
  static constexpr int kRows = 8 * NB;
  static constexpr int kPerSM = NB == 1 ? 3 : 2;   // CTAs
  static constexpr int kStages = NB == 1 ? 2 : 3;  // tiles of a warp's ring
  static constexpr int kGrid = kSMs * kPerSM;
};
constexpr int kMostCtas = Shape<1>::kGrid;

// A probability is held as p = 2^(s - m + kLift), and m may lag behind the
// true maximum by kLag, so that p < 2^15.  For the second product it is
// multiplied by its page's V scale over a power of two above the largest so far
// and taken as the sum of two f16 values.  The second one is subnormal where the
// weight is under 2^-2, so that the sum is off by 2^-23 of the weight or by
// 2^-25, whichever is more (2^-36 of the largest probability, which has at least
// 2^12, times the largest scale).  Weights under kNormal, rare but for sharp
// distributions, go through products of their own, raised by 2^28 each time,
// as one f16 value: off by 2^-11 of themselves, which is under 2^-25, too.
constexpr float kLift = 12.0f, kLag = 3.0f, kNormal = 0x1p-14f;

// n / d for n < 2^31 (a multiplication by the reciprocal, rounded up).
struct Divisor {
  uint32_t mul, shift;
  Divisor(uint32_t d = 1) {
    shift = 0;
    while ((uint64_t(1) << shift) < d) shift++;
    mul = uint32_t(((uint64_t(1) << 32) * ((uint64_t(1) << shift) - d)) / d + 1);
  }
  __device__ uint32_t operator()(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
};

// What a CTA leaves behind: its error bits, and the item that it has the first
// but not the last part of (parts = 0: none).
struct Note {
  uint32_t errors;
  int32_t parts;   // of the item, in this CTA and the next ones
  int32_t second;  // the first part is in this CTA's second slot
  int32_t b, h, rt;
};

struct AttendArgs {
  CUtensorMap k_map, v_map;  // of the pools as rows of d codes, in tiles of 16
  const uint16_t *q;
  const uint8_t *kp, *vp;
  const float *ks, *vs;
  const int32_t *table, *len;
  uint16_t *out;
  float *lse;
  uint32_t *status;
  Note *notes;   // [grid]: what each CTA of k_attend leaves for k_join
  float *parts;  // [2 * grid][rows of an item][D + 2]
  int64_t q_seq, q_tok, q_head;
  int B, T, Hq, H, G, rows, RT, HR, d, bt, n_blocks, stride;  // rows: T * G; RT: items of them; HR: heads x RT
  float scale_log2;  // scale * log2(e)
  Divisor by_bt;
  bool plain;
};

template <int D>
struct Tile {
  uint8_t k[kTok * D], v[kTok * D];
};

template <int D, int NB>
struct Smem {
  static constexpr int kRows = Shape<NB>::kRows, kStages = Shape<NB>::kStages;
  Tile<D> ring[kWarps][kStages];
  float ks[kWarps][kStages][kTok], vs[kWarps][kStages][kTok];  // PLAIN: the first two of each
  float o[2][kRows * D / 2];  // where warps hand their outputs over, half of the channels at a time
  float m[kWarps][kRows], l[kWarps][kRows];
  uint64_t full[kWarps][kStages];
  uint32_t valid[kWarps][kStages];
  int64_t sum[kWarps][2], prefix;
  int most[kWarps], b;
  uint32_t errors, dead;
  int len[kLens];
};

// Where 16-byte chunk c of row r lies in a tile: the swizzle of a tiled copy
// with rows of 128 (64) bytes.  Eight lanes that read together take, of K, the
// even or the odd chunks of two rows, of V, the chunks 2i, 2i+1 of four rows
// of one parity: no bank conflict (two-way for V where D is 64).
template <int D>
__device__ inline int chunk_at(int r, int c) {
  return r * D + ((D == 128 ? c ^ (r & 7) : c ^ (r >> 1 & 3)) << 4);
}

template <int N>
__device__ inline void copy_async(uint32_t dst, const void *src, bool ok) {
  const int n = ok ? N : 0;  // the rest is filled with zeros
  if (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(n) : "memory");
}

__device__ inline void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of 16-bit elements, lane i with elements 2 (i % 4) and one more of row i / 4, transposed.
__device__ inline uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Two fp32 operations in one instruction.
__device__ inline float2 add2(float2 a, float2 b) {
  float2 y;
  asm("{.reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; add.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d;}"
      : "=f"(y.x), "=f"(y.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return y;
}
__device__ inline float2 mul2(float2 a, float2 b) {
  float2 y;
  asm("{.reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mul.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d;}"
      : "=f"(y.x), "=f"(y.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return y;
}

__device__ inline float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Codes in the low (H = 0) or high half of w -> two f16.
template <int FMT, int H>
__device__ inline uint32_t halves_of(uint32_t w) {
  uint32_t r;
  if (FMT == CG_CACHE_E4M3) {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(H ? w >> 16 : w)));
  } else {  // 0x64uu is 1024 + u; w holds code + 128
    const __half2 x = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    uint32_t p = __byte_perm(w, 0x64646464u, H ? 0x4342 : 0x4140);
    const __half2 y = __hsub2(*reinterpret_cast<__half2 *>(&p), x);
    r = *reinterpret_cast<const uint32_t *>(&y);
  }
  return r;
}

template <int FMT>
__device__ inline uint32_t biased(uint32_t w) {
  return FMT == CG_CACHE_INT8 ? w ^ 0x80808080u : w;
}

__device__ inline uint32_t pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Which bytes are an e4m3 NaN.
__device__ inline uint32_t nan_bytes(uint32_t w) { return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu); }

// A walk over the units of a call, from one item (sequence, head, row block) to the next.
struct Walk {
  int b, h, rt, tile, tiles, len;
};

__device__ inline int clamped_length(const AttendArgs &a, int b) {
  return int(max(int64_t(0), min(int64_t(a.len[b]), int64_t(a.stride) * a.bt)));
}

__device__ inline int length(const AttendArgs &a, const int *kept, int b) {
  return a.B <= kLens ? kept[b] : clamped_length(a, b);
}

__device__ inline int tiles_of(int len) { return int((uint32_t(len) + kUnit - 1) / kUnit); }

__device__ inline void set_seq(const AttendArgs &a, const int *kept, Walk &w) {
  w.len = length(a, kept, w.b);
  w.tiles = tiles_of(w.len);
}

// The next item; the caller knows that there is one.
__device__ inline void next_item(const AttendArgs &a, const int *kept, Walk &w) {
  w.tile = 0;
  if (++w.rt < a.RT) return;
  w.rt = 0;
  if (++w.h < a.H) return;
  w.h = 0;
  do {
    w.b++;
    set_seq(a, kept, w);
  } while (w.tiles == 0);
}

// Channels c0 .. c0 + N - 1 of a finished row.
template <bool BF16, int N>
__device__ inline void write_row(const AttendArgs &a, int b, int h, int r, const float (&x)[N], int c0, float m,
                                 float l, bool lead) {
  const int t = r / a.G;
  const int64_t row = (int64_t(b) * a.T + t) * a.Hq + h * a.G + r % a.G;
  const float f = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    if (c0 + i >= a.d) continue;
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; k++)
      w[k] = uint32_t(elem_of<BF16>(x[i + 2 * k] * f)) | uint32_t(elem_of<BF16>(x[i + 2 * k + 1] * f)) << 16;
    *reinterpret_cast<uint4 *>(a.out + row * a.d + c0 + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (lead && a.lse) a.lse[row] = l == 0.0f ? -INFINITY : (m - kLift + log2f(l)) * 0.6931471805599453f;
}

// PLAIN: pages are a multiple of 16 tokens and a row has D channels, so that
// half a warp's tile lies in one page (one table entry, one scale) and is one
// tiled copy.  Other shapes copy 8 or 16 bytes a lane: on pages of 64 and D
// channels 131072 tokens of 8 heads take 61 us the first way and 76 us the
// second.
template <int FMT, int D, int NB, bool BF16, bool PLAIN>
__global__ void __launch_bounds__(kThreads, Shape<NB>::kPerSM) k_attend(const __grid_constant__ AttendArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem<D, NB> &sm = *reinterpret_cast<Smem<D, NB> *>(smem_raw);
  constexpr int kRows = Shape<NB>::kRows, kStages = Shape<NB>::kStages;
  constexpr int kJ = D / 16;       // tiles of 16 channels
  constexpr int kChunks = D / 16;  // 16-byte chunks of a row
  constexpr int kMine = D / 8;     // channels of a lane in the second product: kMine g ...
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x == 0) {
    sm.errors = sm.dead = 0;
    a.notes[blockIdx.x].parts = 0;
  }
  // The items of the call and what they cost: their units and kIn.  Where items
  // are few and short each has a CTA of its own.
  const int per = (a.B + kThreads - 1) / kThreads, b0 = threadIdx.x * per, b1 = min(a.B, b0 + per);
  int64_t cost = 0, items = 0;
  int most = 0;
  bool bad_len = false;
  for (int b = b0; b < b1; b++) {
    const int n = a.len[b], fit = clamped_length(a, b), tiles = tiles_of(fit);
    bad_len |= n != fit;
    if (a.B <= kLens) sm.len[b] = fit;
    cost += tiles ? tiles + kIn : 0;
    items += tiles > 0;
    most = max(most, tiles);
  }
  cost *= a.HR, items *= a.HR;
  int64_t cost_to = cost, items_to = items;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, cost_to, o), z = __shfl_up_sync(0xffffffffu, items_to, o);
    if (lane >= o) cost_to += y, items_to += z;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 31) sm.sum[warp][0] = cost_to, sm.sum[warp][1] = items_to, sm.most[warp] = most;
  if (PLAIN && lane == 0) {
    for (int s = 0; s < kStages; s++) bar_init(&sm.full[warp][s], 2);
    bar_init_fence();
  }
  if (!PLAIN && a.d < D) {  // channels that no copy fills
    uint4 *z = reinterpret_cast<uint4 *>(sm.ring[warp]);
    for (int i = lane; i < int(sizeof(sm.ring[warp]) / 16); i += 32) z[i] = make_uint4(0, 0, 0, 0);
  }
  __syncthreads();
  int64_t total = 0, n_items = 0;
#pragma unroll
  for (int w = 0; w < kWarps; w++) {
    if (w < warp) cost_to += sm.sum[w][0], items_to += sm.sum[w][1];
    total += sm.sum[w][0], n_items += sm.sum[w][1];
    most = max(most, sm.most[w]);
  }
  const bool single = most <= kShort && n_items <= gridDim.x;  // a CTA per item
  if (single) total = n_items, cost = items, cost_to = items_to;
  const int64_t before = cost_to - cost;
  if (blockIdx.x == 0 && bad_len) atomicOr(&sm.errors, kStBadArg);
  for (int b = blockIdx.x; b < a.B; b += gridDim.x)  // sequences with nothing in them
    if (length(a, sm.len, b) == 0) {
      const int64_t rows = int64_t(a.T) * a.Hq, at = b * rows;
      for (int64_t i = threadIdx.x; i < rows * a.d / 8; i += kThreads)
        reinterpret_cast<uint4 *>(a.out + at * a.d)[i] = make_uint4(0, 0, 0, 0);
      if (a.lse)
        for (int64_t i = threadIdx.x; i < rows; i += kThreads) a.lse[at + i] = -INFINITY;
    }
  const int64_t ctas = min(int64_t(gridDim.x), total);
  if (blockIdx.x >= ctas) {
    __syncthreads();
    if (threadIdx.x == 0) a.notes[blockIdx.x].errors = sm.errors;
    return;
  }
  const int64_t lo = total * blockIdx.x / ctas, hi = total * (blockIdx.x + 1) / ctas;
  auto cost_of = [&](int tiles) { return single ? (tiles > 0) : tiles ? tiles + kIn : 0; };
  if (lo >= before && lo < before + cost) {  // one thread's sequences hold the first unit
    int64_t at = before;
    int b = b0;
    for (;; b++) {
      const int64_t n = int64_t(cost_of(tiles_of(length(a, sm.len, b)))) * a.HR;
      if (lo < at + n) break;
      at += n;
    }
    sm.b = b;
    sm.prefix = at;
  }
  __syncthreads();

  Walk cur;
  cur.b = sm.b;
  set_seq(a, sm.len, cur);
  int item_cost = cost_of(cur.tiles);
  const int item0 = int((lo - sm.prefix) / item_cost);
  cur.h = item0 / a.RT, cur.rt = item0 % a.RT;
  int64_t item_lo = sm.prefix + int64_t(item0) * item_cost;  // where the item's cost begins
  // A run [lo, hi) of costs has the tiles whose costs lie in it; an item's
  // first kIn costs are no tiles.
  const int skip = single ? 0 : kIn;
  cur.tile = max(0, int(lo - item_lo) - skip);
  int units = 0;  // tiles of the run
  if (single) {
    units = cur.tiles;
  } else {
    int64_t at = lo;
    Walk w = cur;
    int64_t w_lo = item_lo;
    int w_cost = item_cost;
    while (at < hi) {  // item by item
      const int64_t end = min(hi, w_lo + w_cost);
      units += int(max(int64_t(0), end - w_lo - kIn) - max(int64_t(0), at - w_lo - kIn));
      at = end;
      if (at < hi) {
        w_lo += w_cost;
        next_item(a, sm.len, w);
        w_cost = w.tiles + kIn;
      }
    }
  }
  Walk ahead = cur;

  // The page of row `lane` of the warp's tile in the unit that `ahead` stands
  // at; PLAIN: that of the lane's half of the tile.
  const int d = PLAIN ? D : a.d;
  const int64_t page_elems = int64_t(a.H) * a.bt * d;
  int page = 0, slot = 0, page_h = 0, have_rows = 0;
  bool wanted = false;
  auto find_page = [&]() {  // nothing here waits for the entry: the next copy does
    const uint32_t tok0 = uint32_t(ahead.tile) * kUnit + warp * kTok, tok = tok0 + (PLAIN ? lane & 16 : lane);
    page_h = ahead.h;
    have_rows = ahead.len - int(tok0);
    wanted = tok < uint32_t(ahead.len);
    if (wanted) {
      const uint32_t blk = a.by_bt(tok);
      slot = int(tok - blk * a.bt);
      page = a.table[int64_t(ahead.b) * a.stride + blk];
    }
  };
  auto issue = [&](int s) {
    Tile<D> &st = sm.ring[warp][s];
    const bool ok = wanted && uint32_t(page) < uint32_t(a.n_blocks);
    if (wanted && !ok) atomicOr(&sm.errors, kStBadArg);
    const int64_t sc_at = ok ? int64_t(page) * a.H + page_h : 0;
    uint32_t valid = __ballot_sync(0xffffffffu, ok);
    if (PLAIN) {  // the rows that are there, of the pages that are right
      if (have_rows < kTok) valid &= have_rows <= 0 ? 0u : (1u << have_rows) - 1;
      const int half = lane >> 4;
      if ((lane & 15) < 2)
        copy_async<4>(smem_of((lane & 1 ? sm.vs : sm.ks)[warp][s] + half), (lane & 1 ? a.vs : a.ks) + sc_at, ok);
      if ((lane & 15) == 0) {
        bar_expect(&sm.full[warp][s], ok ? 2 * 16 * D : 0);
        if (ok) {
          const int y = (page * a.H + page_h) * a.bt + slot;  // a row of the pool
          tma_2d(smem_of(st.k + half * 16 * D), &a.k_map, &sm.full[warp][s], 0, y);
          tma_2d(smem_of(st.v + half * 16 * D), &a.v_map, &sm.full[warp][s], 0, y);
        }
      }
    } else {
      copy_async<4>(smem_of(&sm.ks[warp][s][lane]), a.ks + sc_at, ok);
      copy_async<4>(smem_of(&sm.vs[warp][s][lane]), a.vs + sc_at, ok);
      const int64_t off = ok ? page * page_elems + (int64_t(page_h) * a.bt + slot) * d : 0;
      const int c = lane % kChunks, r0 = lane / kChunks;
      constexpr int kStep = 32 / kChunks;  // rows of one copy
#pragma unroll
      for (int i = 0; i < kTok / kStep; i++) {
        const int r = i * kStep + r0, to = chunk_at<D>(r, c);
        const bool have = valid >> r & 1;
        int64_t at = __shfl_sync(0xffffffffu, off, r) + c * 16;
        if (!have) at = 0;
        if (c * 16 < d) {
          if ((d & 15) == 0) {
            copy_async<16>(smem_of(st.k + to), a.kp + at, have);
            copy_async<16>(smem_of(st.v + to), a.vp + at, have);
          } else {
            copy_async<8>(smem_of(st.k + to), a.kp + at, have);
            copy_async<8>(smem_of(st.v + to), a.vp + at, have);
            if (c * 16 + 8 < d) {
              copy_async<8>(smem_of(st.k + to + 8), a.kp + (have ? at + 8 : 0), have);
              copy_async<8>(smem_of(st.v + to + 8), a.vp + (have ? at + 8 : 0), have);
            }
          }
        }
      }
    }
    if (lane == 0) sm.valid[warp][s] = valid;
  };
  int issued = 0;
  find_page();
#pragma unroll
  for (int s = 0; s < kStages - 1; s++) {
    if (issued < units) {
      issue(s);
      issued++;
      if (issued < units) {
        if (++ahead.tile == ahead.tiles) next_item(a, sm.len, ahead);
        find_page();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }

  // A lane has, of each block n of eight rows, rows 8 n + 2 t and 8 n + 2 t + 1
  // (.x and .y): scores of positions g and g + 8 of each 16, outputs of
  // channels kMine g ..., o[j][n][2 c + i] being channel 2 j + c of row i.
  uint32_t q[NB][kJ][2];
  float o[kJ][NB][4];
  float2 m[NB], l[NB], sc[NB];
  int last[NB][2], v_exp = 1;  // O is in units of 2^(v_exp - 127), the largest V scale so far
  bool first = true;
  int seg = 0;  // items begun before
  uint32_t phase = 0;
  int slot_now = 0, slot_next = kStages - 1;  // of the ring
  for (int u = 0; u < units; u++) {
    const int h = cur.h, r0 = cur.rt * kRows;
    if (first) {  // a new item: its query rows
      first = false;
#pragma unroll
      for (int n = 0; n < NB; n++) {
        const int r = r0 + 8 * n + g, tt = r / a.G;
        const bool ok = r < a.rows;
        const uint16_t *src = a.q + cur.b * a.q_seq + tt * a.q_tok + int64_t(h * a.G + r % a.G) * a.q_head;
        uint4 w[D / 32];
#pragma unroll
        for (int c = 0; c < D / 32; c++) {
          const int ch = D / 4 * t + 8 * c;
          w[c] = ok && ch < a.d ? *reinterpret_cast<const uint4 *>(src + ch) : make_uint4(0, 0, 0, 0);
        }
        float scale = a.scale_log2;
        if (BF16) {  // to f16, raised to its top: off by at most 2^-39 of the row's largest
          uint32_t top = 0;
#pragma unroll
          for (int c = 0; c < D / 32; c++) {
            const uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
            for (int k = 0; k < 4; k++) top = max(top, max(x[k] << 16 & 0x7fff0000u, x[k] & 0x7fff0000u));
          }
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int f = min(253, max(1, 268 - int(top >> 23)));
          const float up = __int_as_float(f << 23);
          scale *= __int_as_float((254 - f) << 23);
#pragma unroll
          for (int c = 0; c < D / 32; c++) {
            uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
            for (int k = 0; k < 4; k++)
              x[k] = pack(__uint_as_float(x[k] << 16) * up, __uint_as_float(x[k] & 0xffff0000u) * up);
            w[c] = make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
#pragma unroll
        for (int c = 0; c < D / 32; c++)
          q[n][2 * c][0] = w[c].x, q[n][2 * c][1] = w[c].y, q[n][2 * c + 1][0] = w[c].z, q[n][2 * c + 1][1] = w[c].w;
        // this lane has loaded row g of the block and keeps the state of rows 2 t, 2 t + 1
        sc[n] = make_float2(__shfl_sync(0xffffffffu, scale, 8 * t), __shfl_sync(0xffffffffu, scale, 8 * t + 4));
#pragma unroll
        for (int i = 0; i < 2; i++) {
          const int ri = r0 + 8 * n + 2 * t + i;
          last[n][i] = ri < a.rows ? cur.len - a.T + ri / a.G : 0x7fffffff;  // a row of padding may see anything
        }
        m[n] = make_float2(-INFINITY, -INFINITY);
        l[n] = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < kJ; j++) o[j][n][0] = o[j][n][1] = o[j][n][2] = o[j][n][3] = 0.0f;
      }
      v_exp = 1;
    }

    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    const int s = slot_now;
    bool landed = true;
    if (PLAIN) landed = bar_wait(&sm.full[warp][s], phase, &sm.dead);
    if (!landed) atomicOr(&sm.errors, kStTimeout);
    __syncwarp();
    if (++slot_now == kStages) slot_now = 0, phase ^= 1;
    if (issued < units) {
      issue(slot_next);
      issued++;
      if (issued < units) {
        if (++ahead.tile == ahead.tiles) next_item(a, sm.len, ahead);
        find_page();
      }
    }
    slot_next = slot_next + 1 == kStages ? 0 : slot_next + 1;
    asm volatile("cp.async.commit_group;" ::: "memory");

    Tile<D> &st = sm.ring[warp][s];
    const uint32_t valid = sm.valid[warp][s];
    const uint32_t tok0 = uint32_t(cur.tile) * kUnit + warp * kTok;
    if (PLAIN && valid != 0xffffffffu && valid) {  // what lies behind the last position must not reach a product: 0 * NaN
#pragma unroll
      for (int i = 0; i < kTok * kChunks / 32; i++) {
        const int r = (i * 32 + lane) / kChunks;
        if (!(valid >> r & 1)) reinterpret_cast<uint4 *>(st.v)[i * 32 + lane] = make_uint4(0, 0, 0, 0);
      }
      fence_async();
      __syncwarp();
    }
    if (valid) {
      constexpr int kT = kTok / 16;
      // S^T = K Q^T
      float x[kT][NB][4];  // [..][2 half + i]: position 16 tt + 8 half + g, row i
#pragma unroll
      for (int tt = 0; tt < kT; tt++)
#pragma unroll
        for (int n = 0; n < NB; n++) x[tt][n][0] = x[tt][n][1] = x[tt][n][2] = x[tt][n][3] = 0.0f;
#pragma unroll
      for (int c = 0; c < D / 64; c++)
#pragma unroll
        for (int tt = 0; tt < kT; tt++) {
          const uint4 w0 = *reinterpret_cast<const uint4 *>(st.k + chunk_at<D>(16 * tt + g, D / 64 * t + c));
          const uint4 w1 = *reinterpret_cast<const uint4 *>(st.k + chunk_at<D>(16 * tt + 8 + g, D / 64 * t + c));
          const uint32_t y0[4] = {w0.x, w0.y, w0.z, w0.w}, y1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
          for (int k = 0; k < 4; k++) {
            const uint32_t z0 = biased<FMT>(y0[k]), z1 = biased<FMT>(y1[k]);
            const uint32_t f[4] = {halves_of<FMT, 0>(z0), halves_of<FMT, 0>(z1), halves_of<FMT, 1>(z0), halves_of<FMT, 1>(z1)};
#pragma unroll
            for (int n = 0; n < NB; n++) mma(x[tt][n], f, q[n][4 * c + k][0], q[n][4 * c + k][1]);
          }
        }
      // what turns a product into a score, and V's scale, for positions 16 tt + 8 half + g
      float ks[kT][2], vs[kT][2];
#pragma unroll
      for (int tt = 0; tt < kT; tt++)
#pragma unroll
        for (int half = 0; half < 2; half++) {
          ks[tt][half] = sm.ks[warp][s][PLAIN ? tt : 16 * tt + 8 * half + g];
          vs[tt][half] = sm.vs[warp][s][PLAIN ? tt : 16 * tt + 8 * half + g];
        }
#pragma unroll
      for (int tt = 0; tt < kT; tt++)
#pragma unroll
        for (int half = 0; half < 2; half++)
#pragma unroll
          for (int n = 0; n < NB; n++) {
            const float2 y = mul2(make_float2(x[tt][n][2 * half], x[tt][n][2 * half + 1]),
                                  make_float2(ks[tt][half] * sc[n].x, ks[tt][half] * sc[n].y));
            x[tt][n][2 * half] = y.x, x[tt][n][2 * half + 1] = y.y;
          }
      // whether every position is there and every row sees it
      const bool whole = valid == 0xffffffffu && int(tok0) + kTok - 1 <= cur.len - a.T;
      auto sees = [&](int p, int most_seen) { return (valid >> p & 1) && int(tok0) + p <= most_seen; };
      if (!whole) {
#pragma unroll
        for (int tt = 0; tt < kT; tt++)
#pragma unroll
          for (int n = 0; n < NB; n++)
#pragma unroll
            for (int i = 0; i < 4; i++)
              if (!sees(16 * tt + 8 * (i >> 1) + g, last[n][i & 1])) x[tt][n][i] = -INFINITY;
      }
      float vmax = fabsf(vs[0][0]);
#pragma unroll
      for (int tt = 0; tt < kT; tt++) vmax = fmaxf(vmax, PLAIN ? fabsf(vs[tt][0]) : fmaxf(fabsf(vs[tt][0]), fabsf(vs[tt][1])));
      if (!PLAIN) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, o));
      }
      const int e = min(254, int(__float_as_uint(vmax) >> 23) + 1);
      bool moved = e > v_exp;  // the same in every lane
      const float down = !moved ? 1.0f : e - v_exp > 126 ? 0.0f : __int_as_float((127 + v_exp - e) << 23);
      v_exp = max(v_exp, e);
      float2 keep[NB];
#pragma unroll
      for (int n = 0; n < NB; n++) {
        float2 top = make_float2(x[0][n][0], x[0][n][1]);
#pragma unroll
        for (int tt = 0; tt < kT; tt++) {
          top.x = fmaxf(top.x, fmaxf(x[tt][n][0], x[tt][n][2]));
          top.y = fmaxf(top.y, fmaxf(x[tt][n][1], x[tt][n][3]));
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          top.x = fmaxf(top.x, __shfl_xor_sync(0xffffffffu, top.x, o));
          top.y = fmaxf(top.y, __shfl_xor_sync(0xffffffffu, top.y, o));
        }
        keep[n] = make_float2(1.0f, 1.0f);
        if (top.x > m[n].x + kLag) keep[n].x = ex2(m[n].x - top.x), m[n].x = top.x, moved = true;
        if (top.y > m[n].y + kLag) keep[n].y = ex2(m[n].y - top.y), m[n].y = top.y, moved = true;
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int n = 0; n < NB; n++) {
          l[n] = mul2(l[n], keep[n]);
          const float2 f = mul2(keep[n], make_float2(down, down));
#pragma unroll
          for (int j = 0; j < kJ; j++) o[j][n][0] *= f.x, o[j][n][1] *= f.y, o[j][n][2] *= f.x, o[j][n][3] *= f.y;
        }
      }
      const float unit = __int_as_float((254 - v_exp) << 23);
      float least = INFINITY;  // of the probabilities
#pragma unroll
      for (int n = 0; n < NB; n++) {
        const float2 base = make_float2(kLift - (m[n].x == -INFINITY ? 0.0f : m[n].x), kLift - (m[n].y == -INFINITY ? 0.0f : m[n].y));
#pragma unroll
        for (int tt = 0; tt < kT; tt++)
#pragma unroll
          for (int half = 0; half < 2; half++) {
            float2 y = add2(make_float2(x[tt][n][2 * half], x[tt][n][2 * half + 1]), base);
            y = make_float2(ex2(y.x), ex2(y.y));
            l[n] = add2(l[n], y);
            const float v = vs[tt][half] * unit;
            y = mul2(y, make_float2(v, v));
            x[tt][n][2 * half] = y.x, x[tt][n][2 * half + 1] = y.y;
            least = fminf(least, fminf(fabsf(y.x), fabsf(y.y)));
          }
      }
      if (!whole) {  // 0 * NaN
#pragma unroll
        for (int tt = 0; tt < kT; tt++)
#pragma unroll
          for (int n = 0; n < NB; n++)
#pragma unroll
            for (int i = 0; i < 4; i++)
              if (!sees(16 * tt + 8 * (i >> 1) + g, last[n][i & 1])) x[tt][n][i] = 0.0f;
      }
      // P^T as an operand, and what its rounding left over
      uint32_t hi_p[kT][NB][2], lo_p[kT][NB][2];
      auto to_half = [&](auto keep_small) {
#pragma unroll
        for (int tt = 0; tt < kT; tt++)
#pragma unroll
          for (int n = 0; n < NB; n++)
#pragma unroll
            for (int half = 0; half < 2; half++) {
              float p0 = x[tt][n][2 * half], p1 = x[tt][n][2 * half + 1];
              if (!keep_small.value) p0 = fabsf(p0) < kNormal ? 0.0f : p0, p1 = fabsf(p1) < kNormal ? 0.0f : p1;
              const uint32_t w = pack(p0, p1);
              const float2 back = __half22float2(*reinterpret_cast<const __half2 *>(&w));
              hi_p[tt][n][half] = transposed(w);
              lo_p[tt][n][half] = transposed(pack(p0 - back.x, p1 - back.y));
            }
      };
      const bool small = __any_sync(0xffffffffu, least < kNormal);
      if (small)
        to_half(std::false_type());
      else
        to_half(std::true_type());

      // O^T += V^T P^T, sixteen positions at a time
      constexpr int kWords = D / 32;  // words of a token that a lane takes
      auto load_v = [&](int tt, uint32_t (&w)[4][kWords]) {  // positions 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int r = 16 * tt + 2 * t + (i & 1) + 8 * (i >> 1);
          if (D == 128) {
            const uint4 y = *reinterpret_cast<const uint4 *>(st.v + chunk_at<D>(r, g));
            w[i][0] = y.x, w[i][1] = y.y, w[i][kWords - 2] = y.z, w[i][kWords - 1] = y.w;
          } else {
            const uint2 y = *reinterpret_cast<const uint2 *>(st.v + chunk_at<D>(r, g >> 1) + 8 * (g & 1));
            w[i][0] = y.x, w[i][1] = y.y;
          }
        }
      };
      // the operands of channels 4 k, 4 k + 1 (f[0]) and 4 k + 2, 4 k + 3 (f[1])
      auto operand = [&](const uint32_t (&w)[4][kWords], int k, uint32_t (&f)[2][4]) {
        uint32_t z[4];
#pragma unroll
        for (int i = 0; i < 4; i++) z[i] = biased<FMT>(w[i][k]);
        const uint32_t a01 = __byte_perm(z[0], z[1], 0x5140), a23 = __byte_perm(z[0], z[1], 0x7362);
        const uint32_t b01 = __byte_perm(z[2], z[3], 0x5140), b23 = __byte_perm(z[2], z[3], 0x7362);
        f[0][0] = halves_of<FMT, 0>(a01), f[0][1] = halves_of<FMT, 1>(a01), f[0][2] = halves_of<FMT, 0>(b01), f[0][3] = halves_of<FMT, 1>(b01);
        f[1][0] = halves_of<FMT, 0>(a23), f[1][1] = halves_of<FMT, 1>(a23), f[1][2] = halves_of<FMT, 0>(b23), f[1][3] = halves_of<FMT, 1>(b23);
      };
      bool odd = false;
#pragma unroll
      for (int tt = 0; tt < kT; tt++) {
        uint32_t w[4][kWords];
        load_v(tt, w);
        if (FMT == CG_CACHE_E4M3 && !whole && a.T > 1) {
          // A NaN code behind a row's last position must not reach that row
          // through 0 * NaN: such codes are taken out of the product, and a
          // product of "is NaN" and "sees" says which outputs are NaN.
          uint32_t any = 0;
#pragma unroll
          for (int i = 0; i < 4; i++)
#pragma unroll
            for (int k = 0; k < kWords; k++) any |= nan_bytes(w[i][k]);
          if (__any_sync(0xffffffffu, any != 0)) {
            odd = true;
            constexpr uint32_t kOne = 0x3c00u;
            uint32_t see[NB][2];  // of row g: positions 2 t, 2 t + 1 and 2 t + 8, 2 t + 9
#pragma unroll
            for (int n = 0; n < NB; n++)
#pragma unroll
              for (int half = 0; half < 2; half++) {
                const int p = 16 * tt + 8 * half + 2 * t;
                const int l0 = __shfl_sync(0xffffffffu, last[n][0], g >> 1), l1 = __shfl_sync(0xffffffffu, last[n][1], g >> 1);
                const int mine = g & 1 ? l1 : l0;
                see[n][half] = (sees(p, mine) ? kOne : 0) | (sees(p + 1, mine) ? kOne << 16 : 0);
              }
#pragma unroll
            for (int k = 0; k < kWords; k++) {
              uint32_t z[4];
#pragma unroll
              for (int i = 0; i < 4; i++) z[i] = nan_bytes(w[i][k]), w[i][k] &= ~z[i];
#pragma unroll
              for (int c = 0; c < 2; c++) {
                auto pair = [&](int i, int byte) {
                  return (z[i] >> (8 * byte) & 1 ? kOne : 0) | (z[i + 1] >> (8 * byte) & 1 ? kOne << 16 : 0);
                };
                const uint32_t f[4] = {pair(0, 2 * c), pair(0, 2 * c + 1), pair(2, 2 * c), pair(2, 2 * c + 1)};
#pragma unroll
                for (int n = 0; n < NB; n++) {
                  float hit[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                  mma(hit, f, see[n][0], see[n][1]);
#pragma unroll
                  for (int i = 0; i < 4; i++)
                    if (hit[i] > 0.0f) o[2 * k + c][n][i] = __int_as_float(0x7fffffff);
                }
              }
            }
          }
        }
#pragma unroll
        for (int k = 0; k < kWords; k++) {
          uint32_t f[2][4];
          operand(w, k, f);
#pragma unroll
          for (int c = 0; c < 2; c++)
#pragma unroll
            for (int n = 0; n < NB; n++) {
              mma(o[2 * k + c][n], f[c], hi_p[tt][n][0], hi_p[tt][n][1]);
              mma(o[2 * k + c][n], f[c], lo_p[tt][n][0], lo_p[tt][n][1]);
            }
        }
      }
      if (small) {
        float fall = 1.0f;
#pragma unroll 1
        for (int pass = 0; pass < 4; pass++) {  // to 2^-126
          fall *= 0x1p-28f;
          bool have = false;
#pragma unroll
          for (int tt = 0; tt < kT; tt++)
#pragma unroll
            for (int n = 0; n < NB; n++)
#pragma unroll
              for (int i = 0; i < 4; i++) {  // what the last product had goes, the rest is raised
                x[tt][n][i] = fabsf(x[tt][n][i]) < kNormal ? x[tt][n][i] * 0x1p28f : 0.0f;
                have |= x[tt][n][i] != 0.0f;
              }
          if (!__any_sync(0xffffffffu, have)) break;
          to_half(std::false_type());
#pragma unroll
          for (int k = 0; k < kWords; k++) {
            float y[2][NB][4] = {};
#pragma unroll
            for (int tt = 0; tt < kT; tt++) {
              uint32_t w[4][kWords], f[2][4];
              load_v(tt, w);
              if (odd)
#pragma unroll
                for (int i = 0; i < 4; i++) w[i][k] &= ~nan_bytes(w[i][k]);
              operand(w, k, f);
#pragma unroll
              for (int c = 0; c < 2; c++)
#pragma unroll
                for (int n = 0; n < NB; n++) mma(y[c][n], f[c], hi_p[tt][n][0], hi_p[tt][n][1]);
            }
#pragma unroll
            for (int c = 0; c < 2; c++)
#pragma unroll
              for (int n = 0; n < NB; n++)
#pragma unroll
                for (int i = 0; i < 4; i++) o[2 * k + c][n][i] += y[c][n][i] * fall;
          }
        }
      }
    }

    const bool end = cur.tile + 1 == cur.tiles || u + 1 == units;
    if (end) {
      // The four warps' parts of the item, joined in a fixed order.
#pragma unroll
      for (int n = 0; n < NB; n++) {
        float2 y = l[n];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) y.x += __shfl_xor_sync(0xffffffffu, y.x, o), y.y += __shfl_xor_sync(0xffffffffu, y.y, o);
        if (g == 0) {
          sm.m[warp][8 * n + 2 * t] = m[n].x, sm.m[warp][8 * n + 2 * t + 1] = m[n].y;
          sm.l[warp][8 * n + 2 * t] = y.x, sm.l[warp][8 * n + 2 * t + 1] = y.y;
        }
      }
      __syncthreads();
      float top[NB][2], sum[NB][2];
#pragma unroll
      for (int n = 0; n < NB; n++)
#pragma unroll
        for (int i = 0; i < 2; i++) {
          const int r = 8 * n + 2 * t + i;
          top[n][i] = -INFINITY;
          for (int w = 0; w < kWarps; w++) top[n][i] = fmaxf(top[n][i], sm.m[w][r]);
          sum[n][i] = 0.0f;
          for (int w = 0; w < kWarps; w++)
            sum[n][i] += sm.l[w][r] * (sm.m[w][r] == -INFINITY ? 0.0f : ex2(sm.m[w][r] - top[n][i]));
          const float mine = i ? m[n].y : m[n].x;
          const float f = (mine == -INFINITY ? 0.0f : ex2(mine - top[n][i])) * __int_as_float(v_exp << 23);
#pragma unroll
          for (int j = 0; j < kJ; j++) o[j][n][i] *= f, o[j][n][2 + i] *= f;
        }
#pragma unroll
      for (int w = kWarps / 2; w; w >>= 1)  // warps w .. 2w-1 hand theirs to 0 .. w-1
#pragma unroll
        for (int j0 = 0; j0 < kJ; j0 += kJ / 2) {
          if (warp >= w && warp < 2 * w)
#pragma unroll
            for (int j = 0; j < kJ / 2; j++)
#pragma unroll
              for (int n = 0; n < NB; n++)
                *reinterpret_cast<float4 *>(&sm.o[warp - w][((j * NB + n) * 32 + lane) * 4]) =
                    make_float4(o[j0 + j][n][0], o[j0 + j][n][1], o[j0 + j][n][2], o[j0 + j][n][3]);
          __syncthreads();
          if (warp < w)
#pragma unroll
            for (int j = 0; j < kJ / 2; j++)
#pragma unroll
              for (int n = 0; n < NB; n++) {
                const float4 y = *reinterpret_cast<const float4 *>(&sm.o[warp][((j * NB + n) * 32 + lane) * 4]);
                o[j0 + j][n][0] += y.x, o[j0 + j][n][1] += y.y, o[j0 + j][n][2] += y.z, o[j0 + j][n][3] += y.w;
              }
          __syncthreads();
        }
      // who has tiles of this item
      const int64_t first_tile = item_lo + skip, last_tile = item_lo + item_cost - 1;
      const int64_t c0 = ((first_tile + 1) * ctas - 1) / total, c1 = ((last_tile + 1) * ctas - 1) / total;
      if (warp == 0) {
        // slot 1: the CTA's last part, where another came before it
        const bool second = seg > 0;
        float *part = a.parts + (2 * int64_t(blockIdx.x) + second) * kRows * (D + 2);
#pragma unroll
        for (int n = 0; n < NB; n++)
#pragma unroll
          for (int i = 0; i < 2; i++) {
            const int r = 8 * n + 2 * t + i;
            float y[kMine];
#pragma unroll
            for (int c = 0; c < kMine; c++) y[c] = o[c / 2][n][2 * (c & 1) + i];
            if (c0 == c1) {
              if (r0 + r < a.rows) write_row<BF16>(a, cur.b, h, r0 + r, y, kMine * g, top[n][i], sum[n][i], g == 0);
            } else {
#pragma unroll
              for (int c = 0; c < kMine; c += 4)
                *reinterpret_cast<float4 *>(part + r * D + kMine * g + c) = make_float4(y[c], y[c + 1], y[c + 2], y[c + 3]);
              if (g == 0) part[kRows * D + r] = top[n][i], part[kRows * D + kRows + r] = sum[n][i];
            }
          }
        if (c0 != c1 && lane == 0 && int64_t(blockIdx.x) == c0) {
          Note &note = a.notes[blockIdx.x];
          note.parts = int(c1 - c0 + 1), note.second = second, note.b = cur.b, note.h = h, note.rt = cur.rt;
        }
      }
      first = true;
      seg++;
      item_lo += item_cost;
      if (u + 1 < units) {
        next_item(a, sm.len, cur);
        item_cost = cost_of(cur.tiles);
      }
    } else {
      cur.tile++;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  if (sm.dead)  // what is in flight gets a moment to land
    for (int i = 0; i < 1000; i++) __nanosleep(1000);
  if (threadIdx.x == 0) a.notes[blockIdx.x].errors = sm.errors;
}

// Joins the parts of items that several CTAs had: one CTA per CTA that has the
// first part of such an item, and four rows; a warp per row, four channels a
// lane, sixteen parts' loads in flight.  It is launched with the first kernel
// and waits for its end here.
template <int D, int NB, bool BF16>
__global__ void __launch_bounds__(128) k_join(const __grid_constant__ AttendArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kRows = Shape<NB>::kRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && blockIdx.y == 0) {  // the status of the call
    __shared__ uint32_t s_errors;
    if (threadIdx.x == 0) s_errors = 0;
    __syncthreads();
    uint32_t e = 0;
    for (int i = threadIdx.x; i < int(gridDim.x); i += 128) e |= __ldcg(&a.notes[i].errors);
    if (e) atomicOr(&s_errors, e);
    __syncthreads();
    if (threadIdx.x == 0) *a.status = s_errors;
  }
  const Note note = a.notes[blockIdx.x];
  const int r = blockIdx.y * 4 + warp, row = note.rt * kRows + r;
  if (note.parts == 0 || row >= a.rows) return;
  auto part = [&](int i) { return a.parts + (2 * (int64_t(blockIdx.x) + i) + (i == 0 ? note.second : 0)) * kRows * (D + 2); };
  float top = -INFINITY, sum = 0.0f, y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int base = 0; base < note.parts; base += 32) {
    const int n = min(32, note.parts - base);
    float m = -INFINITY, l = 0.0f;  // lane i: of part base + i
    if (lane < n) m = __ldcg(part(base + lane) + kRows * D + r), l = __ldcg(part(base + lane) + kRows * D + kRows + r);
    float now = m;
#pragma unroll
    for (int o = 16; o; o >>= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, o));
    now = fmaxf(now, top);
    const float keep = top == -INFINITY ? 0.0f : ex2(top - now);
    const float w = m == -INFINITY ? 0.0f : ex2(m - now);
    top = now;
    sum *= keep;
#pragma unroll
    for (int k = 0; k < 4; k++) y[k] *= keep;
    float lw = l * w;  // of a part that saw nothing 0, of one with a NaN a NaN
#pragma unroll
    for (int o = 16; o; o >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, o);
    sum += lw;
    for (int i0 = 0; i0 < n; i0 += 16) {
      float4 v[16];
#pragma unroll
      for (int i = 0; i < 16; i++)
        if (i0 + i < n && lane * 4 < D) v[i] = __ldcg(reinterpret_cast<const float4 *>(part(base + i0 + i) + r * D) + lane);
#pragma unroll
      for (int i = 0; i < 16; i++)
        if (i0 + i < n) {
          const float f = __shfl_sync(0xffffffffu, w, i0 + i);
          if (lane * 4 < D) y[0] += f * v[i].x, y[1] += f * v[i].y, y[2] += f * v[i].z, y[3] += f * v[i].w;
        }
    }
  }
  const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int t = row / a.G;
  const int64_t at = (int64_t(note.b) * a.T + t) * a.Hq + note.h * a.G + row % a.G;
  if (lane * 4 < a.d) {
    const uint32_t w0 = uint32_t(elem_of<BF16>(y[0] * f)) | uint32_t(elem_of<BF16>(y[1] * f)) << 16;
    const uint32_t w1 = uint32_t(elem_of<BF16>(y[2] * f)) | uint32_t(elem_of<BF16>(y[3] * f)) << 16;
    *reinterpret_cast<uint2 *>(a.out + at * a.d + lane * 4) = make_uint2(w0, w1);
  }
  if (lane == 0 && a.lse) a.lse[at] = sum == 0.0f ? -INFINITY : (top - kLift + log2f(sum)) * 0.6931471805599453f;
}

int blocks(const cg_cache *c, const cg_attend *t) { return int64_t(t->q_tokens) * (t->Hq / c->H) <= 8 ? 1 : 2; }

int row_tiles(const cg_cache *c, const cg_attend *t) {
  const int rows = 8 * blocks(c, t);
  return int((int64_t(t->q_tokens) * (t->Hq / c->H) + rows - 1) / rows);
}

bool attend_ok(const cg_cache *c, const cg_attend *t) {
  if (!cache8_ok(c) || !t || t->n_seq < 1 || t->q_tokens < 1 || t->Hq < 1 || t->Hq % c->H || t->table_stride < 1 ||
      (t->dtype != CG_F16 && t->dtype != CG_BF16) || !std::isfinite(t->scale) || !(t->scale > 0.0f))
    return false;
  for (int64_t s : t->q_stride)
    if (s % 8) return false;
  return int64_t(t->table_stride) * c->block_tokens <= (1 << 30) && t->n_seq <= (1 << 20) && t->q_tokens <= (1 << 16) && t->Hq <= 65535 &&
         int64_t(t->q_tokens) * (t->Hq / c->H) <= (1 << 28) && int64_t(t->n_seq) * c->H * row_tiles(c, t) <= (1 << 28);
}

// the status word, then the notes
constexpr uint64_t kNotes = 256 + ((sizeof(Note) * kMostCtas + 255) & ~uint64_t(255));

int padded(int d) { return d <= 64 ? 64 : 128; }

template <int FMT, int D, int NB, bool BF16, bool PLAIN>
cudaError_t launch_kernels(const AttendArgs &a, unsigned grid, cudaStream_t st) {
  constexpr int kSmem = int(sizeof(Smem<D, NB>));
  const cudaError_t e = cudaFuncSetAttribute(k_attend<FMT, D, NB, BF16, PLAIN>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  k_attend<FMT, D, NB, BF16, PLAIN><<<grid, kThreads, kSmem, st>>>(a);
  const cudaError_t e2 = launch_early(k_join<D, NB, BF16>, dim3(grid, unsigned((min(8 * NB, a.rows) + 3) / 4)), dim3(128), 0, st, a);
  return e2 != cudaSuccess ? e2 : cudaGetLastError();
}

template <int FMT, int D, int NB>
cudaError_t launch_type(const AttendArgs &a, bool bf16, int64_t units, cudaStream_t st) {
  const unsigned grid = unsigned(units < Shape<NB>::kGrid ? units : Shape<NB>::kGrid);
  if (a.plain)
    return bf16 ? launch_kernels<FMT, D, NB, true, true>(a, grid, st) : launch_kernels<FMT, D, NB, false, true>(a, grid, st);
  return bf16 ? launch_kernels<FMT, D, NB, true, false>(a, grid, st) : launch_kernels<FMT, D, NB, false, false>(a, grid, st);
}

template <int FMT>
cudaError_t launch_format(const AttendArgs &a, bool bf16, int64_t units, cudaStream_t st) {
  const bool one = a.rows <= 8;
  // (64 channels and pages of 64, four readers of 131072: 139 us as they are, 266 us padded to 128)
  if (a.d <= 64) return one ? launch_type<FMT, 64, 1>(a, bf16, units, st) : launch_type<FMT, 64, 2>(a, bf16, units, st);
  return one ? launch_type<FMT, 128, 1>(a, bf16, units, st) : launch_type<FMT, 128, 2>(a, bf16, units, st);
}

}  // namespace
}  // namespace cg

extern "C" size_t cg_cache_workspace_bytes(const cg_cache *cache, const cg_attend *attend) {
  using namespace cg;
  if (!attend_ok(cache, attend)) return 0;
  return size_t(kNotes + 4 * uint64_t(2 * kMostCtas) * 8 * blocks(cache, attend) * (padded(cache->d) + 2));
}

extern "C" cg_status cg_cache_attend(const cg_cache *cache, const cg_attend *attend, const void *q_dev,
                                     const void *k_pool, const void *v_pool, const float *k_scale,
                                     const float *v_scale, const int32_t *table_dev, const int32_t *len_dev,
                                     void *out_dev, float *lse_dev, void *ws_dev, size_t ws_bytes, void *stream) {
  using namespace cg;
  if (!attend_ok(cache, attend) || !q_dev || !k_pool || !v_pool || !k_scale || !v_scale || !table_dev || !len_dev ||
      !out_dev || !ws_dev)
    return CG_ERR_INVALID_ARG;
  if (!is_aligned(q_dev, 16) || !is_aligned(k_pool, 16) || !is_aligned(v_pool, 16) || !is_aligned(out_dev, 16) ||
      !is_aligned(k_scale, 4) || !is_aligned(v_scale, 4) || !is_aligned(table_dev, 4) || !is_aligned(len_dev, 4) ||
      !is_aligned(lse_dev, 4) || !is_aligned(ws_dev, 256) ||
      ws_bytes < cg_cache_workspace_bytes(cache, attend))
    return CG_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t *ws = static_cast<uint8_t *>(ws_dev);
  AttendArgs a{};
  a.q = static_cast<const uint16_t *>(q_dev);
  a.kp = static_cast<const uint8_t *>(k_pool), a.vp = static_cast<const uint8_t *>(v_pool);
  a.ks = k_scale, a.vs = v_scale, a.table = table_dev, a.len = len_dev;
  a.out = static_cast<uint16_t *>(out_dev), a.lse = lse_dev;
  a.status = reinterpret_cast<uint32_t *>(ws);
  a.notes = reinterpret_cast<Note *>(ws + 256);
  a.parts = reinterpret_cast<float *>(ws + kNotes);
  a.q_seq = attend->q_stride[0], a.q_tok = attend->q_stride[1], a.q_head = attend->q_stride[2];
  a.B = attend->n_seq, a.T = attend->q_tokens, a.Hq = attend->Hq, a.H = cache->H, a.d = cache->d;
  a.G = a.Hq / a.H, a.rows = a.T * a.G, a.RT = row_tiles(cache, attend), a.HR = a.H * a.RT;
  a.bt = cache->block_tokens, a.n_blocks = cache->n_blocks, a.stride = attend->table_stride;
  a.scale_log2 = attend->scale * 1.4426950408889634f;
  a.by_bt = Divisor(uint32_t(a.bt));
  const int64_t most = (int64_t(a.stride) * a.bt + kUnit - 1) / kUnit;  // units of an item
  const int64_t items = int64_t(a.B) * a.HR, units = most >= kMostCtas ? kMostCtas : items * most;
  const int64_t rows = int64_t(a.n_blocks) * a.H * a.bt;
  a.plain = a.bt % 16 == 0 && (a.d == 64 || a.d == 128) && rows <= 0x7fffffff;
  if (a.plain) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return CG_ERR_CUDA;
    const cuuint64_t dims[2] = {cuuint64_t(a.d), cuuint64_t(rows)}, strides[1] = {cuuint64_t(a.d)};
    const cuuint32_t box[2] = {cuuint32_t(a.d), 16}, ones[2] = {1, 1};
    for (int i = 0; i < 2; i++)
      if (encode(i ? &a.v_map : &a.k_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(i ? a.vp : a.kp), dims, strides, box,
                 ones, CU_TENSOR_MAP_INTERLEAVE_NONE, a.d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return CG_ERR_CUDA;
  }
  const bool bf16 = attend->dtype == CG_BF16;
  const cudaError_t e = cache->format == CG_CACHE_E4M3 ? launch_format<CG_CACHE_E4M3>(a, bf16, units, st)
                                                       : launch_format<CG_CACHE_INT8>(a, bf16, units, st);
  return e == cudaSuccess ? CG_OK : CG_ERR_CUDA;
}
