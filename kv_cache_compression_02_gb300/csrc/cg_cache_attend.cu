// cg_cache_attend.cu -- cg_cache_attend: new tokens attend over 8-bit pages.
//
// For one KV head of one sequence the G = Hq / H query heads of the T new
// tokens are T * G rows that read the same keys and values, so they are rows
// of one matrix product.  Sixteen rows are a tile of mma.sync m16n8k16 (f16
// operands, fp32 sums): codes of either format are exact in f16, page scales
// are applied outside the products, on the scores (K) and on the
// probabilities (V).
//
// What bounds it is the read of the codes: 2 d bytes per token and head
// against 4 T G d operations, so the tensor cores of tcgen05, which take their
// operands from shared memory in one format, would only add a pass that
// converts codes there.  The codes go from shared memory to registers once,
// each thread 16 bytes of a row at a time, and become the operands of
// mma.sync as they are: both products leave the order of their summed index
// free, so a thread takes 16 consecutive channels of a token (K) or of two
// tokens (V) for the fragments of four or sixteen products.
//
// Work is cut into units of 128 positions of one item (sequence, head, row
// tile), and the units of the whole call are dealt in equal runs to as many
// CTAs as fit on the GPU: a long context is shared by all SMs, short ones are
// packed.  A CTA that covers only a part of an item leaves its running
// maximum, sum and output in the workspace, and a second kernel, already
// waiting when the first one ends, joins the parts in their order: the result
// does not depend on timing.
#include <type_traits>

#include "cg_cache.cuh"

namespace cg {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTok = 32;               // positions of a warp's tile
constexpr int kUnit = kTok * kWarps;   // positions of a unit
constexpr int kRows = 16;              // query rows of an item
constexpr int kStages = 2;             // tiles in flight per warp
constexpr int kPerSM = 2;              // CTAs
constexpr int kGrid = kSMs * kPerSM;
constexpr int kShort = 8;               // units of an item that one CTA takes where items are few

// A probability is held as p = 2^(s - m + kLift), and m may lag behind the
// true maximum by kLag, so that p < 2^15.  For the second product it is
// multiplied by its page's V scale over the largest so far and rounded to f16:
// 11 bits from kNormal up.  Smaller ones, rare but for sharp distributions,
// go through products of their own, raised by 2^28 each time.
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
  const uint16_t *q;
  const uint8_t *kp, *vp;
  const float *ks, *vs;
  const int32_t *table, *len;
  uint16_t *out;
  float *lse;
  uint32_t *status;
  Note *notes;      // [kGrid]: what each CTA of k_attend leaves for k_join
  float *parts;     // [2 * kGrid][kRows][D + 2]
  int64_t q_seq, q_tok, q_head;
  int B, T, Hq, H, G, RT, HR, d, bt, n_blocks, stride;  // RT: row tiles; HR: heads x row tiles
  float scale_log2;  // scale * log2(e)
  Divisor by_bt;
};

template <int D>
struct Stage {
  uint8_t k[kTok * D], v[kTok * D];
  float ks[kTok], vs[kTok];
};

template <int D>
struct Smem {
  Stage<D> ring[kWarps][kStages];
  float o[2][kRows * D];  // where warps hand their outputs over
  float m[kWarps][kRows], l[kWarps][kRows];
  uint32_t valid[kWarps][kStages];
  int64_t sum[kWarps][2], start, prefix;
  int most[kWarps], b;
  uint32_t errors;
};

// Where 16-byte chunk c of row r lies in a tile.  The reads are: K, chunks
// 0-3 (or 4-7) of rows 2i, 2i+1 by eight lanes; V, the chunks 2i, 2i+1 of
// four rows of one parity.  With this swizzle neither has a bank conflict.
template <int D>
__device__ inline int chunk_at(int r, int c) {
  if (D == 128) return r * 128 + ((c ^ ((r & 6) ^ ((r & 1) << 2))) << 4);
  return (r >> 1) * 128 + (((((r & 1) << 2) | c) ^ (r & 6)) << 4);
}

__device__ inline uint32_t smem_of(const void *p) { return uint32_t(__cvta_generic_to_shared(p)); }

template <int N>
__device__ inline void copy_async(uint32_t dst, const void *src, bool ok) {
  const int n = ok ? N : 0;  // the rest is filled with zeros
  if (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(n) : "memory");
}

__device__ inline void copy_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ inline void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ inline float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

__device__ inline float min3(float a, float b, float c) {
  float y;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// Two fp32 operations in one instruction.
__device__ inline float2 fma2(float2 a, float2 b, float2 c) {
  float2 y;
  asm("{.reg .b64 a, b, c, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7};"
      " fma.rn.f32x2 d, a, b, c; mov.b64 {%0, %1}, d;}"
      : "=f"(y.x), "=f"(y.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return y;
}
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

// A walk over the units of a call, from one item (sequence, head, row tile) to the next.
struct Walk {
  int b, h, rt, tile, tiles, len;
};

__device__ inline int length(const AttendArgs &a, int b) {
  return int(max(int64_t(0), min(int64_t(a.len[b]), int64_t(a.stride) * a.bt)));
}

__device__ inline int tiles_of(int len) { return int((uint32_t(len) + kUnit - 1) / kUnit); }

__device__ inline void set_seq(const AttendArgs &a, Walk &w) {
  w.len = length(a, w.b);
  w.tiles = tiles_of(w.len);
}

// The next item; the caller knows that there is one.
__device__ inline void next_item(const AttendArgs &a, Walk &w) {
  w.tile = 0;
  if (++w.rt < a.RT) return;
  w.rt = 0;
  if (++w.h < a.H) return;
  w.h = 0;
  do {
    w.b++;
    set_seq(a, w);
  } while (w.tiles == 0);
}

__device__ inline void step(const AttendArgs &a, Walk &w) {
  if (++w.tile == w.tiles) next_item(a, w);
}

// One row's outputs: lane t of a quad holds channels D/4 t .. D/4 t + D/4 - 1
// of row g in o[j][0], o[j][1] and of row g + 8 in o[j][2], o[j][3].
template <int D>
__device__ inline float out_at(const float (&o)[D / 8][4], int half, int i) {
  return o[i % (D / 8)][2 * half + i / (D / 8)];
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
// half a warp's tile lies in one page (one table entry, one scale and one
// address for sixteen rows) and no chunk of it is ragged.  MEASURE
template <int FMT, int D, bool BF16, bool PLAIN>
__global__ void __launch_bounds__(kThreads, kPerSM) k_attend(const AttendArgs a) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem<D> &sm = *reinterpret_cast<Smem<D> *>(smem_raw);
  constexpr int kNT = D / 8;       // output column tiles
  constexpr int kChunks = D / 16;  // 16-byte chunks of a row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x == 0) {
    sm.errors = 0;
    a.notes[blockIdx.x].parts = 0;
  }
  // The items of the call and what they cost.  An item costs its units and
  // one more (its queries' way in, the warps' join and the way out take about
  // as long).  Where items are few and short each has a CTA of its own.
  const int per = (a.B + kThreads - 1) / kThreads, b0 = threadIdx.x * per, b1 = min(a.B, b0 + per);
  int64_t cost = 0, items = 0;
  int most = 0;
  bool bad_len = false;
  for (int b = b0; b < b1; b++) {
    const int n = a.len[b];
    bad_len |= n < 0 || int64_t(n) > int64_t(a.stride) * a.bt;
    const int tiles = tiles_of(length(a, b));
    cost += tiles ? tiles + 1 : 0;
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
    if (length(a, b) == 0) {
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
  auto cost_of = [&](int tiles) { return single ? (tiles > 0) : tiles ? tiles + 1 : 0; };
  if (lo >= before && lo < before + cost) {  // one thread's sequences hold the first unit
    int64_t at = before;
    int b = b0;
    for (;; b++) {
      const int64_t n = int64_t(cost_of(tiles_of(length(a, b)))) * a.HR;
      if (lo < at + n) break;
      at += n;
    }
    sm.b = b;
    sm.prefix = at;
  }
  if (!PLAIN && a.d < D) {  // channels that no copy fills
    uint4 *z = reinterpret_cast<uint4 *>(sm.ring[warp]);
    for (int i = lane; i < int(sizeof(sm.ring[warp]) / 16); i += 32) z[i] = make_uint4(0, 0, 0, 0);
  }
  __syncthreads();

  Walk cur;
  cur.b = sm.b;
  set_seq(a, cur);
  int item_cost = cost_of(cur.tiles);
  const int item0 = int((lo - sm.prefix) / item_cost);
  cur.h = item0 / a.RT, cur.rt = item0 % a.RT;
  int64_t item_lo = sm.prefix + int64_t(item0) * item_cost;  // where the item's cost begins
  // A run [lo, hi) of costs has the tiles whose costs lie in it; an item's
  // first cost is no tile.
  const int skip = single ? 0 : 1;
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
      units += int(max(int64_t(0), end - w_lo - 1) - max(int64_t(0), at - w_lo - 1));
      at = end;
      if (at < hi) {
        w_lo += w_cost;
        next_item(a, w);
        w_cost = w.tiles + 1;
      }
    }
  }
  Walk ahead = cur;

  // The page of row `lane` of the warp's tile in the unit that `ahead` stands
  // at; PLAIN: that of the lane's half of the tile.
  const int d = PLAIN ? D : a.d;
  const int64_t page_elems = int64_t(a.H) * a.bt * d;
  int page = -1, slot = 0, page_h = 0, have_rows = 0;
  auto find_page = [&]() {
    const uint32_t tok0 = uint32_t(ahead.tile) * kUnit + warp * kTok, tok = tok0 + (PLAIN ? lane & 16 : lane);
    page = -1;
    page_h = ahead.h;
    have_rows = ahead.len - int(tok0);
    if (tok < uint32_t(ahead.len)) {
      const uint32_t blk = a.by_bt(tok);
      slot = int(tok - blk * a.bt);
      page = a.table[int64_t(ahead.b) * a.stride + blk];
      if (uint32_t(page) >= uint32_t(a.n_blocks)) {
        atomicOr(&sm.errors, kStBadArg);
        page = -1;
      }
    }
  };
  auto issue = [&](int s) {
    Stage<D> &st = sm.ring[warp][s];
    const bool ok = page >= 0;
    const int64_t off = ok ? page * page_elems + (int64_t(page_h) * a.bt + slot) * d : 0;
    const int64_t sc_at = ok ? int64_t(page) * a.H + page_h : 0;
    const int c = lane % kChunks, r0 = lane / kChunks;
    const uint32_t pages = __ballot_sync(0xffffffffu, ok);
    uint32_t valid = pages;
    if (PLAIN) {  // the rows that are there, of the pages that are right
      valid &= have_rows >= kTok ? 0xffffffffu : have_rows <= 0 ? 0u : (1u << have_rows) - 1;
      if ((lane & 15) < 2) copy_async<4>(smem_of((lane & 1 ? st.vs : st.ks) + (lane >> 4)), (lane & 1 ? a.vs : a.ks) + sc_at, ok);
    } else {
      copy_async<4>(smem_of(&st.ks[lane]), a.ks + sc_at, ok);
      copy_async<4>(smem_of(&st.vs[lane]), a.vs + sc_at, ok);
    }
    if (lane == 0) sm.valid[warp][s] = valid;
    constexpr int kStep = 32 / kChunks;  // rows of one copy
    if (PLAIN && valid == 0xffffffffu) {  // all there: addresses that differ by constants
      const int64_t h0 = __shfl_sync(0xffffffffu, off, 0) + r0 * D + c * 16, h1 = __shfl_sync(0xffffffffu, off, 16) + r0 * D + c * 16;
      const uint8_t *k0 = a.kp + h0, *k1 = a.kp + h1, *v0 = a.vp + h0, *v1 = a.vp + h1;
#pragma unroll
      for (int i = 0; i < kTok / kStep; i++) {
        const int to = chunk_at<D>(i * kStep + r0, c), at = i * kStep % 16 * D;
        copy_async16(smem_of(st.k + to), (i * kStep < 16 ? k0 : k1) + at);
        copy_async16(smem_of(st.v + to), (i * kStep < 16 ? v0 : v1) + at);
      }
      return;
    }
    const int64_t half0 = __shfl_sync(0xffffffffu, off, 0) + r0 * d + c * 16;
    const int64_t half1 = __shfl_sync(0xffffffffu, off, 16) + r0 * d + c * 16;
#pragma unroll
    for (int i = 0; i < kTok / kStep; i++) {
      const int r = i * kStep + r0, to = chunk_at<D>(r, c);
      const bool have = valid >> r & 1;
      if (PLAIN) {
        int64_t at = (i * kStep < 16 ? half0 : half1) + i * kStep % 16 * D;
        if (!have) at = 0;
        copy_async<16>(smem_of(st.k + to), a.kp + at, have);
        copy_async<16>(smem_of(st.v + to), a.vp + at, have);
      } else {
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
  };
  int issued = 0;
  find_page();
#pragma unroll
  for (int s = 0; s < kStages - 1; s++) {
    if (issued < units) {
      issue(s);
      issued++;
      if (issued < units) {
        step(a, ahead);
        find_page();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }

  uint32_t q[D / 16][4];
  float o[kNT][4], m[2], sc[2];
  float2 l[2];  // sums of the even and the odd positions
  int last[2], v_exp = 1;  // O is in units of 2^(v_exp - 127), the largest V scale so far
  bool first = true;
  int seg = 0;  // items begun before
  int slot_now = 0, slot_next = kStages - 1;  // of the ring
  for (int u = 0; u < units; u++) {
    const int h = cur.h, r0 = cur.rt * kRows;
    if (first) {  // a new item: its query rows
      first = false;
#pragma unroll
      for (int half = 0; half < 2; half++) {
        const int r = r0 + g + 8 * half, tt = r / a.G;
        const bool ok = r < a.T * a.G;
        const uint16_t *src = a.q + cur.b * a.q_seq + tt * a.q_tok + int64_t(h * a.G + r % a.G) * a.q_head;
        last[half] = ok ? cur.len - a.T + tt : 0x7fffffff;  // a row of padding may see anything
        uint4 w[D / 32];
#pragma unroll
        for (int c = 0; c < D / 32; c++) {  // channels 64 (c / 2) + 16 t + 8 (c % 2) ...
          const int ch = 64 * (c >> 1) + 16 * t + 8 * (c & 1);
          w[c] = ok && ch < a.d ? *reinterpret_cast<const uint4 *>(src + ch) : make_uint4(0, 0, 0, 0);
        }
        sc[half] = a.scale_log2;
        if (BF16) {  // to f16, exactly but for what is under 2^-38 of the row's largest
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
          sc[half] *= __int_as_float((254 - f) << 23);
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
        for (int c = 0; c < D / 64; c++) {
          q[4 * c][half] = w[2 * c].x, q[4 * c][half + 2] = w[2 * c].y;
          q[4 * c + 1][half] = w[2 * c].z, q[4 * c + 1][half + 2] = w[2 * c].w;
          q[4 * c + 2][half] = w[2 * c + 1].x, q[4 * c + 2][half + 2] = w[2 * c + 1].y;
          q[4 * c + 3][half] = w[2 * c + 1].z, q[4 * c + 3][half + 2] = w[2 * c + 1].w;
        }
        m[half] = -INFINITY;
        l[half] = make_float2(0.0f, 0.0f);
      }
#pragma unroll
      for (int j = 0; j < kNT; j++) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
      v_exp = 1;
    }

    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();
    const int s = slot_now;
    slot_now = slot_now + 1 == kStages ? 0 : slot_now + 1;
    if (issued < units) {
      issue(slot_next);
      issued++;
      if (issued < units) {
        step(a, ahead);
        find_page();
      }
    }
    slot_next = slot_next + 1 == kStages ? 0 : slot_next + 1;
    asm volatile("cp.async.commit_group;" ::: "memory");

    const Stage<D> &st = sm.ring[warp][s];
    const uint32_t valid = sm.valid[warp][s];
    const uint32_t tok0 = uint32_t(cur.tile) * kUnit + warp * kTok;
    if (valid) {
      // S = Q K^T: positions 8 n + 2 t, 8 n + 2 t + 1 of rows g and g + 8
      constexpr int kN = kTok / 8;
      float x[kN][4], vs[kN][2];
#pragma unroll
      for (int n = 0; n < kN; n++) {
        x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.0f;
#pragma unroll
        for (int c = 0; c < D / 64; c++) {
          const uint4 w = *reinterpret_cast<const uint4 *>(st.k + chunk_at<D>(8 * n + g, 4 * c + t));
          const uint32_t y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int k = 0; k < 4; k++) {
            const uint32_t z = biased<FMT>(y[k]);
            mma(x[n], q[4 * c + k], halves_of<FMT, 0>(z), halves_of<FMT, 1>(z));
          }
        }
      }
      float f[kN / 2][2];  // PLAIN: what turns a product into a score, for each half of the tile and of the rows
#pragma unroll
      for (int n = 0; n < kN; n++) {
        if (PLAIN) {
          const float ks = st.ks[n >> 1];
          f[n >> 1][0] = ks * sc[0], f[n >> 1][1] = ks * sc[1];
          vs[n][0] = vs[n][1] = st.vs[n >> 1];
        } else {
          const float2 ks = *reinterpret_cast<const float2 *>(&st.ks[8 * n + 2 * t]);
          const float2 v2 = *reinterpret_cast<const float2 *>(&st.vs[8 * n + 2 * t]);
          vs[n][0] = v2.x, vs[n][1] = v2.y;
          x[n][0] *= ks.x * sc[0], x[n][1] *= ks.y * sc[0];
          x[n][2] *= ks.x * sc[1], x[n][3] *= ks.y * sc[1];
          f[n >> 1][0] = f[n >> 1][1] = 1.0f;
        }
      }
      // whether every position is there and every row sees it
      const bool whole = valid == 0xffffffffu && int(tok0) + kTok - 1 <= cur.len - a.T;
      uint32_t seen = 0xffffu;  // bit 4 n + 2 half + i
      if (!whole) {
        seen = 0;
#pragma unroll
        for (int n = 0; n < kN; n++)
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const int p = 8 * n + 2 * t + (i & 1);
            const bool sees = (valid >> p & 1) && int(tok0) + p <= last[i >> 1];
            seen |= uint32_t(sees) << (4 * n + i);
            x[n][i] = sees ? x[n][i] * f[n >> 1][i >> 1] : -INFINITY;
          }
#pragma unroll
        for (int n = 0; n < kN / 2; n++) f[n][0] = f[n][1] = 1.0f;
      }
      float keep[2];
      bool moved = false;
#pragma unroll
      for (int half = 0; half < 2; half++) {
        float top = -INFINITY;
#pragma unroll
        for (int n = 0; n < kN; n += 2) {
          const float y = max3(x[n][2 * half], x[n][2 * half + 1], fmaxf(x[n + 1][2 * half], x[n + 1][2 * half + 1]));
          top = fmaxf(top, y * f[n >> 1][half]);
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        keep[half] = 1.0f;
        if (top > m[half] + kLag) {
          keep[half] = ex2(m[half] - top);
          m[half] = top;
          moved = true;
        }
      }
      float vmax = fabsf(vs[0][0]);
#pragma unroll
      for (int n = PLAIN ? 2 : 0; n < kN; n += PLAIN ? 2 : 1) vmax = fmaxf(vmax, fmaxf(fabsf(vs[n][0]), fabsf(vs[n][1])));
      if (!PLAIN) {
        vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, 1));
        vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, 2));
      }
      const int e = min(254, int(__float_as_uint(vmax) >> 23) + 1);
      float down = 1.0f;
      if (e > v_exp) {  // the same in every lane
        down = e - v_exp > 126 ? 0.0f : __int_as_float((127 + v_exp - e) << 23);
        v_exp = e;
        moved = true;
      }
      if (__any_sync(0xffffffffu, moved)) {
        l[0].x *= keep[0], l[0].y *= keep[0], l[1].x *= keep[1], l[1].y *= keep[1];
        const float f0 = keep[0] * down, f1 = keep[1] * down;
#pragma unroll
        for (int j = 0; j < kNT; j++) o[j][0] *= f0, o[j][1] *= f0, o[j][2] *= f1, o[j][3] *= f1;
      }
      const float unit = __int_as_float((254 - v_exp) << 23);
      float least = INFINITY;  // of the probabilities
#pragma unroll
      for (int half = 0; half < 2; half++) {
        const float base = kLift - (m[half] == -INFINITY ? 0.0f : m[half]);
#pragma unroll
        for (int n = 0; n < kN; n++) {
          float2 y = make_float2(x[n][2 * half], x[n][2 * half + 1]);
          const float g1 = f[n >> 1][half];
          y = fma2(y, make_float2(g1, g1), make_float2(base, base));
          y = make_float2(ex2(y.x), ex2(y.y));
          l[half] = add2(l[half], y);
          y = mul2(y, make_float2(vs[n][0] * unit, vs[n][1] * unit));
          x[n][2 * half] = y.x, x[n][2 * half + 1] = y.y;
          least = min3(least, fabsf(y.x), fabsf(y.y));
        }
      }
      if (!whole) {  // 0 * NaN
#pragma unroll
        for (int n = 0; n < kN; n++)
#pragma unroll
          for (int i = 0; i < 4; i++)
            if (!(seen >> (4 * n + i) & 1)) x[n][i] = 0.0f;
      }
      uint32_t pf[kN / 2][4];
      auto to_half = [&](auto keep_small) {
#pragma unroll
        for (int n = 0; n < kN; n++)
#pragma unroll
          for (int half = 0; half < 2; half++) {
            float p0 = x[n][2 * half], p1 = x[n][2 * half + 1];
            if (!keep_small.value) p0 = fabsf(p0) < kNormal ? 0.0f : p0, p1 = fabsf(p1) < kNormal ? 0.0f : p1;
            pf[n >> 1][2 * (n & 1) + half] = pack(p0, p1);
          }
      };
      const bool small = __any_sync(0xffffffffu, least < kNormal);
      if (small)
        to_half(std::false_type());
      else
        to_half(std::true_type());

      // O += P V, sixteen positions at a time: column tile j is channel (D / 8) g + j
      constexpr int kWords = D / 32;  // words of a token that a lane takes
      auto load_v = [&](int s16, uint32_t (&w)[4][kWords]) {  // positions 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int r = 16 * s16 + 2 * t + (i & 1) + 8 * (i >> 1);
          if (D == 128) {
            const uint4 y = *reinterpret_cast<const uint4 *>(st.v + chunk_at<D>(r, g));
            w[i][0] = y.x, w[i][1] = y.y, w[i][kWords - 2] = y.z, w[i][kWords - 1] = y.w;
          } else {
            const uint2 y = *reinterpret_cast<const uint2 *>(st.v + chunk_at<D>(r, g >> 1) + 8 * (g & 1));
            w[i][0] = y.x, w[i][1] = y.y;
          }
        }
      };
      // the products of four column tiles with P
      auto product = [&](const uint32_t (&w)[4][kWords], int k, const uint32_t (&p)[4], float (&c)[4][4]) {
        uint32_t z[4];
#pragma unroll
        for (int i = 0; i < 4; i++) z[i] = biased<FMT>(w[i][k]);
        const uint32_t a01 = __byte_perm(z[0], z[1], 0x5140), a23 = __byte_perm(z[0], z[1], 0x7362);
        const uint32_t b01 = __byte_perm(z[2], z[3], 0x5140), b23 = __byte_perm(z[2], z[3], 0x7362);
        mma(c[0], p, halves_of<FMT, 0>(a01), halves_of<FMT, 0>(b01));
        mma(c[1], p, halves_of<FMT, 1>(a01), halves_of<FMT, 1>(b01));
        mma(c[2], p, halves_of<FMT, 0>(a23), halves_of<FMT, 0>(b23));
        mma(c[3], p, halves_of<FMT, 1>(a23), halves_of<FMT, 1>(b23));
      };
      bool odd = false;
#pragma unroll
      for (int s16 = 0; s16 < kN / 2; s16++) {
        uint32_t w[4][kWords];
        load_v(s16, w);
        if (FMT == CG_CACHE_E4M3 && !whole && a.T > 1) {
          // A NaN code behind a row's last position must not reach that row
          // through 0 * NaN: such codes are taken out of the product, and a
          // product of "sees" and "is NaN" says which outputs are NaN.
          uint32_t any = 0;
#pragma unroll
          for (int i = 0; i < 4; i++)
#pragma unroll
            for (int k = 0; k < kWords; k++) any |= __vcmpeq4(w[i][k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
          odd |= __any_sync(0xffffffffu, any != 0);
        }
        if (odd) {
          const uint32_t one = 0x3c00u;
          uint32_t sees[4];
#pragma unroll
          for (int n = 0; n < 2; n++)
#pragma unroll
            for (int half = 0; half < 2; half++) {
              const uint32_t b = seen >> (4 * (2 * s16 + n) + 2 * half);
              sees[2 * n + half] = (b & 1 ? one : 0) | (b & 2 ? one << 16 : 0);
            }
#pragma unroll
          for (int k = 0; k < kWords; k++) {
            uint32_t z[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
              z[i] = __vcmpeq4(w[i][k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
              w[i][k] &= ~z[i];
            }
#pragma unroll
            for (int c = 0; c < 4; c++) {
              const uint32_t n0 = (z[0] >> (8 * c) & 1 ? one : 0) | (z[1] >> (8 * c) & 1 ? one << 16 : 0);
              const uint32_t n1 = (z[2] >> (8 * c) & 1 ? one : 0) | (z[3] >> (8 * c) & 1 ? one << 16 : 0);
              float hit[4] = {0.0f, 0.0f, 0.0f, 0.0f};
              mma(hit, sees, n0, n1);
#pragma unroll
              for (int i = 0; i < 4; i++)
                if (hit[i] > 0.0f) o[4 * k + c][i] = __int_as_float(0x7fffffff);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < kWords; k++) product(w, k, pf[s16], reinterpret_cast<float(&)[4][4]>(o[4 * k]));
      }
      if (small) {
        float fall = 1.0f;
#pragma unroll 1
        for (int pass = 0; pass < 4; pass++) {  // to 2^-126
          fall *= 0x1p-28f;
          bool have = false;
#pragma unroll
          for (int n = 0; n < kN; n++)
#pragma unroll
            for (int i = 0; i < 4; i++) {  // what the last product had goes, the rest is raised
              x[n][i] = fabsf(x[n][i]) < kNormal ? x[n][i] * 0x1p28f : 0.0f;
              have |= x[n][i] != 0.0f;
            }
          if (!__any_sync(0xffffffffu, have)) break;
          to_half(std::false_type());
#pragma unroll
          for (int s16 = 0; s16 < kN / 2; s16++) {
            uint32_t w[4][kWords];
            load_v(s16, w);
#pragma unroll
            for (int k = 0; k < kWords; k++) {
              if (odd)
#pragma unroll
                for (int i = 0; i < 4; i++) w[i][k] &= ~__vcmpeq4(w[i][k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
              float y[4][4] = {};
              product(w, k, pf[s16], y);
#pragma unroll
              for (int c = 0; c < 4; c++)
#pragma unroll
                for (int i = 0; i < 4; i++) o[4 * k + c][i] += y[c][i] * fall;
            }
          }
        }
      }
    }

    const bool end = cur.tile + 1 == cur.tiles || u + 1 == units;
    if (end) {
      // The four warps' parts of the item, joined in a fixed order.
#pragma unroll
      for (int half = 0; half < 2; half++) {
        float y = l[half].x + l[half].y;
        y += __shfl_xor_sync(0xffffffffu, y, 1);
        y += __shfl_xor_sync(0xffffffffu, y, 2);
        if (t == 0) sm.m[warp][g + 8 * half] = m[half], sm.l[warp][g + 8 * half] = y;
      }
      __syncthreads();
      float top[2], sum[2];
#pragma unroll
      for (int half = 0; half < 2; half++) {
        const int r = g + 8 * half;
        top[half] = -INFINITY;
        for (int w = 0; w < kWarps; w++) top[half] = fmaxf(top[half], sm.m[w][r]);
        sum[half] = 0.0f;
        for (int w = 0; w < kWarps; w++)
          sum[half] += sm.l[w][r] * (sm.m[w][r] == -INFINITY ? 0.0f : ex2(sm.m[w][r] - top[half]));
        const float f = (m[half] == -INFINITY ? 0.0f : ex2(m[half] - top[half])) * __int_as_float(v_exp << 23);
#pragma unroll
        for (int j = 0; j < kNT; j++) o[j][2 * half] *= f, o[j][2 * half + 1] *= f;
      }
#pragma unroll
      for (int w = kWarps / 2; w; w >>= 1) {  // warps w .. 2w-1 hand theirs to 0 .. w-1
        if (warp >= w && warp < 2 * w)
#pragma unroll
          for (int j = 0; j < kNT; j++)
            *reinterpret_cast<float4 *>(&sm.o[warp - w][(j * 32 + lane) * 4]) = make_float4(o[j][0], o[j][1], o[j][2], o[j][3]);
        __syncthreads();
        if (warp < w)
#pragma unroll
          for (int j = 0; j < kNT; j++) {
            const float4 y = *reinterpret_cast<const float4 *>(&sm.o[warp][(j * 32 + lane) * 4]);
            o[j][0] += y.x, o[j][1] += y.y, o[j][2] += y.z, o[j][3] += y.w;
          }
        __syncthreads();
      }
      // who has tiles of this item
      const int64_t first_tile = item_lo + skip, last_tile = item_lo + item_cost - 1;
      const int64_t c0 = ((first_tile + 1) * ctas - 1) / total, c1 = ((last_tile + 1) * ctas - 1) / total;
      if (c0 == c1) {
        if (warp == 0)
#pragma unroll
          for (int half = 0; half < 2; half++) {
            const int r = r0 + g + 8 * half;
            float y[D / 4];
#pragma unroll
            for (int i = 0; i < D / 4; i++) y[i] = out_at<D>(o, half, i);
            if (r < a.T * a.G) write_row<BF16>(a, cur.b, h, r, y, D / 4 * t, top[half], sum[half], t == 0);
          }
      } else if (warp == 0) {
        // slot 1: the CTA's last part, where another came before it
        const bool second = seg > 0;
        float *part = a.parts + (2 * int64_t(blockIdx.x) + second) * kRows * (D + 2);
#pragma unroll
        for (int half = 0; half < 2; half++) {
          const int r = g + 8 * half;
#pragma unroll
          for (int i = 0; i < D / 4; i += 4)
            *reinterpret_cast<float4 *>(part + r * D + D / 4 * t + i) =
                make_float4(out_at<D>(o, half, i), out_at<D>(o, half, i + 1), out_at<D>(o, half, i + 2), out_at<D>(o, half, i + 3));
          if (t == 0) part[kRows * D + r] = top[half], part[kRows * D + kRows + r] = sum[half];
        }
        if (lane == 0 && int64_t(blockIdx.x) == c0) {
          Note &note = a.notes[blockIdx.x];
          note.parts = int(c1 - c0 + 1), note.second = second, note.b = cur.b, note.h = h, note.rt = cur.rt;
        }
      }
      first = true;
      seg++;
      item_lo += item_cost;
      if (u + 1 < units) {
        next_item(a, cur);
        item_cost = cost_of(cur.tiles);
      }
    } else {
      cur.tile++;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0) a.notes[blockIdx.x].errors = sm.errors;
}

// Joins the parts of items that several CTAs had: one CTA per CTA that has the
// first part of such an item, and four rows; a warp per row, four channels a
// lane, sixteen parts' loads in flight.  It is launched with the first kernel
// and waits for its end here.
template <int D, bool BF16>
__global__ void __launch_bounds__(128) k_join(const AttendArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
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
  if (note.parts == 0 || row >= a.T * a.G) return;
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

int row_tiles(const cg_cache *c, const cg_attend *t) {
  return int((int64_t(t->q_tokens) * (t->Hq / c->H) + kRows - 1) / kRows);
}

bool attend_ok(const cg_cache *c, const cg_attend *t) {
  if (!cache8_ok(c) || !t || t->n_seq < 1 || t->q_tokens < 1 || t->Hq < 1 || t->Hq % c->H || t->table_stride < 1 ||
      (t->dtype != CG_F16 && t->dtype != CG_BF16) || !std::isfinite(t->scale) || !(t->scale > 0.0f))
    return false;
  for (int64_t s : t->q_stride)
    if (s % 8) return false;
  return t->n_seq <= (1 << 20) && t->q_tokens <= (1 << 16) && t->Hq <= 65535 &&
         int64_t(t->q_tokens) * (t->Hq / c->H) <= (1 << 28) && int64_t(t->n_seq) * c->H * row_tiles(c, t) <= (1 << 28);
}

constexpr uint64_t kNotes = 256 + ((sizeof(Note) * kGrid + 255) & ~uint64_t(255));  // the status word, then the notes

int padded(int d) { return d <= 64 ? 64 : 128; }

template <int FMT, int D, bool BF16, bool PLAIN>
cudaError_t launch_kernel(const AttendArgs &a, unsigned grid, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(k_attend<FMT, D, BF16, PLAIN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             int(sizeof(Smem<D>)));
  if (e != cudaSuccess) return e;
  k_attend<FMT, D, BF16, PLAIN><<<grid, kThreads, sizeof(Smem<D>), st>>>(a);
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, unsigned((min(kRows, a.T * a.G) + 3) / 4)), cfg.blockDim = dim3(128), cfg.stream = st;
  cfg.attrs = &early, cfg.numAttrs = 1;
  const cudaError_t e2 = cudaLaunchKernelEx(&cfg, k_join<D, BF16>, a);
  return e2 != cudaSuccess ? e2 : cudaGetLastError();
}

template <int FMT, int D, bool BF16>
cudaError_t launch(const AttendArgs &a, unsigned grid, cudaStream_t st) {
  return a.bt % 16 == 0 && a.d == D ? launch_kernel<FMT, D, BF16, true>(a, grid, st)
                                    : launch_kernel<FMT, D, BF16, false>(a, grid, st);
}

template <int FMT>
cudaError_t launch_format(const AttendArgs &a, bool bf16, unsigned grid, cudaStream_t st) {
  if (a.d <= 64) return bf16 ? launch<FMT, 64, true>(a, grid, st) : launch<FMT, 64, false>(a, grid, st);
  return bf16 ? launch<FMT, 128, true>(a, grid, st) : launch<FMT, 128, false>(a, grid, st);
}

}  // namespace
}  // namespace cg

extern "C" size_t cg_cache_workspace_bytes(const cg_cache *cache, const cg_attend *attend) {
  using namespace cg;
  if (!attend_ok(cache, attend)) return 0;
  return size_t(kNotes + 4 * uint64_t(2 * kGrid) * kRows * (padded(cache->d) + 2));
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
  a.G = a.Hq / a.H, a.RT = row_tiles(cache, attend), a.HR = a.H * a.RT;
  a.bt = cache->block_tokens, a.n_blocks = cache->n_blocks, a.stride = attend->table_stride;
  a.scale_log2 = attend->scale * 1.4426950408889634f;
  a.by_bt = Divisor(uint32_t(a.bt));
  const int64_t most = (int64_t(a.stride) * a.bt + kUnit - 1) / kUnit;  // units of an item
  const int64_t items = int64_t(a.B) * a.HR;
  const unsigned grid = unsigned(most >= kGrid || items * most >= kGrid ? kGrid : items * most);
  const bool bf16 = attend->dtype == CG_BF16;
  const cudaError_t e = cache->format == CG_CACHE_E4M3 ? launch_format<CG_CACHE_E4M3>(a, bf16, grid, st)
                                                       : launch_format<CG_CACHE_INT8>(a, bf16, grid, st);
  return e == cudaSuccess ? CG_OK : CG_ERR_CUDA;
}
