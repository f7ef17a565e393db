// cg_cross_few.cu -- cg_cross_attend for few query rows: one or a few tokens of
// each sequence attend to the states of an encoder or a loaded context.
//
// For one KV head of one sequence the up to 16 rows (queries x Hq / H) are one
// matrix.  Both products are taken transposed on mma.sync m16n8k16, S^T = K Q^T
// and O^T = V^T P^T, so that positions and channels fill the side of 16 and
// eight rows waste nothing.  P goes into the second product as two values of the
// rows' type, so that a weight is off by at most 2^-16 (bf16) or 2^-20 (f16) of
// itself, or by half of f16's least step: 2^-32 of the largest.
//
// What bounds it is the read of the keys and values.  A warp works by itself: it
// has tiles of 32 positions copied (TMA) two tiles ahead, a running maximum, sum
// and output of its own, and no barrier with the others.  The tiles of all items
// (sequence, KV head) are dealt in equal runs to all warps of the GPU; what a warp
// has of an item that others share goes to the workspace, and a second kernel,
// launched with the first, joins the parts in their order.
#include "cg_cross_few.cuh"

#include "cg_cache.cuh"
#include "cg_tc.cuh"
#include "cg_tma.cuh"

namespace cg {
namespace {

constexpr int kTok = 32;    // positions of a tile
constexpr int kStages = 2;  // tiles of a warp's ring
constexpr int kIn = 3;      // what an item's way in and out costs, in tiles
constexpr float kLift = 7.0f, kLag = 8.0f;  // p = 2^(s - m + kLift) < 2^15, m at most kLag under the maximum

template <int D>
struct Shape {
  static constexpr int kWarps = D == 64 ? 12 : 6;  // 192 KB of tiles
  static constexpr int kThreads = 32 * kWarps, kRuns = kSMs * kWarps;
};
constexpr int kMostRuns = Shape<64>::kRuns;

// An item that a warp has the first but not the last part of (parts = 0: none).
struct Note {
  int32_t parts;   // in this warp and the next ones
  int32_t second;  // the first part is in this warp's second slot
  int32_t b, h;
};

struct FewArgs {
  CUtensorMap k_map, v_map;
  const uint16_t *q;
  const int32_t *cu_q, *k_begin, *k_len;
  uint16_t *out;
  float *lse;
  uint32_t *status, *errors;  // errors: [kSMs], of each CTA
  Note *notes;                // [runs]
  float *parts;               // [2 * runs][kFewRows][D + 2]
  int64_t q_row, q_head;
  int n_seq, Hq, H, G, d, max_q, max_k, n_q, n_k;
  float scale_log2;  // scale * log2(e)
};

template <int D>
struct Smem {
  static constexpr int kChunks = D / 64;  // of 64 channels: 128 bytes, a swizzled row
  uint8_t ring[Shape<D>::kWarps][kStages][2][kChunks][kTok * 128];  // K and V
  uint64_t full[Shape<D>::kWarps][kStages];
  int64_t before[Shape<D>::kThreads], sum[Shape<D>::kWarps];
  uint32_t errors, dead;
};

struct Seq {
  int q0, nq, k0, nk, tiles;  // tiles: 0 where there is nothing to do
};

__device__ inline bool load_seq(const FewArgs &a, int b, Seq &s) {
  s.q0 = a.cu_q[b], s.k0 = a.k_begin[b], s.nk = a.k_len[b];
  const int q1 = a.cu_q[b + 1];
  s.nq = q1 - s.q0;
  const bool ok = s.q0 >= 0 && q1 >= s.q0 && q1 <= a.n_q && s.nq <= a.max_q && s.k0 >= 0 && s.nk >= 0 && s.nk <= a.max_k && int64_t(s.k0) + s.nk <= a.n_k;
  if (!ok) s.nq = 0;
  s.tiles = s.nq > 0 ? (s.nk + kTok - 1) / kTok : 0;
  return ok;
}

struct Walk {
  Seq s;
  int b, h, tile;
};

// The next item; the caller knows that there is one.
__device__ inline void next_item(const FewArgs &a, Walk &w) {
  w.tile = 0;
  if (++w.h < a.H) return;
  w.h = 0;
  do load_seq(a, ++w.b, w.s);
  while (w.s.tiles == 0);
}

template <bool BF16>
__device__ inline void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four 8 x 8 matrices; lanes 8 i ... 8 i + 7 give the addresses of the rows of the i-th.
template <bool TRANS>
__device__ inline void load_matrices(uint32_t (&x)[4], uint32_t at) {
  if (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at) : "memory");
}

// An 8 x 8 matrix of 16-bit elements, lane i with elements 2 (i % 4) and one more of row i / 4, transposed.
__device__ inline uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// NB: blocks of eight query rows.
template <int D, int NB, bool BF16>
__global__ void __launch_bounds__(Shape<D>::kThreads, 1) k_few(const __grid_constant__ FewArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem<D> &sm = *reinterpret_cast<Smem<D> *>(smem_raw);
  constexpr int kWarps = Shape<D>::kWarps, kThreads = Shape<D>::kThreads, kChunks = Smem<D>::kChunks, kJ = D / 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int me = blockIdx.x * kWarps + warp;  // this warp's run

  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x == 0) sm.errors = sm.dead = 0;
  if (lane == 0) {
    a.notes[me].parts = 0;
    for (int s = 0; s < kStages; s++) bar_init(&sm.full[warp][s], 1);
    bar_init_fence();
  }
  // What the items of the call cost: their tiles and kIn.
  const int per = (a.n_seq + kThreads - 1) / kThreads, b0 = threadIdx.x * per, b1 = min(a.n_seq, b0 + per);
  int64_t cost = 0;
  bool bad = false;
  for (int b = b0; b < b1; b++) {
    Seq s;
    bad |= !load_seq(a, b, s);
    cost += s.tiles ? s.tiles + kIn : 0;
  }
  cost *= a.H;
  int64_t cost_to = cost;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, cost_to, o);
    if (lane >= o) cost_to += y;
  }
  if (lane == 31) sm.sum[warp] = cost_to;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; w++) {
    if (w < warp) cost_to += sm.sum[w];
    total += sm.sum[w];
  }
  sm.before[threadIdx.x] = cost_to - cost;
  if (blockIdx.x == 0 && bad) atomicOr(&sm.errors, kStBadArg);
  for (int b = blockIdx.x; b < a.n_seq; b += gridDim.x) {  // queries that see no key
    Seq s;
    load_seq(a, b, s);
    if (s.nq == 0 || s.nk > 0) continue;
    const int64_t rows = int64_t(s.nq) * a.Hq, at = int64_t(s.q0) * a.Hq;
    for (int64_t i = threadIdx.x; i < rows * a.d / 8; i += kThreads) reinterpret_cast<uint4 *>(a.out + at * a.d)[i] = make_uint4(0, 0, 0, 0);
    if (a.lse)
      for (int64_t i = threadIdx.x; i < rows; i += kThreads) a.lse[at + i] = -INFINITY;
  }
  __syncthreads();
  const int64_t runs = min(int64_t(gridDim.x) * kWarps, total);
  if (me < runs) {
    const int64_t lo = total * me / runs, hi = total * (me + 1) / runs;
    // the item that holds the first cost
    int l = 0, n = kThreads;  // the last thread whose sequences begin at or before lo is one of l .. l + n - 1
    while (n > 1) {
      const int half = n / 2;
      if (sm.before[l + half] <= lo)
        l += half, n -= half;
      else
        n = half;
    }
    Walk cur;
    int64_t prefix = sm.before[l];
    for (cur.b = l * per;; cur.b++) {
      load_seq(a, cur.b, cur.s);
      const int64_t all = int64_t(cur.s.tiles ? cur.s.tiles + kIn : 0) * a.H;
      if (lo < prefix + all) break;
      prefix += all;
    }
    int item_cost = cur.s.tiles + kIn;
    cur.h = int((lo - prefix) / item_cost);
    int64_t item_lo = prefix + int64_t(cur.h) * item_cost;  // where the item's cost begins
    cur.tile = max(0, int(lo - item_lo) - kIn);
    // a run has the tiles whose costs lie in it; an item's first kIn costs are no tiles
    int tiles = 0;
    {
      Walk w = cur;
      int64_t at = lo, w_lo = item_lo;
      while (at < hi) {
        const int w_cost = w.s.tiles + kIn;
        const int64_t end = min(hi, w_lo + w_cost);
        tiles += int(max(int64_t(0), end - w_lo - kIn) - max(int64_t(0), at - w_lo - kIn));
        at = end;
        if (at < hi) {
          w_lo += w_cost;
          next_item(a, w);
        }
      }
    }
    Walk ahead = cur;
    int issued = 0;
    auto issue = [&](int s) {
      if (lane == 0) {
        bar_expect(&sm.full[warp][s], 2 * kChunks * kTok * 128);
        const int y = ahead.s.k0 + ahead.tile * kTok;
#pragma unroll
        for (int c = 0; c < kChunks; c++) {
          tma_3d(smem_of(sm.ring[warp][s][0][c]), &a.k_map, &sm.full[warp][s], 64 * c, y, ahead.h);
          tma_3d(smem_of(sm.ring[warp][s][1][c]), &a.v_map, &sm.full[warp][s], 64 * c, y, ahead.h);
        }
      }
      if (++issued < tiles && ++ahead.tile == ahead.s.tiles) next_item(a, ahead);
    };
#pragma unroll
    for (int s = 0; s < kStages; s++)
      if (issued < tiles) issue(s);

    // A lane has, of each block n of eight rows, rows 8 n + 2 t and 8 n + 2 t + 1
    // (.x and .y): scores of positions g and g + 8 of each 16, outputs of channels
    // 16 j + g and 16 j + g + 8.
    uint32_t q[NB][kJ][2];
    float o[kJ][NB][4];
    float2 m[NB], sum[NB];
    bool first = true;
    int seg = 0;  // items begun before
    uint32_t phase = 0;
    int s = 0;
    // where this lane's rows of the matrices lie: K's of positions lane % 16, V's alike, 8 channels to the right for the upper half or every other eight
    const int k_row = lane & 15, k_ch = lane >> 4, v_row = (lane & 7) + (lane >> 4 << 3), v_ch = lane >> 3 & 1;
    for (int u = 0; u < tiles; u++) {
      const int rows = cur.s.nq * a.G;
      if (first) {
        first = false;
#pragma unroll
        for (int n = 0; n < NB; n++) {
          const int r = 8 * n + g;
          const uint16_t *src = a.q + (int64_t(cur.s.q0) + r / a.G) * a.q_row + int64_t(cur.h * a.G + r % a.G) * a.q_head;
#pragma unroll
          for (int j = 0; j < kJ; j++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
              const int ch = 16 * j + 8 * i + 2 * t;
              q[n][j][i] = r < rows && ch < a.d ? *reinterpret_cast<const uint32_t *>(src + ch) : 0;
            }
          m[n] = make_float2(-INFINITY, -INFINITY), sum[n] = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int j = 0; j < kJ; j++) o[j][n][0] = o[j][n][1] = o[j][n][2] = o[j][n][3] = 0.0f;
        }
      }
      if (!bar_wait(&sm.full[warp][s], phase, &sm.dead)) {
        atomicOr(&sm.errors, kStTimeout);
        break;
      }
      __syncwarp();
      const int left = cur.s.nk - cur.tile * kTok;  // positions from the tile's first on
      if (left < kTok) {  // what lies behind the last one must not reach a product: 0 * NaN
        for (int i = lane; i < (kTok - left) * 8 * kChunks; i += 32) {
          const int r = left + i / (8 * kChunks), c = i % (8 * kChunks);
          reinterpret_cast<uint4 *>(sm.ring[warp][s][1][c / 8] + r * 128)[c % 8] = make_uint4(0, 0, 0, 0);
        }
        fence_async();
        __syncwarp();
      }
      const uint32_t k_at = smem_of(sm.ring[warp][s][0][0]), v_at = smem_of(sm.ring[warp][s][1][0]);
      // S^T = K Q^T
      float x[2][NB][4];  // [..][2 half + i]: position 16 tt + 8 half + g, row i
#pragma unroll
      for (int tt = 0; tt < 2; tt++)
#pragma unroll
        for (int n = 0; n < NB; n++) x[tt][n][0] = x[tt][n][1] = x[tt][n][2] = x[tt][n][3] = 0.0f;
#pragma unroll
      for (int j = 0; j < kJ; j++)
#pragma unroll
        for (int tt = 0; tt < 2; tt++) {
          const int r = 16 * tt + k_row, c = 2 * j + k_ch;
          uint32_t f[4];
          load_matrices<false>(f, k_at + (c >> 3) * (kTok * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
#pragma unroll
          for (int n = 0; n < NB; n++) mma<BF16>(x[tt][n], f, q[n][j][0], q[n][j][1]);
        }
      if (left < kTok) {
#pragma unroll
        for (int tt = 0; tt < 2; tt++)
#pragma unroll
          for (int n = 0; n < NB; n++)
#pragma unroll
            for (int i = 0; i < 4; i++)
              if (16 * tt + 8 * (i >> 1) + g >= left) x[tt][n][i] = -INFINITY;
      }
      bool moved = false;
      float2 keep[NB];
#pragma unroll
      for (int n = 0; n < NB; n++) {
        float2 top = make_float2(fmaxf(fmaxf(x[0][n][0], x[0][n][2]), fmaxf(x[1][n][0], x[1][n][2])),
                                 fmaxf(fmaxf(x[0][n][1], x[0][n][3]), fmaxf(x[1][n][1], x[1][n][3])));
#pragma unroll
        for (int e = 4; e < 32; e <<= 1) {
          top.x = fmaxf(top.x, __shfl_xor_sync(0xffffffffu, top.x, e));
          top.y = fmaxf(top.y, __shfl_xor_sync(0xffffffffu, top.y, e));
        }
        top.x *= a.scale_log2, top.y *= a.scale_log2;
        keep[n] = make_float2(1.0f, 1.0f);
        if (top.x > m[n].x + kLag) keep[n].x = ex2(m[n].x - top.x), m[n].x = top.x, moved = true;
        if (top.y > m[n].y + kLag) keep[n].y = ex2(m[n].y - top.y), m[n].y = top.y, moved = true;
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int n = 0; n < NB; n++) {
          sum[n] = mul2(sum[n], keep[n]);
#pragma unroll
          for (int j = 0; j < kJ; j++) o[j][n][0] *= keep[n].x, o[j][n][1] *= keep[n].y, o[j][n][2] *= keep[n].x, o[j][n][3] *= keep[n].y;
        }
      }
      // P^T as an operand, and what it leaves over: the tensor cores have the time.  It
      // is taken a little less than it is, so that the rest is above 0 where P is, too,
      // and an infinite value of V stays what it is.  In f16 a P under kHalved is
      // subnormal, or nearly: a little less may round to P itself, and it is taken in
      // halves (off by 2^-25 either way; both are above 0 where P is above 2^-23).
      uint32_t p[2][NB][2], rest[2][NB][2];
      constexpr float kLess = BF16 ? 1.0f - 0x1p-8f : 1.0f - 0x1p-10f, kHalved = 0x1p-13f;
      auto less = [&](float2 y) {
        const float2 f = make_float2(!BF16 && y.x < kHalved ? 0.5f : kLess, !BF16 && y.y < kHalved ? 0.5f : kLess);
        return mul2(y, f);
      };
      const float2 sl = make_float2(a.scale_log2, a.scale_log2);
#pragma unroll
      for (int n = 0; n < NB; n++) {
        const float2 base = make_float2(kLift - (m[n].x == -INFINITY ? 0.0f : m[n].x), kLift - (m[n].y == -INFINITY ? 0.0f : m[n].y));
#pragma unroll
        for (int tt = 0; tt < 2; tt++)
#pragma unroll
          for (int half = 0; half < 2; half++) {
            float2 y = fma2(make_float2(x[tt][n][2 * half], x[tt][n][2 * half + 1]), sl, base);
            y = make_float2(ex2(y.x), ex2(y.y));
            sum[n] = add2(sum[n], y);
            const float2 z = less(y);
            const uint32_t w = pack<BF16>(z.x, z.y);
            p[tt][n][half] = transposed(w);
            rest[tt][n][half] = transposed(pack<BF16>(y.x - elem<BF16>(uint16_t(w)), y.y - elem<BF16>(uint16_t(w >> 16))));
          }
      }
      // O^T += V^T P^T
#pragma unroll
      for (int j = 0; j < kJ; j++)
#pragma unroll
        for (int tt = 0; tt < 2; tt++) {
          const int r = 16 * tt + v_row, c = 2 * j + v_ch;
          uint32_t f[4];
          load_matrices<true>(f, v_at + (c >> 3) * (kTok * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
#pragma unroll
          for (int n = 0; n < NB; n++) {
            mma<BF16>(o[j][n], f, p[tt][n][0], p[tt][n][1]);
            mma<BF16>(o[j][n], f, rest[tt][n][0], rest[tt][n][1]);
          }
        }
      __syncwarp();
      if (issued < tiles) issue(s);
      if (++s == kStages) s = 0, phase ^= 1;

      if (cur.tile + 1 == cur.s.tiles || u + 1 == tiles) {  // the end of the item, or of what this warp has of it
        // who has tiles of this item
        const int64_t c0 = ((item_lo + kIn + 1) * runs - 1) / total, c1 = ((item_lo + item_cost) * runs - 1) / total;
        const bool second = seg > 0;  // slot 1: the warp's last part, where another came before it
        float *part = a.parts + (2 * int64_t(me) + second) * kFewRows * (D + 2);
#pragma unroll
        for (int n = 0; n < NB; n++) {
          float2 y = sum[n];
#pragma unroll
          for (int e = 4; e < 32; e <<= 1) y.x += __shfl_xor_sync(0xffffffffu, y.x, e), y.y += __shfl_xor_sync(0xffffffffu, y.y, e);
          if (c0 == c1) {
            const float2 f = make_float2(y.x == 0.0f ? 0.0f : 1.0f / y.x, y.y == 0.0f ? 0.0f : 1.0f / y.y);
            const int r = 8 * n + g;
            const int64_t at = (int64_t(cur.s.q0) + r / a.G) * a.Hq + cur.h * a.G + r % a.G;
#pragma unroll
            for (int j = 0; j < kJ; j++)
#pragma unroll
              for (int half = 0; half < 2; half++) {
                const uint32_t w = transposed(pack<BF16>(o[j][n][2 * half] * f.x, o[j][n][2 * half + 1] * f.y));
                const int ch = 16 * j + 8 * half + 2 * t;
                if (r < rows && ch < a.d) *reinterpret_cast<uint32_t *>(a.out + at * a.d + ch) = w;
              }
            if (g == 0 && a.lse)
#pragma unroll
              for (int i = 0; i < 2; i++) {
                const int ri = 8 * n + 2 * t + i;
                const float l = i ? y.y : y.x, mm = i ? m[n].y : m[n].x;
                if (ri < rows)
                  a.lse[(int64_t(cur.s.q0) + ri / a.G) * a.Hq + cur.h * a.G + ri % a.G] = l == 0.0f ? -INFINITY : (mm - kLift + log2f(l)) * 0.6931471805599453f;
              }
          } else {
#pragma unroll
            for (int j = 0; j < kJ; j++)
#pragma unroll
              for (int i = 0; i < 4; i++) part[(8 * n + 2 * t + (i & 1)) * D + 16 * j + 8 * (i >> 1) + g] = o[j][n][i];
            if (g == 0) {
              float *ml = part + kFewRows * D + 8 * n + 2 * t;
              ml[0] = m[n].x, ml[1] = m[n].y, ml[kFewRows] = y.x, ml[kFewRows + 1] = y.y;
            }
          }
        }
        if (c0 != c1 && lane == 0 && me == c0) {
          Note &note = a.notes[me];
          note.parts = int(c1 - c0 + 1), note.second = second, note.b = cur.b, note.h = cur.h;
        }
        first = true;
        seg++;
        item_lo += item_cost;
        if (u + 1 < tiles) {
          next_item(a, cur);
          item_cost = cur.s.tiles + kIn;
        }
      } else {
        cur.tile++;
      }
    }
  }
  __syncthreads();
  if (sm.dead)  // what is in flight gets a moment to land
    for (int i = 0; i < 1000; i++) __nanosleep(1000);
  if (threadIdx.x == 0) a.errors[blockIdx.x] = sm.errors;
}

// Joins the parts of items that several warps had: a CTA per warp that has the
// first part of such an item, and four rows; a warp per row, four channels a
// lane, eight parts' loads in flight.  It is launched with the first kernel and waits for its end here.
template <int D, bool BF16>
__global__ void __launch_bounds__(128) k_few_join(const __grid_constant__ FewArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && blockIdx.y == 0) {  // the status of the call
    uint32_t e = 0;
    for (int i = threadIdx.x; i < int(kSMs); i += 128) e |= __ldcg(&a.errors[i]);
    __shared__ uint32_t s_errors;
    if (threadIdx.x == 0) s_errors = 0;
    __syncthreads();
    if (e) atomicOr(&s_errors, e);
    __syncthreads();
    if (threadIdx.x == 0) *a.status = s_errors;
  }
  const Note note = a.notes[blockIdx.x];
  if (note.parts == 0) return;
  const int q0 = a.cu_q[note.b], rows = (a.cu_q[note.b + 1] - q0) * a.G;
  auto part = [&](int i) { return a.parts + (2 * (int64_t(blockIdx.x) + i) + (i == 0 ? note.second : 0)) * kFewRows * (D + 2); };
  const int r = blockIdx.y * 4 + warp;
  if (r >= rows) return;
  float top = -INFINITY, sum = 0.0f, y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int base = 0; base < note.parts; base += 32) {
    const int n = min(32, note.parts - base);
    float m = -INFINITY, l = 0.0f;  // lane i: of part base + i
    if (lane < n) m = __ldcg(part(base + lane) + kFewRows * D + r), l = __ldcg(part(base + lane) + kFewRows * (D + 1) + r);
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
    float lw = l * w;
#pragma unroll
    for (int o = 16; o; o >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, o);
    sum += lw;
    for (int i0 = 0; i0 < n; i0 += 8) {
      float4 v[8];
#pragma unroll
      for (int i = 0; i < 8; i++)
        if (i0 + i < n && lane * 4 < D) v[i] = __ldcg(reinterpret_cast<const float4 *>(part(base + i0 + i) + r * D) + lane);
#pragma unroll
      for (int i = 0; i < 8; i++)
        if (i0 + i < n) {
          const float f = __shfl_sync(0xffffffffu, w, i0 + i);
          if (lane * 4 < D) y[0] += f * v[i].x, y[1] += f * v[i].y, y[2] += f * v[i].z, y[3] += f * v[i].w;
        }
    }
  }
  const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int64_t at = (int64_t(q0) + r / a.G) * a.Hq + note.h * a.G + r % a.G;
  if (lane * 4 < a.d)
    *reinterpret_cast<uint2 *>(a.out + at * a.d + lane * 4) = make_uint2(pack<BF16>(y[0] * f, y[1] * f), pack<BF16>(y[2] * f, y[3] * f));
  if (lane == 0 && a.lse) a.lse[at] = sum == 0.0f ? -INFINITY : (top - kLift + log2f(sum)) * 0.6931471805599453f;
}

int padded(int d) { return d <= 64 ? 64 : 128; }

// the status word, the CTAs' errors, then the notes
constexpr uint64_t kErrors = 256, kNotes = kErrors + ((4 * kSMs + 255) & ~uint64_t(255)), kParts = kNotes + ((sizeof(Note) * kMostRuns + 255) & ~uint64_t(255));

template <int D, int NB, bool BF16>
cudaError_t launch(const FewArgs &a, cudaStream_t st) {
  constexpr int kSmem = int(sizeof(Smem<D>));
  static_assert(kSmem <= 227 * 1024, "fits in an SM");
  const cudaError_t e = cudaFuncSetAttribute(k_few<D, NB, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  k_few<D, NB, BF16><<<kSMs, Shape<D>::kThreads, kSmem, st>>>(a);
  const cudaError_t e2 = launch_early(k_few_join<D, BF16>, dim3(Shape<D>::kRuns, unsigned((a.max_q * a.G + 3) / 4)), dim3(128), 0, st, a);
  return e2 != cudaSuccess ? e2 : cudaGetLastError();
}

template <int D>
cudaError_t launch_rows(const FewArgs &a, bool bf16, cudaStream_t st) {
  const bool one = a.max_q * a.G <= 8;
  if (one) return bf16 ? launch<D, 1, true>(a, st) : launch<D, 1, false>(a, st);
  return bf16 ? launch<D, 2, true>(a, st) : launch<D, 2, false>(a, st);
}

}  // namespace

uint64_t few_bytes(const cg_prompt &p) { return kParts + 4 * uint64_t(2 * kMostRuns) * kFewRows * (padded(p.d) + 2); }

cg_status cross_few(const cg_prompt &p, const void *q_dev, const void *k_dev, const void *v_dev, const int32_t *cu_q_dev,
                    const int32_t *k_begin_dev, const int32_t *k_len_dev, void *out_dev, float *lse_dev, uint8_t *ws, cudaStream_t st) {
  FewArgs a{};
  a.q = static_cast<const uint16_t *>(q_dev);
  a.cu_q = cu_q_dev, a.k_begin = k_begin_dev, a.k_len = k_len_dev;
  a.out = static_cast<uint16_t *>(out_dev), a.lse = lse_dev;
  a.status = reinterpret_cast<uint32_t *>(ws), a.errors = reinterpret_cast<uint32_t *>(ws + kErrors);
  a.notes = reinterpret_cast<Note *>(ws + kNotes), a.parts = reinterpret_cast<float *>(ws + kParts);
  a.q_row = p.q_stride[0], a.q_head = p.q_stride[1];
  a.n_seq = p.n_seq, a.Hq = p.Hq, a.H = p.H, a.G = p.Hq / p.H, a.d = p.d;
  a.max_q = p.max_q, a.max_k = p.max_k, a.n_q = p.n_q, a.n_k = p.n_k;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  if (p.n_k > 0 && (!make_map(&a.k_map, k_dev, p.d, p.n_k, p.k_stride[0], kTok, p.H, p.k_stride[1], 1) ||
                    !make_map(&a.v_map, v_dev, p.d, p.n_k, p.v_stride[0], kTok, p.H, p.v_stride[1], 1)))
    return CG_ERR_INVALID_ARG;  // strides that a tensor map cannot have
  const bool bf16 = p.dtype == CG_BF16;
  const cudaError_t e = p.d <= 64 ? launch_rows<64>(a, bf16, st) : launch_rows<128>(a, bf16, st);
  return e == cudaSuccess ? CG_OK : CG_ERR_CUDA;
}

}  // namespace cg
