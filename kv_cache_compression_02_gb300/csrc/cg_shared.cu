// cg_shared.cu -- cg_shared_attend: new tokens of sequences that share a prefix.
//
// The rows of all readers of a prefix that read the same KV head (members x T x
// Hq / H of them) are one matrix Q, and the prefix is gone over once for up to
// 256 of its rows:  S = Q K^T, P = 2^(S - max), O = P V, in tiles of 128 rows and
// 128 positions on tcgen05.  What a sequence has to itself is left to the
// kernels of cg_cache_attend, and the two parts, each with its maximum m and sum
// l, are joined: with M = max m_i, l = sum l_i 2^(m_i - M), out = sum O_i 2^(m_i -
// M) / l.
//
// Codes of either format are exact in f16, which is what the products take.  A
// bf16 query row is raised to the top of f16's range by a power of two.  K's
// page scales are applied to the scores, V's to the probabilities, over a power
// of two above the largest scale so far (O is scaled when that grows).  P is
// rounded to f16: a weight is off by at most 2^-11 of itself or 2^-31 of the
// largest times the largest scale, whichever is more (the largest has at least
// 2^7, and half of the spacing of f16's subnormals is 2^-25).  What the rounding
// leaves would take a product of its own, as in cg_cache_attend: built so, in the
// columns that S leaves free, the two calls below take 145 us each back to back, not
// 112 and 106.  Outputs against 64 bits, relative: f16 3.0e-4 (a 32-bit form
// rounded once 2.1e-4), bf16 1.7e-3 as that form.
//
// A CTA has two tiles of rows, a and b, whose softmax warpgroups take turns with
// the products; where an item has up to 128 rows, a and b are the same rows
// and take the even and the odd tiles of positions.  Warps: 0-3 and 4-7 the
// softmax of a and b, one row a thread; 8-11 turn codes into operands in shared
// memory; 12 and 13 look up pages and scales, a tile each in turns; 14 has the
// codes copied; 15 issues the products.
//
//   operands:  K(0) | K(1) V(0) | K(2) V(1) | ...
//   products:  S_a(0) S_b(0) | PV_a(j) S_a(j+1) PV_b(j) S_b(j+1) | ...
//   a = b:     S_a(0) | S_b(1) PV_a(0) | S_a(2) PV_b(1) | ...
//
// The tiles of positions of all items (group, KV head, 256 rows) are dealt in
// equal runs to one CTA per SM.  What a CTA has of an item goes to the workspace;
// beside this kernel the own parts are worked on, as far as SMs are free, and one
// join at the end puts all of it together.
//
// What bounds it: for many rows the products (4 d operations a row and position)
// and the softmax between them, for few rows the turning of codes into operands,
// which comes before the read of the codes.  64 readers of 32768 tokens, 64 heads
// on 8, d = 128, 20 to 2000 tokens of their own, e4m3: 109 us, of which the
// prefix takes 71 (0.97 PFLOP/s; 27 tiles of 256 rows a CTA at 2.1 us, 10 us of
// set-up); without sharing 698 us.  16 readers of 131072 tokens, int8: 103
// us (2.6 TB/s of distinct codes).  The roles of a scheduler's four warps differ,
// so that their code has to fit its instruction cache together: with loops unrolled
// whole the two calls took 155 and 182 us where they then took 115 and 109.
#include "cg_shared.cuh"

#include "cg_cache.cuh"
#include "cg_tc.cuh"
#include "cg_tma.cuh"

namespace cg {
namespace {

constexpr int kThreads = 512;
// Registers a thread: 512 are launched with 128 each (2 * 192 + 72 + 56 = 4 * 128).
constexpr int kSoftRegs = 192, kConvRegs = 72, kOtherRegs = 56;
constexpr int kTile = 128;  // rows of a tile, positions of a tile
constexpr int kRows = 2 * kTile;
constexpr int kGrid = kSMs;
constexpr int kStages = 3;   // operand tiles of K or V
constexpr int kRaw = 4;      // tiles of codes
constexpr int kLookers = 2;  // warps that look them up
constexpr int kPlan = 1024;
// p = 2^(s - m + kLift) < 2^15, m at most kLag under the maximum.  The parts that
// these are joined with have kOwnLift.  (With 12 and 3 here O is scaled more often:
// 64 readers of 32768 tokens take 115.5 us, with 7 and 8 112, back to back.)
constexpr float kLift = 7.0f, kLag = 8.0f, kOwnLift = 12.0f;
// What an item costs: kIn for its way in and out, and for each tile of positions.
constexpr int kIn = 10, kFull = 4, kSplit = 2;

struct alignas(16) Note {
  uint32_t errors;
  int32_t parts;   // of the item that this CTA has the first but not the last part of, or 0
  int32_t second;  // the first part is in this CTA's second slot
  int32_t e0, row0, rows, head;  // as in Todo
  int32_t reserved;
};

struct SharedArgs {
  const uint16_t *q;
  const uint8_t *kp, *vp;
  const float *ks, *vs;
  const int32_t *table, *len;
  uint16_t *out;
  float *lse;
  const int32_t *cu, *member, *shared;  // the caller's groups
  uint32_t *status, *bad;
  int32_t *any;  // whether some group counts
  int32_t *owner, *first;  // of a sequence: its entry in the groups, and the pages that it shares
  int32_t *seq;            // of an entry: its sequence, or -1
  int32_t *keys, *lead;    // of a group: its positions (0: nothing to do), and a sequence whose row of the table has them
  float *own, *own_ml;     // of each row [B][T][Hq]: what its sequence has to itself, not normalised, with maximum and sum
  float *pre, *pre_ml;     // the same of the prefix where one CTA had all of it; else the sum is -1 and the parts have it
  Note *notes;
  float *parts;  // [2 * kGrid][kRows][D + 2]
  int64_t q_seq, q_tok, q_head;
  int n_groups, n_members, B, T, Hq, H, G, TG, d, bt, n_blocks, stride, chunk;  // TG: rows of a sequence and KV head; chunk: positions copied at a time
  float scale_log2;  // scale * log2(e)
  bool bf16;
};

// Pages and scales of a tile of positions, for each EACH of them.
template <int EACH>
struct Info {
  static constexpr int kCount = kTile / EACH;
  int64_t row[kCount];  // where a position's codes begin, or -1
  float ks[kCount], vs[kCount];
  uint32_t valid[4];
  int v_exp, whole;
};

// What is to be done for a part of an item.
struct Todo {
  int n, split;      // tiles of positions; n < 0: the end
  int e0, row0, rows;  // the group's first entry; the block's first row, and the group's rows
  int head, slot;    // KV head; slot of the workspace, or -1: the item is whole
};

template <int D, int EACH>
struct Smem {
  static constexpr bool RAW = EACH > 1;
  static constexpr int kInfo = EACH == 8 ? 4 : 6;  // tiles whose pages and scales are known (as there is room)
  static constexpr int kChunks = D / 64;  // of 64 channels: 128 bytes, a swizzled row
  uint8_t q[2][kChunks][kTile * 128];
  uint8_t kv[kStages][kChunks][kTile * 128];
  uint8_t raw[RAW ? kRaw : 1][RAW ? kTile * D : 16];
  Info<EACH> info[kInfo];
  float ml[kTile][2];  // split: b's maximum and sum, for a
  int ml_exp;
  uint64_t todo_full[2], todo_empty[2], info_full[kInfo], info_empty[kInfo], q_full, q_empty, kv_full[kStages], kv_empty[kStages], raw_full[kRaw], raw_empty[kRaw], s_full[2],
      p_full[2][2], o_full[2], ml_full, ml_empty;
  Todo todo[2];
  uint32_t tmem, errors, dead;
  int most[kThreads / 32], g;
  int64_t sum[kThreads / 32][2], prefix;
};

// ---- the plan: who takes part -----------------------------------------------------
// An entry of a group counts where it is the first to name its sequence and every
// new token of the sequence sees the whole prefix; the others read their
// positions by themselves.
__global__ void __launch_bounds__(kPlan) k_shared_plan(const SharedArgs a) {
  asm volatile("griddepcontrol.launch_dependents;");
  constexpr int kKept = 8192;  // sequences whose entries are kept here (64 of them: 4.2 us, in global memory 4.7)
  __shared__ int s_owner[kKept];
  int *const owner = a.B <= kKept ? s_owner : a.owner;
  for (int b = threadIdx.x; b < a.B; b += kPlan) owner[b] = 0x7fffffff, a.first[b] = 0;
  bool bad = false, fall = false, any = false;
  for (int g = threadIdx.x; g < a.n_groups; g += kPlan) {
    const int e0 = a.cu[g], e1 = a.cu[g + 1], pages = a.shared[g];
    a.keys[g] = 0, a.lead[g] = 0x7fffffff;
    fall |= e0 < 0 || e1 < e0 || e1 > a.n_members;
    bad |= pages < 0 || pages > a.stride;
  }
  fall = __syncthreads_or(fall);
  if (!fall) {
    const int e0 = a.cu[0], e1 = a.cu[a.n_groups];
    for (int e = e0 + threadIdx.x; e < e1; e += kPlan) {
      const int b = a.member[e];
      if (uint32_t(b) < uint32_t(a.B))
        atomicMin(&owner[b], e);
      else
        bad = true;
    }
    __syncthreads();
    for (int e = e0 + threadIdx.x; e < e1; e += kPlan) {
      const int b = a.member[e];
      int takes = -1;
      if (uint32_t(b) < uint32_t(a.B)) {
        if (*static_cast<volatile int *>(&owner[b]) != e) {
          bad = true;
        } else {
          const int64_t len = max(int64_t(0), min(int64_t(a.len[b]), int64_t(a.stride) * a.bt));
          int g = 0, hi = a.n_groups;  // the last group that begins at or before e
          while (hi - g > 1) {
            const int mid = g + (hi - g) / 2;
            if (a.cu[mid] <= e)
              g = mid;
            else
              hi = mid;
          }
          const int pages = a.shared[g];
          const int64_t keys = int64_t(pages) * a.bt;
          if (pages > 0 && pages <= a.stride && len - a.T + 1 >= keys) {
            takes = b;
            any = true;
            a.first[b] = pages;
            a.keys[g] = int(keys);
            atomicMin(&a.lead[g], b);
          }
        }
      }
      a.seq[e] = takes;
    }
  }
  bad = __syncthreads_or(bad || fall);
  any = __syncthreads_or(any);
  if (threadIdx.x == 0) *a.bad = bad ? kStBadArg : 0, *a.any = any;
}

// ---- items --------------------------------------------------------------------------
// Item (g, h, q): rows 256 q ... of group g, KV head h.
struct Group {
  int rows, tiles, blocks;
};

__device__ inline Group load_group(const SharedArgs &a, int g) {
  Group s;
  const int keys = a.keys[g];
  s.rows = keys > 0 ? (a.cu[g + 1] - a.cu[g]) * a.TG : 0;
  s.blocks = (s.rows + kRows - 1) / kRows, s.tiles = (keys + kTile - 1) / kTile;
  return s;
}

__device__ inline bool is_split(const Group &s, int q) { return s.rows - q * kRows <= kTile; }

__device__ inline int tile_cost(const Group &s, int q) { return is_split(s, q) ? kSplit : kFull; }

__device__ inline int64_t item_cost(const Group &s, int q, int skip) { return skip ? kIn + int64_t(s.tiles) * tile_cost(s, q) : 1; }

__device__ inline int64_t head_cost(const Group &s, int skip) {
  return s.blocks == 0 ? 0 : skip ? (s.blocks - 1) * (kIn + int64_t(s.tiles) * kFull) + item_cost(s, s.blocks - 1, 1) : s.blocks;
}

struct Part {
  int g, h, q, j0, n;
  int64_t first, last;  // where the costs of the item's first and last tile begin
};

// The parts of a CTA's run [lo, hi), one after the other.
struct Run {
  Group s;
  int g, h, q;
  int64_t lo;  // where the item's cost begins
  int64_t at, hi;
  int skip;  // 1: items have their costs; 0: each is one

  __device__ bool next(const SharedArgs &a, Part &p) {
    while (at < hi) {
      // a tile belongs to the run in which its cost begins
      const int64_t cost = item_cost(s, q, skip), end = min(hi, lo + cost);
      const int each = tile_cost(s, q);
      auto tiles_before = [&](int64_t x) { return int(max(int64_t(0), x - lo - kIn + each - 1) / each); };
      p.j0 = skip ? tiles_before(at) : 0;
      p.n = (skip ? tiles_before(end) : s.tiles) - p.j0;
      p.g = g, p.h = h, p.q = q;
      p.first = lo + (skip ? kIn : 0), p.last = p.first + (skip ? int64_t(s.tiles - 1) * each : 0);
      at = end;
      if (at < hi) {
        lo += cost;
        if (++q == s.blocks) {
          q = 0;
          if (++h == a.H) {
            h = 0;
            do s = load_group(a, ++g);
            while (s.blocks == 0);
          }
        }
      }
      if (p.n > 0) return true;
    }
    return false;
  }
};

// Codes in the low (HALF = 0) or high half of w -> two f16.
template <int FMT, int HALF>
__device__ inline uint32_t halves_of(uint32_t w) {
  uint32_t r;
  if (FMT == CG_CACHE_E4M3) {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(HALF ? w >> 16 : w)));
  } else {  // 0x64uu is 1024 + u; w holds code + 128
    const __half2 x = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    uint32_t p = __byte_perm(w, 0x64646464u, HALF ? 0x4342 : 0x4140);
    const __half2 y = __hsub2(*reinterpret_cast<__half2 *>(&p), x);
    r = *reinterpret_cast<const uint32_t *>(&y);
  }
  return r;
}

template <int FMT>
__device__ inline uint4 operands_of(uint2 w) {  // eight codes
  if (FMT == CG_CACHE_INT8) w.x ^= 0x80808080u, w.y ^= 0x80808080u;
  return make_uint4(halves_of<FMT, 0>(w.x), halves_of<FMT, 1>(w.x), halves_of<FMT, 0>(w.y), halves_of<FMT, 1>(w.y));
}

// Waits for what tm_load is to bring; x is not used before.
__device__ inline void tm_landed(uint32_t (&x)[32]) {
#define CG_W8(i) "+r"(x[i]), "+r"(x[i + 1]), "+r"(x[i + 2]), "+r"(x[i + 3]), "+r"(x[i + 4]), "+r"(x[i + 5]), "+r"(x[i + 6]), "+r"(x[i + 7])
  asm volatile("tcgen05.wait::ld.sync.aligned;" : CG_W8(0), CG_W8(8), CG_W8(16), CG_W8(24) : : "memory");
#undef CG_W8
}

// 16 columns of this thread's lane, waited for.
__device__ inline void tm_load16(uint32_t addr, uint32_t (&x)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
               "tcgen05.wait::ld.sync.aligned;"
               : CG_R8(x, 0), CG_R8(x, 8)
               : "r"(addr)
               : "memory");
}

// The larger of two values, or NaN where one of them is.
__device__ inline float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Copies `bytes`, a multiple of 16, to shared memory.
__device__ inline void copy_bulk(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes),
               "r"(smem_of(bar))
               : "memory");
}

// EACH positions have one scale and lie together: 16 or 8 where pages are multiples
// of that, else 1.  With 16 and 8 (RAW) codes are copied, `chunk` positions (a power
// of two up to 128 that divides a page) at a time; with 1 they are loaded a position
// and eight channels at a time, and scales are applied on a way of their own (a
// context of 32768 tokens and 16 readers in pages of 32: 45 us, of 24: 54, of 7: 61).
template <int FMT, int D, int EACH>
__global__ void __launch_bounds__(kThreads, 1) k_shared(const __grid_constant__ SharedArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  constexpr bool RAW = EACH > 1;
  constexpr int kWith = RAW ? EACH : 16;  // positions that the softmax takes together
  constexpr int kInfo = Smem<D, EACH>::kInfo;
  Smem<D, EACH> &sm = *reinterpret_cast<Smem<D, EACH> *>(smem_raw);
  constexpr int kChunks = Smem<D, EACH>::kChunks;
  constexpr uint32_t kTileBytes = kChunks * kTile * 128;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  status_cleared();  // the plan is there
  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x == 0) {
    sm.errors = sm.dead = 0;
    a.notes[blockIdx.x].parts = 0;
    bar_init(&sm.q_full, 8), bar_init(&sm.q_empty, 1);
    for (int i = 0; i < 2; i++) bar_init(&sm.todo_full[i], 1), bar_init(&sm.todo_empty[i], 14);  // 14 warps read it
    for (int i = 0; i < kInfo; i++) bar_init(&sm.info_full[i], 1), bar_init(&sm.info_empty[i], 1);
    for (int i = 0; i < kStages; i++) bar_init(&sm.kv_full[i], 4), bar_init(&sm.kv_empty[i], 1);
    for (int i = 0; i < kRaw; i++) bar_init(&sm.raw_full[i], 1), bar_init(&sm.raw_empty[i], 4);
    for (int t = 0; t < 2; t++) bar_init(&sm.s_full[t], 1), bar_init(&sm.p_full[t][0], 4), bar_init(&sm.p_full[t][1], 4), bar_init(&sm.o_full[t], 1);
    bar_init(&sm.ml_full, 4), bar_init(&sm.ml_empty, 4);
    bar_init_fence();
  }
  if (warp == 15) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_of(&sm.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // The items of the call and what they cost.
  const int per = (a.n_groups + kThreads - 1) / kThreads, g0 = threadIdx.x * per, g1 = min(a.n_groups, g0 + per);
  int64_t cost = 0, items = 0;
  int most = 0;
  for (int g = g0; g < g1; g++) {
    const Group s = load_group(a, g);
    cost += head_cost(s, 1) * a.H, items += int64_t(s.blocks) * a.H;
    if (s.blocks) most = max(most, s.tiles);
  }
  int64_t cost_to = cost, items_to = items;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, cost_to, o), z = __shfl_up_sync(0xffffffffu, items_to, o);
    if (lane >= o) cost_to += y, items_to += z;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 31) sm.sum[warp][0] = cost_to, sm.sum[warp][1] = items_to, sm.most[warp] = most;
  tm_before();
  __syncthreads();
  tm_after();
  int64_t total = 0, n_items = 0;
  for (int w = 0; w < kThreads / 32; w++) {
    if (w < warp) cost_to += sm.sum[w][0], items_to += sm.sum[w][1];
    total += sm.sum[w][0], n_items += sm.sum[w][1];
    most = max(most, sm.most[w]);
  }
  const int skip = most <= 1 && n_items <= gridDim.x ? 0 : 1;  // 0: a CTA per item
  if (!skip) total = n_items, cost = items, cost_to = items_to;
  const int64_t before = cost_to - cost;
  // No run is shorter than a tile, so that each has one of every item that goes through
  // it: the join takes a part from every CTA between those of the first and last tile.
  const int64_t ctas = min(int64_t(gridDim.x), skip ? total / kFull : total);
  const int64_t lo = ctas ? total * blockIdx.x / ctas : 0, hi = ctas ? total * (blockIdx.x + 1) / ctas : 0;
  const bool busy = int64_t(blockIdx.x) < ctas;
  if (busy && lo >= before && lo < before + cost) {  // one thread's groups hold the first cost
    int64_t at = before;
    int g = g0;
    for (;; g++) {
      const int64_t n = head_cost(load_group(a, g), skip) * a.H;
      if (lo < at + n) break;
      at += n;
    }
    sm.g = g;
    sm.prefix = at;
  }
  __syncthreads();
  const uint32_t tmem = sm.tmem;

  if (busy) {
    if (warp >= 12) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
      if (warp < 12 + kLookers) {
        // ---- pages and scales ----
        Run run;
        Part p;
        run.at = lo, run.hi = hi, run.skip = skip, run.g = sm.g;
        run.s = load_group(a, run.g);
        const int64_t head = head_cost(run.s, skip), rest0 = lo - sm.prefix;
        run.h = int(rest0 / head);
        const int64_t rest = rest0 - run.h * head;
        run.q = int(min(int64_t(run.s.blocks) - 1, rest / (skip ? kIn + int64_t(run.s.tiles) * kFull : 1)));
        run.lo = sm.prefix + run.h * head + run.q * (skip ? kIn + int64_t(run.s.tiles) * kFull : 1);
        int turn = 0, seg = 0, slot = 0, who = 0;
        uint32_t todo_phase = 1, phase = 1;  // the first pass over a ring finds it empty
        bool ok = true;
        while (ok) {
          const bool more = run.next(a, p);
          if (warp == 12) {
            if (!(ok = bar_wait(&sm.todo_empty[turn], todo_phase, &sm.dead))) break;
            if (lane == 0) {
              Todo &todo = sm.todo[turn];
              if (!more) {
                todo.n = -1;
              } else {
                // who has tiles of this item
                const int64_t c0 = ((p.first + 1) * ctas - 1) / total, c1 = ((p.last + 1) * ctas - 1) / total;
                todo.n = p.n;
                todo.e0 = a.cu[p.g], todo.row0 = p.q * kRows, todo.rows = (a.cu[p.g + 1] - a.cu[p.g]) * a.TG;
                todo.split = todo.rows - todo.row0 <= kTile;
                todo.head = p.h;
                todo.slot = c0 == c1 ? -1 : 2 * int(blockIdx.x) + (seg > 0);  // slot 1: the run's last part
                if (c0 != c1 && int64_t(blockIdx.x) == c0) {
                  Note &note = a.notes[blockIdx.x];
                  note.parts = int(c1 - c0 + 1), note.second = seg > 0, note.e0 = todo.e0, note.row0 = todo.row0, note.rows = todo.rows, note.head = p.h;
                }
              }
              bar_arrive(&sm.todo_full[turn]);
            }
            __syncwarp();
            seg++;
            turn ^= 1;
            if (turn == 0) todo_phase ^= 1;
          }
          if (!more) break;
          const int keys = a.keys[p.g];
          const int32_t *row = a.table + int64_t(a.lead[p.g]) * a.stride;
          constexpr int kCount = Info<EACH>::kCount, kMine = (kCount + 31) / 32;
          int page[kMine], at[kMine];  // of the warp's next tile
          auto look = [&](int j) {
#pragma unroll
            for (int k = 0; k < kMine; k++) {
              const int i = 32 * k + lane, tok = (p.j0 + j) * kTile + i * EACH, blk = tok / a.bt;
              const bool there = i < kCount && tok < keys;
              at[k] = there ? tok - blk * a.bt : -1;
              page[k] = there ? row[blk] : -1;
            }
          };
          int mine = warp - 12 - who;
          if (mine < 0) mine += kLookers;
          if (mine < p.n) look(mine);
          for (int j = 0; j < p.n; j++) {
            if (j == mine) {
              float ks[kMine], vs[kMine], top = 0.0f;
              int64_t begin[kMine];
              bool good[kMine];
#pragma unroll
              for (int k = 0; k < kMine; k++) {
                good[k] = uint32_t(page[k]) < uint32_t(a.n_blocks);
                if (at[k] >= 0 && !good[k]) atomicOr(&sm.errors, kStBadArg);
                const int64_t sc = good[k] ? int64_t(page[k]) * a.H + p.h : 0;
                ks[k] = good[k] ? a.ks[sc] : 0.0f, vs[k] = good[k] ? a.vs[sc] : 0.0f;
                begin[k] = good[k] ? page_row(page[k], a.H, p.h, a.bt, at[k], a.d) : -1;
              }
              mine += kLookers;
              if (mine < p.n) look(mine);
              if (!(ok = bar_wait(&sm.info_empty[slot], phase, &sm.dead))) break;
              Info<EACH> &in = sm.info[slot];
              int whole = 1;
#pragma unroll
              for (int k = 0; k < kMine; k++) {
                const int i = 32 * k + lane;
                const uint32_t valid = __ballot_sync(0xffffffffu, good[k]);
                whole &= valid == (kCount < 32 ? (1u << kCount % 32) - 1 : 0xffffffffu);
                if (i < kCount) in.row[i] = begin[k], in.ks[i] = ks[k], in.vs[i] = vs[k];
                top = fmaxf(top, fabsf(vs[k]));
                if (RAW) {
                  constexpr int kBits = 32 / EACH;  // of `valid`, for a word of positions
                  uint32_t word = 0;
#pragma unroll
                  for (int b = 0; b < kBits; b++) word |= (valid >> (kBits * (lane & 3) + b) & 1 ? (1u << EACH % 32) - 1 : 0) << b * EACH;
                  if (lane < 4) in.valid[lane] = word;
                } else if (lane == 0) {
                  in.valid[k] = valid;
                }
              }
              const int e = __reduce_max_sync(0xffffffffu, min(254, int(__float_as_uint(top) >> 23) + 1));
              if (lane == 0) in.v_exp = e, in.whole = whole;
              __syncwarp();
              if (lane == 0) bar_arrive(&sm.info_full[slot]);
            }
            if (++who == kLookers) who = 0;
            if (++slot == kInfo) slot = 0, phase ^= 1;
          }
        }
      } else if (warp == 14) {
        // ---- copies of codes ----
        int turn = 0, k_slot = 0, v_slot = 0, at = 0;
        uint32_t todo_phase = 0, k_phase = 0, v_phase = 0, raw_phase = 1;
        bool ok = true;
        const int chunk = a.chunk;  // lane l has the l-th
        const uint32_t bytes = uint32_t(chunk) * a.d;
        auto copy = [&](const uint8_t *pool, int slot, uint32_t phase) {
          if (!(ok = bar_wait(&sm.info_full[slot], phase, &sm.dead))) return;
          if (!(ok = bar_wait(&sm.raw_empty[at], raw_phase, &sm.dead))) return;
          const int64_t begin = lane < kTile / chunk ? sm.info[slot].row[RAW ? lane * (chunk / EACH) : 0] : -1;
          const uint32_t there = __ballot_sync(0xffffffffu, begin >= 0);
          if (lane == 0) bar_expect(&sm.raw_full[at], __popc(there) * bytes);
          __syncwarp();
          if (begin >= 0) copy_bulk(smem_of(sm.raw[RAW ? at : 0] + lane * bytes), pool + begin, bytes, &sm.raw_full[at]);
          if (++at == kRaw) at = 0, raw_phase ^= 1;
        };
        for (;;) {
          if (!(ok = bar_wait(&sm.todo_full[turn], todo_phase, &sm.dead))) break;
          const int n = sm.todo[turn].n;
          __syncwarp();
          if (lane == 0) bar_arrive(&sm.todo_empty[turn]);
          turn ^= 1;
          if (turn == 0) todo_phase ^= 1;
          if (n < 0) break;
#pragma unroll 1
          for (int i = 0; RAW && i < 2 * n && ok; i++) {
            const bool is_v = i == 2 * n - 1 || (i > 0 && i % 2 == 0);
            copy(is_v ? a.vp : a.kp, is_v ? v_slot : k_slot, is_v ? v_phase : k_phase);
            if (is_v) {
              if (++v_slot == kInfo) v_slot = 0, v_phase ^= 1;
            } else {
              if (++k_slot == kInfo) k_slot = 0, k_phase ^= 1;
            }
          }
          if (!ok) break;
        }
      } else {
        // ---- products ----
        constexpr uint32_t kCommon = 1u << 4 | uint32_t(kTile >> 4) << 24;  // f16 operands, fp32 sums
        constexpr uint32_t kS = kCommon | uint32_t(kTile >> 3) << 17, kO = kCommon | 1u << 16 | uint32_t(D >> 3) << 17;
        constexpr uint32_t kChunk = kTile * 128 >> 4, kStage = kTileBytes >> 4;
        const uint32_t q_lo = operand_lo(sm.q[0], 16), k_lo = operand_lo(sm.kv[0], 16), v_lo = operand_lo(sm.kv[0], kTile * 128);
        int stage = 0, turn = 0, slot = 0;
        uint32_t kv_phase = 0, q_phase = 0, todo_phase = 0, p_phase[2] = {0, 0};
        // A wait that runs out is seen between parts only (the others end at once, and what
        // is issued meanwhile stays within the CTA's own memory): without a way out of the
        // loops the compiler sees that the warp stays together, and what the products take
        // comes from uniform registers.
        auto s_product = [&](int t, int q, int st) {  // S_t = Q_q K^T
          const uint32_t a0 = q_lo + q * kStage, b0 = k_lo + st * kStage;
          if (elected()) {
#pragma unroll
            for (int k = 0; k < D / 16; k++)
              mma_ss(tmem + t * kTile, a0 + k / 4 * kChunk + k % 4 * 2, b0 + k / 4 * kChunk + k % 4 * 2, kS, k > 0);
            mma_commit(&sm.s_full[t]);
          }
        };
        auto take = [&]() {  // the next operand tile
          const int st = stage;
          bar_wait(&sm.kv_full[st], kv_phase, &sm.dead);
          if (++stage == kStages) stage = 0, kv_phase ^= 1;
          return st;
        };
        for (;;) {
          const bool there = bar_wait(&sm.todo_full[turn], todo_phase, &sm.dead);
          if (!__all_sync(0xffffffffu, there)) break;
          const int n = __shfl_sync(0xffffffffu, sm.todo[turn].n, 0), split = __shfl_sync(0xffffffffu, sm.todo[turn].split, 0);
          __syncwarp();
          if (lane == 0) bar_arrive(&sm.todo_empty[turn]);
          turn ^= 1;
          if (turn == 0) todo_phase ^= 1;
          if (n < 0) break;
          bar_wait(&sm.q_full, q_phase, &sm.dead);
          q_phase ^= 1;
          {
            const int ks = take();
            tm_after();
            s_product(0, 0, ks);
            if (!split) s_product(1, 1, ks);
            if (elected()) {
              mma_commit(&sm.kv_empty[ks]);
              if (n == 1) mma_commit(&sm.q_empty);
            }
          }
          for (int j = 0; j < n; j++) {
            const bool more = j + 1 < n;
            int ks = 0;
            if (more) {
              ks = take();
              if (split) {  // the other tile's: P(j-1), which it overwrites, is behind PV(j-1)
                tm_after();
                s_product(j + 1 & 1, 0, ks);
              }
            }
            const int vs = take();
#pragma unroll
            for (int t = 0; t < 2; t++) {
              if (split && t != (j & 1)) continue;
              const uint32_t b0 = v_lo + vs * kStage;
#pragma unroll
              for (int half = 0; half < 2; half++) {  // O_t += P_t V
                bar_wait(&sm.p_full[t][half], p_phase[t], &sm.dead);
                tm_after();
                if (elected())
#pragma unroll
                  for (int k = half * 4; k < half * 4 + 4; k++)
                    mma_ts(tmem + 2 * kTile + t * kTile, tmem + t * kTile + k * 8, b0 + k * (2048 >> 4), kO, j > split || k > 0);
              }
              p_phase[t] ^= 1;
              if (more && !split)
                s_product(t, t, ks);
              else if ((!more || (split && j + 2 == n)) && elected())
                mma_commit(&sm.o_full[t]);
            }
            if (elected()) {
              mma_commit(&sm.kv_empty[vs]);
              mma_commit(&sm.info_empty[slot]);
              if (more) mma_commit(&sm.kv_empty[ks]);
              if (j + 2 == n) mma_commit(&sm.q_empty);
            }
            if (++slot == kInfo) slot = 0;
          }
        }
      }
    } else if (warp >= 8) {
      // ---- codes into operands ----
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
      const int ct = threadIdx.x - 256;
      int stage = 0, turn = 0, k_slot = 0, v_slot = 0, at = 0;
      uint32_t kv_phase = 1, todo_phase = 0, k_phase = 0, v_phase = 0, raw_phase = 0;
      bool ok = true;
      constexpr int kUnits = D / 8, kStep = 128 / kUnits;  // eight codes each, of a row
      const int u = ct % kUnits, r0 = ct / kUnits;
      for (;;) {
        if (!(ok = bar_wait(&sm.todo_full[turn], todo_phase, &sm.dead))) break;
        const int n = sm.todo[turn].n;
        __syncwarp();
        if (lane == 0) bar_arrive(&sm.todo_empty[turn]);
        turn ^= 1;
        if (turn == 0) todo_phase ^= 1;
        if (n < 0) break;
#pragma unroll 1
        for (int i = 0; i < 2 * n; i++) {
          const bool is_v = i == 2 * n - 1 || (i > 0 && i % 2 == 0);
          const Info<EACH> &in = sm.info[is_v ? v_slot : k_slot];
          if (RAW) {  // (who had the codes copied has seen the tile's pages)
            if (!(ok = bar_wait(&sm.raw_full[at], raw_phase, &sm.dead))) break;
          } else {
            if (!(ok = bar_wait(&sm.info_full[is_v ? v_slot : k_slot], is_v ? v_phase : k_phase, &sm.dead))) break;
          }
          const uint8_t *pool = is_v ? a.vp : a.kp, *from = sm.raw[RAW ? at : 0] + r0 * a.d + u * 8;
          const bool there = u * 8 < a.d, whole = in.whole;
          uint8_t *to = sm.kv[stage][u >> 3] + r0 * 128 + (((u & 7) ^ (r0 & 7)) << 4);  // (kStep is a multiple of 8)
          constexpr int kBatch = RAW ? kUnits : 8;  // (codes from shared memory: all of them before the wait; from global memory: 8)
#pragma unroll 1
          for (int h = 0; h < kUnits; h += kBatch) {
            uint2 w[kBatch];
            if (RAW && a.d == D) {
#pragma unroll
              for (int k = 0; k < kBatch; k++) w[k] = *reinterpret_cast<const uint2 *>(from + (h + k) * kStep * D);
            } else {
#pragma unroll
              for (int k = 0; k < kBatch; k++) {
                const int r = (h + k) * kStep;
                if (RAW) {
                  w[k] = there ? *reinterpret_cast<const uint2 *>(from + r * a.d) : make_uint2(0, 0);
                } else {
                  const int64_t begin = in.row[RAW ? 0 : r0 + r];
                  w[k] = there && begin >= 0 ? *reinterpret_cast<const uint2 *>(pool + begin + u * 8) : make_uint2(0, 0);
                }
              }
            }
            if (RAW) {
              if (!whole) {  // nothing was copied there
#pragma unroll
                for (int k = 0; k < kBatch; k++) {
                  const int r = r0 + (h + k) * kStep;
                  if (!(in.valid[r / 32] >> (r & 31) & 1)) w[k] = make_uint2(0, 0);
                }
              }
              __syncwarp();
              if (lane == 0) bar_arrive(&sm.raw_empty[at]);
            }
            if (h == 0 && !(ok = bar_wait(&sm.kv_empty[stage], kv_phase, &sm.dead))) break;
#pragma unroll
            for (int k = 0; k < kBatch; k++) *reinterpret_cast<uint4 *>(to + (h + k) * kStep * 128) = operands_of<FMT>(w[k]);
          }
          if (!ok) break;
          fence_async();
          __syncwarp();
          if (lane == 0) bar_arrive(&sm.kv_full[stage]);
          if (++stage == kStages) stage = 0, kv_phase ^= 1;
          if (++at == kRaw) at = 0, raw_phase ^= 1;
          if (is_v) {
            if (++v_slot == kInfo) v_slot = 0, v_phase ^= 1;
          } else {
            if (++k_slot == kInfo) k_slot = 0, k_phase ^= 1;
          }
        }
        if (!ok) break;
      }
    } else {
      // ---- softmax: a row a thread ----
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
      const int t = warp >> 2, r = threadIdx.x & (kTile - 1);
      const uint32_t lanes = uint32_t(warp & 3) << 21;  // the warp's lanes of TMEM
      const uint32_t s_at = tmem + lanes + t * kTile, o_at = tmem + lanes + 2 * kTile + t * kTile;
      uint32_t s_phase = 0, o_phase = 0, todo_phase = 0, q_phase = 1, info_phase = 0, ml_phase = 0;
      int turn = 0, slot = 0;
      bool ok = true;
      for (;;) {
        if (!(ok = bar_wait(&sm.todo_full[turn], todo_phase, &sm.dead))) break;
        const Todo &todo = sm.todo[turn];
        const int n = todo.n;
        const bool split = todo.split;
        if (n < 0) break;
        // the query row
        const int row = todo.row0 + (split ? 0 : t * kTile) + r;
        const int b = row < todo.rows ? a.seq[todo.e0 + row / a.TG] : -1;
        const int tok = row % a.TG / a.G, head = todo.head * a.G + row % a.G;  // TG is a multiple of G
        float sc = a.scale_log2;
        {
          const uint16_t *src = a.q + b * a.q_seq + tok * a.q_tok + head * a.q_head;
          uint4 w[D / 8];
#pragma unroll
          for (int c = 0; c < D / 8; c++) w[c] = b >= 0 && c * 8 < a.d ? *reinterpret_cast<const uint4 *>(src + c * 8) : make_uint4(0, 0, 0, 0);
          if (a.bf16) {  // to f16, raised to its top: off by at most 2^-39 of the row's largest
            uint32_t top = 0;
#pragma unroll
            for (int c = 0; c < D / 8; c++) {
              const uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
              for (int k = 0; k < 4; k++) top = max(top, max(x[k] << 16 & 0x7fff0000u, x[k] & 0x7fff0000u));
            }
            const int f = min(253, max(1, 268 - int(top >> 23)));
            const float up = __int_as_float(f << 23);
            sc *= __int_as_float((254 - f) << 23);
#pragma unroll
            for (int c = 0; c < D / 8; c++) {
              uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
              for (int k = 0; k < 4; k++)
                x[k] = pack<false>(__uint_as_float(x[k] << 16) * up, __uint_as_float(x[k] & 0xffff0000u) * up);
              w[c] = make_uint4(x[0], x[1], x[2], x[3]);
            }
          }
          if (!(ok = bar_wait(&sm.q_empty, q_phase, &sm.dead))) break;
          q_phase ^= 1;
          if (!split || t == 0) {
#pragma unroll
            for (int c = 0; c < D / 8; c++) *reinterpret_cast<uint4 *>(sm.q[t][c >> 3] + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = w[c];
            fence_async();
          }
          __syncwarp();
          if (lane == 0) bar_arrive(&sm.q_full);
        }
        float m = -INFINITY;
        float2 l = make_float2(0.0f, 0.0f);
        int v_exp = 1;  // O is in units of 2^(v_exp - 127), the largest V scale so far
        int done = 0;   // tiles of this thread's
        for (int j = 0; j < n; j++) {
          const Info<EACH> &in = sm.info[slot];
          const uint32_t full = info_phase;
          uint64_t *const info_full = &sm.info_full[slot];
          if (++slot == kInfo) slot = 0, info_phase ^= 1;
          if (split && t != (j & 1)) continue;
          if (!(ok = bar_wait(info_full, full, &sm.dead))) break;
          if (!(ok = bar_wait(&sm.s_full[t], s_phase, &sm.dead))) break;
          s_phase ^= 1;
          tm_after();
          const int whole = in.whole;
          if (!RAW || !whole) {  // in the way of the loops below: scales of single positions (K's), and positions that are not there
#pragma unroll 1
            for (int c = 0; c < 4; c++) {
              uint32_t y[32];
              tm_load(s_at + 32 * c, y);
              tm_landed(y);
              const uint32_t valid = in.valid[c];
#pragma unroll
              for (int i = 0; i < 32; i++) {
                if (!RAW) y[i] = __float_as_uint(__uint_as_float(y[i]) * (in.ks[RAW ? 0 : 32 * c + i] * sc));
                if (!(valid >> i & 1)) y[i] = 0xff800000u;
              }
              tm_store32(s_at + 32 * c, y);
            }
            tm_wait_st();
          }
          // What turns a product into a score: a page's scale times the row's.  It is
          // not 0, so that what is masked stays at -inf (a page's codes are 0 where its scale is);
          // a NaN stays one.
          auto scale_of = [&](int i) { return RAW ? max_nan(in.ks[RAW ? i : 0] * sc, 0x1p-126f) : 1.0f; };
          uint32_t x[4][32];
#pragma unroll
          for (int c = 0; c < 4; c++) tm_load(s_at + 32 * c, x[c]);
#pragma unroll
          for (int c = 0; c < 4; c++) tm_landed(x[c]);
          float now = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; c++)
#pragma unroll
            for (int h = 0; h < 32 / kWith; h++) {
              auto at = [&](int i) { return __uint_as_float(x[c][kWith * h + i]); };
              float top[2] = {fmaxf(at(0), at(1)), fmaxf(at(2), at(3))};
#pragma unroll
              for (int i = 4; i < kWith; i += 4) top[0] = max3(top[0], at(i), at(i + 1)), top[1] = max3(top[1], at(i + 2), at(i + 3));
              now = fmaxf(now, fmaxf(top[0], top[1]) * scale_of(32 / kWith * c + h));
            }
          const bool moved = now > m + kLag;
          const float keep = moved ? ex2(m - now) : 1.0f;
          if (moved) m = now;
          float scale_o = keep;
          const int e = in.v_exp;
          if (e > v_exp) {  // the same in every thread
            scale_o *= e - v_exp > 126 ? 0.0f : __int_as_float((127 + v_exp - e) << 23);
            v_exp = e;
          }
          if (done > 0 && __any_sync(0xffffffffu, scale_o != 1.0f)) {
            l = mul2(l, make_float2(keep, keep));
#pragma unroll 1
            for (int c = 0; c < D / 16; c++) {
              uint32_t y[16];
              tm_load16(o_at + 16 * c, y);
#pragma unroll
              for (int i = 0; i < 16; i++) y[i] = __float_as_uint(__uint_as_float(y[i]) * scale_o);
              tm_store16(o_at + 16 * c, y);
            }
          }
          done++;
          const float base = kLift - (m == -INFINITY ? 0.0f : m), unit = __int_as_float((254 - v_exp) << 23);
          float2 sums[4] = {};
#pragma unroll
          for (int c = 0; c < 4; c++) {
            uint32_t pk[16];
#pragma unroll
            for (int h = 0; h < 32 / kWith; h++) {
              const int group = 32 / kWith * c + h;
              const float f = scale_of(group), v = RAW ? in.vs[RAW ? group : 0] * unit : 0.0f;
#pragma unroll
              for (int i = kWith / 2 * h; i < kWith / 2 * (h + 1); i++) {
                float2 y = make_float2(__uint_as_float(x[c][2 * i]), __uint_as_float(x[c][2 * i + 1]));
                y = RAW ? fma2(y, make_float2(f, f), make_float2(base, base)) : add2(y, make_float2(base, base));
                y = make_float2(ex2(y.x), ex2(y.y));
                sums[i & 3] = add2(sums[i & 3], y);
                if (RAW) {
                  y = mul2(y, make_float2(v, v));
                } else {
                  const float2 v2 = *reinterpret_cast<const float2 *>(&in.vs[RAW ? 0 : 32 * c + 2 * i]);
                  y = mul2(y, make_float2(v2.x * unit, v2.y * unit));
                }
                pk[i] = pack<false>(y.x, y.y);
              }
            }
            tm_store16(s_at + 16 * c, pk);
            if (c & 1) {  // half of P is there
              tm_wait_st();
              tm_before();
              __syncwarp();
              if (lane == 0) bar_arrive(&sm.p_full[t][c >> 1]);
            }
          }
          l = add2(l, add2(add2(sums[0], sums[1]), add2(sums[2], sums[3])));
        }
        if (!ok) break;
        float sum = l.x + l.y;
        m += kOwnLift - kLift;
        if (done > 0) {
          if (!(ok = bar_wait(&sm.o_full[t], o_phase, &sm.dead))) break;
          o_phase ^= 1;
          tm_after();
        }
        const int slot_out = todo.slot;
        const bool whole = slot_out < 0;
        float f_mine = __int_as_float(v_exp << 23), f_other = 0.0f;
        if (split && t == 1) {  // hands over to a
          sm.ml[r][0] = m, sm.ml[r][1] = sum;
          if (r == 0) sm.ml_exp = v_exp;
          tm_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&sm.ml_full), bar_arrive(&sm.todo_empty[turn]);
          if (!(ok = bar_wait(&sm.ml_empty, ml_phase, &sm.dead))) break;
          ml_phase ^= 1;
        } else {
          bool both = false;
          if (split) {
            if (!(ok = bar_wait(&sm.ml_full, ml_phase, &sm.dead))) break;
            ml_phase ^= 1;
            tm_after();
            const float mb = sm.ml[r][0], lb = sm.ml[r][1], top = fmaxf(m, mb);
            both = n > 1;
            const float ka = m == -INFINITY ? 0.0f : ex2(m - top), kb = mb == -INFINITY ? 0.0f : ex2(mb - top);
            f_mine *= ka;
            f_other = kb * __int_as_float(sm.ml_exp << 23);
            sum = sum * ka + lb * kb;
            m = top;
          }
          const int64_t at = (int64_t(b) * a.T + tok) * a.Hq + head;
          float *part = a.parts + int64_t(slot_out) * kRows * (D + 2);
#pragma unroll 1
          for (int c = 0; c < D / 32; c++) {
            uint32_t y[32];
            tm_load(o_at + 32 * c, y);
            tm_landed(y);
#pragma unroll
            for (int i = 0; i < 32; i++) y[i] = __float_as_uint(__uint_as_float(y[i]) * f_mine);
            if (both) {
              uint32_t z[32];
              tm_load(o_at + kTile + 32 * c, z);
              tm_landed(z);
#pragma unroll
              for (int i = 0; i < 32; i++) y[i] = __float_as_uint(__uint_as_float(y[i]) + __uint_as_float(z[i]) * f_other);
            }
            if (whole) {
              if (b >= 0)
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                  if (32 * c + i < a.d) *reinterpret_cast<uint4 *>(a.pre + at * a.d + 32 * c + i) = make_uint4(y[i], y[i + 1], y[i + 2], y[i + 3]);
            } else if (b >= 0) {  // four channels of 32 rows lie together
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<uint4 *>(part + ((8 * c + i / 4) * kRows + t * kTile + r) * 4) = make_uint4(y[i], y[i + 1], y[i + 2], y[i + 3]);
            }
          }
          tm_before();
          if (b >= 0) {
            if (!whole) part[kRows * D + t * kTile + r] = m, part[kRows * (D + 1) + t * kTile + r] = sum;
            a.pre_ml[2 * at] = m, a.pre_ml[2 * at + 1] = whole ? sum : -1.0f;
          }
          __syncwarp();
          if (lane == 0) {
            if (split) bar_arrive(&sm.ml_empty);
            bar_arrive(&sm.todo_empty[turn]);
          }
        }
        turn ^= 1;
        if (turn == 0) todo_phase ^= 1;
      }
    }
  }
  __syncwarp();
  tm_before();
  __syncthreads();
  tm_after();
  if (sm.dead)  // what is in flight gets a moment to land
    for (int i = 0; i < 1000; i++) __nanosleep(1000);
  if (warp == 15) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  if (threadIdx.x == 0) a.notes[blockIdx.x].errors = sm.errors | (sm.dead ? kStTimeout : 0);
}

// A finished row's channels 4 c ...
__device__ inline void write_row(const SharedArgs &a, int64_t at, int c, float4 y, float top, float sum) {
  const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
  if (c * 4 < a.d) {
    const uint2 w = a.bf16 ? make_uint2(pack<true>(y.x * f, y.y * f), pack<true>(y.z * f, y.w * f))
                           : make_uint2(pack<false>(y.x * f, y.y * f), pack<false>(y.z * f, y.w * f));
    *reinterpret_cast<uint2 *>(a.out + at * a.d + c * 4) = w;
  }
  if (c == 0 && a.lse) a.lse[at] = sum == 0.0f ? -INFINITY : (top - kOwnLift + log2f(sum)) * 0.6931471805599453f;
}

// Rows whose prefix one CTA had: a warp per row, by the whole grid.
template <int D>
__device__ void join_whole(const SharedArgs &a, int64_t first, int64_t step) {
  const int lane = threadIdx.x & 31;
  const int64_t rows = int64_t(a.n_members) * a.T * a.Hq, of_one = int64_t(a.T) * a.Hq;
  const int e0 = a.cu[0], e1 = a.cu[a.n_groups];
  for (int64_t r = first; r < rows; r += step) {
    const int64_t e = r / of_one;
    if (e < e0 || e >= e1) continue;
    const int b = __ldcg(&a.seq[e]);
    if (b < 0) continue;
    const int64_t at = b * of_one + r % of_one;
    const float pl = __ldcg(&a.pre_ml[2 * at + 1]);
    if (pl < 0.0f) continue;
    const float pm = __ldcg(&a.pre_ml[2 * at]), om = __ldcg(&a.own_ml[2 * at]), ol = __ldcg(&a.own_ml[2 * at + 1]), top = fmaxf(pm, om);
    const float wp = pm == -INFINITY ? 0.0f : ex2(pm - top), wo = om == -INFINITY ? 0.0f : ex2(om - top);
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (lane * 4 < a.d) {
      const float4 p = __ldcg(reinterpret_cast<const float4 *>(a.pre + at * a.d) + lane);
      y = make_float4(p.x * wp, p.y * wp, p.z * wp, p.w * wp);
      if (om != -INFINITY) {
        const float4 o = __ldcg(reinterpret_cast<const float4 *>(a.own + at * a.d) + lane);
        y.x += o.x * wo, y.y += o.y * wo, y.z += o.z * wo, y.w += o.w * wo;
      }
    }
    write_row(a, at, lane, y, top, pl * wp + ol * wo);
  }
}

// Joins the parts of items that several CTAs had, with what each sequence has
// to itself: eight rows a CTA, four channels a thread.  First the rows' maxima
// and sums, then the outputs, eight parts' loads in flight.  The last kWholeY
// CTAs of each column look after the other rows.
constexpr int kWholeY = 4;

template <int D>
__global__ void __launch_bounds__(2 * D) k_shared_join(const __grid_constant__ SharedArgs a) {
  status_cleared();
  if (blockIdx.x == 0 && blockIdx.y == 0) {  // the status of the call, with that of the kernels before
    __shared__ uint32_t s_errors;
    if (threadIdx.x == 0) s_errors = __ldcg(a.bad);
    __syncthreads();
    uint32_t e = 0;
    for (int i = threadIdx.x; i < int(gridDim.x); i += 2 * D) e |= __ldcg(&a.notes[i].errors);
    if (e) atomicOr(&s_errors, e);
    __syncthreads();
    if (threadIdx.x == 0 && s_errors) atomicOr(a.status, s_errors);
  }
  if (blockIdx.y >= kRows / 8) {
    constexpr int kWarps = 2 * D / 32;
    if (__ldcg(a.any))
      join_whole<D>(a, (int64_t(blockIdx.y - kRows / 8) * gridDim.x + blockIdx.x) * kWarps + threadIdx.x / 32, int64_t(kWholeY) * gridDim.x * kWarps);
    return;
  }
  // what the kernels before the last one have written is read past the L1 cache
  union {
    int4 words[2];
    Note note;
  } u;
  u.words[0] = __ldcg(reinterpret_cast<const int4 *>(a.notes + blockIdx.x)), u.words[1] = __ldcg(reinterpret_cast<const int4 *>(a.notes + blockIdx.x) + 1);
  const Note &note = u.note;
  if (note.parts == 0 || note.row0 + int(blockIdx.y) * 8 >= note.rows) return;
  const int rr = threadIdx.x % 8, r = blockIdx.y * 8 + rr, c = threadIdx.x / 8, row = note.row0 + r;
  const int b = row < note.rows ? __ldcg(&a.seq[note.e0 + row / a.TG]) : -1;
  auto part = [&](int i) { return a.parts + (2 * (int64_t(blockIdx.x) + i) + (i == 0 ? note.second : 0)) * kRows * (D + 2); };
  float4 v[8];  // the first parts' outputs are on their way before their weights are known
  auto load = [&](int base) {
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (base + i < note.parts) v[i] = __ldcg(reinterpret_cast<const float4 *>(part(base + i)) + c * kRows + r);
  };
  load(0);
  __shared__ float s_m[kGrid][8], s_l[kGrid][8];  // of each part
  for (int i = c; i < note.parts; i += D / 4) {
    const float *p = part(i);
    s_m[i][rr] = __ldcg(p + kRows * D + r), s_l[i][rr] = __ldcg(p + kRows * (D + 1) + r);
  }
  const int64_t at = b >= 0 ? (int64_t(b) * a.T + row % a.TG / a.G) * a.Hq + note.head * a.G + row % a.G : 0;
  const float own_m = b >= 0 ? __ldcg(&a.own_ml[2 * at]) : -INFINITY, own_l = b >= 0 ? __ldcg(&a.own_ml[2 * at + 1]) : 0.0f;
  float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (own_m != -INFINITY && c * 4 < a.d) y = __ldcg(reinterpret_cast<const float4 *>(a.own + at * a.d + c * 4));
  __syncthreads();
  float top = own_m;
  for (int i = 0; i < note.parts; i++) top = fmaxf(top, s_m[i][rr]);
  const float own_w = own_m == -INFINITY ? 0.0f : ex2(own_m - top);
  float sum = own_l * own_w;
  for (int i = 0; i < note.parts; i++) sum += s_l[i][rr] * (s_m[i][rr] == -INFINITY ? 0.0f : ex2(s_m[i][rr] - top));
  if (b < 0) return;
  y.x *= own_w, y.y *= own_w, y.z *= own_w, y.w *= own_w;
  for (int base = 0; base < note.parts; base += 8) {
    if (base > 0) load(base);
#pragma unroll
    for (int i = 0; i < 8; i++)
      if (base + i < note.parts) {
        const float m = s_m[base + i][rr], w = m == -INFINITY ? 0.0f : ex2(m - top);
        y.x += w * v[i].x, y.y += w * v[i].y, y.z += w * v[i].z, y.w += w * v[i].w;
      }
  }
  write_row(a, at, c, y, top, sum);
}

bool groups_ok(const cg_cache *c, const cg_attend *t, const cg_groups *g) {
  return attend_args_ok(c, t) && g && g->n_groups >= 0 && g->n_groups <= (1 << 20) && g->n_members >= 0 && g->n_members <= (1 << 20) &&
         int64_t(g->n_members) * t->q_tokens * (t->Hq / c->H) <= (1 << 30);
}

int padded(int d) { return d <= 64 ? 64 : 128; }

struct Places {
  uint64_t bad, owner, first, seq, keys, lead, own, own_ml, pre, pre_ml, notes, parts, bytes;
};

Places places(const cg_cache *c, const cg_attend *t, const cg_groups *g) {
  Places w{};
  const uint64_t rows = uint64_t(t->n_seq) * t->q_tokens * t->Hq;
  w.bad = attend_own_bytes(c, t);
  w.bad = pad256(w.bad);
  w.owner = w.bad + 256;
  w.first = w.owner + pad256(4 * uint64_t(t->n_seq));
  w.seq = w.first + pad256(4 * uint64_t(t->n_seq));
  w.keys = w.seq + pad256(4 * uint64_t(g->n_members));
  w.lead = w.keys + pad256(4 * uint64_t(g->n_groups));
  w.own = w.lead + pad256(4 * uint64_t(g->n_groups));
  w.own_ml = w.own + pad256(4 * rows * c->d);
  w.pre = w.own_ml + pad256(8 * rows);
  w.pre_ml = w.pre + pad256(4 * rows * c->d);
  w.notes = w.pre_ml + pad256(8 * rows);
  w.parts = w.notes + pad256(sizeof(Note) * kGrid);
  w.bytes = w.parts + 4 * uint64_t(2 * kGrid) * kRows * (padded(c->d) + 2);
  return w;
}

template <int FMT, int D, int EACH>
cudaError_t launch(const SharedArgs &a, cudaStream_t st) {
  constexpr int kSmem = int(sizeof(Smem<D, EACH>));
  static_assert(kSmem <= 227 * 1024, "fits in an SM");
  const cudaError_t e = cudaFuncSetAttribute(k_shared<FMT, D, EACH>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  return launch_early(k_shared<FMT, D, EACH>, dim3(kGrid), dim3(kThreads), kSmem, st, a);
}

template <int FMT>
cudaError_t launch_format(const SharedArgs &a, cudaStream_t st) {
  const int each = a.bt % 16 == 0 ? 16 : a.bt % 8 == 0 ? 8 : 1;
  if (a.d <= 64) return each == 16 ? launch<FMT, 64, 16>(a, st) : each == 8 ? launch<FMT, 64, 8>(a, st) : launch<FMT, 64, 1>(a, st);
  return each == 16 ? launch<FMT, 128, 16>(a, st) : each == 8 ? launch<FMT, 128, 8>(a, st) : launch<FMT, 128, 1>(a, st);
}

}  // namespace
}  // namespace cg

extern "C" size_t cg_shared_workspace_bytes(const cg_cache *cache, const cg_attend *attend, const cg_groups *groups) {
  using namespace cg;
  if (!groups_ok(cache, attend, groups)) return 0;
  return size_t(places(cache, attend, groups).bytes);
}

extern "C" cg_status cg_shared_attend(const cg_cache *cache, const cg_attend *attend, const cg_groups *groups, const void *q_dev,
                                      const void *k_pool, const void *v_pool, const float *k_scale, const float *v_scale,
                                      const int32_t *table_dev, const int32_t *len_dev, void *out_dev, float *lse_dev,
                                      void *ws_dev, size_t ws_bytes, void *stream) {
  using namespace cg;
  if (!groups_ok(cache, attend, groups) || !q_dev || !k_pool || !v_pool || !k_scale || !v_scale || !table_dev || !len_dev || !out_dev || !ws_dev)
    return CG_ERR_INVALID_ARG;
  // groups without entries may be NULL
  if ((groups->n_groups > 0 && (!groups->cu_group_dev || !groups->shared_dev)) || (groups->n_members > 0 && !groups->member_dev))
    return CG_ERR_INVALID_ARG;
  if (!is_aligned(q_dev, 16) || !is_aligned(k_pool, 16) || !is_aligned(v_pool, 16) || !is_aligned(out_dev, 16) || !is_aligned(k_scale, 4) ||
      !is_aligned(v_scale, 4) || !is_aligned(table_dev, 4) || !is_aligned(len_dev, 4) || !is_aligned(lse_dev, 4) || !is_aligned(ws_dev, 256) ||
      !is_aligned(groups->cu_group_dev, 4) || !is_aligned(groups->member_dev, 4) || !is_aligned(groups->shared_dev, 4))
    return CG_ERR_INVALID_ARG;
  const Places w = places(cache, attend, groups);
  if (ws_bytes < w.bytes) return CG_ERR_INVALID_ARG;
  if (groups->n_groups == 0 || groups->n_members == 0)
    return cg_cache_attend(cache, attend, q_dev, k_pool, v_pool, k_scale, v_scale, table_dev, len_dev, out_dev, lse_dev, ws_dev, ws_bytes, stream);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t *ws = static_cast<uint8_t *>(ws_dev);
  SharedArgs a{};
  a.q = static_cast<const uint16_t *>(q_dev);
  a.kp = static_cast<const uint8_t *>(k_pool), a.vp = static_cast<const uint8_t *>(v_pool);
  a.ks = k_scale, a.vs = v_scale, a.table = table_dev, a.len = len_dev;
  a.out = static_cast<uint16_t *>(out_dev), a.lse = lse_dev;
  a.cu = groups->cu_group_dev, a.member = groups->member_dev, a.shared = groups->shared_dev;
  a.status = reinterpret_cast<uint32_t *>(ws), a.bad = reinterpret_cast<uint32_t *>(ws + w.bad);
  a.any = reinterpret_cast<int32_t *>(ws + w.bad + 4);
  a.pre = reinterpret_cast<float *>(ws + w.pre), a.pre_ml = reinterpret_cast<float *>(ws + w.pre_ml);
  a.owner = reinterpret_cast<int32_t *>(ws + w.owner), a.first = reinterpret_cast<int32_t *>(ws + w.first);
  a.seq = reinterpret_cast<int32_t *>(ws + w.seq), a.keys = reinterpret_cast<int32_t *>(ws + w.keys);
  a.lead = reinterpret_cast<int32_t *>(ws + w.lead);
  a.own = reinterpret_cast<float *>(ws + w.own), a.own_ml = reinterpret_cast<float *>(ws + w.own_ml);
  a.notes = reinterpret_cast<Note *>(ws + w.notes), a.parts = reinterpret_cast<float *>(ws + w.parts);
  a.q_seq = attend->q_stride[0], a.q_tok = attend->q_stride[1], a.q_head = attend->q_stride[2];
  a.n_groups = groups->n_groups, a.n_members = groups->n_members;
  a.B = attend->n_seq, a.T = attend->q_tokens, a.Hq = attend->Hq, a.H = cache->H, a.G = a.Hq / a.H, a.TG = a.T * a.G, a.d = cache->d;
  a.bt = cache->block_tokens, a.n_blocks = cache->n_blocks, a.stride = attend->table_stride;
  a.scale_log2 = attend->scale * 1.4426950408889634f;
  a.bf16 = attend->dtype == CG_BF16;
  a.chunk = kTile;
  while (a.bt % a.chunk) a.chunk /= 2;
  k_shared_plan<<<1, kPlan, 0, st>>>(a);
  cudaError_t e = cache->format == CG_CACHE_E4M3 ? launch_format<CG_CACHE_E4M3>(a, st) : launch_format<CG_CACHE_INT8>(a, st);
  if (e != cudaSuccess) return CG_ERR_CUDA;
  const cg_status rc = attend_own(cache, attend, a.first, a.own, a.own_ml, q_dev, k_pool, v_pool, k_scale, v_scale, table_dev, len_dev, out_dev,
                                  lse_dev, ws, st);
  if (rc != CG_OK) return rc;
  e = a.d <= 64 ? launch_early(k_shared_join<64>, dim3(kGrid, kRows / 8 + kWholeY), dim3(2 * 64), 0, st, a)
                : launch_early(k_shared_join<128>, dim3(kGrid, kRows / 8 + kWholeY), dim3(2 * 128), 0, st, a);
  return e == cudaSuccess ? launched() : CG_ERR_CUDA;
}
