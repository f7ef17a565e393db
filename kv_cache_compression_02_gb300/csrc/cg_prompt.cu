// cg_prompt.cu -- cg_prompt_attend: causal attention of packed prompts.
//
// The G = Hq / H query heads that share a KV head are rows of one matrix: row
// r of a tile of 128 is token r / G, head r % G (128 / G tokens, whole ones).
// An item is two such tiles, a and b, of one sequence and KV head; it goes over
// its keys in tiles of 128, and per tile and 128 rows there are two products of
// 128 x 128 x d on tcgen05: S = Q K^T into TMEM, and O += P V with P, the
// probabilities in the rows' type, read back from TMEM.
//
// What bounds it is those products (4 d operations a visible pair); the
// exponentials come next.  So the two tiles take turns: while the tensor cores
// work for one, a warpgroup computes the other's probabilities, one row a
// thread.  Warps: 0-3 and 4-7 the softmax of tiles a and b, 8 the loads (TMA),
// 9 the products, 10 looks after V's tiles that some row sees a part of only.
// TMEM: S of both tiles (P lies over S), O of both.
//
//   products:  S_a(0) S_b(0) | PV_a(j) S_a(j+1) PV_b(j) S_b(j+1) ...
//   softmax a: waits for S_a(j): maximum, exponentials, P_a(j); O_a is scaled
//              only when a maximum grows by more than 2^8
//
// A product is issued when its operands are there; tcgen05 runs them in the
// order of issue, so S_a(j+1) may overwrite P_a(j) behind PV_a(j), and S_a(j+1)
// being done says that O_a rests.
//
// P is rounded to the rows' type: a product takes both operands in one type, and
// what the rounding leaves would need a product of its own, three where there
// are two and the tensor cores are what is short.  Sums, maxima and O are fp32,
// and the sum takes P unrounded.  Errors of the outputs against 64 bits,
// relative: bf16 2.1e-3 (a 32-bit form whose outputs are rounded once 1.6e-3),
// f16 2.8e-4 (2.1e-4); with P rounded, under the same maxima, and all else in 64
// bits they are the same.
//
// The key tiles of all items are dealt in equal runs to one CTA per SM: the
// causal triangle needs no other balance, and a short question on a long
// context takes the whole GPU.  What a CTA has of an item that others share goes
// to the workspace as maximum, sum and output, and a second kernel joins the
// parts in their order.
//
// Measured, ten calls in a graph: 8192 tokens, 32 heads on 8, d = 128: 369 us,
// 1.5 PFLOP/s (the products are busy for two thirds of the time; what is left is
// a tile's chain of maximum, exponentials and hand-over; called back to back for
// longer, under the power limit, 398 us or 1.38 PFLOP/s).  77 queries of 64 heads on 32845
// keys: 82 us.  Rows of up to 64 channels have operands of 64 (8192 tokens, d =
// 64: 278 us; padded to 128 they take 360).
#include "cg_cache.cuh"
#include "cg_cross_few.cuh"
#include "cg_tc.cuh"
#include "cg_tma.cuh"

namespace cg {
namespace {

constexpr int kThreads = 384;
// Registers a thread: 384 are launched with 168 each; the softmax warpgroups
// take 216, which the third leaves them (2 * 216 + 72 = 3 * 168).
constexpr int kSoftRegs = 216, kOtherRegs = 72;
constexpr int kTile = 128;   // rows of a tile, keys of a tile
constexpr int kRows = 2 * kTile;
constexpr int kGrid = kSMs;
// Items are not split, but have a CTA each, where none is longer than one key
// tile, or than kShort and they fill a third of the GPU (64 items of four: 17.4
// us, dealt in runs 20.6; but 16 of four: 21.2 and 16.7).
constexpr int kShort = 4;
constexpr float kLift = 7.0f, kLag = 8.0f;  // p = 2^(s - m + kLift) < 2^15, m at most kLag under the maximum

struct Note {
  uint32_t errors;
  int32_t parts;   // of the item that this CTA has the first but not the last part of, or 0
  int32_t second;  // the first part is in this CTA's second slot
  int32_t b, h, q;
};

struct PromptArgs {
  CUtensorMap q_map, k_map, v_map;
  const int32_t *cu_q, *cu_k, *k_len;  // CROSS: cu_k is where each sequence's keys begin, k_len how many they are
  uint16_t *out;
  float *lse;
  uint32_t *status;
  Note *notes;
  float *parts;  // [2 * kGrid][kRows][D + 2]
  int n_seq, Hq, H, G, TG, W, d, max_q, max_k, n_q, n_k;  // TG: tokens of a tile; W: of an item
  float scale_log2;  // scale * log2(e)
};

// What a part's products and softmax need to know.
struct Todo {
  int cnt[2], tok[2];   // as in Part; cnt[0] < 0: the end
  int nq, nk, keys;     // keys: from the part's first on
  int q0, head, slot;   // head: the first query head; slot of the workspace, or -1: the item is whole
  int cut;              // the part's first key tile that not every row sees all of
  int careful;
};

// A product takes 0 * V for keys that a row does not see, which must not be
// NaN.  V's cut tiles are looked through for values that are not finite while
// the products run; where there is one, the CTA goes over its run once more,
// carefully: in cut tiles such values become 0 before the product, and the
// first keys that had one, of each channel, are kept for the way out.
template <int D>
struct Odd {
  uint16_t nan[D], up[D], down[D];  // NaN, inf, -inf: keys from the first cut tile on; 0xffff: none
};

template <int D>
struct Smem {
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kChunks = D / 64;  // of 64 channels: 128 bytes, a swizzled row
  uint8_t q[2][kChunks][kTile * 128];
  uint8_t kv[kStages][kChunks][kTile * 128];
  uint64_t todo_full[2], todo_empty[2], q_full, q_empty, kv_full[kStages], kv_empty[kStages], v_ok[kStages], odd_full[2], s_full[2], p_full[2][2], o_full[2];  // p_full: of the first and the second 64 keys
  uint8_t out[8][32 * 128];  // a softmax warp's rows on their way out, 64 channels at a time
  Odd<D> odd[2];             // of the parts, by their turns
  uint32_t any_odd[2];
  Todo todo[2];              // the parts of the run, by turns, from the loading warp to the others
  uint32_t tmem, errors, dead, again;  // again: the run is to be gone over once more
  int most[kThreads / 32], b;
  int64_t sum[kThreads / 32][2], prefix;
};

// ---- items ------------------------------------------------------------------
// sum of floor((a i + b) / 128), i < n; a < 2^16, b >= 0
__device__ inline int64_t tiles_sum(int64_t n, uint32_t a, int64_t b) {
  int64_t r = (n - 1) * n / 2 * (a / kTile) + n * (b / kTile);
  uint32_t m = kTile, c = uint32_t(b % kTile);
  a %= kTile;
  while (n > 0) {  // as points under a line, with the axes exchanged at each turn
    const uint64_t top = uint64_t(a) * n + c;
    if (top < m) break;
    const bool small = top >> 32 == 0;
    n = small ? uint32_t(top) / m : int64_t(top / m);
    c = small ? uint32_t(top) % m : uint32_t(top % m);
    const uint32_t t = m;
    m = a, a = t;
    r += (n - 1) * n / 2 * (a / m) + n * (c / m);
    a %= m, c %= m;
  }
  return r;
}

struct Seq {
  int q0, nq, k0, nk, items;
};

template <bool CROSS>
__device__ inline bool load_seq(const PromptArgs &a, int b, Seq &s) {
  s.q0 = a.cu_q[b], s.k0 = a.cu_k[b];
  const int q1 = a.cu_q[b + 1];
  const int64_t k1 = CROSS ? int64_t(s.k0) + a.k_len[b] : a.cu_k[b + 1];
  s.nq = q1 - s.q0, s.nk = int(k1 - s.k0);
  const bool ok = s.q0 >= 0 && q1 >= s.q0 && q1 <= a.n_q && s.nq <= a.max_q && s.k0 >= 0 && k1 >= s.k0 && k1 <= a.n_k && s.nk <= a.max_k;
  if (!ok) s.nq = 0;
  s.items = (s.nq + a.W - 1) / a.W;
  return ok;
}

// Key tiles that tokens before `tok` of a sequence see; at least one, so that
// every row gets an output.
template <bool CROSS>
__device__ inline int key_tiles(const Seq &s, int tok) {
  const int64_t seen = CROSS ? int64_t(s.nk) : min(int64_t(s.nk), int64_t(s.nk) - s.nq + tok);
  return seen <= kTile ? 1 : int((seen + kTile - 1) / kTile);
}

// What an item costs: kIn for its way in and out and kTileCost for each key
// tile (measured: 4.8 and 1.4 us; rows in one tile only cost nearly as much as
// rows in both, for then the turns do not fill up).
constexpr int kTileCost = 2, kIn = 7;

// What the items before item i of a sequence and head cost.
template <bool CROSS>
__device__ inline int64_t cost_before(const PromptArgs &a, const Seq &s, int i) {
  if (CROSS) return int64_t(i) * (key_tiles<true>(s, 0) * kTileCost + kIn);
  const bool all = i == s.items && i > 0;  // the last item may be a short one
  const int64_t n = all ? i - 1 : i;
  const int64_t base = int64_t(s.nk) - s.nq;  // item j < items - 1 sees base + (j + 1) W keys
  const int64_t ones = max(int64_t(0), min(n, base > kTile ? int64_t(0) : (kTile - base) / a.W));
  return n * kIn + kTileCost * (ones + tiles_sum(n - ones, a.W, base + (ones + 1) * a.W + kTile - 1)) + (all ? key_tiles<false>(s, s.nq) * kTileCost + kIn : 0);
}

// How many equal runs the costs of a call's items are dealt in: the CTAs that
// there are, or, where all items cost about the same, a few fewer, so that
// each item has a whole number of runs.  Then the items that read the same
// keys are at the same keys at the same time, and HBM gives them once (77
// queries of 64 heads on 32845 keys: 82 us on 144 CTAs, 87 us on 152).
__device__ inline int64_t aligned_runs(int64_t ctas, int64_t items, int64_t total, int64_t most) {
  if (items == 0 || items > ctas || total * 20 < items * most * 19) return ctas;
  const int64_t whole = ctas / items * items;
  return whole * 10 >= ctas * 9 ? whole : ctas;
}

struct Walk {
  Seq s;
  int b, h, q, n;  // item q of sequence b, head h, with n key tiles
  int64_t lo;       // where its cost begins
};

template <bool CROSS>
__device__ inline void set_item(const PromptArgs &a, Walk &w) {
  w.n = key_tiles<CROSS>(w.s, int(min(int64_t(w.s.nq), (int64_t(w.q) + 1) * a.W)));
}

// The next item; the caller knows that there is one.
template <bool CROSS>
__device__ inline void next_item(const PromptArgs &a, Walk &w, int skip) {
  w.lo += skip ? w.n * kTileCost + kIn : 1;
  if (++w.q == w.s.items) {
    w.q = 0;
    if (++w.h == a.H) {
      w.h = 0;
      do {
        w.b++;
        load_seq<CROSS>(a, w.b, w.s);
      } while (w.s.items == 0);
    }
  }
  set_item<CROSS>(a, w);
}

// A part of an item: key tiles j0 .. j0 + max(cnt) - 1, of which tile a of the rows
// has the first cnt[0] and tile b the first cnt[1].
struct Part {
  int b, h, q, q0, nq, k0, nk, j0, tok[2], cnt[2];
  int64_t first, last;  // where the costs of the item's first and last key tile begin
};

// The parts of a CTA's run [lo, hi), one after the other.
template <bool CROSS>
struct Run {
  Walk w;
  int64_t at, hi;
  int skip;  // 1: items have their costs; 0: each is one

  __device__ bool next(const PromptArgs &a, Part &p) {
    while (at < hi) {
      // a key tile belongs to the run in which its cost begins
      const int64_t cost = skip ? w.n * kTileCost + kIn : 1, end = min(hi, w.lo + cost);
      auto tiles_before = [&](int64_t x) { return int(max(int64_t(0), x - w.lo - kIn + kTileCost - 1)) / kTileCost; };
      const int j0 = skip ? tiles_before(at) : 0, j1 = skip ? tiles_before(end) : w.n;
      p.b = w.b, p.h = w.h, p.q = w.q, p.q0 = w.s.q0, p.nq = w.s.nq, p.k0 = w.s.k0, p.nk = w.s.nk, p.j0 = j0;
      p.first = w.lo + (skip ? kIn : 0), p.last = p.first + (skip ? (w.n - 1) * kTileCost : 0);
      for (int t = 0; t < 2; t++) {
        p.tok[t] = w.q * a.W + t * a.TG;
        const int n = p.tok[t] < w.s.nq ? key_tiles<CROSS>(w.s, min(w.s.nq, p.tok[t] + a.TG)) : 0;
        p.cnt[t] = max(0, min(j1, n) - j0);
      }
      at = end;
      if (at < hi) next_item<CROSS>(a, w, skip);
      if (j1 > j0) return true;
    }
    return false;
  }
};

// ---- the kernel -----------------------------------------------------------------
// CROSS: every query of a sequence sees all of its keys, which others may share
// and read at the same time.  Beside the lengths, only what a row sees last and
// what is done about values of V that are not finite differ.
template <int D, bool BF16, bool CROSS>
__global__ void __launch_bounds__(kThreads, 1) k_prompt(const __grid_constant__ PromptArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem<D> &sm = *reinterpret_cast<Smem<D> *>(smem_raw);
  constexpr int kStages = Smem<D>::kStages, kChunks = Smem<D>::kChunks;
  constexpr uint32_t kTileBytes = kChunks * kTile * 128;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x == 0) {
    sm.errors = sm.dead = sm.again = 0;
    a.notes[blockIdx.x].parts = 0;
    bar_init(&sm.q_full, 1), bar_init(&sm.q_empty, 1);
    for (int i = 0; i < 2; i++) bar_init(&sm.todo_full[i], 1), bar_init(&sm.todo_empty[i], 10), bar_init(&sm.odd_full[i], 1);  // ten warps read it
    for (int i = 0; i < kStages; i++) bar_init(&sm.kv_full[i], 1), bar_init(&sm.kv_empty[i], 1 + (i & 1)), bar_init(&sm.v_ok[i], 1);  // odd stages hold V
    for (int t = 0; t < 2; t++) bar_init(&sm.s_full[t], 1), bar_init(&sm.p_full[t][0], kTile / 32), bar_init(&sm.p_full[t][1], kTile / 32), bar_init(&sm.o_full[t], 1);
    bar_init_fence();
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_of(&sm.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // The items of the call and what they cost.
  const int per = (a.n_seq + kThreads - 1) / kThreads, b0 = threadIdx.x * per, b1 = min(a.n_seq, b0 + per);
  int64_t cost = 0, items = 0;
  int most = 0;
  bool bad = false;
  for (int b = b0; b < b1; b++) {
    Seq s;
    bad |= !load_seq<CROSS>(a, b, s);
    if (s.items == 0) continue;
    cost += cost_before<CROSS>(a, s, s.items) * a.H;
    items += int64_t(s.items) * a.H;
    most = max(most, key_tiles<CROSS>(s, s.nq));
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
  const bool few = most <= 1 || (most <= kShort && 3 * n_items >= gridDim.x);
  const int skip = few && n_items <= gridDim.x ? 0 : 1;  // 0: a CTA per item
  if (!skip) total = n_items, cost = items, cost_to = items_to;
  const int64_t before = cost_to - cost;
  if (blockIdx.x == 0 && bad) atomicOr(&sm.errors, kStBadArg);
  // No run but the first is shorter than a key tile, so that each has one of every item
  // that goes through it: the join takes a part from every CTA between those of the first
  // and last tile.  (Rounded up, an odd total leaves the first run one unit of cost; that
  // lies in the first item's way in, where no tile begins.)
  int64_t ctas = min(int64_t(gridDim.x), skip ? (total + kTileCost - 1) / kTileCost : total);
  if (skip) ctas = aligned_runs(ctas, n_items, total, int64_t(most) * kTileCost + kIn);
  const int64_t lo = ctas ? total * blockIdx.x / ctas : 0, hi = ctas ? total * (blockIdx.x + 1) / ctas : 0;
  const bool busy = int64_t(blockIdx.x) < ctas;
  if (busy && lo >= before && lo < before + cost) {  // one thread's sequences hold the first cost
    int64_t at = before;
    int b = b0;
    for (;; b++) {
      Seq s;
      load_seq<CROSS>(a, b, s);
      const int64_t n = s.items == 0 ? 0 : (skip ? cost_before<CROSS>(a, s, s.items) : s.items) * a.H;
      if (lo < at + n) break;
      at += n;
    }
    sm.b = b;
    sm.prefix = at;
  }
  __syncthreads();
  const uint32_t tmem = sm.tmem;

  if (busy) {
    if (warp >= 8) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
      if (warp == 8) {
      // ---- loads ----
      Run<CROSS> run;
      Part p;
      run.at = lo, run.hi = hi, run.skip = skip;
      Walk &w = run.w;
      w.b = sm.b;
      load_seq<CROSS>(a, w.b, w.s);
      const int64_t head = skip ? cost_before<CROSS>(a, w.s, w.s.items) : w.s.items;
      w.h = int((lo - sm.prefix) / head);
      const int64_t rest = lo - sm.prefix - w.h * head;
      int l = 0, n = w.s.items;  // the last item that begins at or before `rest` is one of l .. l + n - 1
      while (n > 1) {            // 32 of them at a time
        const int step = (n + 31) / 32, at = l + lane * step;
        const bool behind = lane > 0 && (at >= l + n || (skip ? cost_before<CROSS>(a, w.s, at) : at) > rest);
        const uint32_t first = __ballot_sync(0xffffffffu, behind);
        const int k = first ? __ffs(first) - 2 : 31;
        n = min(step, l + n - (l + k * step));
        l += k * step;
      }
      w.q = l;
      w.lo = sm.prefix + w.h * head + (skip ? cost_before<CROSS>(a, w.s, l) : l);
      set_item<CROSS>(a, w);
      if (lane == 0) {
        int stage = 0, turn = 0, seg = 0;
        uint32_t kv_phase = 1, q_phase = 1, todo_phase = 1;  // the first pass over a ring finds it empty
        bool ok = true;
        const uint32_t q_bytes = uint32_t(kChunks) * 128 * a.G * a.TG;
        const Run<CROSS> begin = run;
        int careful = 0;
        for (;;) {
          const bool more = run.next(a, p);
          if (!(ok = bar_wait(&sm.todo_empty[turn], todo_phase, &sm.dead))) break;
          Todo &todo = sm.todo[turn];
          if (!more) {
            if (!careful) {  // once all is done: is it to be gone over again?
              if (!(ok = bar_wait(&sm.todo_empty[turn ^ 1], turn ? todo_phase ^ 1 : todo_phase, &sm.dead))) break;
              if (*static_cast<volatile uint32_t *>(&sm.again)) {
                careful = 1;
                run = begin;
                seg = 0;
                continue;
              }
            }
            todo.cnt[0] = todo.cnt[1] = -1;
            bar_arrive(&sm.todo_full[turn]);
            break;
          }
          todo.careful = careful;
          // who has key tiles of this item
          const int64_t c0 = ((p.first + 1) * ctas - 1) / total, c1 = ((p.last + 1) * ctas - 1) / total;
          for (int t = 0; t < 2; t++) todo.cnt[t] = p.cnt[t], todo.tok[t] = p.tok[t];
          todo.nq = p.nq, todo.nk = p.nk, todo.keys = p.nk - p.j0 * kTile, todo.q0 = p.q0, todo.head = p.h * a.G;
          const int least = (CROSS ? p.nk - 1 : min(p.nk - 1, p.nk - p.nq + p.tok[p.cnt[0] > 0 ? 0 : 1])) - p.j0 * kTile;  // the last key of the first row
          todo.cut = max(0, least + 1) / kTile;
          todo.slot = c0 == c1 ? -1 : 2 * int(blockIdx.x) + (seg > 0);  // slot 1: the run's last part
          bar_arrive(&sm.todo_full[turn]);
          if (c0 != c1 && int64_t(blockIdx.x) == c0) {
            Note &note = a.notes[blockIdx.x];
            note.parts = int(c1 - c0 + 1), note.second = seg > 0, note.b = p.b, note.h = p.h, note.q = p.q;
          }
          seg++;
          turn ^= 1;
          if (turn == 0) todo_phase ^= 1;
          const int n = max(p.cnt[0], p.cnt[1]);
          if (!(ok = bar_wait(&sm.q_empty, q_phase, &sm.dead))) break;
          q_phase ^= 1;
          bar_expect(&sm.q_full, q_bytes * ((p.cnt[0] > 0) + (p.cnt[1] > 0)));
          for (int t = 0; t < 2; t++)
            if (p.cnt[t] > 0)
              for (int c = 0; c < kChunks; c++) tma_3d(smem_of(sm.q[t][c]), &a.q_map, &sm.q_full, 64 * c, p.h * a.G, p.q0 + p.tok[t]);
          for (int j = 0; j < 2 * n && ok; j++) {  // K, V, K, V ...
            if (!(ok = bar_wait(&sm.kv_empty[stage], kv_phase, &sm.dead))) break;
            bar_expect(&sm.kv_full[stage], kTileBytes);
            const CUtensorMap *map = j & 1 ? &a.v_map : &a.k_map;
            for (int c = 0; c < kChunks; c++)
              tma_3d(smem_of(sm.kv[stage][c]), map, &sm.kv_full[stage], 64 * c, p.k0 + (p.j0 + j / 2) * kTile, p.h);
            if (++stage == kStages) stage = 0, kv_phase ^= 1;
          }
        }
      }
    } else if (warp == 9) {
      // ---- products ----
      constexpr uint32_t kType = BF16 ? 1u : 0u;
      constexpr uint32_t kCommon = 1u << 4 | kType << 7 | kType << 10 | uint32_t(kTile >> 4) << 24;
      constexpr uint32_t kS = kCommon | uint32_t(kTile >> 3) << 17, kO = kCommon | 1u << 16 | uint32_t(D >> 3) << 17;
      constexpr uint32_t kChunk = kTile * 128 >> 4, kStage = kTileBytes >> 4;
      const uint32_t q_lo = operand_lo(sm.q[0], 16), k_lo = operand_lo(sm.kv[0], 16), v_lo = operand_lo(sm.kv[0], kTile * 128);
      int stage = 0, turn = 0;
      uint32_t kv_phase = 0, q_phase = 0, todo_phase = 0, p_phase[2] = {0, 0}, v_phases = 0;
      bool ok = true;
      auto advance = [&] {
        if (++stage == kStages) stage = 0, kv_phase ^= 1;
      };
      auto s_product = [&](int t, int st) {  // S_t = Q_t K^T
        const uint32_t a0 = q_lo + t * kStage, b0 = k_lo + st * kStage;
        if (elected()) {
#pragma unroll
          for (int k = 0; k < D / 16; k++)
            mma_ss(tmem + t * kTile, a0 + k / 4 * kChunk + k % 4 * 2, b0 + k / 4 * kChunk + k % 4 * 2, kS, k > 0);
          mma_commit(&sm.s_full[t]);
        }
      };
      for (;;) {
        if (!(ok = bar_wait(&sm.todo_full[turn], todo_phase, &sm.dead))) break;
        const int cnt[2] = {sm.todo[turn].cnt[0], sm.todo[turn].cnt[1]}, cut = sm.todo[turn].cut, keys = sm.todo[turn].keys, careful = sm.todo[turn].careful;
        __syncwarp();
        if (lane == 0) bar_arrive(&sm.todo_empty[turn]);
        turn ^= 1;
        if (turn == 0) todo_phase ^= 1;
        if (cnt[0] < 0) break;
        const int n = max(cnt[0], cnt[1]);
        if (!(ok = bar_wait(&sm.q_full, q_phase, &sm.dead))) break;
        q_phase ^= 1;
        if (!(ok = bar_wait(&sm.kv_full[stage], kv_phase, &sm.dead))) break;
        tm_after();
#pragma unroll
        for (int t = 0; t < 2; t++)
          if (cnt[t] > 0) s_product(t, stage);
        if (elected()) {
          mma_commit(&sm.kv_empty[stage]);
          if (n == 1) mma_commit(&sm.q_empty);
        }
        advance();
        for (int j = 0; j < n && ok; j++) {
          const int vs = stage;
          const uint32_t v_phase = kv_phase;
          advance();
          const int ks = stage;
          const uint32_t k_phase = kv_phase;
          const bool more = j + 1 < n;
          if (!(ok = bar_wait(&sm.kv_full[vs], v_phase, &sm.dead))) break;
          if (careful ? j >= cut : keys - j * kTile < kTile) {  // V is being put right
            if (!(ok = bar_wait(&sm.v_ok[vs], v_phases >> vs & 1, &sm.dead))) break;
            v_phases ^= 1u << vs;
          }
          if (more && !(ok = bar_wait(&sm.kv_full[ks], k_phase, &sm.dead))) break;
#pragma unroll
          for (int t = 0; t < 2; t++) {
            if (j >= cnt[t]) continue;
            const uint32_t b0 = v_lo + vs * kStage;
#pragma unroll
            for (int half = 0; half < 2; half++) {  // O_t += P_t V
              if (!(ok = bar_wait(&sm.p_full[t][half], p_phase[t], &sm.dead))) break;
              tm_after();
              if (elected())
#pragma unroll
                for (int k = half * 4; k < half * 4 + 4; k++)
                  mma_ts(tmem + 2 * kTile + t * kTile, tmem + t * kTile + k * 8, b0 + k * (2048 >> 4), kO, j > 0 || k > 0);
            }
            if (!ok) break;
            p_phase[t] ^= 1;
            if (j + 1 < cnt[t])
              s_product(t, ks);
            else if (elected())
              mma_commit(&sm.o_full[t]);
          }
          if (!ok) break;
          if (elected()) {
            mma_commit(&sm.kv_empty[vs]);
            if (more) mma_commit(&sm.kv_empty[ks]);
            if (j + 2 == n) mma_commit(&sm.q_empty);
          }
          if (more) advance();
        }
        if (!ok) break;
      }
      } else if (warp == 10) {
        // ---- V of cut tiles ----
        int stage = 0, turn = 0;
        uint32_t kv_phase = 0, todo_phase = 0;
        bool ok = true;
        constexpr int kMine = D / 32;  // channels of a lane
        constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u;
        for (;;) {
          if (!(ok = bar_wait(&sm.todo_full[turn], todo_phase, &sm.dead))) break;
          const int n = max(sm.todo[turn].cnt[0], sm.todo[turn].cnt[1]), keys = sm.todo[turn].keys, cut = sm.todo[turn].cut;
          const bool careful = sm.todo[turn].careful;
          uint32_t nan[kMine], up[kMine], down[kMine];
          bool any = false;
#pragma unroll
          for (int k = 0; k < kMine; k++) nan[k] = up[k] = down[k] = 0xffffu;
          for (int j = 0; j < n; j++) {
            const int vs = stage + 1;  // K is at `stage`
            if (!(ok = bar_wait(&sm.kv_full[vs], kv_phase, &sm.dead))) break;
            if (j >= cut) {
              const int left = min(kTile, keys - j * kTile);  // keys of the tile
              uint4 *v = reinterpret_cast<uint4 *>(sm.kv[vs][0]);
              if (left < kTile) {  // nothing behind the last key
                for (int i = lane; i < kTile * 8 * kChunks; i += 32)
                  if (i / 8 % kTile >= left) v[i] = make_uint4(0, 0, 0, 0);
                fence_async();
                __syncwarp();
                if (!careful && lane == 0) bar_arrive(&sm.v_ok[vs]);
              }
              if (!CROSS) {  // (no row sees a part of the keys that are left)
                uint32_t top = 0;
#pragma unroll 8
                for (int i = lane; i < kTile * 8 * kChunks; i += 32) {
                  const uint4 w = v[i];
                  top = __vmaxu2(top, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
                }
                const bool odd = __any_sync(0xffffffffu, max(top & 0xffffu, top >> 16) >= kInf);
                if (odd && !careful) sm.again = 1;
                if (odd && careful) {
                  any = true;
                  for (int r = 0; r < left; r++)
#pragma unroll
                    for (int k = 0; k < kMine; k++) {
                      const int ch = lane * kMine + k;
                      uint16_t *x = reinterpret_cast<uint16_t *>(sm.kv[vs][ch / 64] + r * 128 + ((ch % 64 / 8 ^ (r & 7)) << 4)) + ch % 8;
                      const uint32_t w = *x, at = uint32_t(j - cut) * kTile + r;
                      if ((w & 0x7fffu) < kInf) continue;
                      if ((w & 0x7fffu) > kInf)
                        nan[k] = min(nan[k], at);
                      else if (w >> 15)
                        down[k] = min(down[k], at);
                      else
                        up[k] = min(up[k], at);
                      *x = 0;
                    }
                  fence_async();
                }
                __syncwarp();
                if (careful && lane == 0) bar_arrive(&sm.v_ok[vs]);
              }
            }
            if (lane == 0) bar_arrive(&sm.kv_empty[vs]);
            stage += 2;
            if (stage == kStages) stage = 0, kv_phase ^= 1;
          }
          if (!ok || n < 0) break;
          if (any)
#pragma unroll
            for (int k = 0; k < kMine; k++) {
              const int ch = lane * kMine + k;
              sm.odd[turn].nan[ch] = uint16_t(nan[k]), sm.odd[turn].up[ch] = uint16_t(up[k]), sm.odd[turn].down[ch] = uint16_t(down[k]);
            }
          if (lane == 0) sm.any_odd[turn] = any;
          __syncwarp();
          if (careful && lane == 0) bar_arrive(&sm.odd_full[turn]);
          if (lane == 0) bar_arrive(&sm.todo_empty[turn]);
          turn ^= 1;
          if (turn == 0) todo_phase ^= 1;
        }
      }
    } else {
      // ---- softmax: a row a thread ----
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
      const int t = warp >> 2, r = threadIdx.x & (kTile - 1);
      const uint32_t row = uint32_t(warp & 3) << 21;  // the warp's lanes of TMEM
      const uint32_t s_at = tmem + row + t * kTile, o_at = tmem + row + 2 * kTile + t * kTile;
      uint32_t s_phase = 0, o_phase = 0, todo_phase = 0, odd_phase = 0;
      int turn = 0;
      bool ok = true;
      const int my_tok = r / a.G;
      const float2 sc = make_float2(a.scale_log2, a.scale_log2);
      for (;;) {
        if (!(ok = bar_wait(&sm.todo_full[turn], todo_phase, &sm.dead))) break;
        const Todo &todo = sm.todo[turn];
        const int cnt = todo.cnt[0] < 0 ? -1 : todo.cnt[t];
        // the last key seen, from the part's first
        const int last = CROSS ? todo.keys - 1 : min(todo.nk - 1, todo.nk - todo.nq + todo.tok[t] + my_tok) - (todo.nk - todo.keys);
        if (cnt < 0) break;
        float m = -INFINITY;
        float2 l = make_float2(0.0f, 0.0f);
        for (int j = 0; j < cnt; j++) {
          if (!(ok = bar_wait(&sm.s_full[t], s_phase, &sm.dead))) break;
          s_phase ^= 1;
          tm_after();
          uint32_t x[kTile];
#pragma unroll
          for (int i = 0; i < 4; i++) tm_load(s_at + 32 * i, x + 32 * i);
          tm_wait_ld();
          const int lim = last - j * kTile;
          if (__any_sync(0xffffffffu, lim < kTile - 1)) {
#pragma unroll
            for (int i = 0; i < kTile; i++)
              if (i > lim) x[i] = 0xff800000u;
          }
          float top[4];
#pragma unroll
          for (int i = 0; i < 4; i++) top[i] = fmaxf(__uint_as_float(x[i]), __uint_as_float(x[i + 4]));
#pragma unroll
          for (int i = 8; i < kTile; i += 8)
#pragma unroll
            for (int k = 0; k < 4; k++) top[k] = max3(top[k], __uint_as_float(x[i + 2 * k]), __uint_as_float(x[i + 2 * k + 1]));
          const float now = max3(top[0], top[1], fmaxf(top[2], top[3])) * a.scale_log2;
          const bool moved = now > m + kLag;
          const float keep = moved ? ex2(m - now) : 1.0f;
          if (moved) m = now;
          if (j > 0 && __any_sync(0xffffffffu, moved)) {
            l = mul2(l, make_float2(keep, keep));
#pragma unroll
            for (int c = 0; c < D / 32; c++) {
              uint32_t y[32];
              tm_load(o_at + 32 * c, y);
              tm_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; i++) y[i] = __float_as_uint(__uint_as_float(y[i]) * keep);
              tm_store32(o_at + 32 * c, y);
            }
          }
          const float base = kLift - (m == -INFINITY ? 0.0f : m);
          float2 sums[4] = {};
#pragma unroll
          for (int c = 0; c < 4; c++) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; i++) {
              float2 y = make_float2(__uint_as_float(x[32 * c + 2 * i]), __uint_as_float(x[32 * c + 2 * i + 1]));
              y = fma2(y, sc, make_float2(base, base));
              y = make_float2(ex2(y.x), ex2(y.y));
              sums[i & 3] = add2(sums[i & 3], y);
              pk[i] = pack<BF16>(y.x, y.y);
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
        const float sum = l.x + l.y;
        const bool some = cnt > 0;
        if (some) {
          if (!(ok = bar_wait(&sm.o_full[t], o_phase, &sm.dead))) break;
          o_phase ^= 1;
          tm_after();
        }
        // what the loop above did not need
        const int tok = todo.tok[t] + my_tok, slot = todo.slot, last_cut = last - todo.cut * kTile;
        const bool mine = my_tok < a.TG && tok < todo.nq;
        const int64_t at = (int64_t(todo.q0) + tok) * a.Hq + todo.head + r % a.G;
        bool odd = false;
        if (todo.careful) {
          if (!(ok = bar_wait(&sm.odd_full[turn], odd_phase >> turn & 1, &sm.dead))) break;
          odd_phase ^= 1u << turn;
          odd = sm.any_odd[turn];
        }
        const bool whole = slot < 0;
        float *part = a.parts + int64_t(slot) * kRows * (D + 2);
        const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
        const uint32_t live = __ballot_sync(0xffffffffu, mine);
#pragma unroll
        for (int c2 = 0; c2 < D / 64; c2++) {
#pragma unroll
          for (int c = 2 * c2; c < 2 * c2 + 2; c++) {
            uint32_t y[32];
            if (some) {
              tm_load(o_at + 32 * c, y);
              tm_wait_ld();
            } else {
#pragma unroll
              for (int i = 0; i < 32; i++) y[i] = 0;
            }
            if (odd) {  // rare
#pragma unroll
              for (int i = 0; i < 32; i++) {
                const Odd<D> &w = sm.odd[turn];
                const int ch = 32 * c + i;
                auto seen = [&](uint16_t key) { return key != 0xffff && last_cut >= int(key); };
                if (seen(w.nan[ch])) y[i] = 0x7fffffffu;
                if (seen(w.up[ch])) y[i] = __float_as_uint(__uint_as_float(y[i]) + INFINITY);
                if (seen(w.down[ch])) y[i] = __float_as_uint(__uint_as_float(y[i]) - INFINITY);
              }
            }
            if (whole) {  // to the warp's rows of 128 bytes, swizzled
#pragma unroll
              for (int i = 0; i < 32; i += 8) {
                uint32_t w4[4];
#pragma unroll
                for (int k = 0; k < 4; k++) w4[k] = pack<BF16>(__uint_as_float(y[i + 2 * k]) * f, __uint_as_float(y[i + 2 * k + 1]) * f);
                const int chunk = c % 2 * 4 + i / 8;
                *reinterpret_cast<uint4 *>(sm.out[warp] + lane * 128 + ((chunk ^ (lane & 7)) << 4)) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
              }
            } else if (mine) {  // four channels of 32 rows lie together
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<uint4 *>(part + ((8 * c + i / 4) * kRows + t * kTile + r) * 4) = make_uint4(y[i], y[i + 1], y[i + 2], y[i + 3]);
            }
          }
          if (whole) {  // eight lanes write 128 bytes of a row
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; i++) {
              const int rr = 4 * i + lane / 8, chunk = lane % 8, ch = 64 * c2 + 8 * chunk;
              const int64_t to = __shfl_sync(0xffffffffu, at, rr);
              if ((live >> rr & 1) && ch < a.d)
                *reinterpret_cast<uint4 *>(a.out + to * a.d + ch) = *reinterpret_cast<const uint4 *>(sm.out[warp] + rr * 128 + ((chunk ^ (rr & 7)) << 4));
            }
            __syncwarp();
          }
        }
        tm_before();
        if (mine) {
          if (whole) {
            if (a.lse) a.lse[at] = sum == 0.0f ? -INFINITY : (m - kLift + log2f(sum)) * 0.6931471805599453f;
          } else {
            part[kRows * D + t * kTile + r] = m, part[kRows * (D + 1) + t * kTile + r] = sum;
          }
        }
        __syncwarp();
        if (lane == 0) bar_arrive(&sm.todo_empty[turn]);
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
  if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  if (threadIdx.x == 0) a.notes[blockIdx.x].errors = sm.errors | (sm.dead ? kStTimeout : 0);
}

// Joins the parts of items that several CTAs had: for a CTA that has the first
// part of such an item, eight rows a CTA, four channels a thread.  It is
// launched with the first kernel and waits for its end here.
template <int D, bool BF16>
__global__ void __launch_bounds__(2 * D, 2048 / (2 * D)) k_prompt_join(const __grid_constant__ PromptArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.x == 0 && blockIdx.y == 0) {  // the status of the call
    __shared__ uint32_t s_errors;
    if (threadIdx.x == 0) s_errors = 0;
    __syncthreads();
    uint32_t e = 0;
    for (int i = threadIdx.x; i < int(gridDim.x); i += 2 * D) e |= __ldcg(&a.notes[i].errors);
    if (e) atomicOr(&s_errors, e);
    __syncthreads();
    if (threadIdx.x == 0) *a.status = s_errors;
  }
  const Note note = a.notes[blockIdx.x];
  if (note.parts == 0) return;
  const int r = blockIdx.y * 8 + threadIdx.x % 8, c = threadIdx.x / 8, t = r / kTile, rt = r % kTile;
  const int tok = note.q * a.W + t * a.TG + rt / a.G, q0 = a.cu_q[note.b];
  if (rt / a.G >= a.TG || tok >= a.cu_q[note.b + 1] - q0) return;
  auto part = [&](int i) { return a.parts + (2 * (int64_t(blockIdx.x) + i) + (i == 0 ? note.second : 0)) * kRows * (D + 2); };
  float top = -INFINITY, sum = 0.0f, y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int base = 0; base < note.parts; base += 2) {
    float m[2], l[2], now = top;
    float4 v[2];
#pragma unroll
    for (int i = 0; i < 2; i++)
      if (base + i < note.parts) {
        const float *p = part(base + i);
        m[i] = __ldcg(p + kRows * D + r), l[i] = __ldcg(p + kRows * (D + 1) + r);
        v[i] = __ldcg(reinterpret_cast<const float4 *>(p) + c * kRows + r);
        now = fmaxf(now, m[i]);
      }
    const float keep = top == -INFINITY ? 0.0f : ex2(top - now);
    top = now;
    sum *= keep;
#pragma unroll
    for (int k = 0; k < 4; k++) y[k] *= keep;
#pragma unroll
    for (int i = 0; i < 2; i++)
      if (base + i < note.parts) {
        const float w = m[i] == -INFINITY ? 0.0f : ex2(m[i] - now);
        sum += w * l[i];
        y[0] += w * v[i].x, y[1] += w * v[i].y, y[2] += w * v[i].z, y[3] += w * v[i].w;
      }
  }
  const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int64_t at = (int64_t(q0) + tok) * a.Hq + note.h * a.G + rt % a.G;
  if (c * 4 < a.d) *reinterpret_cast<uint2 *>(a.out + at * a.d + c * 4) = make_uint2(pack<BF16>(y[0] * f, y[1] * f), pack<BF16>(y[2] * f, y[3] * f));
  if (c == 0 && a.lse) a.lse[at] = sum == 0.0f ? -INFINITY : (top - kLift + log2f(sum)) * 0.6931471805599453f;
}

// The status of a call without queries: only its offsets are looked at.
template <bool CROSS>
__global__ void __launch_bounds__(kThreads) k_prompt_none(const int32_t *cu_q, const int32_t *cu_k, const int32_t *k_len, int n_seq, int max_q, int max_k, int n_q, int n_k,
                                                          uint32_t *status) {
  PromptArgs a{};
  a.cu_q = cu_q, a.cu_k = cu_k, a.k_len = k_len, a.max_q = max_q, a.max_k = max_k, a.n_q = n_q, a.n_k = n_k, a.W = 1;
  bool bad = false;
  for (int b = threadIdx.x; b < n_seq; b += kThreads) {
    Seq s;
    bad |= !load_seq<CROSS>(a, b, s);
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) *status = bad ? kStBadArg : 0;
}

bool prompt_ok(const cg_prompt *p) {
  if (!p || p->n_seq < 1 || p->n_seq > 65535 || p->H < 1 || p->Hq < 1 || p->Hq > 65535 || p->Hq % p->H ||
      p->Hq / p->H > 128 || p->d < 8 || p->d > 128 || p->d % 8 || (p->dtype != CG_F16 && p->dtype != CG_BF16) ||
      p->max_q < 0 || p->max_k < 0 || p->n_q < 0 || p->n_k < 0 || p->n_q > (1 << 30) || p->n_k > (1 << 30) || !std::isfinite(p->scale) || !(p->scale > 0.0f))
    return false;
  for (int i = 0; i < 2; i++)
    if (p->q_stride[i] % 8 || p->k_stride[i] % 8 || p->v_stride[i] % 8) return false;
  return true;
}

int padded(int d) { return d <= 64 ? 64 : 128; }

// the status word, then the notes
constexpr uint64_t kNotes = 256 + ((sizeof(Note) * kGrid + 255) & ~uint64_t(255));

template <int D, bool BF16, bool CROSS>
cudaError_t launch(const PromptArgs &a, unsigned grid, cudaStream_t st) {
  constexpr int kSmem = int(sizeof(Smem<D>));
  static_assert(kSmem <= 227 * 1024, "fits in an SM");
  const cudaError_t e = cudaFuncSetAttribute(k_prompt<D, BF16, CROSS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  k_prompt<D, BF16, CROSS><<<grid, kThreads, kSmem, st>>>(a);
  const cudaError_t e2 = launch_early(k_prompt_join<D, BF16>, dim3(grid, kRows / 8), dim3(2 * D), 0, st, a);
  return e2 != cudaSuccess ? e2 : cudaGetLastError();
}

size_t workspace_bytes(const cg_prompt &p) {
  const uint64_t bytes = kNotes + 4 * uint64_t(2 * kGrid) * kRows * (padded(p.d) + 2);
  return size_t(bytes > few_bytes(p) ? bytes : few_bytes(p));
}

// Both calls: k_first is cu_k, or (CROSS) where each sequence's keys begin.
template <bool CROSS>
cg_status attend(const cg_prompt *prompt, const void *q_dev, const void *k_dev, const void *v_dev, const int32_t *cu_q_dev,
                 const int32_t *k_first_dev, const int32_t *k_len_dev, void *out_dev, float *lse_dev, void *ws_dev, size_t ws_bytes, void *stream) {
  // arrays without rows may be NULL
  if (!prompt_ok(prompt) || ((!q_dev || !out_dev) && prompt->n_q > 0) || ((!k_dev || !v_dev) && prompt->n_k > 0) || !cu_q_dev || !k_first_dev ||
      (CROSS && !k_len_dev) || !ws_dev)
    return CG_ERR_INVALID_ARG;
  if (!is_aligned(q_dev, 16) || !is_aligned(k_dev, 16) || !is_aligned(v_dev, 16) || !is_aligned(out_dev, 16) ||
      !is_aligned(cu_q_dev, 4) || !is_aligned(k_first_dev, 4) || !is_aligned(k_len_dev, 4) || !is_aligned(lse_dev, 4) || !is_aligned(ws_dev, 256) ||
      ws_bytes < workspace_bytes(*prompt))
    return CG_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t *ws = static_cast<uint8_t *>(ws_dev);
  const cg_prompt &p = *prompt;
  if (p.max_q == 0 || p.n_q == 0) {
    k_prompt_none<CROSS><<<1, kThreads, 0, st>>>(cu_q_dev, k_first_dev, k_len_dev, p.n_seq, p.max_q, p.max_k, p.n_q, p.n_k, reinterpret_cast<uint32_t *>(ws));
    return launched();
  }
  PromptArgs a{};
  a.cu_q = cu_q_dev, a.cu_k = k_first_dev, a.k_len = k_len_dev;
  a.out = static_cast<uint16_t *>(out_dev), a.lse = lse_dev;
  a.status = reinterpret_cast<uint32_t *>(ws);
  a.notes = reinterpret_cast<Note *>(ws + 256);
  a.parts = reinterpret_cast<float *>(ws + kNotes);
  a.n_seq = p.n_seq, a.Hq = p.Hq, a.H = p.H, a.G = p.Hq / p.H, a.TG = kTile / a.G, a.W = 2 * a.TG, a.d = p.d;
  a.max_q = p.max_q, a.max_k = p.max_k, a.n_q = p.n_q, a.n_k = p.n_k;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  bool ok = make_map(&a.q_map, q_dev, p.d, p.Hq, p.q_stride[1], a.G, p.n_q, p.q_stride[0], a.TG);
  if (p.n_k > 0) {
    ok = ok && make_map(&a.k_map, k_dev, p.d, p.n_k, p.k_stride[0], kTile, p.H, p.k_stride[1], 1);
    ok = ok && make_map(&a.v_map, v_dev, p.d, p.n_k, p.v_stride[0], kTile, p.H, p.v_stride[1], 1);
  } else {  // no key is seen: what is loaded in its place is masked
    ok = ok && make_map(&a.k_map, q_dev, p.d, p.n_q, p.q_stride[0], kTile, p.Hq, p.q_stride[1], 1);
    a.v_map = a.k_map;
  }
  if (!ok) return CG_ERR_INVALID_ARG;  // strides that a tensor map cannot have
  const bool bf16 = p.dtype == CG_BF16;
  if (CROSS && int64_t(p.max_q) * a.G <= kFewRows)
    return cross_few(p, q_dev, k_dev, v_dev, cu_q_dev, k_first_dev, k_len_dev, out_dev, lse_dev, ws, st);
  const cudaError_t e = p.d <= 64 ? (bf16 ? launch<64, true, CROSS>(a, kGrid, st) : launch<64, false, CROSS>(a, kGrid, st))
                                  : (bf16 ? launch<128, true, CROSS>(a, kGrid, st) : launch<128, false, CROSS>(a, kGrid, st));
  return e == cudaSuccess ? CG_OK : CG_ERR_CUDA;
}

}  // namespace
}  // namespace cg

extern "C" size_t cg_prompt_workspace_bytes(const cg_prompt *prompt) {
  using namespace cg;
  if (!prompt_ok(prompt)) return 0;
  return workspace_bytes(*prompt);
}

extern "C" cg_status cg_prompt_attend(const cg_prompt *prompt, const void *q_dev, const void *k_dev,
                                      const void *v_dev, const int32_t *cu_q_dev, const int32_t *cu_k_dev,
                                      void *out_dev, float *lse_dev, void *ws_dev, size_t ws_bytes, void *stream) {
  return cg::attend<false>(prompt, q_dev, k_dev, v_dev, cu_q_dev, cu_k_dev, nullptr, out_dev, lse_dev, ws_dev, ws_bytes, stream);
}

extern "C" cg_status cg_cross_attend(const cg_prompt *prompt, const void *q_dev, const void *k_dev, const void *v_dev,
                                     const int32_t *cu_q_dev, const int32_t *k_begin_dev, const int32_t *k_len_dev,
                                     void *out_dev, float *lse_dev, void *ws_dev, size_t ws_bytes, void *stream) {
  return cg::attend<true>(prompt, q_dev, k_dev, v_dev, cu_q_dev, k_begin_dev, k_len_dev, out_dev, lse_dev, ws_dev, ws_bytes, stream);
}
