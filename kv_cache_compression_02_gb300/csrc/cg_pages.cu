// cg_pages.cu -- the bookkeeping of pages that sequences share: extend, fork,
// free, copy and compact.
//
// A fork or a compaction has a plan, made by one CTA (a scan over the reference
// counts, in order, so that no order of atomics can change the result), and a
// step over the whole GPU that carries it out: table rows, counts, and the
// pages that move.  That kernel is launched with the plan and waits for it.
// Measured, ten calls in a graph: 64 branches of a 32-layer cache with 8 KV heads
// (free, fork, extend; 235 MB written) 67.5 us, a third of its pages compacted
// (169 MB) 34.5 us.
#include "cg_cache.cuh"

namespace cg {
namespace {

constexpr int kPlan = 1024;   // threads of a plan's CTA
constexpr int kMove = 256;    // threads of a CTA that moves pages
constexpr int kMoveBytes = 32768;  // of one page, moved by one CTA at a time

// Workspace: the status word, then what a plan tells the apply step.
struct Book {
  uint32_t *status;   // status bits
  int4 *plan;         // of a fork or a compaction: x: it holds and is carried out, y: pages that move, z: live pages
  int32_t *marks;     // [n_seqs]
  int32_t *src, *dst, *rank;  // [most]: moved pages, where they go, a number for each
};

struct PageArgs {
  int32_t *refs, *table, *len;
  int n_seqs, stride, n_blocks, bt, n;
  const int32_t *a, *b;  // the call's own lists
  Book w;
};

struct MoveArgs {
  uint8_t *const *pools;
  float *const *scales;
  uint64_t page_bytes;
  int n_pools, H, n_blocks, parts;  // parts: pieces of kMoveBytes of a page
  int lanes;                        // threads that move a piece
  const int32_t *src, *dst;
  int n;  // entries of a copy
  uint32_t *status;
};

uint64_t book_bytes(const cg_pages *p, uint64_t most, uint8_t *at, Book *w) {
  const uint64_t marks = pad256(4 * uint64_t(p ? p->n_seqs : 0)), list = pad256(4 * most);
  if (w) {
    w->status = reinterpret_cast<uint32_t *>(at);
    w->plan = reinterpret_cast<int4 *>(at + 16);
    w->marks = reinterpret_cast<int32_t *>(at + 256);
    w->src = reinterpret_cast<int32_t *>(at + 256 + marks);
    w->dst = reinterpret_cast<int32_t *>(at + 256 + marks + list);
    w->rank = reinterpret_cast<int32_t *>(at + 256 + marks + 2 * list);
  }
  return 256 + marks + 3 * list;
}

// Exclusive sum over the CTA's threads, and the total.
template <typename T>
__device__ T scan(T v, T *total) {
  __shared__ T s_warp[kPlan / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  T w = lane < kPlan / 32 ? s_warp[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const T before = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0);
  __syncthreads();  // s_warp may be written again
  return x - v + (warp ? before : 0);
}

// The lowest `want` free pages, in order, to list[]; returns how many there are of them.
__device__ int find_free(const int32_t *refs, int n_blocks, int want, int32_t *list) {
  int got = 0;
  for (int64_t base = 0; base < n_blocks && got < want; base += 4 * kPlan) {
    const int64_t p = base + 4 * threadIdx.x;
    int f[4], n = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) n += f[i] = p + i < n_blocks && refs[p + i] == 0;
    int total, r = got + scan(n, &total);
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (f[i]) {
        if (r < want) list[r] = int32_t(p + i);
        r++;
      }
    got += total;
  }
  __syncthreads();
  return min(got, want);
}

// Whether a pool or scale array is null or misaligned.  A plan looks before
// anything is changed: what carries it out need not.  A thread's first entries
// are loaded where the plan begins and looked at where it ends, so that their
// latency is not added to the plan's.
struct PoolCheck {
  uintptr_t pool = 16, scale = 16;
  __device__ void load(const MoveArgs &m, int i) {
    if (i >= m.n_pools) return;
    pool = reinterpret_cast<uintptr_t>(m.pools[i]);
    if (m.scales) scale = reinterpret_cast<uintptr_t>(m.scales[i]);
  }
  __device__ bool bad(const MoveArgs &m) {  // among this thread's share of the entries
    bool any = false;
    for (int i = threadIdx.x;;) {
      any |= !pool || (pool & 15) || !scale || (scale & 3);
      if ((i += kPlan) >= m.n_pools) return any;
      load(m, i);
    }
  }
};

__device__ inline int pages_of(int64_t len, int bt) { return int((len + bt - 1) / bt); }

// extend: a = sequences, b = new lengths
__global__ void __launch_bounds__(kPlan) k_extend(const PageArgs g) {
  const Book &w = g.w;
  for (int i = threadIdx.x; i < g.n_seqs; i += kPlan) w.marks[i] = 0;
  __syncthreads();
  bool bad = false;
  int64_t sum = 0;
  for (int base = 0; base < g.n; base += kPlan) {
    const int i = base + threadIdx.x;
    int64_t lacks = 0;
    if (i < g.n) {
      const int s = g.a[i];
      if (uint32_t(s) >= uint32_t(g.n_seqs)) {
        bad = true;
      } else {
        const int64_t len = g.len[s], next = g.b[i];
        if (atomicExch(&w.marks[s], 1) || len < 0 || next < len || next > int64_t(g.stride) * g.bt)
          bad = true;
        else
          lacks = pages_of(next, g.bt) - pages_of(len, g.bt);
      }
    }
    int64_t total;
    const int64_t r = sum + scan(lacks, &total);
    if (i < g.n) w.rank[i] = int(min(r, int64_t(g.n_blocks)));  // one past the pages is only read where there is no room
    sum += total;
  }
  bad = __syncthreads_or(bad);
  const int want = int(min(sum, int64_t(g.n_blocks) + 1));
  const bool room = !bad && want <= g.n_blocks && find_free(g.refs, g.n_blocks, want, w.src) == want;
  if (threadIdx.x == 0) *w.status = bad ? kStBadArg : room ? 0 : kStCapacity;
  if (!room) return;
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x >> 5; i < g.n; i += kPlan / 32) {  // a warp per sequence
    const int s = g.a[i], have = pages_of(g.len[s], g.bt), need = pages_of(g.b[i], g.bt);
    for (int j = have + lane; j < need; j += 32) {
      const int p = w.src[w.rank[i] + j - have];
      g.table[int64_t(s) * g.stride + j] = p;
      g.refs[p] = 1;
    }
    __syncwarp();
    if (lane == 0) g.len[s] = g.b[i];
  }
}

// fork: a = parents, b = children
__global__ void __launch_bounds__(kPlan) k_fork_plan(const PageArgs g, const MoveArgs m) {
  const Book &w = g.w;
  asm volatile("griddepcontrol.launch_dependents;");
  PoolCheck pools;
  if (g.n > 0) pools.load(m, threadIdx.x);
  for (int i = threadIdx.x; i < g.n_seqs; i += kPlan) w.marks[i] = 0;
  __syncthreads();
  bool bad = false;
  for (int i = threadIdx.x; i < g.n; i += kPlan) {
    const int p = g.a[i], c = g.b[i];
    if (uint32_t(p) >= uint32_t(g.n_seqs) || uint32_t(c) >= uint32_t(g.n_seqs))
      bad = true;
    else if (g.len[c] != 0 || atomicExch(&w.marks[c], 1))
      bad = true;
  }
  bad = __syncthreads_or(bad);
  int want = 0;
  if (!bad) {
    for (int base = 0; base < g.n; base += kPlan) {
      const int i = base + threadIdx.x;
      int part = 0;
      if (i < g.n) {
        const int p = g.a[i];
        const int64_t len = g.len[p];
        if (w.marks[p] || len < 0 || len > int64_t(g.stride) * g.bt)
          bad = true;
        else
          part = len % g.bt != 0;
      }
      int total;
      const int r = want + scan(part, &total);
      if (i < g.n) w.rank[i] = part ? r : -1;
      if (part) w.src[r] = g.table[int64_t(g.a[i]) * g.stride + g.len[g.a[i]] / g.bt];
      want += total;
    }
    bad = __syncthreads_or(bad || (want > 0 && pools.bad(m)));
  }
  if (!bad)  // every page of a parent must be one: a warp per pair
    for (int i = threadIdx.x >> 5; i < g.n; i += kPlan / 32) {
      const int32_t *row = g.table + int64_t(g.a[i]) * g.stride;
      const int used = pages_of(g.len[g.a[i]], g.bt);
      for (int j = threadIdx.x & 31; j < used; j += 32) bad |= uint32_t(row[j]) >= uint32_t(g.n_blocks);
    }
  bad = __syncthreads_or(bad);
  const bool room = !bad && find_free(g.refs, g.n_blocks, min(want, g.n_blocks), w.dst) == want;
  if (threadIdx.x == 0) {
    *w.status = bad ? kStBadArg : room ? 0 : kStCapacity;
    *w.plan = make_int4(room, want, 0, 0);
  }
}

// A fork's pair i: the child's row, counts and length, by one CTA.
__device__ void fork_row(const PageArgs &g, int i) {
  const Book &w = g.w;
  const int len = g.len[g.a[i]], used = pages_of(len, g.bt), r = w.rank[i];
  const int32_t *row = g.table + int64_t(g.a[i]) * g.stride;
  int32_t *to = g.table + int64_t(g.b[i]) * g.stride;
  for (int j = threadIdx.x; j < g.stride; j += kMove) {
    int p = -1;
    if (j < used) {
      p = row[j];
      if (r >= 0 && j == used - 1)
        g.refs[p = w.dst[r]] = 1;
      else
        atomicAdd(&g.refs[p], 1);
    }
    to[j] = p;
  }
  if (threadIdx.x == 0) g.len[g.b[i]] = len;
}

// free: a = sequences, one CTA each
__global__ void __launch_bounds__(kMove) k_free(const PageArgs g) {
  const int s = g.a[blockIdx.x];
  status_cleared();
  if (uint32_t(s) >= uint32_t(g.n_seqs)) {
    if (threadIdx.x == 0) atomicOr(g.w.status, kStBadArg);
    return;
  }
  __shared__ int s_len;
  if (threadIdx.x == 0) s_len = atomicExch(&g.len[s], 0);  // of several CTAs for one sequence, one gets its length
  __syncthreads();
  const int64_t len = s_len;
  if (len == 0) return;
  int used = pages_of(len, g.bt);
  if (len < 0 || used > g.stride) {
    if (threadIdx.x == 0) atomicOr(g.w.status, kStBadArg);
    used = len < 0 ? 0 : g.stride;
  }
  int32_t *row = g.table + int64_t(s) * g.stride;
  for (int j = threadIdx.x; j < used; j += kMove) {
    const int p = row[j];
    row[j] = -1;
    if (uint32_t(p) >= uint32_t(g.n_blocks)) {
      atomicOr(g.w.status, kStBadArg);
    } else if (atomicSub(&g.refs[p], 1) <= 0) {
      atomicAdd(&g.refs[p], 1);
      atomicOr(g.w.status, kStCorrupt);
    }
  }
}

// compact: src = pages that move, dst = where to; rank[p] is the number of
// page p's move, as a hole (p < n_live) or a mover, or -1.  marks is not used.
__global__ void __launch_bounds__(kPlan, 1) k_compact_plan(const PageArgs g, const MoveArgs m, int32_t *n_live_out, int32_t *moved_refs) {
  const Book &w = g.w;
  asm volatile("griddepcontrol.launch_dependents;");
  PoolCheck pools;
  pools.load(m, threadIdx.x);
  int mine = 0, n_live;
#pragma unroll 8
  for (int64_t p = threadIdx.x; p < g.n_blocks; p += kPlan) mine += g.refs[p] > 0;
  scan(mine, &n_live);
  constexpr int kEach = 8;  // pages of a thread at a time
  int holes = 0, movers = 0;
  for (int64_t base = 0; base < g.n_blocks; base += kEach * kPlan) {
    const int64_t p0 = base + kEach * threadIdx.x;
    int refs[kEach];
    int64_t both = 0;  // holes, and movers above
#pragma unroll
    for (int i = 0; i < kEach; i++) refs[i] = p0 + i < g.n_blocks ? g.refs[p0 + i] : 0;
    auto is_hole = [&](int i) { return p0 + i < n_live && refs[i] <= 0; };
    auto is_mover = [&](int i) { return p0 + i >= n_live && refs[i] > 0; };
#pragma unroll
    for (int i = 0; i < kEach; i++) both += int64_t(is_hole(i)) | int64_t(is_mover(i)) << 32;
    int64_t sum;
    const int64_t to = scan(both, &sum);
    int rh = holes + int(to & 0xffffffff), rm = movers + int(to >> 32);
#pragma unroll
    for (int i = 0; i < kEach; i++) {
      if (p0 + i >= g.n_blocks) continue;
      w.rank[p0 + i] = is_hole(i) ? rh : is_mover(i) ? rm : -1;
      if (is_hole(i)) w.dst[rh++] = int32_t(p0 + i);
      if (is_mover(i)) w.src[rm] = int32_t(p0 + i), moved_refs[rm++] = refs[i];
    }
    holes += int(sum & 0xffffffff), movers += int(sum >> 32);
  }
  const bool bad = __syncthreads_or(movers > 0 && pools.bad(m));
  if (threadIdx.x == 0) {
    *w.status = bad ? kStBadArg : 0;
    *w.plan = make_int4(!bad, movers, n_live, 0);
    if (!bad) *n_live_out = n_live;
  }
}

// A compaction's counts and table, by the whole grid.
__device__ void compact_book(const PageArgs &g, int n_live, int32_t *refs_out, int32_t *table_out, const int32_t *moved_refs) {
  const Book &w = g.w;
  const int64_t entries = int64_t(g.n_seqs) * g.stride, step = int64_t(gridDim.x) * kMove;
  for (int64_t i = int64_t(blockIdx.x) * kMove + threadIdx.x; i < g.n_blocks; i += step) {
    const int r = w.rank[i];
    refs_out[i] = i >= n_live ? 0 : r >= 0 ? moved_refs[r] : g.refs[i];
  }
  for (int64_t i = int64_t(blockIdx.x) * kMove + threadIdx.x; i < entries; i += step) {
    int p = g.table[i];
    if (p >= g.n_blocks || (p >= 0 && (w.rank[p] >= 0) != (p >= n_live)))
      atomicOr(w.status, kStBadArg);  // no page, or a free one
    else if (p >= n_live)
      p = w.dst[w.rank[p]];
    table_out[i] = p;
  }
}

enum What { kCopy, kFork, kCompact };

// Pages src[i] -> dst[i] of every pool, with their scales, and the rest of
// what a plan asks for.  Bound by HBM: a CTA moves 32 KB at a time, each thread
// with eight 16-byte loads in flight; pages of up to 16 KB take a warp each
// (150 pages of 16 KB in 64 pools: 53 us, a CTA each 70 us; of 8 KB: 28 and 42
// us; 64 KB pages go at the copy peak, 6.8 TB/s).
template <What W, typename V>
__global__ void __launch_bounds__(kMove) k_move(const MoveArgs g, const PageArgs b, int32_t *refs_out, int32_t *table_out,
                                                const int32_t *moved_refs) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 plan = W == kCopy ? make_int4(1, g.n, 0, 0) : *b.w.plan;
  if (!plan.x) return;
  if (W == kFork)
    for (int i = blockIdx.x; i < b.n; i += gridDim.x) fork_row(b, i);
  if (W == kCompact) compact_book(b, plan.z, refs_out, table_out, moved_refs);
  const int64_t units = int64_t(g.n_pools) * plan.y * g.parts;
  constexpr int kVecs = kMoveBytes / int(sizeof(V));
  const int64_t page_vecs = int64_t(g.page_bytes / sizeof(V));
  const int lane = threadIdx.x % g.lanes, per_cta = kMove / g.lanes;
  for (int64_t u = int64_t(blockIdx.x) * per_cta + threadIdx.x / g.lanes; u < units; u += int64_t(gridDim.x) * per_cta) {
    const int part = int(u % g.parts), pool = int(u / g.parts % g.n_pools);
    const int64_t i = u / g.parts / g.n_pools;
    const int s = g.src[i], t = g.dst[i];
    if (uint32_t(s) >= uint32_t(g.n_blocks) || uint32_t(t) >= uint32_t(g.n_blocks)) {
      if (lane == 0) atomicOr(g.status, kStBadArg);
      continue;
    }
    uint8_t *base = g.pools[pool];
    if (W == kCopy && (!base || (reinterpret_cast<uintptr_t>(base) & 15))) {
      if (lane == 0) atomicOr(g.status, kStBadArg);
      continue;
    }
    const V *from = reinterpret_cast<const V *>(base + g.page_bytes * uint64_t(s)) + int64_t(part) * kVecs;
    V *to = reinterpret_cast<V *>(base + g.page_bytes * uint64_t(t)) + int64_t(part) * kVecs;
    const int m = int(min(int64_t(kVecs), page_vecs - int64_t(part) * kVecs));
    int x = lane;
    for (; x + 7 * g.lanes < m; x += 8 * g.lanes) {
      V v[8];
#pragma unroll
      for (int k = 0; k < 8; k++) v[k] = from[x + k * g.lanes];
#pragma unroll
      for (int k = 0; k < 8; k++) to[x + k * g.lanes] = v[k];
    }
    for (; x < m; x += g.lanes) to[x] = from[x];
    if (part == 0 && g.scales) {
      float *sc = g.scales[pool];
      if (W == kCopy && (!sc || (reinterpret_cast<uintptr_t>(sc) & 3))) {
        if (lane == 0) atomicOr(g.status, kStBadArg);
      } else {
        for (int h = lane; h < g.H; h += g.lanes) sc[int64_t(t) * g.H + h] = sc[int64_t(s) * g.H + h];
      }
    }
  }
}

bool pages_ok(const cg_cache *c, const cg_pages *p) {
  return cache_ok(c) && p && p->n_seqs >= 1 && p->table_stride >= 1 && p->refs_dev && p->table_dev && p->len_dev &&
         is_aligned(p->refs_dev, 4) && is_aligned(p->table_dev, 4) && is_aligned(p->len_dev, 4);
}

bool pools_ok(const cg_cache *c, void *const *pools, float *const *scales) {
  return pools && is_aligned(pools, 8) && is_aligned(scales, 8) && (scales || c->format == CG_CACHE_F16);
}

bool ws_ok(const void *ws, size_t bytes, size_t need) { return ws && is_aligned(ws, 256) && bytes >= need; }

uint64_t most_of(const cg_cache *c, int32_t n) { return uint64_t(c->n_blocks > n ? c->n_blocks : n); }

PageArgs page_args(const cg_cache *c, const cg_pages *p, int32_t n, const int32_t *a, const int32_t *b, void *ws) {
  PageArgs g{};
  g.refs = p->refs_dev, g.table = p->table_dev, g.len = p->len_dev;
  g.n_seqs = p->n_seqs, g.stride = p->table_stride, g.n_blocks = c->n_blocks, g.bt = c->block_tokens, g.n = n;
  g.a = a, g.b = b;
  book_bytes(p, most_of(c, n), static_cast<uint8_t *>(ws), &g.w);
  return g;
}

// What a move of up to n pages needs to know.
MoveArgs move_args(const cg_cache *c, void *const *pools, float *const *scales, const int32_t *src, const int32_t *dst, int32_t n, void *ws) {
  MoveArgs m{};
  m.pools = reinterpret_cast<uint8_t *const *>(pools);
  m.scales = scales;
  m.page_bytes = page_bytes(c);
  m.n_pools = 2 * c->L, m.H = c->H, m.n_blocks = c->n_blocks;
  m.parts = int((m.page_bytes + kMoveBytes - 1) / kMoveBytes);
  m.lanes = m.page_bytes <= 16384 ? 32 : kMove;
  m.src = src, m.dst = dst, m.n = n;
  m.status = static_cast<uint32_t *>(ws);
  return m;
}

// Launches k_move behind a plan (or k_clear).
template <What W>
cg_status move_pages(const MoveArgs &m, const PageArgs &g, int32_t *refs_out, int32_t *table_out, const int32_t *moved_refs, cudaStream_t st) {
  const int64_t units = int64_t(m.n) * m.n_pools * m.parts, ctas = (units * m.lanes + kMove - 1) / kMove, most = kSMs * 8;
  const dim3 grid(unsigned(ctas < most ? ctas : most)), block(kMove);
  const cudaError_t e = m.page_bytes % 16 == 0 ? launch_early(k_move<W, uint4>, grid, block, 0, st, m, g, refs_out, table_out, moved_refs)
                                               : launch_early(k_move<W, uint2>, grid, block, 0, st, m, g, refs_out, table_out, moved_refs);
  return e == cudaSuccess ? launched() : CG_ERR_CUDA;
}

}  // namespace
}  // namespace cg

using namespace cg;

extern "C" size_t cg_pages_workspace_bytes(const cg_cache *cache, const cg_pages *pages, int32_t n) {
  if (!cache_ok(cache) || n < 0 || (pages && !pages_ok(cache, pages))) return 0;
  // compaction keeps one list more
  return size_t(book_bytes(pages, most_of(cache, n), nullptr, nullptr) + pad256(4 * uint64_t(cache->n_blocks)));
}

extern "C" cg_status cg_pages_extend(const cg_cache *cache, const cg_pages *pages, int32_t n, const int32_t *seq_dev,
                                     const int32_t *new_len_dev, void *ws_dev, size_t ws_bytes, void *stream) {
  if (!pages_ok(cache, pages) || n < 0 || (n > 0 && (!seq_dev || !new_len_dev)) || !is_aligned(seq_dev, 4) ||
      !is_aligned(new_len_dev, 4) || !ws_ok(ws_dev, ws_bytes, cg_pages_workspace_bytes(cache, pages, n)))
    return CG_ERR_INVALID_ARG;
  k_extend<<<1, kPlan, 0, static_cast<cudaStream_t>(stream)>>>(page_args(cache, pages, n, seq_dev, new_len_dev, ws_dev));
  return launched();
}

extern "C" cg_status cg_pages_fork(const cg_cache *cache, const cg_pages *pages, void *const *pools_dev,
                                   float *const *scales_dev, int32_t n, const int32_t *parent_dev,
                                   const int32_t *child_dev, void *ws_dev, size_t ws_bytes, void *stream) {
  if (!pages_ok(cache, pages) || !pools_ok(cache, pools_dev, scales_dev) || n < 0 || (n > 0 && (!parent_dev || !child_dev)) ||
      !is_aligned(parent_dev, 4) || !is_aligned(child_dev, 4) ||
      !ws_ok(ws_dev, ws_bytes, cg_pages_workspace_bytes(cache, pages, n)))
    return CG_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const PageArgs g = page_args(cache, pages, n, parent_dev, child_dev, ws_dev);
  const MoveArgs m = move_args(cache, pools_dev, scales_dev, g.w.src, g.w.dst, n, ws_dev);
  k_fork_plan<<<1, kPlan, 0, st>>>(g, m);
  if (n == 0) return launched();
  return move_pages<kFork>(m, g, nullptr, nullptr, nullptr, st);
}

extern "C" cg_status cg_pages_free(const cg_cache *cache, const cg_pages *pages, int32_t n, const int32_t *seq_dev,
                                   void *ws_dev, size_t ws_bytes, void *stream) {
  if (!pages_ok(cache, pages) || n < 0 || (n > 0 && !seq_dev) || !is_aligned(seq_dev, 4) ||
      !ws_ok(ws_dev, ws_bytes, cg_pages_workspace_bytes(cache, pages, n)))
    return CG_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  k_clear<<<1, 32, 0, st>>>(static_cast<uint32_t *>(ws_dev));
  if (n == 0) return launched();
  const cudaError_t e = launch_early(k_free, dim3(unsigned(n)), dim3(kMove), 0, st, page_args(cache, pages, n, seq_dev, nullptr, ws_dev));
  return e == cudaSuccess ? launched() : CG_ERR_CUDA;
}

extern "C" cg_status cg_pages_copy(const cg_cache *cache, void *const *pools_dev, float *const *scales_dev, int32_t n,
                                   const int32_t *src_dev, const int32_t *dst_dev, void *ws_dev, size_t ws_bytes,
                                   void *stream) {
  if (!cache_ok(cache) || !pools_ok(cache, pools_dev, scales_dev) || n < 0 || (n > 0 && (!src_dev || !dst_dev)) ||
      !is_aligned(src_dev, 4) || !is_aligned(dst_dev, 4) || !ws_ok(ws_dev, ws_bytes, 256))
    return CG_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  k_clear<<<1, 32, 0, st>>>(static_cast<uint32_t *>(ws_dev));
  if (n == 0) return launched();
  return move_pages<kCopy>(move_args(cache, pools_dev, scales_dev, src_dev, dst_dev, n, ws_dev), PageArgs{}, nullptr, nullptr, nullptr, st);
}

extern "C" cg_status cg_pages_compact(const cg_cache *cache, const cg_pages *pages, void *const *pools_dev,
                                      float *const *scales_dev, int32_t *refs_out_dev, int32_t *table_out_dev,
                                      int32_t *n_live_dev, void *ws_dev, size_t ws_bytes, void *stream) {
  if (!pages_ok(cache, pages) || !pools_ok(cache, pools_dev, scales_dev) || !refs_out_dev || !table_out_dev ||
      !n_live_dev || !is_aligned(refs_out_dev, 4) || !is_aligned(table_out_dev, 4) || !is_aligned(n_live_dev, 4) ||
      !ws_ok(ws_dev, ws_bytes, cg_pages_workspace_bytes(cache, pages, 0)))
    return CG_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const PageArgs g = page_args(cache, pages, 0, nullptr, nullptr, ws_dev);
  int32_t *moved_refs = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(ws_dev) +
                                                    book_bytes(pages, most_of(cache, 0), nullptr, nullptr));
  // at most half of the pages move
  const MoveArgs m = move_args(cache, pools_dev, scales_dev, g.w.src, g.w.dst, (cache->n_blocks + 1) / 2, ws_dev);
  k_compact_plan<<<1, kPlan, 0, st>>>(g, m, n_live_dev, moved_refs);
  return move_pages<kCompact>(m, g, refs_out_dev, table_out_dev, moved_refs, st);
}
