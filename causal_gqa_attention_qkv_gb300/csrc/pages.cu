// Pages of a paged cache (include/pages.h): reserve, fork, free, copy, compact.
//
// Which pages a call takes is a question of ranks: the k-th page asked for is
// the k-th lowest page with reference count 0.  The plan kernel answers it with
// one cluster of 8 CTAs: each of its warps owns one run of consecutive pages and
// one of the call's list, counts the free pages (ballots, kept in registers) and
// the pages its rows ask for; the counts are added up over the warps and, through
// distributed shared memory, over the CTAs, and each free page is written to its
// rank in a list.  No atomics decide anything, so the result is the same every
// time, and one launch of one cluster needs no counters in memory.  It is bound by
// latency: three or four cluster barriers and the chain list -> lengths -> table ->
// pages (256 rows over 20000 pages: 8.0 us, 0.3 MB).
//
// The bytes are moved by a second kernel, 16 bytes per thread and 8 in flight,
// in units of 32 KB, so that few pages still spread over many SMs.  Bound by
// HBM: each copied byte is read once and written once (1400 bf16 pages of 64 x 8 x
// 128 entries: 112.8 us, 6.5 TB/s; 4 or 2 loads in flight measured the same).
#include "kernels.cuh"
#include "../../include/pages.h"

namespace gb300 {

namespace {

constexpr int kCluster = 8;
constexpr int kPlanThreads = 1024;                            // of a plan's CTA, at most
constexpr int kSmallPlan = 256;                               // of a small one
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kCopyThreads = 256;
constexpr int kCopyInFlight = 8;                              // 16-byte loads per thread
constexpr int kUnitChunks = kCopyThreads * kCopyInFlight;     // 16-byte chunks per unit
constexpr int64_t kMaxPages = 1 << 24;

// Scratch behind the workspace header, int32: results of a plan, then lists.
enum { kOk = 0, kMoves = 1, kLive = 2, kScratchHead = 64 };
struct Scratch {
  int32_t* head;
  int32_t* list;   // [pages] free pages by rank; compact: where moved pages go
  int32_t* moved;  // [pages] compact: the pages that move, by rank
  int32_t* remap;  // [pages] compact: new number of the pages >= the live count
  int32_t* mark;   // [rows] the position in the call's list that claimed the row, or -1
  int32_t* off;    // [rows] fork: pages asked for by the entries of the call's list before i
};
size_t scratch_ints(int64_t pages, int64_t rows) { return (size_t)(kScratchHead + 3 * pages + 2 * rows); }
Scratch carve(void* ws, int64_t pages, int64_t rows) {
  Scratch s;
  s.head = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + kWsHeader);
  s.list = s.head + kScratchHead;
  s.moved = s.list + pages;
  s.remap = s.moved + pages;
  s.mark = s.remap + pages;
  s.off = s.mark + rows;
  return s;
}

enum PlanOp { kReserve, kFork, kCompact };

struct PlanPar {
  int32_t* table;
  int32_t* ref;
  int32_t* lens;
  const int32_t* rows;  // reserve: rows; fork: destinations
  const int32_t* arg;   // reserve: new tokens; fork: sources
  int32_t n, num_rows, ppr, num_pages, log2_page;
  Scratch s;
  int32_t* status;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Shared- and global-memory writes before it are visible to the cluster after it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int peer_load(const int* p, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return (int)v;
}

// This warp's run of pages, 128 at a time: bit l of word e is set when page
// q + 32 e + l is free.
__device__ __forceinline__ void load_refs(const int32_t* ref, int q, int p1, int lane, int (&v)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = q + 32 * e + lane < p1 ? __ldcg(ref + q + 32 * e + lane) : 1;
}
__device__ __forceinline__ void free_words(const int (&v)[4], uint32_t (&m)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) m[e] = __ballot_sync(0xffffffffu, v[e] <= 0);
}

struct PlanSmem {
  int warp[kPlanWarps];
  int total;  // free pages of this CTA's runs (published)
  int below;  // compact: those below the live count (published)
  int need;   // pages that this CTA's rows ask for (published)
  int bad;    // a row of this CTA's share is refused (published)
  int scan[kPlanWarps];
};

// Sum over the CTA's warps of the warps' values, and the sum before this warp.
__device__ __forceinline__ int sum_warps(int v, int* slots, int warp, int lane, int* before) {
  __syncthreads();  // the slots' previous values have been read
  if (lane == 0) slots[warp] = v;
  __syncthreads();
  const int w = lane < (int)blockDim.x >> 5 ? slots[lane] : 0;
  *before = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
  return __reduce_add_sync(0xffffffffu, w);
}

// Entry i of a call's list by itself (one warp): is it acceptable, how many
// pages does it ask for; reserve: table entries [first, last), and which of the
// first 32 are open.
struct RowFacts {
  int row, first, last, need;
  uint32_t open;
  bool ok;
};
template <int OP>
__device__ __forceinline__ RowFacts row_facts(const PlanPar& p, int row, int arg, int lane) {
  RowFacts f = {row, 0, 0, 0, 0u, row >= 0 && row < p.num_rows};
  if (OP == kFork) f.ok = f.ok && arg >= 0 && arg < p.num_rows;
  if (!f.ok) return f;
  const int page = 1 << p.log2_page;
  const int64_t c = __ldcg(p.lens + (OP == kFork ? arg : row));
  const int64_t last = (c + (OP == kFork ? 0 : arg) + page - 1) >> p.log2_page;
  f.ok = c >= 0 && (OP == kFork || arg >= 0) && last <= p.ppr;
  if (!f.ok) return f;
  f.last = (int)last;
  if constexpr (OP == kReserve) {
    const int32_t* t = p.table + (int64_t)row * p.ppr;
    f.first = (int)((c + page - 1) >> p.log2_page);
    for (int e0 = f.first; e0 < f.last; e0 += 32) {
      const uint32_t m = __ballot_sync(0xffffffffu, e0 + lane < f.last && __ldcg(t + e0 + lane) == -1);
      if (e0 == f.first) f.open = m;
      f.need += __popc(m);
    }
  } else {
    const int32_t* t = p.table + (int64_t)arg * p.ppr;
    const int dst = __ldcg(p.table + (int64_t)row * p.ppr);
    uint32_t worst = 0;  // largest page number, -1 the largest of all
#pragma unroll 4
    for (int e = lane; e < f.last; e += 32) worst = max(worst, (uint32_t)__ldcg(t + e));
    f.ok = __all_sync(0xffffffffu, dst == -1 && worst < (uint32_t)p.num_pages);
    f.need = (c & (page - 1)) != 0 ? 1 : 0;
  }
  return f;
}

template <int OP>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads, 1) plan_kernel(const PlanPar p) {
  __shared__ PlanSmem sm;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = cluster_rank();
  const int warps = blockDim.x >> 5, gwarp = (int)rank * warps + warp, nwarps = kCluster * warps;
  // The copy kernel of the same call may start early: it waits before it reads.  A
  // reservation is followed by kernels that read the caller's tables and lengths as
  // settled (some before their wait), so they start when it has completed.
  if constexpr (OP != kReserve) launch_dependents();
  grid_dependency_wait();
  // this warp's run of pages and (reserve, fork) of the call's list
  const int run = ((p.num_pages + nwarps - 1) / nwarps + 31) & ~31;
  const int p0 = min((int64_t)gwarp * run, (int64_t)p.num_pages), p1 = min(p0 + run, p.num_pages);
  const int share = (p.n + nwarps - 1) / nwarps;
  const int i0 = (int)min((int64_t)gwarp * share, (int64_t)p.n), i1 = min(i0 + share, p.n);
  if (threadIdx.x == 0) sm.bad = 0;
  // Loads that depend on nothing go first: the run's first 128 counts (more in
  // none but pools of over 32768 pages) and the warp's first list entry.
  int refs[4];
  uint32_t head[4];
  RowFacts f0 = {};
  bool bad = false;
  int sum = 0;  // pages the warp's entries ask for, cut at 2^25: that many are refused (there are 2^24 pages at
                // most), and 32 of them fit 32 bits
  if constexpr (OP == kCompact) {
    load_refs(p.ref, p0, p1, lane, refs);
  } else {
    const int row = i0 < i1 ? p.rows[i0] : -1, arg = i0 < i1 ? p.arg[i0] : -1;
    load_refs(p.ref, p0, p1, lane, refs);
    for (int i = gwarp * 32 + lane; i < p.n; i += nwarps * 32) {
      const int r = p.rows[i];
      if (r >= 0 && r < p.num_rows) p.s.mark[r] = -1;
      if constexpr (OP == kFork) {
        const int src = p.arg[i];
        if (src >= 0 && src < p.num_rows) p.s.mark[src] = -1;
      }
    }
    for (int i = i0; i < i1; ++i) {
      const RowFacts f = i == i0 ? row_facts<OP>(p, row, arg, lane) : row_facts<OP>(p, p.rows[i], p.arg[i], lane);
      if (i == i0) f0 = f;
      if (OP == kFork && lane == 0) p.s.off[i] = sum;
      bad = bad || !f.ok;
      sum = min(sum + f.need, 1 << 25);
    }
  }
  free_words(refs, head);
  // f(first page, free pages among the 32 from there) over the warp's run
  auto words = [&](auto f) {
    for (int q = p0; q < p1; q += 128) {
      uint32_t m[4] = {head[0], head[1], head[2], head[3]};
      if (q != p0) {
        int v[4];
        load_refs(p.ref, q, p1, lane, v);
        free_words(v, m);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (q + 32 * e < p1) f(q + 32 * e, m[e]);
    }
  };
  int mine = 0, before_warp;
  words([&](int, uint32_t m) { mine += __popc(m); });
  const int cta_free = sum_warps(mine, sm.warp, warp, lane, &before_warp);
  if (threadIdx.x == 0) sm.total = cta_free;
  cluster_sync();  // marks are cleared, counts published

  int total_free = 0, before = before_warp;  // free pages in all, and before this warp's run
#pragma unroll
  for (uint32_t r = 0; r < kCluster; ++r) {
    const int t = peer_load(&sm.total, r);
    total_free += t;
    if (r < rank) before += t;
  }

  if constexpr (OP == kCompact) {
    const int live = p.num_pages - total_free;
    int below = 0, unused;
    words([&](int q, uint32_t m) {
      if (q < live) below += __popc(live - q < 32 ? m & ((1u << (live - q)) - 1u) : m);
    });
    const int cta_below = sum_warps(below, sm.scan, warp, lane, &unused);
    if (threadIdx.x == 0) sm.below = cta_below;
    cluster_sync();
    int moves = 0;  // free pages below the live count = pages in use behind it
#pragma unroll
    for (uint32_t r = 0; r < kCluster; ++r) moves += peer_load(&sm.below, r);
    words([&](int q, uint32_t m) {
      const int pg = q + lane;
      const bool in = pg < p1;
      const bool free = m >> lane & 1;
      const int frank = before + __popc(m & ((1u << lane) - 1u));  // free pages before pg
      if (free && pg < live) p.s.list[frank] = pg;
      if (in && !free && pg >= live) p.s.moved[pg - frank - live + moves] = pg;
      if (in && pg >= live) p.s.remap[pg] = pg;
      before += __popc(m);
    });
    cluster_sync();  // both lists are complete (and every peer's counts read)
    for (int k = gwarp * 32 + lane; k < moves; k += nwarps * 32) {
      const int from = __ldcg(p.s.moved + k), to = __ldcg(p.s.list + k);
      p.s.remap[from] = to;
      p.ref[to] = p.ref[from];
      p.ref[from] = 0;
    }
    if (gwarp == 0 && lane == 0) {
      p.s.head[kMoves] = moves;
      p.s.head[kLive] = live;
    }
    return;
  } else {
    for (int i = i0 + lane; i < i1; i += 32) {  // a row listed twice is claimed once
      const int row = p.rows[i];
      if (row >= 0 && row < p.num_rows && atomicCAS(p.s.mark + row, -1, i) != -1) bad = true;
    }
    if constexpr (OP == kFork) {
      cluster_sync();  // every destination is marked
      for (int i = gwarp * 32 + lane; i < p.n; i += nwarps * 32) {
        const int src = p.arg[i];
        if (src >= 0 && src < p.num_rows && __ldcg(p.s.mark + src) != -1) bad = true;  // a source that is a destination
      }
    }
    int before_need;
    const int cta_need = sum_warps(sum, sm.scan, warp, lane, &before_need);
    if (bad) sm.bad = 1;
    if (threadIdx.x == 0) sm.need = cta_need;
    cluster_sync();  // needs and refusals published
    int refused = 0;
    int64_t demand = 0, at = before_need;  // pages asked for in all, and before this warp's entries
#pragma unroll
    for (uint32_t r = 0; r < kCluster; ++r) {
      refused |= peer_load(&sm.bad, r);
      const int t = peer_load(&sm.need, r);
      demand += t;
      if (r < rank) at += t;
    }
    const bool go = !refused && demand <= total_free;  // the same in every CTA
    if (go) {
      words([&](int q, uint32_t m) {
        const int k = before + __popc(m & ((1u << lane) - 1u));
        if ((m >> lane & 1) && k < demand) p.s.list[k] = q + lane;
        before += __popc(m);
      });
      if constexpr (OP == kFork)
        for (int i = i0 + lane; i < i1; i += 32) p.s.off[i] += (int)at;
    }
    if (gwarp == 0 && lane == 0) {
      p.s.head[kOk] = go ? 1 : 0;
      if (!go) set_status(p.status, ATTN_STATUS_PAGES);
    }
    cluster_sync();  // the list is complete; every peer's shared memory has been read
    if (!go) return;
    if constexpr (OP == kReserve) {
      int k = (int)at;
      for (int i = i0; i < i1; ++i) {
        const RowFacts f = i == i0 ? f0 : row_facts<OP>(p, p.rows[i], p.arg[i], lane);
        int32_t* t = p.table + (int64_t)f.row * p.ppr;
        for (int e0 = f.first; e0 < f.last; e0 += 32) {
          const int e = e0 + lane;
          const uint32_t m =
              e0 == f.first ? f.open : __ballot_sync(0xffffffffu, e < f.last && __ldcg(t + e) == -1);
          if (m >> lane & 1) {
            const int pg = __ldcg(p.s.list + k + __popc(m & ((1u << lane) - 1u)));
            t[e] = pg;
            p.ref[pg] = 1;
          }
          k += __popc(m);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- data movement
struct PoolPar {
  uint4* k;
  uint4* v;
  uint32_t* ks;             // E2M1 block scales, else nullptr
  uint32_t* vs;
  int64_t num_slots;
  int32_t slot_chunks;      // 16-byte chunks of one slot (all heads)
  int32_t scale_words;      // 4-byte words of one head's block scales of one slot
  int32_t Hkv, log2_page, num_pages;
};

// Unit u of copying the first `slots` slots of page `from` to page `to`: units
// of kUnitChunks 16-byte chunks over K's then V's entries; the block scales
// (words, one run per head) are shared out among the `units` that exist.
__device__ __forceinline__ void copy_unit(const PoolPar& p, int64_t from, int64_t to, int slots, int u) {
  const int64_t per = (int64_t)slots * p.slot_chunks;  // chunks of K (and of V)
  const int64_t c1 = min(per * 2, (int64_t)(u + 1) * kUnitChunks);
  const int64_t base_f = (from << p.log2_page) * p.slot_chunks, base_t = (to << p.log2_page) * p.slot_chunks;
  uint4 x[kCopyInFlight];
#pragma unroll
  for (int e = 0; e < kCopyInFlight; ++e) {
    const int64_t c = (int64_t)u * kUnitChunks + e * kCopyThreads + threadIdx.x;
    if (c < c1) x[e] = c < per ? __ldcs(p.k + base_f + c) : __ldcs(p.v + base_f + c - per);
  }
#pragma unroll
  for (int e = 0; e < kCopyInFlight; ++e) {
    const int64_t c = (int64_t)u * kUnitChunks + e * kCopyThreads + threadIdx.x;
    if (c < c1) (c < per ? p.k + base_t + c : p.v + base_t + c - per)[0] = x[e];
  }
  const int units = (int)((per * 2 + kUnitChunks - 1) / kUnitChunks);
  if (p.ks && u < units) {
    const int run = slots * p.scale_words, words = 2 * p.Hkv * run;  // words of a head; of K and V
    for (int w = u * kCopyThreads + threadIdx.x; w < words; w += units * kCopyThreads) {
      const int head = w / run, at = w - head * run;
      uint32_t* s = head < p.Hkv ? p.ks : p.vs;
      const int64_t row = (int64_t)(head < p.Hkv ? head : head - p.Hkv) * p.num_slots;
      s[(row + (to << p.log2_page)) * p.scale_words + at] = s[(row + (from << p.log2_page)) * p.scale_words + at];
    }
  }
}

struct CopyPar {
  PoolPar pool;
  int32_t units;            // per whole page
  // copy: lists of n pages; compact: the plan's lists
  const int32_t* from;
  const int32_t* to;
  Scratch s;
  // fork, compact
  int32_t* table;
  int32_t* ref;
  int32_t* lens;
  int64_t entries;          // compact: num_rows * ppr
  int32_t ppr;
  int32_t* status;
};

// No kernel below lets its dependents start early (see plan_kernel).
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const CopyPar p) {
  const int i = blockIdx.x / p.units, u = blockIdx.x % p.units;
  grid_dependency_wait();
  const int from = __ldg(p.from + i), to = __ldg(p.to + i);
  if ((uint32_t)from >= (uint32_t)p.pool.num_pages || (uint32_t)to >= (uint32_t)p.pool.num_pages) {
    if (u == 0 && threadIdx.x == 0) set_status(p.status, ATTN_STATUS_PAGES);
    return;
  }
  if (from != to) copy_unit(p.pool, from, to, 1 << p.pool.log2_page, u);
}

__global__ void __launch_bounds__(kCopyThreads) compact_pages_kernel(const CopyPar p) {
  grid_dependency_wait();
  const int moves = __ldcg(p.s.head + kMoves), live = __ldcg(p.s.head + kLive);
  for (int64_t w = blockIdx.x; w < (int64_t)moves * p.units; w += gridDim.x) {
    const int k = (int)(w / p.units);
    copy_unit(p.pool, __ldcg(p.s.moved + k), __ldcg(p.s.list + k), 1 << p.pool.log2_page, (int)(w % p.units));
  }
  for (int64_t e = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; e < p.entries; e += (int64_t)gridDim.x * kCopyThreads) {
    const int pg = p.table[e];
    if (pg >= live && pg < p.pool.num_pages) p.table[e] = __ldcg(p.s.remap + pg);
  }
}

// from: source rows, to: destination rows.
__global__ void __launch_bounds__(kCopyThreads) fork_pages_kernel(const CopyPar p) {
  const int i = blockIdx.x / p.units, u = blockIdx.x % p.units;
  grid_dependency_wait();
  if (__ldcg(p.s.head + kOk) == 0) return;
  const int src = __ldg(p.from + i), dst = __ldg(p.to + i);
  const int c = __ldcg(p.lens + src), whole = c >> p.pool.log2_page, rest = c & ((1 << p.pool.log2_page) - 1);
  const int32_t* ts = p.table + (int64_t)src * p.ppr;
  const int fresh = rest ? __ldcg(p.s.list + __ldcg(p.s.off + i)) : -1;
  if (rest) copy_unit(p.pool, __ldcg(ts + whole), fresh, rest, u);
  if (u != 0) return;
  int32_t* td = p.table + (int64_t)dst * p.ppr;
  for (int e = threadIdx.x; e < p.ppr; e += kCopyThreads) {
    int pg = -1;
    if (e < whole) {
      pg = __ldcg(ts + e);
      atomicAdd(p.ref + pg, 1);
    } else if (e == whole) {
      pg = fresh;
    }
    td[e] = pg;
  }
  if (threadIdx.x == 0) {
    if (rest) p.ref[fresh] = 1;
    p.lens[dst] = c;
  }
}

struct FreePar {
  int32_t* table;
  int32_t* ref;
  int32_t* lens;
  const int32_t* rows;
  int32_t num_rows, ppr, num_pages;
  int32_t* status;
};

// One CTA per listed row.  The exchange hands each entry to one thread only,
// also when a row is listed twice.
__global__ void __launch_bounds__(kCopyThreads) free_pages_kernel(const FreePar p) {
  grid_dependency_wait();
  const int row = __ldg(p.rows + blockIdx.x);
  if ((uint32_t)row >= (uint32_t)p.num_rows) {
    if (threadIdx.x == 0) set_status(p.status, ATTN_STATUS_PAGES);
    return;
  }
  int32_t* t = p.table + (int64_t)row * p.ppr;
  bool bad = false;
  for (int e = threadIdx.x; e < p.ppr; e += kCopyThreads) {
    if (__ldcg(t + e) == -1) continue;
    const int pg = atomicExch(t + e, -1);
    if (pg == -1) continue;
    if ((uint32_t)pg >= (uint32_t)p.num_pages) {
      bad = true;
    } else if (atomicSub(p.ref + pg, 1) <= 0) {
      atomicAdd(p.ref + pg, 1);
      bad = true;
    }
  }
  if (threadIdx.x == 0) p.lens[row] = 0;
  if (bad) set_status(p.status, ATTN_STATUS_PAGES);
}

// ---------------------------------------------------------------- host
int64_t num_pages(const attn_kv_t* kv) { return kv->num_slots / kv->page_size; }

int check_pool(const attn_kv_t* kv, const attn_pages_t* pages) {
  int rc = abi_check_kv(kv);
  if (rc) return rc;
  if (!kv->page_table || num_pages(kv) < 1 || num_pages(kv) > kMaxPages) return ATTN_EINVAL;
  if (!pages) return ATTN_OK;
  if (!pages->page_table || !pages->ref_count || !pages->cache_lens || pages->num_rows < 1 ||
      pages->num_rows > kMaxPages)
    return ATTN_EINVAL;
  return ATTN_OK;
}

bool ws_fits(const void* ws, size_t bytes, size_t need) {
  return ws && (reinterpret_cast<uintptr_t>(ws) & 255) == 0 && bytes >= need;
}

PoolPar pool_of(const attn_config_t* cfg, const attn_kv_t& kv) {
  PoolPar p = {};
  p.k = static_cast<uint4*>(kv.k_cache);
  p.v = static_cast<uint4*>(kv.v_cache);
  const bool f4 = kv.kv_dtype == ATTN_KV_E2M1;
  p.ks = f4 ? static_cast<uint32_t*>(kv.k_block_scale) : nullptr;
  p.vs = f4 ? static_cast<uint32_t*>(kv.v_block_scale) : nullptr;
  p.num_slots = kv.num_slots;
  const int row_bytes = kv.kv_dtype == ATTN_KV_BF16 ? cfg->head_dim * 2 : f4 ? cfg->head_dim / 2 : cfg->head_dim;
  p.slot_chunks = cfg->num_kv_heads * row_bytes / 16;
  p.scale_words = cfg->head_dim / 64;
  p.Hkv = cfg->num_kv_heads;
  p.log2_page = kv_index(kv).log2_page;
  p.num_pages = (int32_t)num_pages(&kv);
  return p;
}

int units_of(const PoolPar& p) {
  return (int)((((int64_t)p.slot_chunks << p.log2_page) * 2 + kUnitChunks - 1) / kUnitChunks);
}

PlanPar plan_of(const attn_kv_t& kv, const attn_pages_t* pages, void* ws) {
  PlanPar p = {};
  p.table = pages->page_table;
  p.ref = pages->ref_count;
  p.lens = pages->cache_lens;
  p.num_rows = pages->num_rows;
  p.ppr = kv.pages_per_req;
  p.num_pages = (int32_t)num_pages(&kv);
  p.log2_page = kv_index(kv).log2_page;
  p.s = carve(ws, p.num_pages, p.num_rows);
  p.status = static_cast<int32_t*>(ws);
  return p;
}

template <int OP>
int launch_plan(const PlanPar& p, cudaStream_t s) {
  // Up to two rows and 128 pages per warp, small CTAs start sooner: a fork of one
  // prompt 8.4 against 10.1 us, a compaction of 6000 pages 47.2 against 48.8; with
  // more rows than that their loads follow one another (384 forks: 24.3 against 17.9).
  const int threads = p.n <= 2 * kCluster * kSmallPlan / 32 && p.num_pages <= 4 * kCluster * kSmallPlan ? kSmallPlan
                                                                                                       : kPlanThreads;
  return launch_dependent(plan_kernel<OP>, dim3(kCluster), dim3(threads), 0, s, p) == cudaSuccess ? ATTN_OK
                                                                                                 : ATTN_ELAUNCH;
}

}  // namespace

}  // namespace gb300

using namespace gb300;

extern "C" {

size_t attn_pages_workspace_size(int64_t max_pages, int32_t max_rows) {
  if (max_pages < 1 || max_pages > kMaxPages || max_rows < 1 || max_rows > kMaxPages) return 0;
  return kWsHeader + align_up(scratch_ints(max_pages, max_rows) * 4, 256);
}

int attn_pages_reserve(const attn_kv_t* kv, const attn_pages_t* pages, const int32_t* rows,
                       const int32_t* new_tokens, int32_t n, void* workspace, size_t ws_bytes, void* stream) {
  int rc = pages ? check_pool(kv, pages) : ATTN_EINVAL;
  if (rc) return rc;
  if (n < 0 || n > pages->num_rows || (n > 0 && (!rows || !new_tokens))) return ATTN_EINVAL;
  if (!ws_fits(workspace, ws_bytes, attn_pages_workspace_size(num_pages(kv), pages->num_rows)))
    return ATTN_EWORKSPACE;
  if ((rc = abi_check_device())) return rc;
  if (n == 0) return ATTN_OK;
  PlanPar p = plan_of(load_kv(kv), pages, workspace);
  p.rows = rows;
  p.arg = new_tokens;
  p.n = n;
  return launch_plan<kReserve>(p, static_cast<cudaStream_t>(stream));
}

int attn_pages_fork(const attn_config_t* cfg, const attn_kv_t* kv, const attn_pages_t* pages,
                    const int32_t* src_rows, const int32_t* dst_rows, int32_t n, void* workspace, size_t ws_bytes,
                    void* stream) {
  int rc = abi_check_config(cfg);
  if (rc) return rc;
  if ((rc = pages ? check_pool(kv, pages) : ATTN_EINVAL)) return rc;
  if (n < 0 || n > pages->num_rows || (n > 0 && (!src_rows || !dst_rows))) return ATTN_EINVAL;
  if (!ws_fits(workspace, ws_bytes, attn_pages_workspace_size(num_pages(kv), pages->num_rows)))
    return ATTN_EWORKSPACE;
  if ((rc = abi_check_device())) return rc;
  if (n == 0) return ATTN_OK;
  const attn_kv_t c = load_kv(kv);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  PlanPar p = plan_of(c, pages, workspace);
  p.rows = dst_rows;
  p.arg = src_rows;
  p.n = n;
  CopyPar q = {};
  q.pool = pool_of(cfg, c);
  q.units = units_of(q.pool);
  if ((int64_t)n * q.units > 0x7fffffff) return ATTN_EINVAL;
  if ((rc = launch_plan<kFork>(p, s))) return rc;
  q.from = src_rows;
  q.to = dst_rows;
  q.s = p.s;
  q.table = p.table;
  q.ref = p.ref;
  q.lens = p.lens;
  q.ppr = p.ppr;
  q.status = p.status;
  return launch_dependent(fork_pages_kernel, dim3((unsigned)(n * q.units)), dim3(kCopyThreads), 0, s, q) == cudaSuccess
             ? ATTN_OK
             : ATTN_ELAUNCH;
}

int attn_pages_free(const attn_kv_t* kv, const attn_pages_t* pages, const int32_t* rows, int32_t n,
                    void* workspace, size_t ws_bytes, void* stream) {
  int rc = pages ? check_pool(kv, pages) : ATTN_EINVAL;
  if (rc) return rc;
  if (n < 0 || (n > 0 && !rows)) return ATTN_EINVAL;
  if (!ws_fits(workspace, ws_bytes, kWsHeader)) return ATTN_EWORKSPACE;
  if ((rc = abi_check_device())) return rc;
  if (n == 0) return ATTN_OK;
  FreePar p;
  p.table = pages->page_table;
  p.ref = pages->ref_count;
  p.lens = pages->cache_lens;
  p.rows = rows;
  p.num_rows = pages->num_rows;
  p.ppr = kv->pages_per_req;
  p.num_pages = (int32_t)num_pages(kv);
  p.status = static_cast<int32_t*>(workspace);
  return launch_dependent(free_pages_kernel, dim3((unsigned)n), dim3(kCopyThreads), 0,
                          static_cast<cudaStream_t>(stream), p) == cudaSuccess
             ? ATTN_OK
             : ATTN_ELAUNCH;
}

int attn_pages_copy(const attn_config_t* cfg, const attn_kv_t* kv, const int32_t* src_pages,
                    const int32_t* dst_pages, int32_t n, void* workspace, size_t ws_bytes, void* stream) {
  int rc = abi_check_config(cfg);
  if (rc) return rc;
  if ((rc = check_pool(kv, nullptr))) return rc;
  if (n < 0 || (n > 0 && (!src_pages || !dst_pages))) return ATTN_EINVAL;
  if (!ws_fits(workspace, ws_bytes, kWsHeader)) return ATTN_EWORKSPACE;
  CopyPar q = {};
  q.pool = pool_of(cfg, load_kv(kv));
  q.units = units_of(q.pool);
  if ((int64_t)n * q.units > 0x7fffffff) return ATTN_EINVAL;
  if ((rc = abi_check_device())) return rc;
  if (n == 0) return ATTN_OK;
  q.from = src_pages;
  q.to = dst_pages;
  q.status = static_cast<int32_t*>(workspace);
  return launch_dependent(copy_pages_kernel, dim3((unsigned)(n * q.units)), dim3(kCopyThreads), 0,
                          static_cast<cudaStream_t>(stream), q) == cudaSuccess
             ? ATTN_OK
             : ATTN_ELAUNCH;
}

int attn_pages_compact(const attn_config_t* cfg, const attn_kv_t* kv, const attn_pages_t* pages, void* workspace,
                       size_t ws_bytes, void* stream) {
  int rc = abi_check_config(cfg);
  if (rc) return rc;
  if ((rc = pages ? check_pool(kv, pages) : ATTN_EINVAL)) return rc;
  if (!ws_fits(workspace, ws_bytes, attn_pages_workspace_size(num_pages(kv), pages->num_rows)))
    return ATTN_EWORKSPACE;
  if ((rc = abi_check_device())) return rc;
  const attn_kv_t c = load_kv(kv);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const PlanPar p = plan_of(c, pages, workspace);
  if ((rc = launch_plan<kCompact>(p, s))) return rc;
  CopyPar q = {};
  q.pool = pool_of(cfg, c);
  q.units = units_of(q.pool);
  q.s = p.s;
  q.table = p.table;
  q.entries = (int64_t)p.num_rows * p.ppr;
  q.ppr = p.ppr;
  q.status = p.status;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return ATTN_ELAUNCH;
  // the number of moves is on the device: a grid that fills the card walks them
  return launch_dependent(compact_pages_kernel, dim3(sms * 8), dim3(kCopyThreads), 0, s, q) == cudaSuccess
             ? ATTN_OK
             : ATTN_ELAUNCH;
}

}  // extern "C"
