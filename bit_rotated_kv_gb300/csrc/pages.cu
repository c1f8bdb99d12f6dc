// The page pool: kv_pages_reserve, kv_seq_fork, kv_seq_free and kv_pages_compact.
//
// A physical page is free when no page-table entry refers to it (page_ref 0), and pages are
// handed out lowest id first: the pool's state is one counter per page, no list whose order
// would depend on the order of atomics, so the same calls give the same tables on every run.
// Forked sequences share whole INT2 pages (a page is written only while the INT2 edge is inside
// it, so a whole one never changes); a page that is half filled and the BF16 windows are copied.
//
// Tables and counts are a few megabytes at most and one cluster of 8 CTAs does them in one launch
// (a scan's barrier inside a cluster costs a fraction of another launch); the rows and pages that
// move are copied by a second, grid-wide launch, which is bound by HBM: each byte is read once
// and written once, 16 bytes per lane, four to eight loads in flight a thread (8 prompts of 4-8 K tokens
// forked to 56 samples: 148 MB in 24 us, 91% of the copy rate; 94 MB of pages moved in 16 us, 86%).  What is
// left is latency: a scan's cluster launch takes 11 to 13 us for 40 K pages (a dozen barriers and dependent
// loads; keeping the counts it has read in registers changed nothing).  Whole calls: free and fork 37 us, free,
// compact and reserve for 64 sequences of 4-8 K 48 us, for 8 of 2 K 20 us.
//
// Order: kernels of this library read the page table before their dependency wait (kv_attn_*), so
// a table must not be written by the launch directly before them.  Each call here is a sequence
// of ordinary launches whose last one does not write the table.
#include <cooperative_groups.h>

#include <mutex>

#include "common.cuh"
#include "launch.h"

namespace cg = cooperative_groups;

namespace kvq {
namespace {

constexpr int kPThreads = 1024;
constexpr int kPWarps = kPThreads / 32;
constexpr int kPCluster = 8;

struct PageParams {
  uint8_t* pages;
  int32_t* table;
  int32_t* ref;
  int32_t* seq_len;
  int32_t* s_quant;
  int32_t* counters;
  uint16_t* sink_k;
  uint16_t* sink_v;
  uint16_t* ring_k;
  uint16_t* ring_v;
  int32_t* status;
  const int32_t* a;      // reserve: n_tokens [B]; fork: src [n]; free: sequences [n]
  const int32_t* b;      // fork: dst [n]
  int n;
  int batch, hkv, s_sink, ring_cap, max_pages, num_pages, page_head;
  int parts;             // fork: CTAs per pair that copy rows
  int32_t* n_live;       // compact
  int32_t* moved;        // compact workspace: count, then source and target lists and the new ids
};

// Block-wide inclusive sum of one T per thread; returns the thread's own prefix, `all` the total.
template <class T>
__device__ __forceinline__ T block_scan(T v, T* warp_sums, T& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    T w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T t = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += t;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  all = warp_sums[kPWarps - 1];
  return v + (warp ? warp_sums[warp - 1] : T(0));
}

// Entries of a table row that hold a page: they are a prefix of it (searched 32 ways at a time).
__device__ __forceinline__ int pages_held(const int32_t* row, int max_pages) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = max_pages;                  // the first empty entry is in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const unsigned full = __ballot_sync(0xffffffffu, at < hi && row[at] >= 0);
    const int k = full == 0xffffffffu ? 32 : __ffs(~full) - 1;
    if (k == 0) return lo;
    hi = min(hi, lo + k * step);
    lo = lo + (k - 1) * step + 1;
  }
  return lo;
}

// Whether pair i of a fork is one: both sequences exist, and its destination is the destination of
// no earlier pair and the source of none.  Called by whole blocks (kBlock) or warps.
template <bool kBlock>
__device__ __forceinline__ bool fork_pair_ok(const PageParams& P, int i) {
  const int src = P.a[i], dst = P.b[i];
  int bad = src < 0 || src >= P.batch || dst < 0 || dst >= P.batch;
#pragma unroll 4
  for (int j = kBlock ? threadIdx.x : threadIdx.x & 31; j < P.n; j += kBlock ? blockDim.x : 32)
    bad |= P.a[j] == dst || (j < i && P.b[j] == dst);
  return kBlock ? !__syncthreads_or(bad) : !__any_sync(0xffffffffu, bad);
}

struct PageShared {
  int warp_sums[kPWarps];
  long long wide_sums[kPWarps];
  int count[2];          // this CTA's counts, read by the others of the cluster
};

// Free pages of the pool go to units 0 .. n - 1 in order, need(u) each, lowest ids first; a unit
// gets all it needs or, from the first one on that the pool cannot serve, none.  end[u] (shared
// memory of every CTA) holds need on entry and its inclusive prefix sum on return; give(u, k, id)
// is called once for the k-th page of unit u.  Returns the number of free pages there were.
template <class Give>
__device__ int hand_out(const PageParams& P, cg::cluster_group& cluster, PageShared& S, int* end, int n, Give give) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = (int)cluster.block_rank();
  // prefix sums of the needs, the same in every CTA (in 64 bits: thousands of sequences may ask for more than
  // any pool has)
  long long before = 0;
  for (int u0 = 0; u0 < n; u0 += kPThreads) {
    long long all;
    const long long v = u0 + tid < n ? end[u0 + tid] : 0;
    const long long upto = block_scan(v, S.wide_sums, all);
    if (u0 + tid < n) end[u0 + tid] = (int)min(before + upto, (long long)INT32_MAX);
    before += all;
  }
  // free pages of this warp's slice of the pool
  const int seg = ((P.num_pages + kPCluster * kPThreads - 1) / (kPCluster * kPThreads)) * 32;
  const long long w0 = (long long)(rank * kPWarps + warp) * seg;
  const int p0 = (int)min((long long)P.num_pages, w0), p1 = (int)min((long long)P.num_pages, w0 + seg);
  int mine = 0;
#pragma unroll 4
  for (int p = p0 + lane; p < p1; p += 32) mine += P.ref[p] == 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  int all;
  const int upto = block_scan(lane == 0 ? mine : 0, S.warp_sums, all);
  if (tid == 0) S.count[0] = all;
  cluster.sync();
  int base = __shfl_sync(0xffffffffu, upto, 0) - mine, free_pages = 0;
  for (int r = 0; r < kPCluster; ++r) {
    const int c = *cluster.map_shared_rank(&S.count[0], r);
    if (r < rank) base += c;
    free_pages += c;
  }
  // units served: a prefix of them
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (end[mid] <= free_pages) lo = mid + 1;
    else hi = mid;
  }
  const int given = lo ? end[lo - 1] : 0;
  for (int q0 = p0; q0 < p1 && base < given; q0 += 32) {
    const int p = q0 + lane;
    const bool f = p < p1 && P.ref[p] == 0;
    const unsigned m = __ballot_sync(0xffffffffu, f);
    const int k = base + __popc(m & ((1u << lane) - 1u));
    if (f && k < given) {
      int a = 0, b = n - 1;                    // the unit with end[u - 1] <= k < end[u]
      while (a < b) {
        const int mid = (a + b) / 2;
        if (end[mid] > k) b = mid;
        else a = mid + 1;
      }
      give(a, k - (a ? end[a - 1] : 0), p);
    }
    base += __popc(m);
  }
  return free_pages;
}

// ---- reserve -----------------------------------------------------------------------------------
__global__ void __cluster_dims__(kPCluster, 1, 1) __launch_bounds__(kPThreads)
    pages_reserve_kernel(const __grid_constant__ PageParams P) {
  extern __shared__ int end[];                 // [batch] needs, then their prefix sums; then [batch] entries held
  __shared__ PageShared S;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int* held = end + P.batch;
  cluster.sync();                              // (every CTA has started: its shared memory can be written)
  for (int u = rank * kPWarps + warp; u < P.batch; u += kPCluster * kPWarps) {
    const long long tokens = P.a[u];
    int need = 0, have = 0;
    if (tokens > 0) {
      const long long want = ((long long)P.seq_len[u] + tokens - P.s_sink + kPage - 1) / kPage;
      if (want > P.max_pages) {
        if (lane == 0) set_status(P.status, KVQ_ERR_BOUNDS);
      } else if (want > 0) {
        have = pages_held(P.table + (size_t)u * P.max_pages, P.max_pages);
        need = max(0, (int)want - have);
      }
    }
    for (int r = lane; r < kPCluster; r += 32) {
      cluster.map_shared_rank(end, r)[u] = need;
      cluster.map_shared_rank(held, r)[u] = have;
    }
  }
  cluster.sync();
  const int free_pages = hand_out(P, cluster, S, end, P.batch, [&](int u, int k, int id) {
    P.table[(size_t)u * P.max_pages + held[u] + k] = id;
    P.ref[id] = 1;
  });
  if (rank == 0 && threadIdx.x == 0 && end[P.batch - 1] > free_pages) set_status(P.status, KVQ_ERR_BOUNDS);
  cluster.sync();
}

// Ends a call whose last kernel wrote the page table (see the head of this file).
__global__ void order_kernel() {}

// ---- fork --------------------------------------------------------------------------------------
__global__ void __cluster_dims__(kPCluster, 1, 1) __launch_bounds__(kPThreads)
    seq_fork_table_kernel(const __grid_constant__ PageParams P) {
  extern __shared__ int end[];                 // [n] prefix sums of the pages needed; then [n] whole pages shared
  __shared__ PageShared S;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), tid = threadIdx.x;
  int* shared_pages = end + P.n;               // -1: not a pair
  cluster.sync();                              // (every CTA has started: its shared memory can be written)
  const int lane = tid & 31, gwarp = rank * kPWarps + (tid >> 5);
  for (int i = gwarp; i < P.n; i += kPCluster * kPWarps) {
    bool ok = fork_pair_ok<false>(P, i);
    int full = -1, need = 0;
    if (ok) {
      const int src = P.a[i], dst = P.b[i];
      const int tokens = max(0, P.s_quant[src] - P.s_sink);
      full = tokens / kPage;
      need = tokens % kPage ? 1 : 0;
      // the destination holds nothing, the source's rows fit its table row
      if (P.seq_len[dst] != 0 || P.table[(size_t)dst * P.max_pages] >= 0 || full + need > P.max_pages) ok = false;
    }
    if (!ok) {
      full = -1;
      need = 0;
      if (lane == 0) set_status(P.status, KVQ_ERR_BOUNDS);
    }
    if (lane < kPCluster) {
      cluster.map_shared_rank(end, lane)[i] = need;
      cluster.map_shared_rank(shared_pages, lane)[i] = full;
    }
  }
  cluster.sync();
  const int free_pages = hand_out(P, cluster, S, end, P.n, [&](int i, int, int id) {
    P.table[(size_t)P.b[i] * P.max_pages + shared_pages[i]] = id;
    P.ref[id] = 1;
  });
  cluster.sync();                              // (counts of free pages are taken before references change)
  // pairs that the pool could serve (from the first one on that it could not, none is) take their shares:
  // a warp takes 128 entries of a pair at once
  for (int i = rank * kPThreads + tid; i < P.n; i += kPCluster * kPThreads) {
    if (shared_pages[i] < 0) continue;
    if (end[i] > free_pages) {
      set_status(P.status, KVQ_ERR_BOUNDS);
    } else {
      const int src = P.a[i], dst = P.b[i];
      P.seq_len[dst] = P.seq_len[src];
      P.s_quant[dst] = P.s_quant[src];
      P.counters[dst] = P.parts;               // the copying CTAs count it back to zero
    }
  }
  const int per_pair = (P.max_pages + 127) / 128;
  for (long long k = gwarp; k < (long long)P.n * per_pair; k += kPCluster * kPWarps) {
    const int i = (int)(k / per_pair), c0 = (int)(k % per_pair) * 128 + lane, full = shared_pages[i];
    if (c0 - lane >= full || end[i] > free_pages) continue;
    const int32_t* from = P.table + (size_t)P.a[i] * P.max_pages;
    int32_t* to = P.table + (size_t)P.b[i] * P.max_pages;
    int id[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) id[x] = c0 + 32 * x < full ? from[c0 + 32 * x] : 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (c0 + 32 * x >= full) continue;
      if ((unsigned)id[x] < (unsigned)P.num_pages) {
        atomicAdd(P.ref + id[x], 1);
        to[c0 + 32 * x] = id[x];
      } else {
        set_status(P.status, KVQ_ERR_BOUNDS);
      }
    }
  }
  cluster.sync();
}

constexpr int kCopyThreads = 256;
constexpr int kRowParts = 4;         // CTAs per (pair, kv head)
constexpr int kRowBatch = 8;         // rows a thread has in flight

__global__ void __launch_bounds__(kCopyThreads) seq_fork_rows_kernel(const __grid_constant__ PageParams P) {
  const int i = blockIdx.y, h = blockIdx.x / kRowParts, part = blockIdx.x % kRowParts;
  if (!fork_pair_ok<true>(P, i)) return;
  const int src = P.a[i], dst = P.b[i], tid = threadIdx.x;
  __shared__ int live;
  if (tid == 0) live = *(volatile int32_t*)(P.counters + dst);
  __syncthreads();
  if (live == 0) return;                       // a pair that was not forked
  if (tid == 0) atomicSub(P.counters + dst, 1);
  const int len = P.seq_len[src], edge = P.s_quant[src];
  // BF16 rows: 16 lanes a row, sink rows first, then the live ring slots
  const int n_sink = min(P.s_sink, len), first = max(edge, P.s_sink), n_ring = min(max(0, len - first), P.ring_cap);
  constexpr int kLanes = kHeadDim * 2 / 16;
  const int sub = tid % kLanes;
  const int rows = n_sink + n_ring;
  const size_t hs = (size_t)src * P.hkv + h, hd = (size_t)dst * P.hkv + h;
  constexpr int kStep = kRowParts * (kCopyThreads / kLanes);
  for (int r0 = part * (kCopyThreads / kLanes) + tid / kLanes; r0 < 2 * rows; r0 += kRowBatch * kStep) {
    uint4 v[kRowBatch];
    uint4* to[kRowBatch];
#pragma unroll
    for (int k = 0; k < kRowBatch; ++k) {
      const int both = r0 + k * kStep, side = both >= rows, r = both - (side ? rows : 0);
      to[k] = nullptr;
      if (both < 2 * rows) {
        const bool in_sink = r < n_sink;
        const size_t slot = in_sink ? r : (size_t)((first + r - n_sink) % P.ring_cap);
        uint16_t* base = in_sink ? (side ? P.sink_v : P.sink_k) : (side ? P.ring_v : P.ring_k);
        const size_t cap = in_sink ? P.s_sink : P.ring_cap;
        v[k] = reinterpret_cast<const uint4*>(base + (hs * cap + slot) * kHeadDim)[sub];
        to[k] = reinterpret_cast<uint4*>(base + (hd * cap + slot) * kHeadDim) + sub;
      }
    }
#pragma unroll
    for (int k = 0; k < kRowBatch; ++k)
      if (to[k]) *to[k] = v[k];
  }
  // the half-filled page
  const int tokens = max(0, edge - P.s_sink);
  if (part == 0 && tokens % kPage) {
    const int ps = P.table[(size_t)src * P.max_pages + tokens / kPage], pd = P.table[(size_t)dst * P.max_pages + tokens / kPage];
    if ((unsigned)ps < (unsigned)P.num_pages && (unsigned)pd < (unsigned)P.num_pages) {
      const uint4* from = reinterpret_cast<const uint4*>(P.pages + ((size_t)ps * P.hkv + h) * P.page_head);
      uint4* to = reinterpret_cast<uint4*>(P.pages + ((size_t)pd * P.hkv + h) * P.page_head);
      for (int k = tid; k < P.page_head / 16; k += kCopyThreads) to[k] = from[k];
    } else if (tid == 0) {
      set_status(P.status, KVQ_ERR_BOUNDS);
    }
  }
}

// ---- free --------------------------------------------------------------------------------------
__global__ void __launch_bounds__(kCopyThreads) seq_free_table_kernel(const __grid_constant__ PageParams P) {
  const int s = P.a[blockIdx.y];
  if (s < 0 || s >= P.batch) {
    if (threadIdx.x == 0 && blockIdx.x == 0) set_status(P.status, KVQ_ERR_BOUNDS);
    return;
  }
  for (int c = blockIdx.x * kCopyThreads + threadIdx.x; c < P.max_pages; c += gridDim.x * kCopyThreads) {
    int32_t* entry = P.table + (size_t)s * P.max_pages + c;
    if (*entry < 0) continue;
    const int id = atomicExch(entry, -1);      // (a sequence listed twice gives its pages up once)
    if (id < 0) continue;
    if (id >= P.num_pages) {
      set_status(P.status, KVQ_ERR_BOUNDS);
    } else if (atomicSub(P.ref + id, 1) <= 0) {
      atomicAdd(P.ref + id, 1);                // a page that nothing held: the counts do not match the tables
      set_status(P.status, KVQ_ERR_BOUNDS);
    }
  }
}

__global__ void __launch_bounds__(kCopyThreads) seq_free_state_kernel(const __grid_constant__ PageParams P) {
  const int i = blockIdx.x * kCopyThreads + threadIdx.x;
  if (i >= P.n) return;
  const int s = P.a[i];
  if (s < 0 || s >= P.batch) return;
  P.seq_len[s] = 0;
  P.s_quant[s] = P.s_sink;
}

// ---- compact -----------------------------------------------------------------------------------
// Live pages are those with a reference; the k-th of them that lies at or above their number moves
// to the k-th free page below it.
__global__ void __cluster_dims__(kPCluster, 1, 1) __launch_bounds__(kPThreads)
    compact_plan_kernel(const __grid_constant__ PageParams P) {
  __shared__ PageShared S;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = (int)cluster.block_rank();
  const int seg = ((P.num_pages + kPCluster * kPThreads - 1) / (kPCluster * kPThreads)) * 32;
  const long long w0 = (long long)(rank * kPWarps + warp) * seg;
  const int p0 = (int)min((long long)P.num_pages, w0), p1 = (int)min((long long)P.num_pages, w0 + seg);
  // how many are live
  int mine = 0, all;
#pragma unroll 4
  for (int p = p0 + lane; p < p1; p += 32) mine += P.ref[p] > 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  (void)block_scan(lane == 0 ? mine : 0, S.warp_sums, all);
  if (tid == 0) S.count[0] = all;
  cluster.sync();
  int n_live = 0;
  for (int r = 0; r < kPCluster; ++r) n_live += *cluster.map_shared_rank(&S.count[0], r);
  // movers of this warp's slice and holes of it (a slice can hold both only around n_live): counts,
  // then ranks
  int movers = 0, holes = 0;
#pragma unroll 4
  for (int p = p0 + lane; p < p1; p += 32) {
    const bool live = P.ref[p] > 0;
    movers += live && p >= n_live;
    holes += !live && p < n_live;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    movers += __shfl_xor_sync(0xffffffffu, movers, o);
    holes += __shfl_xor_sync(0xffffffffu, holes, o);
  }
  int all_m, all_h;
  int bm = block_scan(lane == 0 ? movers : 0, S.warp_sums, all_m);
  int bh = block_scan(lane == 0 ? holes : 0, S.warp_sums, all_h);
  cluster.sync();                              // (the live counts have been read)
  if (tid == 0) {
    S.count[0] = all_m;
    S.count[1] = all_h;
  }
  cluster.sync();
  bm = __shfl_sync(0xffffffffu, bm, 0) - movers;
  bh = __shfl_sync(0xffffffffu, bh, 0) - holes;
  int n_move = 0;
  for (int r = 0; r < kPCluster; ++r) {
    const int cm = *cluster.map_shared_rank(&S.count[0], r), ch = *cluster.map_shared_rank(&S.count[1], r);
    if (r < rank) {
      bm += cm;
      bh += ch;
    }
    n_move += cm;
  }
  int32_t* from = P.moved + 1;
  int32_t* to = from + P.num_pages;
  for (int q0 = p0; q0 < p1; q0 += 32) {
    const int p = q0 + lane;
    const bool live = p < p1 && P.ref[p] > 0;
    const bool m = live && p >= n_live, hole = p < p1 && !live && p < n_live;
    const unsigned mm = __ballot_sync(0xffffffffu, m), mh = __ballot_sync(0xffffffffu, hole);
    const unsigned below = (1u << lane) - 1u;
    if (m) from[bm + __popc(mm & below)] = p;
    if (hole) to[bh + __popc(mh & below)] = p;
    bm += __popc(mm);
    bh += __popc(mh);
  }
  if (rank == 0 && tid == 0) {
    P.moved[0] = n_move;
    *P.n_live = n_live;
  }
  cluster.sync();
  int32_t* renamed = to + P.num_pages;
  for (int k = rank * kPThreads + tid; k < n_move; k += kPCluster * kPThreads) renamed[from[k]] = to[k];
  cluster.sync();
}

__global__ void __launch_bounds__(kCopyThreads) compact_move_kernel(const __grid_constant__ PageParams P) {
  const int n_move = P.moved[0], n_live = *P.n_live, tid = threadIdx.x;
  const int32_t* from = P.moved + 1;
  const int32_t* to = from + P.num_pages;
  const int32_t* renamed = to + P.num_pages;
  const long long entries = (long long)P.batch * P.max_pages;
  for (long long e = (long long)blockIdx.x * kCopyThreads + tid; e < entries; e += (long long)gridDim.x * kCopyThreads) {
    const int id = P.table[e];
    if (id >= n_live) {
      // (a page without a reference that a table names all the same: left, and reported)
      const int now = id < P.num_pages && P.ref[id] > 0 ? renamed[id] : -1;
      if ((unsigned)now < (unsigned)n_live) P.table[e] = now;
      else set_status(P.status, KVQ_ERR_BOUNDS);
    }
  }
  const size_t bytes = (size_t)P.hkv * P.page_head;
  for (int k = blockIdx.x; k < n_move; k += gridDim.x) {
    const uint4* src = reinterpret_cast<const uint4*>(P.pages + (size_t)from[k] * bytes);
    uint4* dst = reinterpret_cast<uint4*>(P.pages + (size_t)to[k] * bytes);
    const int words = (int)(bytes / 16);
    for (int w = tid; w < words; w += 4 * kCopyThreads) {      // four loads in flight a thread
      uint4 v[4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (w + x * kCopyThreads < words) v[x] = src[w + x * kCopyThreads];
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (w + x * kCopyThreads < words) dst[w + x * kCopyThreads] = v[x];
    }
  }
}

__global__ void __launch_bounds__(kCopyThreads) compact_refs_kernel(const __grid_constant__ PageParams P) {
  const int n_move = P.moved[0];
  const int32_t* from = P.moved + 1;
  const int32_t* to = from + P.num_pages;
  for (int k = blockIdx.x * kCopyThreads + threadIdx.x; k < n_move; k += gridDim.x * kCopyThreads) {
    P.ref[to[k]] = P.ref[from[k]];
    P.ref[from[k]] = 0;
  }
}

PageParams page_params(const kvq_config* cfg, const kvq_cache* cache, int32_t* page_ref, int32_t* d_status) {
  PageParams P{};
  P.pages = (uint8_t*)cache->pages;
  P.table = const_cast<int32_t*>(cache->page_table);
  P.ref = page_ref;
  P.seq_len = cache->seq_len;
  P.s_quant = cache->s_quant;
  P.counters = cache->counters;
  P.sink_k = cache->sink_k;
  P.sink_v = cache->sink_v;
  P.ring_k = cache->ring_k;
  P.ring_v = cache->ring_v;
  P.status = d_status;
  P.batch = cfg->batch;
  P.hkv = cfg->n_kv_heads;
  P.s_sink = cfg->s_sink;
  P.ring_cap = cfg->ring_cap;
  P.max_pages = cfg->max_pages_per_seq;
  P.num_pages = cfg->num_pages;
  P.page_head = page_head_bytes(cfg->group_size, cfg->key_l2norm, cfg->key_axis);
  return P;
}

int launched() { return cudaPeekAtLastError() == cudaSuccess ? KVQ_OK : (cudaGetLastError(), KVQ_ERR_CUDA); }

// dynamic shared memory beyond 48 KB, once per (device, kernel)
int allow_smem(const void* kernel, int which) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KVQ_ERR_CUDA;
  static std::mutex mu;
  static unsigned long long done[2] = {};
  std::lock_guard<std::mutex> lock(mu);
  if (!(done[which] & (1ull << dev))) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, KVQ_POOL_MAX_SEQS * 8) != cudaSuccess)
      return KVQ_ERR_CUDA;
    done[which] |= 1ull << dev;
  }
  return KVQ_OK;
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" int kvq_launch_pages_reserve(const kvq_config* cfg, const kvq_cache* cache, int32_t* page_ref,
                                        const int32_t* n_tokens, int32_t* d_status, cudaStream_t stream) {
  if (cfg->batch > KVQ_POOL_MAX_SEQS) return KVQ_ERR_UNSUPPORTED;
  PageParams P = page_params(cfg, cache, page_ref, d_status);
  P.a = n_tokens;
  P.n = cfg->batch;
  const int rc = allow_smem((const void*)pages_reserve_kernel, 0);
  if (rc) return rc;
  pages_reserve_kernel<<<kPCluster, kPThreads, (size_t)cfg->batch * 8, stream>>>(P);
  order_kernel<<<1, 32, 0, stream>>>();
  return launched();
}

extern "C" int kvq_launch_seq_fork(const kvq_config* cfg, const kvq_cache* cache, int32_t* page_ref,
                                   const int32_t* src, const int32_t* dst, int32_t n, int32_t* d_status,
                                   cudaStream_t stream) {
  if (n > KVQ_POOL_MAX_SEQS) return KVQ_ERR_UNSUPPORTED;
  if (n == 0) return KVQ_OK;
  PageParams P = page_params(cfg, cache, page_ref, d_status);
  P.a = src;
  P.b = dst;
  P.n = n;
  P.parts = cfg->n_kv_heads * kRowParts;
  const int rc = allow_smem((const void*)seq_fork_table_kernel, 1);
  if (rc) return rc;
  seq_fork_table_kernel<<<kPCluster, kPThreads, (size_t)n * 8, stream>>>(P);
  seq_fork_rows_kernel<<<dim3(P.parts, n), kCopyThreads, 0, stream>>>(P);
  return launched();
}

extern "C" int kvq_launch_seq_free(const kvq_config* cfg, const kvq_cache* cache, int32_t* page_ref,
                                   const int32_t* seqs, int32_t n, int32_t* d_status, cudaStream_t stream) {
  if (n > KVQ_POOL_MAX_SEQS) return KVQ_ERR_UNSUPPORTED;
  if (n == 0) return KVQ_OK;
  PageParams P = page_params(cfg, cache, page_ref, d_status);
  P.a = seqs;
  P.n = n;
  const int blocks = (int)min(64LL, ((long long)cfg->max_pages_per_seq + kCopyThreads - 1) / kCopyThreads);
  seq_free_table_kernel<<<dim3(blocks, n), kCopyThreads, 0, stream>>>(P);
  seq_free_state_kernel<<<(n + kCopyThreads - 1) / kCopyThreads, kCopyThreads, 0, stream>>>(P);
  return launched();
}

extern "C" size_t kvq_compact_ws_bytes(const kvq_config* cfg) {
  return ((size_t)cfg->num_pages * 3 + 1) * 4;
}

extern "C" int kvq_launch_pages_compact(const kvq_config* cfg, const kvq_cache* cache, int32_t* page_ref,
                                        int32_t* n_live, void* ws, int32_t* d_status, cudaStream_t stream) {
  PageParams P = page_params(cfg, cache, page_ref, d_status);
  P.n_live = n_live;
  P.moved = (int32_t*)ws;
  compact_plan_kernel<<<kPCluster, kPThreads, 0, stream>>>(P);
  compact_move_kernel<<<8 * kSms, kCopyThreads, 0, stream>>>(P);
  compact_refs_kernel<<<kSms, kCopyThreads, 0, stream>>>(P);
  return launched();
}
