// kv_verify_tree and kv_tree_commit: which drafted tokens of a tree are kept, and the cache rows
// that keep them.
//
// Verification is speculative sampling over a tree ([WUSH] and [OSCAR] leave the sampler to the
// serving engine; this is the part of it that decides what the cache keeps).  Walking the nodes
// in index order from the root, a child c of the current node with token x is taken with
// probability min(1, r(x) / q(x)), r the target's distribution at the node less what the missed
// siblings stood for:
//     taken  iff  U_c (Z q(x)) < r(x);      missed:  r <- max(r - Z q, 0),  Z <- sum r
// (q a point mass on x when the drafts carry no distribution).  The token after the last taken
// node is the smallest x with sum_{v <= x} r(v) > U_root sum r.
//
// Every probability is an integer in units of 2^-60 (a float32 p >= 2^-36 is one exactly) and
// every product floor(a b / 2^60), so sums are exact: the result does not depend on the order in
// which 1024 threads and 8 CTAs add, and the same bits give the same token on every run.  Float64
// would need neither but runs at a fortieth of the integer rate on this chip.
//
// What bounds it: latency.  A row of 152 K target probabilities is 0.6 MB, read by one thread
// block cluster (8 CTAs); rows that no decision needs are not read.
#include <cooperative_groups.h>

#include "common.cuh"
#include "launch.h"

namespace cg = cooperative_groups;

namespace kvq {
namespace {

constexpr int kNodes = KVQ_TREE_MAX_NODES;
constexpr int kNodeWords = kNodes / 32;
constexpr unsigned long long kOne = 1ull << 60;

typedef unsigned long long u64;

// floor(a b / 2^60); a, b < 2^63, the product's quotient < 2^64
__device__ __forceinline__ u64 mul60(u64 a, u64 b) {
  return (__umul64hi(a, b) << 4) | ((a * b) >> 60);
}

// p in [0, 1] in units of 2^-60 (the product is exact, the conversion drops what lies below)
__device__ __forceinline__ u64 units(float p) { return __float2ull_rd(p * 0x1p60f); }

struct VerifyParams {
  const int32_t* cu_rows;
  const int32_t* parent;
  const int32_t* token;
  const float* p;
  const float* q;          // nullptr: point-mass drafts
  const float* u;
  long long p_stride, q_stride;
  int vocab;
  int n_rows;
  int batch;
  int32_t* path;
  int32_t* n_accept;
  int32_t* next_token;
  int32_t* status;
};

constexpr int kVThreads = 1024;
constexpr int kVWarps = kVThreads / 32;
constexpr int kVCluster = 8;

struct VerifyShared {
  u64 sum[2][kVWarps];       // per-warp sums of a pass
  u64 total[2];              // this CTA's sum (read by the cluster's other CTAs)
  u64 z[kNodes];             // Z at the misses of the current node (with a draft distribution)
  int gone[kNodes];          // tokens missed at the current node (point-mass drafts)
  float pw[kNodes], qw[kNodes], u[kNodes];
  int token[kNodes];
  int fault;
};

// Sums stop at 4 (a row that is no distribution may hold anything): no addition wraps, and a total
// that reached the stop is reported.
constexpr u64 kTooMuch = 4 * kOne;
__device__ __forceinline__ u64 add_capped(u64 a, u64 b) {
  const u64 t = a + b;
  return t < kTooMuch ? t : kTooMuch;
}
__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = add_capped(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

__global__ void __cluster_dims__(kVCluster, 1, 1) __launch_bounds__(kVThreads)
    verify_tree_kernel(const __grid_constant__ VerifyParams P) {
  __shared__ VerifyShared S;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int b = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  pdl_wait();
  const int first = P.cu_rows[b];
  const int n = P.cu_rows[b + 1] - first;
  if (tid == 0) S.fault = 0;
  __syncthreads();
  // a sequence without rows, or rows that cannot be one tree, ends here (the same decision in
  // every CTA of the cluster)
  bool bad = n < 0 || n > kNodes || first < 0 || first + n > P.n_rows;
  int par[kNodeWords];                         // parents of nodes lane, lane + 32, ...: one copy per warp
#pragma unroll
  for (int w = 0; w < kNodeWords; ++w) {
    const int c = 32 * w + lane;
    par[w] = -2;
    if (!bad && c < n) {
      par[w] = P.parent[first + c];
      if (c == 0 ? par[w] != -1 : (par[w] < 0 || par[w] >= c)) S.fault = 1;
      if (warp == w) {
        const int x = P.token[first + c];
        S.token[c] = x;
        S.u[c] = P.u[first + c];
        if (c > 0) {
          if (x < 0 || x >= P.vocab) {
            S.fault = 1;
          } else if (par[w] >= 0 && par[w] < c) {
            S.pw[c] = P.p[(long long)(first + par[w]) * P.p_stride + x];
            S.qw[c] = P.q ? P.q[(long long)(first + par[w]) * P.q_stride + x] : 1.f;
          }
        }
      }
    }
  }
  __syncthreads();
  bad = bad || S.fault;
  if (bad || n == 0) {
    if (rank == 0) {
      if (!bad || (n > 0 && first >= 0 && first + n <= P.n_rows))
        for (int j = tid; j < n; j += kVThreads) P.path[first + j] = -1;
      if (tid == 0) {
        if (bad) set_status(P.status, KVQ_ERR_BOUNDS);
        P.n_accept[b] = 0;
        P.next_token[b] = -1;
      }
    }
    return;                                     // (uniform over the cluster: nothing waits for it)
  }

  // probabilities outside [0, 1]: larger ones count as 1; negative ones and NaN as 0, reported
  auto clean = [&](float v) {
    if (!(v >= 0.f) || v == INFINITY) {
      set_status(P.status, KVQ_ERR_NONFINITE);
      return 0.f;
    }
    return fminf(v, 1.f);
  };
  auto clean_u = [&](float v) { return v >= 0.f ? fminf(v, 0x1.fffffep-1f) : 0.f; };

  // this warp's contiguous segment of the vocabulary
  const int seg = ((P.vocab + kVCluster * kVWarps * 32 - 1) / (kVCluster * kVWarps * 32)) * 32;
  const int v0 = min(P.vocab, (rank * kVWarps + warp) * seg), v1 = min(P.vocab, v0 + seg);
  int misses = 0;                               // misses of the current node
  bool whole = false;                           // their residual was empty: the weights are p again
  int cur = 0, depth = 1;
  int pass = 0;

  // remaining weight of token v at the current node
  auto weight = [&](int v, float pv, float qv) {
    u64 r = units(clean(pv));
    if (whole) return r;
    if (P.q) {
      const u64 Q = units(clean(qv));
      for (int i = 0; i < misses; ++i) {
        const u64 t = mul60(S.z[i], Q);
        r = r > t ? r - t : 0ull;
      }
    } else {
      for (int i = 0; i < misses; ++i)
        if (S.gone[i] == v) r = 0ull;
    }
    return r;
  };
  // sum over the vocabulary of the remaining weights; S.sum keeps the warps' sums and S.total the
  // CTA's of the last pass (two sets: a pass writes one while others may still read the other)
  auto sum_weights = [&]() {
    const float* pr = P.p + (long long)(first + cur) * P.p_stride;
    const float* qr = P.q ? P.q + (long long)(first + cur) * P.q_stride : nullptr;
    const bool need_q = qr && misses > 0 && !whole;
    u64 acc = 0ull;
#pragma unroll 4
    for (int v = v0 + lane; v < v1; v += 32) acc = add_capped(acc, weight(v, pr[v], need_q ? qr[v] : 0.f));
    acc = warp_sum(acc);
    const int set = pass++ & 1;
    if (lane == 0) S.sum[set][warp] = acc;
    __syncthreads();
    if (warp == 0) {
      const u64 t = warp_sum(S.sum[set][lane]);
      if (lane == 0) S.total[set] = t;
    }
    cluster.sync();
    u64 all = 0ull;
    for (int r = 0; r < kVCluster; ++r) all = add_capped(all, *cluster.map_shared_rank(&S.total[set], r));
    return all;
  };

  // nodes in index order; every warp of every CTA takes the same decisions
  if (rank == 0 && tid == 0) {
    P.path[first] = 0;
    P.next_token[b] = -1;                       // (until the draw below, a cluster barrier later)
  }
  u64 mass = kOne;
  for (int c = 1; c < n; ++c) {
    // the next child of the current node
    int next = n;
#pragma unroll
    for (int w = kNodeWords - 1; w >= 0; --w) {
      unsigned m = __ballot_sync(0xffffffffu, par[w] == cur);
      if (32 * w + 31 < c) m = 0u;
      else if (32 * w < c) m &= ~0u << (c - 32 * w);
      if (m) next = 32 * w + __ffs(m) - 1;
    }
    c = next;
    if (c >= n) break;
    const int x = S.token[c];
    const u64 w = weight(x, S.pw[c], S.qw[c]);
    const u64 want = P.q ? mul60(mass, units(clean(S.qw[c]))) : mass;
    if (mul60(units(clean_u(S.u[c])), want) < w) {
      if (rank == 0 && tid == 0) P.path[first + depth] = c;
      cur = c;
      ++depth;
      misses = 0;
      mass = kOne;
      continue;
    }
    __syncthreads();                            // (nobody still reads the list's next entry)
    if (tid == 0) {
      S.z[misses] = mass;
      S.gone[misses] = x;
    }
    ++misses;
    __syncthreads();
    mass = P.q ? sum_weights() : (mass > w ? mass - w : 0ull);
    if (mass == 0ull) {                         // nothing is left: the draw is from p, no sibling is tried
      whole = true;
      break;
    }
  }
  if (rank == 0)
    for (int j = depth + tid; j < n; j += kVThreads) P.path[first + j] = -1;

  // the token after the last taken node
  u64 total = sum_weights();
  if (total == 0ull && !whole) {
    whole = true;
    total = sum_weights();
  }
  const int set = (pass - 1) & 1;
  if (rank == 0 && tid == 0) P.n_accept[b] = depth;
  if (total == 0ull || total >= kTooMuch) {
    if (rank == 0 && tid == 0) set_status(P.status, KVQ_ERR_NONFINITE);
  } else {
    u64 goal = mul60(units(clean_u(S.u[0])), total);
    for (int r = 0; r < rank; ++r) {
      const u64 t = *cluster.map_shared_rank(&S.total[set], r);
      goal = goal >= t ? goal - t : ~0ull;
      if (goal == ~0ull) break;                 // an earlier CTA holds it
    }
    if (goal != ~0ull && goal < S.total[set]) {
      int owner = -1;
      for (int i = 0; i < kVWarps; ++i) {
        if (goal < S.sum[set][i]) {
          owner = i;
          break;
        }
        goal -= S.sum[set][i];
      }
      if (warp == owner) {
        const float* pr = P.p + (long long)(first + cur) * P.p_stride;
        const float* qr = P.q ? P.q + (long long)(first + cur) * P.q_stride : nullptr;
        const bool need_q = qr && misses > 0 && !whole;
        for (int base = v0; base < v1; base += 32) {
          const int v = base + lane;
          u64 w = v < v1 ? weight(v, pr[v], need_q ? qr[v] : 0.f) : 0ull;
          u64 upto = w;                         // inclusive sum over the lanes
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const u64 t = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += t;
          }
          const unsigned hit = __ballot_sync(0xffffffffu, upto > goal);
          if (hit) {
            if (lane == 0) P.next_token[b] = base + __ffs(hit) - 1;
            break;
          }
          goal -= __shfl_sync(0xffffffffu, upto, 31);
        }
      }
    }
  }
  cluster.sync();                               // the sums stay readable until every CTA is done
}

// ---- the accepted path's rows -----------------------------------------------------------------
struct CommitParams {
  const int32_t* cu_rows;
  const int32_t* path;
  const int32_t* n_accept;
  int32_t* seq_len;
  const int32_t* s_quant;
  uint16_t* sink_k;
  uint16_t* sink_v;
  uint16_t* ring_k;
  uint16_t* ring_v;
  int32_t* status;
  int n_rows, hkv, s_sink, ring_cap;
};

constexpr int kCThreads = 512;
constexpr int kCBatch = 8;           // rows a warp has in flight

// One CTA per sequence, one warp per (kv head, K or V): the rows of the accepted path move down in
// path order.  A row's destination L0 + j is never the source L0 + path[j'] of a later j' > j
// (path[j'] >= j' > j), so loading a batch before storing it is safe in place.
__global__ void __launch_bounds__(kCThreads) tree_commit_kernel(const __grid_constant__ CommitParams P) {
  __shared__ int path[kNodes];
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int first = P.cu_rows[b];
  const int n = P.cu_rows[b + 1] - first;
  const int len = P.seq_len[b], edge = P.s_quant[b], keep = P.n_accept[b];
  const int L0 = len - n;
  int bad = n < 0 || n > kNodes || first < 0 || first + n > P.n_rows || keep < 0 || keep > n || L0 < 0 ||
            edge > max(L0, P.s_sink);
  if (!bad && tid < keep) {
    const int at = P.path[first + tid], before = tid ? P.path[first + tid - 1] : -1;
    path[tid] = at;
    bad = at <= before || at >= n;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) set_status(P.status, KVQ_ERR_BOUNDS);
    return;
  }
  if (tid == 0 && n > 0) P.seq_len[b] = L0 + keep;
  // where token t of kv head h lives
  auto row = [&](int t, int h, int side) {
    uint16_t* sink = side ? P.sink_v : P.sink_k;
    uint16_t* ring = side ? P.ring_v : P.ring_k;
    return t < P.s_sink ? sink + (((size_t)b * P.hkv + h) * P.s_sink + t) * kHeadDim
                        : ring + (((size_t)b * P.hkv + h) * P.ring_cap + t % P.ring_cap) * kHeadDim;
  };
  for (int unit = warp; unit < 2 * P.hkv; unit += kCThreads / 32) {
    const int h = unit >> 1, side = unit & 1;
    for (int j0 = 0; j0 < keep; j0 += kCBatch) {
      uint2 v[kCBatch];
#pragma unroll
      for (int i = 0; i < kCBatch; ++i)
        if (j0 + i < keep && path[j0 + i] != j0 + i)
          v[i] = reinterpret_cast<const uint2*>(row(L0 + path[j0 + i], h, side))[lane];
#pragma unroll
      for (int i = 0; i < kCBatch; ++i)
        if (j0 + i < keep && path[j0 + i] != j0 + i) reinterpret_cast<uint2*>(row(L0 + j0 + i, h, side))[lane] = v[i];
    }
  }
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" int kvq_launch_verify_tree(const kvq_config* cfg, const int32_t* cu_rows, const int32_t* parent,
                                      const int32_t* token, int32_t n_rows, const float* p, int64_t p_stride,
                                      const float* q, int64_t q_stride, int32_t vocab, const float* u, int32_t* path,
                                      int32_t* n_accept, int32_t* next_token, int32_t* d_status, cudaStream_t stream) {
  VerifyParams P{};
  P.cu_rows = cu_rows;
  P.parent = parent;
  P.token = token;
  P.p = p;
  P.q = q;
  P.u = u;
  P.p_stride = p_stride;
  P.q_stride = q_stride;
  P.vocab = vocab;
  P.n_rows = n_rows;
  P.batch = cfg->batch;
  P.path = path;
  P.n_accept = n_accept;
  P.next_token = next_token;
  P.status = d_status;
  return launch_pdl(verify_tree_kernel, dim3(kVCluster, cfg->batch), dim3(kVThreads), 0, stream, P) == cudaSuccess
             ? KVQ_OK
             : KVQ_ERR_CUDA;
}

extern "C" int kvq_launch_tree_commit(const kvq_config* cfg, const kvq_cache* cache, const int32_t* cu_rows,
                                      int32_t n_rows, const int32_t* path, const int32_t* n_accept,
                                      int32_t* d_status, cudaStream_t stream) {
  CommitParams P{};
  P.cu_rows = cu_rows;
  P.path = path;
  P.n_accept = n_accept;
  P.seq_len = cache->seq_len;
  P.s_quant = cache->s_quant;
  P.sink_k = cache->sink_k;
  P.sink_v = cache->sink_v;
  P.ring_k = cache->ring_k;
  P.ring_v = cache->ring_v;
  P.status = d_status;
  P.n_rows = n_rows;
  P.hkv = cfg->n_kv_heads;
  P.s_sink = cfg->s_sink;
  P.ring_cap = cfg->ring_cap;
  return launch_pdl(tree_commit_kernel, dim3(cfg->batch), dim3(kCThreads), 0, stream, P) == cudaSuccess ? KVQ_OK
                                                                                                      : KVQ_ERR_CUDA;
}
