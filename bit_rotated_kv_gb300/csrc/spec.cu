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
// which 4096 threads add, and the same bits give the same token on every run.  (Float64 sums would
// depend on the order, and this chip has few units for them.)
//
// What bounds it: for one sequence, latency -- the sampler's decisions are a chain (8 nodes, 32,000
// tokens: 7.8 us).  For many, integer arithmetic: a row of 152 K target probabilities is 0.6 MB, read by
// one cluster of CTAs, with the draft's row once more for every missed child (64 trees of 16 nodes: 71 us
// for rows that HBM delivers in 11; four of them wait for four sums, one after another).  Rows that no
// decision needs are not read, and the sums of the last miss are those that the draw needs.
#include <cooperative_groups.h>

#include <atomic>

#include "common.cuh"
#include "launch.h"

namespace cg = cooperative_groups;

namespace kvq {
namespace {

constexpr int kNodes = KVQ_TREE_MAX_NODES;
constexpr int kNodeWords = kNodes / 32;
constexpr unsigned long long kOne = 1ull << 60;

typedef unsigned long long u64;

// floor(a b / 2^60); a < 2^63, b < 2^61
__device__ __forceinline__ u64 mul60(u64 a, u64 b) { return __umul64hi(a << 1, b << 3); }

// Probabilities: more than 1 counts as 1; negative values, infinities and NaN as 0, and `odd` is set.
template <int N>
__device__ __forceinline__ void clean(float (&p)[N], bool& odd) {
  uint32_t top = 0u;
#pragma unroll
  for (int k = 0; k < N; ++k) top = max(top, __float_as_uint(p[k]));
  if (top <= 0x7f7fffffu) return;
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (__float_as_uint(p[k]) > 0x7f7fffffu) {
      odd |= __float_as_uint(p[k]) != 0x80000000u;
      p[k] = 0.f;
    }
}
// ... in units of 2^-60: the 24-bit significand (1.0 is 2^23 << 37), what lies below a unit dropped.  (A 64-bit
// float-to-integer conversion does the same, slower: the whole call took 102 instead of 81 us with it.)
__device__ __forceinline__ u64 units(float p) {
  const uint32_t bits = min(__float_as_uint(p), 0x3f800000u);
  return ((u64)((bits & 0x7fffffu) | 0x800000u) << 37) >> min(127u - (bits >> 23), 63u);
}
// ... of a random number: [0, 1)
__device__ __forceinline__ u64 units_below_1(float u) {
  return u >= 0.f ? units(fminf(u, 0x1.fffffep-1f)) : 0ull;
}

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
  int32_t* path;
  int32_t* n_accept;
  int32_t* next_token;
  int32_t* status;
};

constexpr int kVThreads = 256;
constexpr int kVWarps = kVThreads / 32;
// CTAs per sequence.  Most sequences need one sum over their row, a few need one for every missed child, and
// those are what the call waits for: 64 trees over 152 K tokens take 71 us with 16 x 256 threads to a
// sequence, 86 us with 8 x 512, 80 us with 16 x 192, 97 us with 16 x 384.
constexpr int kVCluster = 16;
constexpr int kVChunk = 128;         // tokens a warp takes at once, 4 a lane

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

// A node's row of probabilities less its missed children: with a draft distribution, Z q of each miss;
// without, the missed tokens.
struct Row {
  const float* p;
  const float* q;          // nullptr: not needed
  int misses;              // 0: the row is p
  bool wide;               // rows start on 16 bytes and are read 16 bytes a lane
};

// Four probabilities of a row from token v on (0 from v1 on).
__device__ __forceinline__ float4 load4(const float* row, bool wide, int v, int v1) {
  if (wide && v + 4 <= v1) return __ldg(reinterpret_cast<const float4*>(row + v));
  return make_float4(v < v1 ? __ldg(row + v) : 0.f, v + 1 < v1 ? __ldg(row + v + 1) : 0.f,
                     v + 2 < v1 ? __ldg(row + v + 2) : 0.f, v + 3 < v1 ? __ldg(row + v + 3) : 0.f);
}

// Remaining weights of N tokens from their probabilities, token(k) their ids.  The misses are the outer
// loop: the N chains of products are independent.  Nothing is missed before the first miss, so its Z is 1.
template <bool Q, int N, class Token>
__device__ __forceinline__ void weights(const VerifyShared& S, int misses, float (&pv)[N], float (&qv)[N], Token token,
                                        u64 (&r)[N], bool& odd) {
  clean(pv, odd);
#pragma unroll
  for (int k = 0; k < N; ++k) r[k] = units(pv[k]);
  if (misses == 0) return;
  if (Q) {
    u64 w[N];
    clean(qv, odd);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      w[k] = units(qv[k]);
      r[k] = r[k] > w[k] ? r[k] - w[k] : 0ull;
    }
#pragma unroll 1
    for (int i = 1; i < misses; ++i) {
      const u64 z = S.z[i];
      if (z < kOne) {
        const u64 z4 = z << 4;
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const u64 t = __umul64hi(z4, w[k]);
          r[k] = r[k] > t ? r[k] - t : 0ull;
        }
      } else {                                  // (a row that sums to more than 1)
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const u64 t = mul60(z, w[k]);
          r[k] = r[k] > t ? r[k] - t : 0ull;
        }
      }
    }
  } else {
#pragma unroll 1
    for (int i = 0; i < misses; ++i) {
      const int gone = S.gone[i];
#pragma unroll
      for (int k = 0; k < N; ++k) r[k] = gone == token(k) ? 0ull : r[k];
    }
  }
}

// A probability's units as three limbs of 23, 23 and 14 bits, each the low bits of a float32: adding 1 (2^23)
// and rounding down leaves a limb in the significand, and what it leaves out is exact.  Bits of floats with
// one exponent are integers, so sums of limbs are sums of bits less their number times the exponent's.
// (Eight float instructions for 11 of the integer pipe and a 64-bit sum: 80 -> 71 us for 64 trees of 16 nodes over
// 152 K tokens.)
struct Limbs {
  uint32_t a, b, c;
};
constexpr uint32_t kLimbAB = 0x3f800000u, kLimbC = 0x4b000000u;
__device__ __forceinline__ Limbs limbs(float p) {
  p = __saturatef(p);
  const float y1 = __fadd_rd(p, 1.f), r1 = __fsub_rn(p, __fsub_rn(y1, 1.f));
  const float y2 = __fmaf_rd(r1, 0x1p23f, 1.f), r2 = __fmaf_rn(r1, 0x1p23f, -__fsub_rn(y2, 1.f));
  const float y3 = __fmaf_rd(r2, 0x1p37f, 0x1p23f);
  return {__float_as_uint(y1), __float_as_uint(y2), __float_as_uint(y3)};
}
// The sum of units that sums of limbs stand for, at most kTooMuch.  (a of at least 5 x 2^23 is more than 4
// whatever b and c, which stay below 2^31 either way, are.)
__device__ __forceinline__ u64 limb_sum(uint32_t a, int32_t b, int32_t c) {
  if (a >= 5u << 23) return kTooMuch;
  const long long t = ((long long)a << 37) + ((long long)b << 14) + c;
  return min((u64)t, kTooMuch);
}

// This lane's part of the sum of a row's weights over tokens v0 .. v1 - 1, one warp's.  The next chunk
// is on its way while one is summed.  No miss: sum p; one miss of a drawn draft: sum max(p - q, 0), as Z is
// 1; otherwise token by token.
enum { kPlain, kOneMiss, kMisses, kGone };
template <int kMode>
__device__ __forceinline__ u64 sum_chunks(const VerifyShared& S, const Row& R, int v0, int v1, bool& odd) {
  constexpr bool Q = kMode == kOneMiss || kMode == kMisses;
  constexpr int kBlock = 32;                    // chunks between conversions: 128 limbs below 2^23 each
  int v = v0 + 4 * (threadIdx.x & 31);
  const int chunks = (v1 - v0 + kVChunk - 1) / kVChunk;
  const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
  float4 p = load4(R.p, R.wide, v, v1), q = Q ? load4(R.q, R.wide, v, v1) : none;
  u64 acc = 0ull;
#pragma unroll 1
  for (int i0 = 0; i0 < chunks; i0 += kBlock) {
    uint32_t a = 0u, b = 0u, c = 0u;
    const int here = min(kBlock, chunks - i0);
#pragma unroll 1
    for (int i = 0; i < here; ++i, v += kVChunk) {
      float pv[4] = {p.x, p.y, p.z, p.w}, qv[4] = {q.x, q.y, q.z, q.w};
      p = load4(R.p, R.wide, v + kVChunk, v1);
      if (Q) q = load4(R.q, R.wide, v + kVChunk, v1);
      if constexpr (kMode == kPlain || kMode == kOneMiss) {
        clean(pv, odd);
        if (Q) clean(qv, odd);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const Limbs x = limbs(pv[k]);
          if constexpr (Q) {
            const Limbs y = limbs(fminf(pv[k], qv[k]));
            a += x.a - y.a;
            b += x.b - y.b;
            c += x.c - y.c;
          } else {
            a += x.a;
            b += x.b;
            c += x.c;
          }
        }
      } else {
        u64 w[4];
        weights<Q>(S, R.misses, pv, qv, [&](int k) { return v + k; }, w, odd);
        acc = add_capped(acc, (w[0] + w[1]) + (w[2] + w[3]));   // (4 + 4 at most)
      }
    }
    if constexpr (kMode == kPlain) {
      a -= 4u * here * kLimbAB;
      b -= 4u * here * kLimbAB;
      c -= 4u * here * kLimbC;
    }
    if constexpr (kMode == kPlain || kMode == kOneMiss) acc = add_capped(acc, limb_sum(a, (int32_t)b, (int32_t)c));
  }
  return acc;
}
__device__ __noinline__ u64 sum_part(const VerifyShared& S, const Row R, int v0, int v1, bool& odd) {
  bool bad = false;
  const u64 acc = R.misses == 0   ? sum_chunks<kPlain>(S, R, v0, v1, bad)
                  : !R.q          ? sum_chunks<kGone>(S, R, v0, v1, bad)
                  : R.misses == 1 ? sum_chunks<kOneMiss>(S, R, v0, v1, bad)
                                  : sum_chunks<kMisses>(S, R, v0, v1, bad);
  odd |= bad;
  return acc;
}

__global__ void __launch_bounds__(kVThreads, 4) verify_tree_kernel(const __grid_constant__ VerifyParams P) {
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
  bool bad = n < 0 || n > kNodes || first < 0 || first > P.n_rows - n;
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
      if (!bad || (n > 0 && first >= 0 && first <= P.n_rows - n))
#pragma unroll 1
        for (int j = tid; j < n; j += kVThreads) P.path[first + j] = -1;
      if (tid == 0) {
        if (bad) set_status(P.status, KVQ_ERR_BOUNDS);
        P.n_accept[b] = 0;
        P.next_token[b] = -1;
      }
    }
    return;                                     // (uniform over the cluster: nothing waits for it)
  }

  // this warp's contiguous segment of the vocabulary
  const int per = kVCluster * kVWarps * kVChunk;
  const int seg = ((P.vocab + per - 1) / per) * kVChunk;
  const int v0 = min(P.vocab, (rank * kVWarps + warp) * seg), v1 = min(P.vocab, v0 + seg);
  const bool wide = ((reinterpret_cast<uintptr_t>(P.p) | reinterpret_cast<uintptr_t>(P.q)) & 15) == 0 &&
                    ((P.p_stride | P.q_stride) & 3) == 0;
  bool odd = false;                             // saw a value that is no probability
  int misses = 0;                               // misses of the current node
  bool whole = false;                           // their residual was empty: the weights are p again
  int cur = 0, depth = 1;
  int pass = 0;
  u64 of_rank = 0ull;                           // the last pass's sum of CTA `lane`

  auto row = [&]() {
    return Row{P.p + (long long)(first + cur) * P.p_stride, P.q ? P.q + (long long)(first + cur) * P.q_stride : nullptr,
               whole ? 0 : misses, wide};
  };
  // sum over the vocabulary of the remaining weights; S.sum keeps the warps' sums and S.total the
  // CTA's of the last pass (two sets: a pass writes one while others may still read the other)
  auto sum_weights = [&]() {
    const u64 acc = warp_sum(sum_part(S, row(), v0, v1, odd));
    const int set = pass++ & 1;
    if (lane == 0) S.sum[set][warp] = acc;
    __syncthreads();
    if (warp == 0) {
      const u64 t = warp_sum(lane < kVWarps ? S.sum[set][lane] : 0ull);
      if (lane == 0) S.total[set] = t;
    }
    cluster.sync();
    of_rank = lane < kVCluster ? *cluster.map_shared_rank(&S.total[set], lane) : 0ull;
    return warp_sum(of_rank);
  };

  // nodes in index order; every warp of every CTA takes the same decisions
  if (rank == 0 && tid == 0) {
    P.path[first] = 0;
    P.next_token[b] = -1;                       // (until the draw below, a cluster barrier later)
  }
  u64 mass = kOne;
#pragma unroll 1
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
    u64 at[1];
    float pw[1] = {S.pw[c]}, qw[1] = {S.qw[c]};
    clean(qw, odd);
    const u64 claim = units(qw[0]);             // (1 for point-mass drafts)
    if (P.q) weights<true>(S, misses, pw, qw, [&](int) { return x; }, at, odd);
    else weights<false>(S, misses, pw, qw, [&](int) { return x; }, at, odd);
    const u64 w = at[0];
    if (mul60(mul60(mass, claim), units_below_1(S.u[c])) < w) {
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
#pragma unroll 1
    for (int j = depth + tid; j < n; j += kVThreads) P.path[first + j] = -1;

  // the token after the last taken node (a miss with a draft distribution has left its sums)
  u64 total = P.q && misses > 0 && !whole ? mass : sum_weights();
  if (total == 0ull && !whole) {
    whole = true;
    total = sum_weights();
  }
  const int set = (pass - 1) & 1;
  if (rank == 0 && tid == 0) P.n_accept[b] = depth;
  if (odd) set_status(P.status, KVQ_ERR_NONFINITE);
  if (total == 0ull || total >= kTooMuch) {
    if (rank == 0 && tid == 0) set_status(P.status, KVQ_ERR_NONFINITE);
  } else {
    // the CTA, its warp, the chunk, the lane and the token in which the sum passes the goal
    u64 goal = mul60(total, units_below_1(S.u[0]));
    auto narrow = [&](u64 mine) {               // lane whose sum passes it (goal: what is left there), or -1
      u64 upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 t = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += t;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, upto > goal);
      if (hit) {
        goal -= __shfl_sync(0xffffffffu, upto - mine, __ffs(hit) - 1);
        return __ffs(hit) - 1;
      }
      goal -= __shfl_sync(0xffffffffu, upto, 31);
      return -1;
    };
    if (narrow(of_rank) == rank && narrow(lane < kVWarps ? S.sum[set][lane] : 0ull) == warp) {
      const Row R = row();
      const bool need_q = R.q && R.misses;
#pragma unroll 1
      for (int v = v0 + 4 * lane; v - 4 * lane < v1; v += kVChunk) {
        const float4 a = load4(R.p, wide, v, v1), c = need_q ? load4(R.q, wide, v, v1) : make_float4(0.f, 0.f, 0.f, 0.f);
        float pv[4] = {a.x, a.y, a.z, a.w}, qv[4] = {c.x, c.y, c.z, c.w};
        u64 w[4];
        if (need_q) weights<true>(S, R.misses, pv, qv, [&](int k) { return v + k; }, w, odd);
        else weights<false>(S, R.misses, pv, qv, [&](int k) { return v + k; }, w, odd);
        const int at = narrow((w[0] + w[1]) + (w[2] + w[3]));
        if (at >= 0) {
          if (lane == at) {
            int k = 0;
#pragma unroll
            for (int i = 0; i < 3; ++i)
              if (k == i && goal >= w[i]) {
                goal -= w[i];
                ++k;
              }
            P.next_token[b] = v + k;
          }
          break;
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
  int bad = n < 0 || n > kNodes || first < 0 || first > P.n_rows - n || keep < 0 || keep > n || L0 < 0 ||
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
  P.path = path;
  P.n_accept = n_accept;
  P.next_token = next_token;
  P.status = d_status;
  // clusters of more than 8 CTAs, once per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KVQ_ERR_CUDA;
  static std::atomic<unsigned long long> allowed{0};
  if (!(allowed.load() & (1ull << dev))) {
    if (cudaFuncSetAttribute((const void*)verify_tree_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
      return KVQ_ERR_CUDA;
    allowed.fetch_or(1ull << dev);
  }
  return launch_pdl_cluster(verify_tree_kernel, kVCluster, dim3(kVCluster, cfg->batch), dim3(kVThreads), 0, stream, P) ==
                 cudaSuccess
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
