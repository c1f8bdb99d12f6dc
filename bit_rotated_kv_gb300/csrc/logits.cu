// kv_logits_probs and kv_token_counts: from logits to the probabilities that kv_verify_tree takes, and the counts
// that the penalties go by.
//
//   x = logit + bias;  x = held ? (x > 0 ? x / r : x r) : x;  x -= f n;  x -= n > 0 ? a : 0;  x = allowed ? x : -inf
//   p = exp((x - max x) / T) / sum exp((x - max x) / T)           (T = 0: 1 at the lowest argmax, 0 elsewhere)
// Every operation rounds to float32 by itself (no contraction), sums are float32 in one fixed order.
//
// Bytes bound it: a logit is read once and a probability written once (64 rows of 152 K tokens: 2 + 2 + 4 bytes each
// with the counts), which needs the row on the chip between the two.  A row of 152 K float32 is 0.6 MB, more than an
// SM's shared memory, so a cluster of CTAs takes a row, a contiguous slice each, and they exchange one (maximum, sum) pair
// through distributed shared memory.  At 6.8 TB/s an SM has about thirty instructions a token to spare in all.  Penalties
// are therefore taken without branches (in a history of thousands nearly every warp meets a counted token: behind one they
// took 64 instructions a token, and 64 trees of 16 nodes over 152 K 531 us instead of 221), and loads come in batches that
// are all on their way before the first is used.  Biases and the drafted path touch few tokens: the pass over the slice
// does without them and the tokens concerned are computed again afterwards, by token, so that one that is in both lists is
// right either way.
// What it measured: those 64 x 16 rows 221 us (floor by bytes 106: neither issue, 52%, nor DRAM, 37%, is at its limit; a slice goes
// through shared memory four times, between barriers that are the largest stall), 64 rows of 152 K 25 us (11.5: 768 CTAs, of which
// four an SM, 608, are on the chip at once: a second wave that is mostly empty), 48 rows of 100,003 16 us (3.3: three of four such rows
// begin off a boundary and go token by token), one row of 32 K 4.4 us (a launch and four waits one after another).
#include <cooperative_groups.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "launch.h"

namespace cg = cooperative_groups;

namespace kvq {
namespace {

constexpr int kLThreads = 256;
constexpr int kLWarps = kLThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kBatch = 6;            // fours that a thread asks for at once
constexpr int kNodes = KVQ_TREE_MAX_NODES;
constexpr float kInf = __builtin_huge_valf();

struct LogitParams {
  const void* logits;
  long long l_stride;
  int vocab, per;            // per: tokens of a CTA's slice (a multiple of 32)
  const int32_t* cu_rows;
  const int32_t* parent;
  const int32_t* token;
  int batch, n_rows;
  float* p;
  long long p_stride;
  int32_t* status;
  kvq_logit_rules u;
};

// What the cluster's CTAs read of each other.
struct Share {
  float top;                 // the slice's largest value
  float sum;                 // its sum of exp((x - top) / T)
  int best;                  // T = 0: the lowest token that has it
  int bad;
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

// Four logits as they lie, and as numbers.
template <typename T>
struct Four {
  using Raw = std::conditional_t<sizeof(T) == 4, uint4, uint2>;
  static __device__ __forceinline__ Raw none() {
    if constexpr (sizeof(T) == 4) return make_uint4(0u, 0u, 0u, 0u);
    else return make_uint2(0u, 0u);
  }
  static __device__ __forceinline__ void numbers(const Raw& r, float (&x)[4]) {
    const T* h = reinterpret_cast<const T*>(&r);
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = to_float(h[k]);
  }
};

struct Rules {
  float rep, freq, pres;
  float inv;                 // 1 / rep, to nearest
};
// A value under the penalties of its token; count: as it is kept (or more, with the path's).  x / rep is the product with
// the rounded reciprocal, and its remainder: the quotient to nearest where nothing vanishes on the way (Markstein's theorem).
__device__ __forceinline__ float penalized(const Rules& R, float x, uint32_t count, uint32_t times) {
  const float q = __fmul_rn(x, R.inv);
  float y = x > 0.f ? __fmaf_rn(__fmaf_rn(-q, R.rep, x), R.inv, q) : __fmul_rn(x, R.rep);
  y = __fsub_rn(y, __fmul_rn(R.freq, (float)times));
  y = __fsub_rn(y, times ? R.pres : 0.f);
  return count ? y : x;
}

// (x - r) k of two numbers, each operation rounded
__device__ __forceinline__ float2 scaled_below(float x, float y, float2 minus_r, float2 k) {
  float2 d;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " add.rn.f32x2 x, x, y;\n mul.rn.f32x2 x, x, z;\n mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(x), "f"(y), "f"(minus_r.x), "f"(minus_r.y), "f"(k.x), "f"(k.y));
  return d;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));   // (what is below 2^-126 is 0)
  return y;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The row's sequence: how many of them end at or before it.  A warp looks at 32 ends at a time.
__device__ __forceinline__ int sequences_before(const int32_t* cu_rows, int batch, int row, int lane) {
  int lo = 0, hi = batch;                                // (the answer lies between them)
  if (batch <= 128) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = 32 * k + lane;
      n += __popc(__ballot_sync(0xffffffffu, i < batch && cu_rows[min(i, batch - 1) + 1] <= row));
    }
    return n;
  }
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32, i = lo + (lane + 1) * step - 1;
    const int n = __popc(__ballot_sync(0xffffffffu, i < hi && cu_rows[min(i, batch - 1) + 1] <= row));
    lo = min(lo + n * step, hi);
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
// (for a warp that has written nothing for the others: it need not wait for its stores; 228 us became 221 for 64 x 16 rows)
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <typename T, bool kCounts, bool kMask>
__global__ void __launch_bounds__(kLThreads) logits_kernel(const __grid_constant__ LogitParams P) {
  extern __shared__ __align__(16) float xs[];          // the slice
  __shared__ float wred[kLWarps];
  __shared__ int wbest[kLWarps];
  __shared__ int par[kNodes], tok[kNodes], path[kNodes], n_path_sh;
  __shared__ Share shares[kMaxCluster];                // of every CTA of the cluster, written by it
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = (int)(blockIdx.x / (unsigned)ranks);
  const bool lead = rank == 0 && tid == 0;
  const int v0 = min(P.vocab, rank * P.per), v1 = min(P.vocab, v0 + P.per);
  const int fours = (v1 - v0) >> 2, rest = (v1 - v0) & 3;
  using F = Four<T>;
  using Raw = typename F::Raw;
  const T* l = static_cast<const T*>(P.logits) + (long long)row * P.l_stride;
  const Raw* lw = reinterpret_cast<const Raw*>(l + v0);
  const bool l_wide = (reinterpret_cast<uintptr_t>(l) & (4 * sizeof(T) - 1)) == 0;
  pdl_trigger();
  cluster_arrive_relaxed();                              // (waited for before a CTA writes to another)
  pdl_wait();
  // the first logits and the rest of the slice are on their way while the row's sequence and its rules are found
  Raw r[kBatch];
  if (!kMask) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = tid + k * kLThreads;
      r[k] = F::none();
      if (l_wide && i < fours) r[k] = lw[i];
    }
    for (int v = v0 + 4 * kBatch * kLThreads + tid * (128 / (int)sizeof(T)); v < v1; v += kLThreads * (128 / (int)sizeof(T)))
      prefetch_l2_line(l + v);
  }

  const int b = sequences_before(P.cu_rows, P.batch, row, lane);
  const bool covered = b < P.batch && P.cu_rows[b] >= 0 && P.cu_rows[b] <= row && P.cu_rows[b + 1] > row;
  if (!covered) {                                        // (the same in all CTAs of the cluster)
    if (lead) set_status(P.status, KVQ_ERR_BOUNDS);
    cluster_wait();
    return;
  }
  const int first = P.cu_rows[b], node = row - first;
  const int n = min(P.cu_rows[b + 1], P.n_rows) - first;

  // ---- this row's rules ----
  const kvq_logit_rules& U = P.u;
  Rules R;
  R.rep = U.repetition ? U.repetition[b] : 1.f;
  R.freq = U.frequency ? U.frequency[b] : 0.f;
  R.pres = U.presence ? U.presence[b] : 0.f;
  R.inv = __frcp_rn(R.rep);
  const float heat = U.temperature ? U.temperature[b] : 1.f;
  const bool sound = R.rep >= 0x1p-60f && R.rep <= 0x1p60f && fabsf(R.freq) < kInf && fabsf(R.pres) < kInf && heat >= 0.f && heat < kInf;
  const bool greedy = heat < 0x1p-149f;                  // (0.  Written == 0 the compiler gives bf16 with counts 48 registers instead of 63: 245 us)
  const float k2 = greedy ? 0.f : __fdiv_rn(1.4426950408889634f, fmaxf(heat, 0x1p-120f));   // (1 / T must be a float32)
  const uint16_t* counts = kCounts ? U.counts + (long long)b * U.count_stride : nullptr;
  const uint32_t* mask = nullptr;
  bool fault = false, skip = !sound;                     // skip: a row of zeros
  if (kMask) {
    const int m = U.mask_row ? U.mask_row[row] : row;
    if (m < -1 || m >= U.n_masks) fault = skip = true;
    else if (m >= 0) mask = U.mask + (long long)m * U.mask_stride;
  }
  int b0 = 0, b1 = 0;
  if (U.bias_cu) {
    b0 = U.bias_cu[b];
    b1 = U.bias_cu[b + 1];
    if (b0 < 0 || b1 > U.n_bias || b0 > b1) {
      fault = true;
      b0 = b1 = 0;
    }
  }
  const bool tree = P.parent != nullptr;
  if (tree && n > kNodes) fault = skip = true;

  // ---- the node's path: tokens of the node and its ancestors, roots left out (the last warp; the others go on) ----
  if (tree && !skip && warp == kLWarps - 1) {
    for (int i = lane; i <= node; i += 32) {
      par[i] = P.parent[first + i];
      tok[i] = P.token[first + i];
    }
    __syncwarp();
    if (lane == 0) {
      int at = node, np = 0;
      while (par[at] >= 0 && par[at] < at) {             // (at falls: at most kNodes steps)
        if (tok[at] >= 0 && tok[at] < P.vocab) path[np++] = tok[at];
        else fault = true;
        at = par[at];
      }
      if (par[at] != -1) fault = true;
      n_path_sh = np;
    }
  }
  if (fault && rank == 0) set_status(P.status, KVQ_ERR_BOUNDS);
  if (!sound && lead) set_status(P.status, KVQ_ERR_NONFINITE);

  float* out = P.p + (long long)row * P.p_stride;
  const bool c_wide = (reinterpret_cast<uintptr_t>(counts) & 7) == 0;
  const bool p_wide = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
  float top = -kInf;

  if (!skip) {
    // ---- pass 1: the slice's values, without biases and the path ----
    auto keep = [&](int i, float (&x)[4], uint32_t allowed, uint2 c) {
      if (kCounts) {
        const uint32_t n[4] = {c.x & 0xffffu, c.x >> 16, c.y & 0xffffu, c.y >> 16};
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = penalized(R, x[k], n[k], n[k] & KVQ_COUNT_MOST);
      }
      if (kMask)
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = (allowed >> k) & 1u ? x[k] : -kInf;
      top = fmaxf(fmaxf(fmaxf(top, x[0]), fmaxf(x[1], x[2])), x[3]);   // (drops a NaN: the sum will not)
      *reinterpret_cast<float4*>(xs + 4 * i) = make_float4(x[0], x[1], x[2], x[3]);
    };
    const uint2* cw = reinterpret_cast<const uint2*>(counts + (kCounts ? v0 : 0));
    auto batch = [&](int i0, auto whole) {               // whole: all kBatch of them are there
      uint2 c[kBatch];
      uint32_t m[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * kLThreads;
        m[k] = whole.value || i < fours ? 15u : 0u;
        if (kMask && mask && m[k]) m[k] = (mask[(v0 >> 5) + (i >> 3)] >> (4 * (i & 7))) & 15u;
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * kLThreads;
        c[k] = make_uint2(0u, 0u);
        if ((whole.value && !kMask) || m[k]) {
          if (kMask || i0 != tid) r[k] = lw[i];          // (without a mask the first ones are here)
          if (kCounts) c[k] = __ldg(cw + i);
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * kLThreads;
        if (whole.value || i < fours) {
          float x[4];
          F::numbers(r[k], x);
          keep(i, x, m[k], c[k]);
        }
      }
    };
    const bool wide = l_wide && (!kCounts || c_wide);
    if (wide) {
      int i0 = 0;
      for (; i0 + kBatch * kLThreads <= fours; i0 += kBatch * kLThreads) batch(i0 + tid, std::true_type{});
      if (i0 + tid < fours) batch(i0 + tid, std::false_type{});
    }
    // (rows that do not begin on a boundary, and the slice's last tokens: token by token)
    constexpr int kFew = 3;
    for (int i0 = (wide ? fours : 0) + tid; i0 < fours + (rest > 0); i0 += kFew * kLThreads) {
      uint32_t m[kFew], n[kFew][2];
      float x[kFew][4];
#pragma unroll
      for (int k = 0; k < kFew; ++k) {
        const int i = i0 + k * kLThreads;
        m[k] = i < fours ? 15u : i == fours ? (1u << rest) - 1u : 0u;
        if (kMask && mask && m[k]) m[k] &= mask[(v0 >> 5) + (i >> 3)] >> (4 * (i & 7));
      }
#pragma unroll
      for (int k = 0; k < kFew; ++k) {
        const int v = v0 + 4 * (i0 + k * kLThreads);
        uint32_t c[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool on = (m[k] >> e) & 1u;
          x[k][e] = on ? to_float(l[v + e]) : -kInf;
          c[e] = on && kCounts ? (uint32_t)__ldg(counts + v + e) : 0u;
        }
        n[k][0] = c[0] | c[1] << 16;
        n[k][1] = c[2] | c[3] << 16;
      }
#pragma unroll
      for (int k = 0; k < kFew; ++k) {
        const int i = i0 + k * kLThreads;
        if (i < fours + (rest > 0)) keep(i, x[k], m[k], make_uint2(n[k][0], n[k][1]));
      }
    }
    if (tree || b1 > b0) __syncthreads();
    const int n_path = tree ? n_path_sh : 0;
    if (n_path > 0 || b1 > b0) {
      // ---- tokens of the path and the biases: again, by token ----
      for (int i = tid; i < n_path + (b1 - b0); i += kLThreads) {
        int t;
        if (i < n_path) {
          t = path[i];
        } else {
          const int e = b0 + i - n_path;
          t = U.bias_token[e];
          if (t < 0 || t >= P.vocab || (e > b0 && U.bias_token[e - 1] >= t)) {
            if (rank == 0) set_status(P.status, KVQ_ERR_BOUNDS);
            continue;
          }
        }
        if (t < v0 || t >= v1) continue;
        float x = -kInf;
        if (!mask || ((mask[t >> 5] >> (t & 31)) & 1u)) {
          x = to_float(l[t]);
          const uint32_t c = kCounts ? (uint32_t)counts[t] : 0u;
          int lo = b0, hi = b1;                          // the first entry that is not below t
          while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (U.bias_token[mid] < t) lo = mid + 1;
            else hi = mid;
          }
          if (lo < b1 && U.bias_token[lo] == t) x = __fadd_rn(x, U.bias[lo]);
          uint32_t times = c & KVQ_COUNT_MOST;
          for (int j = 0; j < n_path; ++j) times += path[j] == t;
          x = penalized(R, x, c | times, times);
        }
        xs[t - v0] = x;
      }
      __syncthreads();
      top = -kInf;
#pragma unroll 4
      for (int v = 4 * tid; v < v1 - v0; v += 4 * kLThreads) {
        const float4 x = *reinterpret_cast<const float4*>(xs + v);
        top = fmaxf(fmaxf(fmaxf(top, x.x), fmaxf(x.y, x.z)), x.w);
      }
    }
  }

  // ---- the slice's maximum ----
  top = warp_max(top);
  if (lane == 0) wred[warp] = top;
  __syncthreads();
  top = wred[0];
#pragma unroll
  for (int w = 1; w < kLWarps; ++w) top = fmaxf(top, wred[w]);
  __syncthreads();

  // ---- pass 2: exponentials and their sum, or the lowest token of the maximum ----
  if (!skip && !greedy) {
    const float ref = top == -kInf ? 0.f : top;
    const float2 r2 = make_float2(-ref, -ref), kk = make_float2(k2, k2);
    float s = 0.f;
#pragma unroll 4
    for (int v = 4 * tid; v < v1 - v0; v += 4 * kLThreads) {
      float4 x = *reinterpret_cast<const float4*>(xs + v);
      const float2 y = scaled_below(x.x, x.y, r2, kk), z = scaled_below(x.z, x.w, r2, kk);
      x = make_float4(ex2(y.x), ex2(y.y), ex2(z.x), ex2(z.y));
      *reinterpret_cast<float4*>(xs + v) = x;
      s += (x.x + x.y) + (x.z + x.w);
    }
    s = warp_add(s);
    if (lane == 0) wred[warp] = s;
  } else if (!skip) {
    int best = P.vocab;                                  // (-1: a value that is none)
    for (int v = tid; v < v1 - v0; v += kLThreads) {
      const float x = xs[v];
      if (x == top) best = min(best, v0 + v);
      if (!(x < kInf)) best = -1;
    }
    best = __reduce_min_sync(0xffffffffu, best);
    if (lane == 0) wbest[warp] = best;
  }
  __syncthreads();
  cluster_wait();                                        // (every CTA of the cluster has begun)
  if (warp == 0) {
    const float s = warp_add(!skip && !greedy && lane < kLWarps ? wred[lane] : 0.f);
    const int best = __reduce_min_sync(0xffffffffu, !skip && greedy && lane < kLWarps ? wbest[lane] : P.vocab);
    // (a NaN or an infinity in the slice makes its sum a NaN)
    if (lane < ranks) *cluster.map_shared_rank(&shares[rank], lane) = Share{top, s, best, best < 0 || !(s < kInf)};
  }
  if (warp == 0) cluster_arrive();
  else cluster_arrive_relaxed();
  cluster_wait();
  Share other{-kInf, 0.f, P.vocab, 0};
  if (lane < ranks) other = shares[lane];
  const float whole = warp_max(other.top);
  const float share = other.top == -kInf ? 0.f : ex2((other.top - whole) * k2);
  const float sum = warp_add(other.sum * share);
  const int best = __reduce_min_sync(0xffffffffu, other.top == whole ? other.best : P.vocab);
  const bool none = __any_sync(0xffffffffu, other.bad != 0) || whole == -kInf;
  if (none && !skip && lead) set_status(P.status, KVQ_ERR_NONFINITE);
  const float factor = __fdiv_rn(__shfl_sync(0xffffffffu, share, rank), sum);

  // ---- pass 3: the slice's probabilities ----
  const bool zeros = skip || none;
  if (p_wide) {
#pragma unroll 4
    for (int i = tid; i < fours; i += kLThreads) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      const int v = v0 + 4 * i;
      if (!zeros && !greedy) {
        x = *reinterpret_cast<const float4*>(xs + 4 * i);
        x = make_float4(x.x * factor, x.y * factor, x.z * factor, x.w * factor);
      } else if (!zeros) {
        x = make_float4(v == best ? 1.f : 0.f, v + 1 == best ? 1.f : 0.f, v + 2 == best ? 1.f : 0.f, v + 3 == best ? 1.f : 0.f);
      }
      *reinterpret_cast<float4*>(out + v) = x;
    }
  }
#pragma unroll 4
  for (int i = (p_wide ? 4 * fours : 0) + tid; i < v1 - v0; i += kLThreads)
    out[v0 + i] = zeros ? 0.f : greedy ? (v0 + i == best ? 1.f : 0.f) : xs[i] * factor;
}

// ---- counts ------------------------------------------------------------------------------------
struct CountParams {
  uint16_t* counts;
  long long stride;
  int vocab, kind;
  const int32_t* cu_rows;
  const int32_t* token;
  const int32_t* path;
  const int32_t* n_accept;
  const int32_t* next_token;
  int batch, n_rows;
  int32_t* status;
};

// One 16-bit half of a 32-bit word of counts: what the other half holds is left alone.
struct Half {
  uint32_t* word;
  int shift;
};
__device__ __forceinline__ Half half_of(const CountParams& P, int b, int t) {
  const long long at = (long long)b * P.stride + t;
  return {reinterpret_cast<uint32_t*>(P.counts) + (at >> 1), (int)(at & 1) * 16};
}
// `more` tokens more, up to the most; old: what the word held a moment ago; all: as many as the call may add to it after that.
// (Far from the most an addition will do: of the warps that meet at an answer's most frequent token only one would have
// its exchange accepted at a time.)
__device__ __forceinline__ void add_tokens(const Half& h, uint32_t old, uint32_t more, uint32_t all) {
  if (((old >> h.shift) & KVQ_COUNT_MOST) + all <= KVQ_COUNT_MOST) {
    atomicAdd(h.word, more << h.shift);
    return;
  }
  for (;;) {
    const uint32_t have = (old >> h.shift) & KVQ_COUNT_MOST, room = KVQ_COUNT_MOST - have;
    if (room == 0u) return;
    const uint32_t seen = atomicCAS(h.word, old, old + (min(more, room) << h.shift));   // (no carry: a count stays below its most)
    if (seen == old) return;
    old = seen;
  }
}

constexpr int kPerLane = 4;          // rows of a lane: a warp takes 128 in a row, and their loads are on their way together

// Latency bounds a step's few tokens (a chain of four loads and an atomic); a prompt's many, the random words that they
// mark: 8 K tokens of each of 16 sequences take 6.6 us with the clearing of their counts.  4 K answered tokens of each of 16 take 9 us
// (0.3 MB): 500 warps of 128 rows are 63 CTAs, fewer than half of the SMs.  Equal tokens of a warp are counted
// with one atomic (an answer's most frequent ones meet there).
__global__ void __launch_bounds__(256) count_kernel(const __grid_constant__ CountParams P) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int warp = (int)(blockIdx.x * 8 + (threadIdx.x >> 5)), warps = (P.n_rows + 32 * kPerLane - 1) / (32 * kPerLane);
  int b[kPerLane], t[kPerLane];
  uint32_t all[kPerLane];                                // tokens that the call may count for the sequence
  bool odd = false;
#pragma unroll
  for (int k = 0; k < kPerLane; ++k) {
    b[k] = -1;
    all[k] = ~0u >> 1;
  }
  if (warp < warps) {
    const int r0 = warp * 32 * kPerLane;
    // (an end behind the last row: the rows that there are belong to the sequence all the same)
    if (warp == 0 && lane == 0) odd = __ldg(P.cu_rows + P.batch) > P.n_rows;
    int from[kPerLane];
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      const int r = r0 + 32 * k + lane;
      from[k] = r < P.n_rows ? __ldg((P.path ? P.path : P.token) + r) : -1;
    }
    const int before = sequences_before(P.cu_rows, P.batch, r0, lane);
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      const int r = r0 + 32 * k + lane;
      if (r >= P.n_rows) continue;
      int s = before;
      while (s < P.batch && __ldg(P.cu_rows + s + 1) <= r) ++s;
      const int first = s < P.batch ? __ldg(P.cu_rows + s) : -1;
      if (first < 0 || first > r) {
        odd = true;
        continue;
      }
      t[k] = from[k];
      const int n = __ldg(P.cu_rows + s + 1) - first;    // (more than 0: r is among them)
      all[k] = min((uint32_t)n, 1u << 30) + 1u;
      if (P.path) {
        const int j = r - first;
        if (j == 0 || j >= __ldg(P.n_accept + s)) continue;
        if (from[k] < 0 || from[k] >= n || first > P.n_rows - n) {
          odd = true;
          continue;
        }
        t[k] = __ldg(P.token + first + from[k]);
      }
      b[k] = s;
    }
  } else {
    // the tokens behind the paths: a sequence to a lane (and nothing for the warps that fill the last block up)
    const int s = (warp - warps) * 32 + lane;
    if (P.next_token && s < P.batch) {
      t[0] = __ldg(P.next_token + s);
      b[0] = t[0] == -1 ? -1 : s;
    }
  }
  Half h[kPerLane];
  uint32_t old[kPerLane];
#pragma unroll
  for (int k = 0; k < kPerLane; ++k) {
    if (b[k] >= 0 && (t[k] < 0 || t[k] >= P.vocab)) {
      odd = true;
      b[k] = -1;
    }
    if (b[k] >= 0) {
      h[k] = half_of(P, b[k], t[k]);
      old[k] = *reinterpret_cast<volatile uint32_t*>(h[k].word);
    }
  }
  if (odd) set_status(P.status, KVQ_ERR_BOUNDS);
#pragma unroll
  for (int k = 0; k < kPerLane; ++k) {
    if (P.kind == KVQ_COUNT_PROMPT) {
      const uint32_t bit = 0x8000u << (b[k] >= 0 ? h[k].shift : 0);
      if (b[k] >= 0 && !(old[k] & bit)) atomicOr(h[k].word, bit);
    } else {
      const unsigned long long key = b[k] >= 0 ? (unsigned long long)(b[k] + 1) << 32 | (uint32_t)t[k] : (unsigned long long)lane;
      const unsigned same = __match_any_sync(0xffffffffu, key);
      if (b[k] >= 0 && lane == __ffs(same) - 1) add_tokens(h[k], old[k], __popc(same), all[k]);
    }
  }
}

// Long prompts: a cluster of CTAs takes a sequence.  Each gathers its share of the tokens as bits of the vocabulary in its shared
// memory, then puts a slice of them all together and marks it in one sweep over the slice's counts, which are nobody else's in
// this call.  (Each CTA looking at all of the prompt for the bits of its slice alone took 24 us for 16 of 64 K to 128 K tokens, 12 us so.)
constexpr int kSweepThreads = 1024;
constexpr int kSweepCtas = 8;         // of a sequence
constexpr int kSweepRows = 1 << 16, kSweepEach = 1 << 14;   // (fewer rows, of the call or a sequence, are marked one by one)
__global__ void __launch_bounds__(kSweepThreads) prompt_kernel(const __grid_constant__ CountParams P) {
  extern __shared__ __align__(16) uint32_t bits[];       // the vocabulary's, then the slice's of all CTAs
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int tid = threadIdx.x, b = (int)(blockIdx.x / (unsigned)ranks);
  const int words = (P.vocab + 31) >> 5, per = (words + ranks - 1) / ranks, w0 = min(words, rank * per), w1 = min(words, w0 + per);
  pdl_trigger();
  for (int i = tid; i < words; i += kSweepThreads) bits[i] = 0u;
  pdl_wait();
  const int first = P.cu_rows[b], end = P.cu_rows[b + 1], last = min(end, P.n_rows);
  // rows of no sequence: before the first, behind the last, or where cu_rows falls; ends behind the last row
  bool odd = first < 0 || end < first || end > P.n_rows || (b == 0 && first > 0) || (b == P.batch - 1 && end < P.n_rows);
  __syncthreads();
  if (first >= 0 && first < last) {
    auto mark = [&](int t) {
      if (t >= 0 && t < P.vocab) atomicOr(&bits[t >> 5], 1u << (t & 31));
      else odd = true;
    };
    // four tokens at a time from a boundary on, the others one by one
    const int32_t* from = P.token + first;
    const int n = last - first, head = min(n, (int)(((16 - (reinterpret_cast<uintptr_t>(from) & 15)) & 15) >> 2));
    const int fours = (n - head) >> 2;
    const int4* wide = reinterpret_cast<const int4*>(from + head);
    if (rank == 0 && tid < head) mark(__ldg(from + tid));
    if (rank == 0 && tid < n - head - 4 * fours) mark(__ldg(from + head + 4 * fours + tid));
#pragma unroll 4
    for (int i = rank * kSweepThreads + tid; i < fours; i += ranks * kSweepThreads) {
      const int4 t = __ldg(wide + i);
      mark(t.x);
      mark(t.y);
      mark(t.z);
      mark(t.w);
    }
  }
  if (odd) set_status(P.status, KVQ_ERR_BOUNDS);
  cluster.sync();
  uint32_t* all = bits + words;
  for (int i = tid; i < w1 - w0; i += kSweepThreads) {
    uint32_t x = 0u;
#pragma unroll 4
    for (int r = 0; r < ranks; ++r) x |= *cluster.map_shared_rank(bits + w0 + i, r);
    all[i] = x;
  }
  cluster_arrive();                                      // (this CTA has read the others')
  __syncthreads();
  // two tokens to a word (rows begin on one: the stride is even)
  uint32_t* row = reinterpret_cast<uint32_t*>(P.counts + (long long)b * P.stride) + 16 * (long long)w0;
#pragma unroll 4
  for (int i = tid; i < 16 * (w1 - w0); i += kSweepThreads) {
    const uint32_t two = all[i >> 4] >> (2 * (i & 15)) & 3u;
    if (two) row[i] |= (two & 1u) << 15 | (two & 2u) << 30;   // (no bit stands behind the vocabulary)
  }
  cluster_wait();
}

template <typename T, bool kCounts, bool kMask>
int launch_logits(LogitParams& P, cudaStream_t stream) {
  const auto kernel = logits_kernel<T, kCounts, kMask>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KVQ_ERR_CUDA;
  static std::mutex mu;
  static unsigned long long attr_done = 0;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!(attr_done & (1ull << dev))) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, KVQ_LOGITS_MAX_VOCAB / kMaxCluster * 4) != cudaSuccess ||
          cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return KVQ_ERR_CUDA;
      attr_done |= 1ull << dev;
    }
  }
  // CTAs of a row: slices of at most 13,000 tokens (51 KB: four CTAs of 256 threads on an SM; 64 trees of 16 nodes over
  // 152 K tokens took 231 us so, 245 us in slices of 17 K and 384 threads, 254 in slices of 25 K and 512, 264 in slices of
  // 9.5 K and 256), and more of them while the rows do not fill the SMs
  int c = std::max(1, (P.vocab + 12999) / 13000);
  while (c < kMaxCluster && c * (long long)P.n_rows < kSms && P.vocab / c > 2048) ++c;
  c = std::min(c, kMaxCluster);
  P.per = ((P.vocab + c - 1) / c + 31) / 32 * 32;
  if ((long long)P.n_rows * c > 0x7fffffffLL) return KVQ_ERR_UNSUPPORTED;
  return launch_pdl_cluster(kernel, c, dim3((unsigned)((long long)P.n_rows * c)), dim3(kLThreads), (size_t)P.per * 4, stream, P) ==
                 cudaSuccess
             ? KVQ_OK
             : KVQ_ERR_CUDA;
}
template <typename T>
int launch_logits(LogitParams& P, cudaStream_t stream) {
  if (P.u.mask) return P.u.counts ? launch_logits<T, true, true>(P, stream) : launch_logits<T, false, true>(P, stream);
  return P.u.counts ? launch_logits<T, true, false>(P, stream) : launch_logits<T, false, false>(P, stream);
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" int kvq_launch_logits_probs(const kvq_config* cfg, const kvq_logit_rules* rules, const void* logits,
                                       int32_t logits_type, int64_t l_stride, int32_t vocab, const int32_t* cu_rows,
                                       const int32_t* parent, const int32_t* token, int32_t n_rows, float* p,
                                       int64_t p_stride, int32_t* d_status, cudaStream_t stream) {
  LogitParams P{};
  P.logits = logits;
  P.l_stride = l_stride;
  P.vocab = vocab;
  P.cu_rows = cu_rows;
  P.parent = parent;
  P.token = token;
  P.batch = cfg->batch;
  P.n_rows = n_rows;
  P.p = p;
  P.p_stride = p_stride;
  P.status = d_status;
  if (rules) P.u = *rules;
  if (logits_type == KVQ_LOGITS_F32) return launch_logits<float>(P, stream);
  if (logits_type == KVQ_LOGITS_BF16) return launch_logits<__nv_bfloat16>(P, stream);
  return launch_logits<__half>(P, stream);
}

extern "C" int kvq_launch_token_counts(const kvq_config* cfg, uint16_t* counts, int64_t count_stride, int32_t vocab,
                                       int32_t kind, const int32_t* cu_rows, const int32_t* token, int32_t n_rows,
                                       const int32_t* path, const int32_t* n_accept, const int32_t* next_token,
                                       int32_t* d_status, cudaStream_t stream) {
  const CountParams P{counts, count_stride, vocab, kind, cu_rows, token, path, n_accept, next_token, cfg->batch, n_rows, d_status};
  // long prompts: 16 of 96 K tokens over 152 K take 11.7 us swept and 34.9 one by one, the clearing of their counts among it;
  // 16 of 32 K 10.7 and 13.6, one of 128 K 8.5 and 14.0; 16 of 8 K 10.5 and 6.6, 64 of 8 K 20.8 and 14.5, one of 16 K 7.5 and 5.1,
  // 64 of 1 K over a thousand 9.6 and 4.9
  // (clusters of 16 CTAs: 14.8 for the 16 of 96 K, 7.6 for the one of 128 K)
  if (kind == KVQ_COUNT_PROMPT && vocab <= KVQ_LOGITS_MAX_VOCAB && n_rows >= kSweepRows && n_rows / cfg->batch >= std::max(vocab / 6, kSweepEach)) {
    const int words = (vocab + 31) / 32;
    const size_t smem = 4 * ((size_t)words + (words + kSweepCtas - 1) / kSweepCtas);
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KVQ_ERR_CUDA;
    static std::mutex mu;
    static unsigned long long attr_done = 0;
    {
      std::lock_guard<std::mutex> lock(mu);
      if (!(attr_done & (1ull << dev))) {
        if (cudaFuncSetAttribute(prompt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, KVQ_LOGITS_MAX_VOCAB / 8 + KVQ_LOGITS_MAX_VOCAB / 8 / kSweepCtas) !=
            cudaSuccess)
          return KVQ_ERR_CUDA;
        attr_done |= 1ull << dev;
      }
    }
    if ((long long)cfg->batch * kSweepCtas > 0x7fffffffLL) return KVQ_ERR_UNSUPPORTED;
    return launch_pdl_cluster(prompt_kernel, kSweepCtas, dim3((unsigned)cfg->batch * kSweepCtas), dim3(kSweepThreads), smem, stream, P) == cudaSuccess
               ? KVQ_OK
               : KVQ_ERR_CUDA;
  }
  const long long warps = ((long long)n_rows + 32 * kPerLane - 1) / (32 * kPerLane) + (next_token ? (cfg->batch + 31) / 32 : 0);
  if (warps == 0) return KVQ_OK;
  return launch_pdl(count_kernel, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, stream, P) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
