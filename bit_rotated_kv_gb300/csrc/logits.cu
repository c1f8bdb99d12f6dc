// kv_logits_probs and kv_token_counts: from logits to the probabilities that kv_verify_tree takes, and the counts
// that the penalties go by.
//
//   x = logit + bias;  x = held ? (x > 0 ? x / r : x r) : x;  x -= f n;  x -= n > 0 ? a : 0;  x = allowed ? x : -inf
//   p = exp((x - max x) / T) / sum exp((x - max x) / T)           (T = 0: 1 at the lowest argmax, 0 elsewhere)
// Every operation rounds to float32 by itself (no contraction), sums are float32 in one fixed order.
//
// Bytes bound it: a logit is read once and a probability written once (64 rows of 152 K tokens: 2 + 2 + 4 bytes each
// with the counts), which needs the row on the chip between the two passes.  A row of 152 K float32 is 0.6 MB, more than an
// SM's shared memory, so a cluster of CTAs takes a row, a contiguous slice each, and they exchange one (maximum, sum) pair
// through distributed shared memory.  Biases and the drafted path touch few tokens: the pass over the slice does without them and the
// tokens concerned are computed again afterwards, by token, so that one that is in both lists is right either way.
#include <cooperative_groups.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "launch.h"

namespace cg = cooperative_groups;

namespace kvq {
namespace {

constexpr int kLThreads = 512;
constexpr int kLWarps = kLThreads / 32;
constexpr int kMaxCluster = 16;
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

// Four logits from token v on.
template <typename T>
__device__ __forceinline__ void load_logits(const T* row, bool wide, int v, int v1, float (&x)[4]) {
  if (wide && v + 4 <= v1) {
    if constexpr (sizeof(T) == 4) {
      const float4 t = *reinterpret_cast<const float4*>(row + v);
      x[0] = t.x;
      x[1] = t.y;
      x[2] = t.z;
      x[3] = t.w;
    } else {
      const uint2 t = *reinterpret_cast<const uint2*>(row + v);
      const T* h = reinterpret_cast<const T*>(&t);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = to_float(h[k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = v + k < v1 ? to_float(row[v + k]) : -kInf;
  }
}
__device__ __forceinline__ void load_counts(const uint16_t* row, bool wide, int v, int v1, uint32_t (&n)[4]) {
  if (wide && v + 4 <= v1) {
    const uint2 t = __ldg(reinterpret_cast<const uint2*>(row + v));
    n[0] = t.x & 0xffffu;
    n[1] = t.x >> 16;
    n[2] = t.y & 0xffffu;
    n[3] = t.y >> 16;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) n[k] = v + k < v1 ? (uint32_t)__ldg(row + v + k) : 0u;
  }
}

struct Rules {
  float rep, freq, pres;
};
// n: the token's count as it is kept, times: how often it has been generated.
__device__ __forceinline__ float penalized(const Rules& R, float x, bool held, uint32_t times) {
  if (held) x = x > 0.f ? __fdiv_rn(x, R.rep) : __fmul_rn(x, R.rep);
  if (times) {
    x = __fsub_rn(x, __fmul_rn(R.freq, (float)times));
    x = __fsub_rn(x, R.pres);
  }
  return x;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
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

template <typename T>
__global__ void __launch_bounds__(kLThreads) logits_kernel(const __grid_constant__ LogitParams P) {
  extern __shared__ __align__(16) float xs[];          // the slice
  __shared__ float wred[kLWarps];
  __shared__ int wbest[kLWarps];
  __shared__ int par[kNodes], tok[kNodes], path[kNodes], n_path_sh;
  __shared__ Share mine;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = (int)(blockIdx.x / (unsigned)ranks);
  const bool lead = rank == 0 && tid == 0;
  pdl_trigger();
  pdl_wait();

  // ---- the row's sequence: how many of the sequences end at or before it ----
  int before = 0;
  for (int i0 = 0; i0 < P.batch; i0 += kLThreads) {
    const int i = i0 + tid;
    before += __syncthreads_count(i < P.batch && P.cu_rows[i + 1] <= row);
  }
  const int b = before;
  const bool covered = b < P.batch && P.cu_rows[b] >= 0 && P.cu_rows[b] <= row && P.cu_rows[b + 1] > row;
  if (!covered) {                                        // (the same in all CTAs of the cluster)
    if (lead) set_status(P.status, KVQ_ERR_BOUNDS);
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
  const float heat = U.temperature ? U.temperature[b] : 1.f;
  const bool sound = R.rep > 0.f && R.rep < kInf && fabsf(R.freq) < kInf && fabsf(R.pres) < kInf && heat >= 0.f && heat < kInf;
  const bool greedy = heat < 0x1p-120f;                  // (1 / T must be a float32)
  const float k2 = greedy ? 0.f : __fdiv_rn(1.4426950408889634f, heat);
  const uint16_t* counts = U.counts ? U.counts + (long long)b * U.count_stride : nullptr;
  const uint32_t* mask = nullptr;
  bool fault = false, skip = !sound;                     // skip: a row of zeros
  if (U.mask) {
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

  // ---- the node's path: tokens of the node and its ancestors, roots left out ----
  if (tid == 0) n_path_sh = 0;
  if (tree && !skip) {
    for (int i = tid; i <= node; i += kLThreads) {
      par[i] = P.parent[first + i];
      tok[i] = P.token[first + i];
    }
    __syncthreads();
    if (tid == 0) {
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
  __syncthreads();
  const int n_path = n_path_sh;
  const bool later = n_path > 0 || b1 > b0;              // some tokens are computed again
  if (fault && rank == 0) set_status(P.status, KVQ_ERR_BOUNDS);
  if (!sound && lead) set_status(P.status, KVQ_ERR_NONFINITE);

  const int v0 = min(P.vocab, rank * P.per), v1 = min(P.vocab, v0 + P.per);
  const T* l = static_cast<const T*>(P.logits) + (long long)row * P.l_stride;
  float* out = P.p + (long long)row * P.p_stride;
  const bool l_wide = (reinterpret_cast<uintptr_t>(l) & (4 * sizeof(T) - 1)) == 0;
  const bool c_wide = (reinterpret_cast<uintptr_t>(counts) & 7) == 0;
  const bool p_wide = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
  bool bad = false;
  float top = -kInf;

  // ---- pass 1: the slice's values, without biases and the path ----
  if (!skip) {
#pragma unroll 4
    for (int v = v0 + 4 * tid; v < v1; v += 4 * kLThreads) {
      const uint32_t allowed = mask ? mask[v >> 5] >> (v & 31) : 15u;
      float x[4] = {-kInf, -kInf, -kInf, -kInf};
      if (allowed & 15u) {
        load_logits(l, l_wide, v, v1, x);
        if (counts) {
          uint32_t c[4];
          load_counts(counts, c_wide, v, v1, c);
          if (c[0] | c[1] | c[2] | c[3])
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = penalized(R, x[k], c[k] != 0u, c[k] & KVQ_COUNT_MOST);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (!((allowed >> k) & 1u)) x[k] = -kInf;
          top = fmaxf(top, x[k]);
          if (!later) bad |= !(x[k] < kInf);
        }
      }
      *reinterpret_cast<float4*>(xs + (v - v0)) = make_float4(x[0], x[1], x[2], x[3]);
    }
    if (later) {
      __syncthreads();
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
          int lo = b0, hi = b1;                          // the first entry that is not below t
          while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (U.bias_token[mid] < t) lo = mid + 1;
            else hi = mid;
          }
          if (lo < b1 && U.bias_token[lo] == t) x = __fadd_rn(x, U.bias[lo]);
          const uint32_t c = counts ? (uint32_t)counts[t] : 0u;
          uint32_t times = c & KVQ_COUNT_MOST;
          for (int j = 0; j < n_path; ++j) times += path[j] == t;
          x = penalized(R, x, (c | times) != 0u, times);
        }
        xs[t - v0] = x;
      }
      __syncthreads();
      top = -kInf;
      for (int v = 4 * tid; v < v1 - v0; v += 4 * kLThreads) {
        const float4 x = *reinterpret_cast<const float4*>(xs + v);
        top = fmaxf(fmaxf(fmaxf(top, x.x), fmaxf(x.y, x.z)), x.w);
        bad |= !(x.x < kInf && x.y < kInf && x.z < kInf && x.w < kInf);
      }
    }
  }

  // ---- the slice's maximum ----
  top = warp_max(top);
  if (lane == 0) wred[warp] = top;
  bad = __syncthreads_or(bad);
  top = wred[0];
#pragma unroll
  for (int w = 1; w < kLWarps; ++w) top = fmaxf(top, wred[w]);
  __syncthreads();

  // ---- pass 2: exponentials and their sum, or the lowest token of the maximum ----
  if (!skip && !greedy) {
    const float ref = top == -kInf ? 0.f : top;
    float s = 0.f;
#pragma unroll 4
    for (int v = 4 * tid; v < v1 - v0; v += 4 * kLThreads) {
      float4 x = *reinterpret_cast<const float4*>(xs + v);
      x.x = ex2((x.x - ref) * k2);
      x.y = ex2((x.y - ref) * k2);
      x.z = ex2((x.z - ref) * k2);
      x.w = ex2((x.w - ref) * k2);
      *reinterpret_cast<float4*>(xs + v) = x;
      s += (x.x + x.y) + (x.z + x.w);
    }
    s = warp_add(s);
    if (lane == 0) wred[warp] = s;
  } else if (!skip) {
    int best = P.vocab;
    for (int v = tid; v < v1 - v0; v += kLThreads)
      if (xs[v] == top) best = min(best, v0 + v);
    best = __reduce_min_sync(0xffffffffu, best);
    if (lane == 0) wbest[warp] = best;
  }
  __syncthreads();
  if (tid == 0) {
    float s = 0.f;
    int best = P.vocab;
    if (!skip) {
      if (greedy)
        for (int w = 0; w < kLWarps; ++w) best = min(best, wbest[w]);
      else
        for (int w = 0; w < kLWarps; ++w) s += wred[w];
    }
    mine = Share{top, s, best, bad ? 1 : 0};
  }
  cluster.sync();
  Share other{-kInf, 0.f, P.vocab, 0};
  if (lane < ranks) other = *cluster.map_shared_rank(&mine, lane);
  const float whole = warp_max(other.top);
  const float share = other.top == -kInf ? 0.f : ex2((other.top - whole) * k2);
  const float sum = warp_add(other.sum * share);
  const int best = __reduce_min_sync(0xffffffffu, other.top == whole ? other.best : P.vocab);
  const bool none = __any_sync(0xffffffffu, other.bad != 0) || whole == -kInf;
  if (none && !skip && lead) set_status(P.status, KVQ_ERR_NONFINITE);
  const float factor = __fdiv_rn(__shfl_sync(0xffffffffu, share, rank), sum);

  // ---- pass 3: the slice's probabilities ----
  const bool zeros = skip || none;
#pragma unroll 4
  for (int v = v0 + 4 * tid; v < v1; v += 4 * kLThreads) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!zeros && !greedy) {
      x = *reinterpret_cast<const float4*>(xs + (v - v0));
      x.x *= factor;
      x.y *= factor;
      x.z *= factor;
      x.w *= factor;
    } else if (!zeros) {
      x.x = v == best ? 1.f : 0.f;
      x.y = v + 1 == best ? 1.f : 0.f;
      x.z = v + 2 == best ? 1.f : 0.f;
      x.w = v + 3 == best ? 1.f : 0.f;
    }
    if (p_wide && v + 4 <= v1) {
      *reinterpret_cast<float4*>(out + v) = x;
    } else {
      out[v] = x.x;
      if (v + 1 < v1) out[v + 1] = x.y;
      if (v + 2 < v1) out[v + 2] = x.z;
      if (v + 3 < v1) out[v + 3] = x.w;
    }
  }
  cluster.sync();                                        // (the others have read `mine`)
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

// The sequence of row r: the last one that begins at or before it (cu_rows must cover it).
__device__ __forceinline__ int row_seq(const int32_t* cu_rows, int batch, int r) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(cu_rows + mid) <= r) lo = mid;
    else hi = mid - 1;
  }
  return (__ldg(cu_rows + lo) <= r && r < __ldg(cu_rows + lo + 1)) ? lo : -1;
}

// One token more for a sequence.  16-bit halves of a 32-bit word: what the other half holds is left alone.
__device__ __forceinline__ void count_token(const CountParams& P, int b, int t) {
  const long long at = (long long)b * P.stride + t;
  uint32_t* word = reinterpret_cast<uint32_t*>(P.counts) + (at >> 1);
  const int shift = (int)(at & 1) * 16;
  if (P.kind == KVQ_COUNT_PROMPT) {
    const uint32_t bit = 0x8000u << shift;
    if (!(*reinterpret_cast<volatile uint32_t*>(word) & bit)) atomicOr(word, bit);
    return;
  }
  uint32_t old = *reinterpret_cast<volatile uint32_t*>(word);
  while (((old >> shift) & KVQ_COUNT_MOST) != KVQ_COUNT_MOST) {
    const uint32_t seen = atomicCAS(word, old, old + (1u << shift));   // (a count below its most does not carry)
    if (seen == old) break;
    old = seen;
  }
}

__global__ void __launch_bounds__(256) count_kernel(const __grid_constant__ CountParams P) {
  pdl_trigger();
  pdl_wait();
  const long long total = (long long)P.n_rows + (P.next_token ? P.batch : 0);
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    int b, t;
    if (i < P.n_rows) {
      const int r = (int)i;
      b = row_seq(P.cu_rows, P.batch, r);
      if (b < 0) {
        set_status(P.status, KVQ_ERR_BOUNDS);
        continue;
      }
      int from = r;
      if (P.path) {
        const int first = __ldg(P.cu_rows + b), n = __ldg(P.cu_rows + b + 1) - first, j = r - first;
        if (j == 0 || j >= __ldg(P.n_accept + b)) continue;
        const int node = __ldg(P.path + r);
        if (node < 0 || node >= n || first < 0 || first > P.n_rows - n) {
          set_status(P.status, KVQ_ERR_BOUNDS);
          continue;
        }
        from = first + node;
      }
      t = __ldg(P.token + from);
    } else {
      b = (int)(i - P.n_rows);
      t = __ldg(P.next_token + b);
      if (t == -1) continue;
    }
    if (t < 0 || t >= P.vocab) {
      set_status(P.status, KVQ_ERR_BOUNDS);
      continue;
    }
    count_token(P, b, t);
  }
}

template <typename T>
int launch_logits(LogitParams& P, cudaStream_t stream) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KVQ_ERR_CUDA;
  static std::mutex mu;
  static unsigned long long attr_done = 0;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!(attr_done & (1ull << dev))) {
      if (cudaFuncSetAttribute(logits_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, KVQ_LOGITS_MAX_VOCAB / kMaxCluster * 4) !=
              cudaSuccess ||
          cudaFuncSetAttribute(logits_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return KVQ_ERR_CUDA;
      attr_done |= 1ull << dev;
    }
  }
  // CTAs of a row: slices of at most 20,480 tokens (80 KB: two CTAs on an SM), and more of them while the rows do
  // not fill the SMs
  int c = 1;
  while (c < kMaxCluster && ((P.vocab + c - 1) / c > 20480 || (c * (long long)P.n_rows < kSms && P.vocab / c > 2048))) c *= 2;
  P.per = ((P.vocab + c - 1) / c + 31) / 32 * 32;
  if ((long long)P.n_rows * c > 0x7fffffffLL) return KVQ_ERR_UNSUPPORTED;
  return launch_pdl_cluster(logits_kernel<T>, c, dim3((unsigned)((long long)P.n_rows * c)), dim3(kLThreads),
                            (size_t)P.per * 4, stream, P) == cudaSuccess
             ? KVQ_OK
             : KVQ_ERR_CUDA;
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
  const long long total = (long long)n_rows + (next_token ? cfg->batch : 0);
  if (total == 0) return KVQ_OK;
  const int blocks = (int)std::min((total + 255) / 256, 8LL * kSms);
  return launch_pdl(count_kernel, dim3(blocks), dim3(256), 0, stream, P) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
