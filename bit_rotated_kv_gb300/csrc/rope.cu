// kv_rope_qk: norm of the heads, rotary positions, per-head transform and append of a step's rows.
//
// Source: [WUSH] inference algorithm and [OScaR] algorithm, key and query processing (the transform follows
// the rotation); the norm and the rotation are the models' own.
//   y = w x / sqrt(mean x^2 + eps);  (y_a, y_b) <- s (y_a cos f - y_b sin f, y_b cos f + y_a sin f);  out = T y
// in float32 with one rounding to bf16 at the end.  A phase f is position * freq mod 2^64 (units of 2^-64 turns):
// whole numbers lose nothing at far positions, where a float32 angle of 10^5 radians is off by 2^-8.
//
// This file: the kernel for few rows, on the CUDA cores (rope_tc.cu: the others).  A CTA takes a slice of 32 outputs of one
// matrix and a chunk of the (row, head) pairs that share it: a whole matrix to a CTA would leave most SMs without
// one at a single token (8 kv heads, 3 matrices each), and its 64 KB would be the longest wait of the call.  The
// four slices of a pair each place its row (norm and rotation), which costs less than passing it on would.  Latency
// bounds it (launch, matrix slice, row, destination, one after another): one token of 32 + 8 + 8 heads 2.5 us, sixteen 5.1.
#include "rope.cuh"

#include <algorithm>

namespace kvq {
namespace {

constexpr int kSlice = 32;                        // outputs of a CTA
constexpr int kSlices = kHeadDim / kSlice;
constexpr int kRopeThreads = 4 * kSlice;          // four threads to an output, 32 inputs each
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kMaxRows = 8;                       // pairs of a chunk: more than calls of this kernel come to (5)
constexpr int kRopeSlots = 8 * kSms;              // CTAs that the chunks are made for
static_assert(kRopeTcPairs <= kRopeTcPairsHad && kRopeTcPairsHad * kSlices <= (long long)kRopeSlots * kMaxRows, "pairs of a chunk");
constexpr int kMaxCopies = 8;                     // rows a warp copies

// One warp places a row: norm and rotation, float32, into shared memory.  False when the row or a weight is not finite.
__device__ __forceinline__ bool place_row(const RopeParams& P, const float* w, bool turned, uint2 raw, int pos, float* y, int lane) {
  float x[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xffff0000u), __uint_as_float(raw.y << 16),
                __uint_as_float(raw.y & 0xffff0000u)};
  bool fine = !bf16_pair_odd(raw.x) && !bf16_pair_odd(raw.y);
  if (w) {
    float ss = fmaf(x[3], x[3], fmaf(x[2], x[2], fmaf(x[1], x[1], x[0] * x[0])));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    fine &= ss <= 3.4e38f;
    const float r = fine ? rsqrtf(fmaf(ss, 1.0f / kHeadDim, P.eps)) : __int_as_float(0x7fffffff);
    const float4 w4 = __ldg(reinterpret_cast<const float4*>(w) + lane);
    fine &= max(max(__float_as_uint(fabsf(w4.x)), __float_as_uint(fabsf(w4.y))), max(__float_as_uint(fabsf(w4.z)), __float_as_uint(fabsf(w4.w)))) < 0x7f800000u;
    x[0] *= r * w4.x;
    x[1] *= r * w4.y;
    x[2] *= r * w4.z;
    x[3] *= r * w4.w;
  }
  *reinterpret_cast<float4*>(y + 4 * lane) = make_float4(x[0], x[1], x[2], x[3]);
  fine = __all_sync(0xffffffffu, fine);
  if (turned) {
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = lane + 32 * h;
      if (i < P.half_rot) {
        int a, b;
        rope_pair(P.interleaved, P.half_rot, i, a, b);
        float s, c;
        rope_sincos(__ldg(P.freq + i), pos, s, c);
        s *= P.scale;
        c *= P.scale;
        const float ya = y[a], yb = y[b];
        y[a] = fmaf(ya, c, -(yb * s));
        y[b] = fmaf(yb, c, ya * s);
      }
    }
  }
  return fine;
}

// Rows of values that are copied: a warp takes up to kMaxCopies of them, 16 lanes of 16 bytes each.  Everything that is loaded
// for them is asked for before the first is placed.
__device__ __forceinline__ void copy_rows(const RopeParams& P, int item, int lane) {
  const RotTensor& T = P.r.t[2];
  const int total = T.rows * T.heads;
  constexpr int kEach = kMaxCopies / 2;
  const int p0 = item * P.r.rpw + (lane >> 4), p1 = min(total, (item + 1) * P.r.rpw);
  uint4 x[kEach];
  int row[kEach], head[kEach], b[kEach], at[kEach], sq[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int p = min(p0 + 2 * k, total - 1);
    row[k] = p / T.heads;
    head[k] = p - row[k] * T.heads;
    if (p0 + 2 * k < p1) {
      x[k] = __ldg(reinterpret_cast<const uint4*>(rope_src(P, 2, row[k], head[k])) + (lane & 15));
      b[k] = __ldg(P.r.seq_idx + row[k]);
      at[k] = __ldg(P.r.pos + row[k]);
    } else {
      b[k] = -1;
    }
  }
#pragma unroll
  for (int k = 0; k < kEach; ++k) sq[k] = b[k] >= 0 && b[k] < P.r.batch ? __ldg(P.r.s_quant + b[k]) : -1;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    if (p0 + 2 * k >= p1) continue;
    uint16_t* dst = rot_dst(P.r, T, row[k], head[k], b[k], at[k], (lane & 15) == 0, sq[k]);
    if (dst) __stcg(reinterpret_cast<uint4*>(dst) + (lane & 15), x[k]);
  }
}

__global__ void __launch_bounds__(kRopeThreads) rope_rows_kernel(const __grid_constant__ RopeParams P) {
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if ((int)blockIdx.x >= P.r.dense_total) {
    pdl_wait();
    const int item = ((int)blockIdx.x - P.r.dense_total) * kRopeWarps + warp;
    if (item < P.r.warp_total) copy_rows(P, item, lane);
    return;
  }
  __shared__ __align__(16) float ys[kMaxRows][kHeadDim];
  __shared__ uint16_t* dst_sh[kMaxRows];
  int tt, tile;
  find_item(P.r.n_dense, blockIdx.x, tt, tile);
  const RotTensor& T = P.r.t[tt];
  const int slice = tile % kSlices;
  tile /= kSlices;
  const int pairs = T.rows * T.head_div;
  const int chunks = (pairs + P.r.rt - 1) / P.r.rt;
  const int mh = tile / chunks, p0 = (tile % chunks) * P.r.rt, np = min(P.r.rt, pairs - p0);
  // this thread's part of output o's matrix row: four threads share it, 16-byte pieces in turn (shared memory
  // then serves the four from different banks)
  const int o = kSlice * slice + (tid >> 2), part = tid & 3;
  float t[32];
  if (T.mode == ROT_WHT) {
#pragma unroll
    for (int j = 0; j < 32; ++j) t[j] = hadamard_sign(o, 16 * (j >> 2) + 4 * part + (j & 3)) * kInvSqrtDim;
  } else {
    const float4* m = reinterpret_cast<const float4*>(T.mat + ((size_t)mh * kHeadDim + o) * kHeadDim);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float4 v = __ldg(m + 4 * j + part);
      t[4 * j] = v.x;
      t[4 * j + 1] = v.y;
      t[4 * j + 2] = v.z;
      t[4 * j + 3] = v.w;
    }
  }
  pdl_wait();
  // a warp's rows (warp, warp + 4) are both asked for before the first is placed, and lane k finds out where the
  // k-th goes: one after another, each row's four dependent loads would be waited for in turn
  constexpr int kMine = kMaxRows / kRopeWarps;
  const int32_t* rpos = P.rpos[tt];
  uint2 raw[kMine];
  int pos[kMine];
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const int j = warp + kRopeWarps * k;
    int row, head;
    tile_row(T, mh, p0 + min(j, np - 1), row, head);
    raw[k] = __ldg(reinterpret_cast<const uint2*>(rope_src(P, tt, row, head)) + lane);
    pos[k] = rpos ? __ldg(rpos + row) : 0;
  }
  bool fine = true;                                      // of the lane's own row
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const int j = warp + kRopeWarps * k;
    if (j < np) {
      const bool f = place_row(P, P.norm[tt], rpos != nullptr, raw[k], pos[k], ys[j], lane);
      if (lane == k) fine = f;
    }
  }
  const int own = warp + kRopeWarps * lane;
  if (lane < kMine && own < np) {
    int row, head;
    tile_row(T, mh, p0 + own, row, head);
    const int b = T.is_query ? 0 : __ldg(P.r.seq_idx + row), p = T.is_query ? 0 : __ldg(P.r.pos + row);
    dst_sh[own] = rot_dst(P.r, T, row, head, b, p, slice == 0);
    if (!fine && slice == 0 && dst_sh[own]) set_status(P.r.status, KVQ_ERR_NONFINITE);
  }
  __syncthreads();
  for (int j0 = 0; j0 < np; j0 += 4) {
    float acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      acc[j] = 0.f;
      if (j0 + j < np) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 y = *reinterpret_cast<const float4*>(&ys[j0 + j][16 * i + 4 * part]);
          acc[j] = fmaf(t[4 * i], y.x, acc[j]);
          acc[j] = fmaf(t[4 * i + 1], y.y, acc[j]);
          acc[j] = fmaf(t[4 * i + 2], y.z, acc[j]);
          acc[j] = fmaf(t[4 * i + 3], y.w, acc[j]);
        }
      }
    }
    // sums over the four parts; thread `part` ends with row j0 + part
    const bool up = part & 2, odd = part & 1;
    float u0 = up ? acc[2] : acc[0], u1 = up ? acc[3] : acc[1];
    u0 += __shfl_xor_sync(0xffffffffu, up ? acc[0] : acc[2], 2);
    u1 += __shfl_xor_sync(0xffffffffu, up ? acc[1] : acc[3], 2);
    const float s = (odd ? u1 : u0) + __shfl_xor_sync(0xffffffffu, odd ? u0 : u1, 1);
    uint16_t* dst = j0 + part < np ? dst_sh[j0 + part] : nullptr;
    if (dst) dst[o] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
  }
}

// The copies beside products on the tensor cores, before them (behind them took as long).  16 x 2048 tokens of 8 heads, 67 MB
// read and as many written: 25 us (5.4 TB/s).
__global__ void __launch_bounds__(kRopeThreads, 10) rope_copy_kernel(const __grid_constant__ RopeParams P) {
  pdl_trigger();
  pdl_wait();
  const int item = (int)blockIdx.x * kRopeWarps + (int)(threadIdx.x >> 5);
  if (item < P.r.warp_total) copy_rows(P, item, threadIdx.x & 31);
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" int kvq_launch_rope(const kvq_config* cfg, const kvq_transform* tr, const kvq_rope* rope, const uint16_t* q,
                               int64_t q_stride, uint16_t* q_out, const int32_t* q_pos, int32_t n_q_rows,
                               const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride,
                               const int32_t* seq_idx, const int32_t* pos, const int32_t* rope_pos, int32_t n_kv_rows,
                               const kvq_cache* cache, int32_t* d_status, cudaStream_t stream) {
  RopeParams P{};
  RotParams& R = P.r;
  const int gqa = cfg->n_q_heads / cfg->n_kv_heads;
  const bool had = tr->kind == KVQ_TRANSFORM_HADAMARD;
  R.t[0] = RotTensor{q, n_q_rows, cfg->n_q_heads, had ? ROT_WHT : ROT_DENSE, tr->t_k_inv_t, gqa, 1,
                     q_out, nullptr, nullptr, 0, 0};
  R.t[1] = RotTensor{k, n_kv_rows, cfg->n_kv_heads, had ? ROT_WHT : ROT_DENSE, tr->t_k, 1, 0,
                     nullptr, cache->sink_k, cache->ring_k, 1, 0};
  R.t[2] = RotTensor{v, n_kv_rows, cfg->n_kv_heads, tr->t_v ? ROT_DENSE : ROT_COPY, tr->t_v, 1, 0,
                     nullptr, cache->sink_v, cache->ring_v, 0, 1};
  R.seq_idx = seq_idx;
  R.pos = pos;
  R.seq_len = cache->seq_len;
  R.s_quant = cache->s_quant;
  R.s_sink = cfg->s_sink;
  R.ring_cap = cfg->ring_cap;
  R.batch = cfg->batch;
  R.hkv = cfg->n_kv_heads;
  R.status = d_status;
  P.stride[0] = q_stride;
  P.stride[1] = k_stride;
  P.stride[2] = v_stride;
  if (rope) {
    if (rope->rot_dim > 0) {
      P.rpos[0] = q_pos;
      P.rpos[1] = rope_pos ? rope_pos : pos;
    }
    P.norm[0] = rope->q_norm;
    P.norm[1] = rope->k_norm;
    P.freq = rope->freq;
    P.half_rot = rope->rot_dim / 2;
    P.interleaved = rope->layout == KVQ_ROPE_INTERLEAVED;
    P.scale = rope->scale;
    P.eps = rope->norm_eps;
  }
  long long pairs = 0;
  for (int i = 0; i < 3; ++i) {
    if ((long long)R.t[i].rows * R.t[i].heads > 0x3fffffffLL) return KVQ_ERR_UNSUPPORTED;
    if (R.t[i].mode != ROT_COPY) pairs += (long long)R.t[i].rows * R.t[i].heads;
  }
  const long long copies = R.t[2].mode == ROT_COPY ? (long long)n_kv_rows * cfg->n_kv_heads : 0;
  const long long cslots = 2LL * kSms * 16;
  R.rpw = (int)(copies > cslots ? std::min((copies + cslots - 1) / cslots, (long long)kMaxCopies) : 1);
  R.warp_total = (int)((copies + R.rpw - 1) / R.rpw);
  if (pairs >= (had ? kRopeTcPairsHad : kRopeTcPairs)) {
    // the copies on their own, then the products on the tensor cores
    if (R.warp_total > 0 &&
        launch_pdl(rope_copy_kernel, dim3((unsigned)((R.warp_total + kRopeWarps - 1) / kRopeWarps)), dim3(kRopeThreads), 0, stream, P) !=
            cudaSuccess)
      return KVQ_ERR_CUDA;
    return launch_rope_tc(P, stream);
  }
  // pairs of a chunk: as many as make about eight CTAs an SM of all the slices (128 threads and 4 KB each)
  R.rt = (int)std::max(4LL, (pairs * kSlices + kRopeSlots - 1) / kRopeSlots);
  for (int i = 0; i < 3; ++i) {
    if (R.t[i].mode == ROT_COPY) continue;
    const int chunks = (R.t[i].rows * R.t[i].head_div + R.rt - 1) / R.rt;
    R.n_dense[i] = R.t[i].heads / R.t[i].head_div * chunks * kSlices;
    R.dense_total += R.n_dense[i];
  }
  const unsigned blocks = (unsigned)(R.dense_total + (R.warp_total + kRopeWarps - 1) / kRopeWarps);
  return launch_pdl(rope_rows_kernel, dim3(blocks), dim3(kRopeThreads), 0, stream, P) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}
