// Shared declarations of the kv_rope_qk kernels: the per-call parameters, phases and the rotation of a pair.
#pragma once
#include "rotate.cuh"

namespace kvq {

// r.t[]: queries, keys, values, with the destinations and modes of kv_rotate_qk (rotate.cuh); a row's source is
// t[i].src + row * stride[i] + head * d.
struct RopeParams {
  RotParams r;
  long long stride[3];
  const int32_t* rpos[3];    // position in the text of each row (nullptr: not rotated)
  const float* norm[3];      // RMS norm weights (nullptr: no norm)
  const uint64_t* freq;
  int half_rot;              // rotated pairs
  int interleaved;
  float scale, eps;
};

// Channels of pair i.
__device__ __forceinline__ void rope_pair(int interleaved, int half_rot, int i, int& a, int& b) {
  a = interleaved ? 2 * i : i;
  b = interleaved ? 2 * i + 1 : i + half_rot;
}

// Sine and cosine of a position's phase: the product mod 2^64 is the fraction of a turn, exact for any position;
// its upper 32 bits, taken as a signed number, are half turns in [-1, 1) in units of 2^-31.
__device__ __forceinline__ void rope_sincos(uint64_t freq, int pos, float& s, float& c) {
  const uint64_t phase = freq * (uint64_t)(int64_t)pos;
  sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
}

__device__ __forceinline__ const uint16_t* rope_src(const RopeParams& P, int tt, int row, int head) {
  return P.r.t[tt].src + (long long)row * P.stride[tt] + (long long)head * kHeadDim;
}

// The sign of entry (i, j) of the Walsh-Hadamard matrix (Sylvester's order).
__device__ __forceinline__ float hadamard_sign(int i, int j) {
  return __uint_as_float(0x3f800000u | ((uint32_t)(__popc(i & j) & 1) << 31));
}
// (row, head) pairs from which a call's products run on the tensor cores, where anything of up to a chunk an SM takes
// 7 us (with the launch of copies 7.4).  The CUDA cores take 5.1 us for 18 rows of 32 + 8 + 8 heads (864 pairs), 7.6 for 20,
// 10.1 for 32; 5.2 for 16 rows of 64 + 8 Hadamard heads (1,152), 7.2 for 20, 9.1 for 24.
constexpr long long kRopeTcPairs = 896, kRopeTcPairsHad = 1280;
// ... which this launches (P.r.n_dense is set there; copies are the caller's).
int launch_rope_tc(RopeParams P, cudaStream_t stream);

constexpr float kInvSqrtDim = 0.08838834764831845f;

}  // namespace kvq
