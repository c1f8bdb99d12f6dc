// kv_rope_qk for prefill-sized calls: norm and rotation on the CUDA cores, the per-head products on the tensor
// cores (tcgen05).
//
// A row is read once and written once, 512 bytes a row and head: the 2048-token chunk of 16 sequences with 32 + 8 heads
// moves 671 MB, 99 us at the measured copy rate, which leaves the CUDA cores about 1.6 K clocks and the tensor cores as
// many for 64 rows of an SM.  Both products therefore take two fp16 parts of each operand rather than the integer digits
// of rotate_tc.cu: T row i and x row r are brought under powers of two so that their largest entry lies below 2^15,
// and split as hi + lo, 11 bits each.  hi hi + lo hi + hi lo, summed in float32 by the tensor cores, leaves out 2^-20
// of sum |T_ij x_j| at most (bf16's half step is 2^-8 of the result); three MMAs of 16 inputs instead of nine.  fp16 steps by 2^-24
// at the finest, so an entry is also off by 2^-24 of a row's unit: 2^-37 of its largest entry where the power of two goes by
// that, 2^-22 at worst where a norm's rows share one.  A Walsh-Hadamard matrix is +-1, its 1/sqrt(128) left to the end: two MMAs.
//
// The norm's factor belongs to a row, so the weights take the power of two with it: norm and scaling cost one product a channel.
// Rows far below the norm's epsilon and weights far apart take another way (size_rows).  Sine and cosine are the SFU's (2^-20.9 of
// the pair's length), from phases in whole numbers.  Lanes hold both channels of a pair: eight lanes to a row, two vectors of eight channels each.
//
// Layout: two CTAs on an SM.  A CTA takes a run of chunks of 64 (row, head) pairs.  T hi and lo of its matrix stay in
// TMEM (the A operand, lane = output, 64 columns each); rows come by asynchronous copies two chunks ahead and go through
// swizzled shared memory (B, two buffers of hi and lo); accumulators take two sets of 64 TMEM columns.  Eight warps
// place rows, one issues the MMAs, four write results out through the shared memory that the rows came from, a row's 256
// bytes at a time, two ask for rows, one finds out where they go.
//
// A call of a chunk or less for each SM takes 7 us, half of it the matrix's way into TMEM (through shared memory, asked for before
// the grid ahead has ended).
//
// That chunk of 16 x 2048 tokens takes 211 us with its values' copies, 186 without (3.6 TB/s).  What bounds it are the two
// buffers: a chunk of 64 rows is placed in 3.4 to 3.9 K clocks, its MMAs end 2.3 K later and its results are out of the same buffer 2.4 K
// after that, so that two buffers give a chunk every 4.15 K at best; it is 4.6 K, and those who place wait a quarter of it.  The
// schedulers issue in 63% of the clocks, the shared-memory pipe is busy 65%, DRAM 42%, the tensor cores 30%.  What was tried:
// rows kept in registers a chunk ahead with three buffers 267 us against 217; bulk copies of rows by one warp 289,
// and 96 registers for those who place and 40, 24 for the others 276, against 248.
#include "rope.cuh"
#include "tc.cuh"

#include <algorithm>
#include <mutex>

namespace kvq {
namespace {

// Warps 0-7 place rows, 8-11 write results out, 12 issues the MMAs, 13 and 15 ask for rows, 14 finds out where they
// go.  Registers a thread: 64 at launch (32 warps an SM), shared out again 8 x 88 + 4 x 48 + 4 x 32 = 16 x 64.
constexpr int kRtWarps = 8, kRtOut = 4, kRtMma = 12, kRtLoad = 13, kRtDst = 14;
constexpr int kRtThreads = 512;
constexpr int kPlaceRegs = 88, kOutRegs = 48, kLastRegs = 32;
constexpr int kRtRows = kUmRows;                         // pairs of a chunk (N of every MMA): 64
constexpr int kHalfBuf = kRtRows * kHeadDim * 2;         // hi or lo of a chunk: 16 KB
constexpr int kRtXBuf = 2 * kHalfBuf;
constexpr int kRtRaw = 2 * kRtXBuf;                      // two chunks of rows as they come, 256 bytes each
constexpr int kRtRawBuf = kRtRows * kHeadDim * 2;
constexpr int kRtMeta = kRtRaw + 2 * kRtRawBuf;
constexpr int kMetaSets = 4;
constexpr int kRtFac = kRtMeta + kMetaSets * kRtRows * 8;
constexpr int kRtPos = kRtFac + 2 * kRtRows * 4;
constexpr int kRtNorm = kRtPos + 2 * kRtRows * 4;
constexpr int kRtFreq = kRtNorm + kHeadDim * 4;
// (behind the pairs' frequencies: a frequency of 0)
constexpr int kRtExch = kRtFreq + 66 * 8;                // a T row's largest exponent, by halves
constexpr int kRtRowFac = kRtExch + 2 * kHeadDim * 4;    // what takes an output's power of two back, where they differ
constexpr int kRtUsed = kRtRowFac + kHeadDim * 4;
constexpr int kRtSmem = kRtUsed + 1024;
static_assert(2 * (kRtSmem + 1024) <= 227 * 1024, "two CTAs on an SM");
constexpr uint32_t kRtCols = 256;                        // TMEM: T hi, T lo, two accumulators
constexpr uint32_t kRtLo = 64, kRtAcc = 128;
// kind::f16: D f32, A and B fp16, both K-major, N = 64, M = 128
constexpr uint32_t kRtIdesc = (1u << 4) | ((uint32_t)(kRtRows >> 3) << 17) | ((128u >> 4) << 24);

__device__ __forceinline__ bool rt_elect() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void rt_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(kRtIdesc), "r"(acc)
      : "memory");
}
// Warps of one kind meet at named barriers; one kind waits for another at mbarriers, every wait bounded.
constexpr int kBarPlace = 1, kBarOut = 2, kBarMma = 3;
__device__ __forceinline__ void rt_sync(int id, int warps) { asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(32 * warps) : "memory"); }
__device__ __forceinline__ void rt_init(uint64_t* bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(um_saddr(bar)), "r"(count) : "memory");
}
// What a warp has done, for those who wait for it.
__device__ __forceinline__ void rt_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) um_arrive(bar);
}
__device__ __forceinline__ bool rt_wait(uint64_t* bar, uint32_t parity) {
  if (um_mbar_try(bar, parity)) return true;
  unsigned long long began, now;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(began));
  do {
    if (um_mbar_try(bar, parity)) return true;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(now));
  } while (now - began < 1000000000ull);                 // a second
  return false;
}
// Use n of a pair of barriers (a whole warp waits; after a time-out nobody waits any more: every role runs to its end).
__device__ __forceinline__ bool rt_wait_use(uint64_t* bars, int n, volatile int* abort_sh) {
  if (*abort_sh) return false;
  if (__all_sync(0xffffffffu, rt_wait(bars + (n & 1), (uint32_t)((n >> 1) & 1)))) return true;
  *abort_sh = 1;
  return false;
}
template <int R>
__device__ __forceinline__ void rt_regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void rt_regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float lo16(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi16(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// The leading 11 bits of a float (towards zero): an exact fp16 where it is in fp16's normal range.
__device__ __forceinline__ float lead11(float v) { return __uint_as_float(__float_as_uint(v) & 0xffffe000u); }

// The power of two that brings numbers below 2^(e - 126) below 2^15 (e: an exponent field).
__device__ __forceinline__ int fit_pow2(int e) { return min(max(141 - e, -126), 126); }
__device__ __forceinline__ float pow2(int k) { return __int_as_float((k + 127) << 23); }

// How a lane's two vectors of eight channels form pairs.
enum { kNone, kHalf, kInter, kAny };

// The chunk's place: tensor, matrix, chunk of the matrix.
struct Place {
  int tt, mh, c, cpm;
};
__device__ __forceinline__ Place place_of(const RopeParams& P, int chunk) {
  Place w;
  int item;
  find_item(P.r.n_dense, chunk, w.tt, item);
  const RotTensor& T = P.r.t[w.tt];
  w.cpm = (T.rows * T.head_div + kRtRows - 1) / kRtRows;
  w.mh = item / w.cpm;
  w.c = item % w.cpm;
  return w;
}

// The first chunk of a CTA.  Where CTAs have many chunks (sixteen on average), those whose rows share a token count
// kCostSame, others, which come in shorter pieces and with a sine and cosine each, kCostOwn, and the grid's first half gets
// kShare / 32: of the two CTAs on an SM the first comes to issue more often.  (16 x 2048 tokens, 40 heads: 239 us by chunks
// alone, 230 by 7 : 8 in halves, 215 so.  Where they have few, a chunk more is what counts (3 x 777 tokens: 25.5 us by
// chunks, 28.4 so.)  Both numbers are that shape's: chunks without a norm or a rotation, interleaved or odd layouts, and values under
// T_V cost other than these, and are divided by them all the same.
constexpr int kCostSame = 7, kCostOwn = 8, kShare = 17;
__device__ __forceinline__ int first_chunk(const RopeParams& P, int cta) {
  if (P.r.dense_total < 16 * 2 * kSms) return (int)((long long)P.r.dense_total * cta / gridDim.x);
  long long sum = 0;
  int cost[3];
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    cost[t] = P.r.t[t].head_div > 1 ? kCostSame : kCostOwn;
    sum += (long long)P.r.n_dense[t] * cost[t];
  }
  // (the grid is 2 kSms)
  long long at = sum * (cta <= kSms ? kShare * cta : (32 - kShare) * cta + (2 * kShare - 32) * kSms) / (32 * kSms);
  int c = 0;
#pragma unroll
  for (int t = 0; t < 3; ++t) {
    const long long here = (long long)P.r.n_dense[t] * cost[t], x = min(at, here);
    c += (int)(x / cost[t]);
    at -= x;
  }
  return c;
}

// What a run of chunks of one matrix has in common (in shared memory: read once a chunk, it would cost the loops their
// registers).
struct Seg {
  bool same;                 // a slot's rows are heads of one token
  bool norm;
  bool weighted;             // channels have weights: the norm's, the rotation's factor
  int grow;                  // what weights and rotation may add to a channel's exponent
  bool turned;
  bool wide;                 // weights so far apart, or so far from 1, that every row takes a power of two of its own
  float up, back;            // with a norm: the power of two that rows take
  float least;               // with a norm: rows whose squares sum to less take a power of two of their own (size_rows)
  int most;                  // what a row's power of two may be (with the matrix's it is taken back by 2^-149 or more)
  float t_back;              // takes the matrix's power of two back (and a Hadamard matrix's 1/sqrt(128) in)
};

// Asks for half of a chunk's rows and for their positions, two rows at a time (one warp).  Behind the last row: that row
// again.  (Bulk copies of a token's heads, 1 KB, took one warp 200 clocks each.)
__device__ __forceinline__ void ask_rows(const RopeParams& P, const Place& w, int half, uint32_t raw, uint32_t pos, uint64_t* bar, int lane) {
  const RotTensor& T = P.r.t[w.tt];
  const int lg = __ffs(T.head_div) - 1, last = (T.rows << lg) - 1, mask = T.head_div - 1;
  const uint16_t* src = T.src + (long long)(w.mh << lg) * kHeadDim + 8 * (lane & 15);
  const long long stride = P.stride[w.tt];
  const int r0 = 32 * half + (lane >> 4), p0 = w.c * kRtRows + r0;
  raw += 256u * (uint32_t)r0 + 16u * (uint32_t)(lane & 15);
#pragma unroll 4
  for (int k = 0; k < 16; ++k) {
    const int p = min(p0 + 2 * k, last);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(raw + 512u * k), "l"(src + (p >> lg) * stride + (p & mask) * kHeadDim)
                 : "memory");
  }
  const int32_t* rpos = P.rpos[w.tt];
  if (rpos) {
    const int p = min(w.c * kRtRows + 32 * half + lane, last);
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(pos + 4u * (uint32_t)(32 * half + lane)), "l"(rpos + (p >> lg)) : "memory");
  }
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(um_saddr(bar)) : "memory");
}

// Where pair i stands in the table: the eight lanes of a row, which ask for pairs eight (kInter: four) apart, find theirs
// side by side.
__device__ __forceinline__ int freq_slot(bool inter, int i) { return inter ? (i & 3) * 16 + (i >> 2) : (i & 7) * 8 + (i >> 3); }
// Cosine and sine of a pair's phase.  (Pairs that are not rotated stand in the table with frequency 0.)
__device__ __forceinline__ void phase_sincos(uint32_t freq_at, int pos, float& c, float& s) {
  const uint2 f = lds_v2(freq_at);
  // the upper 32 bits of freq * pos mod 2^64, pos signed
  const uint32_t up = f.y * (uint32_t)pos + __umulhi(f.x, (uint32_t)pos) - (pos < 0 ? f.x : 0u);
  const float x = (float)(int32_t)up * (0x1p-31f * 3.14159265358979f);
  s = __sinf(x);
  c = __cosf(x);
}

// Results of a chunk stand where its rows were (its MMAs are done with them): 16-byte piece c of row r, in what the
// warp that placed the row owns, so that only that warp, which writes the row out, overwrites it with the next.
__device__ __forceinline__ uint32_t out_at(int r, int c) {
  return (uint32_t)((c >> 3) * 8192 + (r >> 3) * 1024 + (r & 7) * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// 16 TMEM lanes x 32 columns: registers 4 k + 2 h + e hold lane (lane >> 2) + 8 h, column 8 k + 2 (lane & 3) + e.
__device__ __forceinline__ void tmem_ld_tiles(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
        "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}

// Two numbers as hi and lo.
__device__ __forceinline__ void split(float x, float y, uint32_t& hi, uint32_t& lo) {
  const float2 v = make_float2(x, y), h = make_float2(lead11(x), lead11(y));
  const float2 l = fma2(h, make_float2(-1.f, -1.f), v);
  hi = half2_bits(h.x, h.y);
  lo = half2_bits(l.x, l.y);
}
__device__ __forceinline__ void sts_v4(uint32_t a, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

// What a lane needs to place its two rows.
struct Lane {
  int r0, sub;               // the slot's first row; the lane of the slot
  int va, vb;                // its vectors of eight channels
  uint32_t at_a, at_b;       // where those of row r0 go in a buffer (row r0 + 1: 128 bytes on, pieces exchanged in twos)
  uint32_t freq_at, freq_step;   // the first of its pairs in the table of frequencies, bytes to the next
};

// The largest of eight lanes' numbers, which share a row.
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// The powers of two of a slot's two rows from their channels as they are after norm and weights.  The one that all rows of a
// normed head share (Seg) is that of the largest numbers such a row can hold: it suits rows whose mean square is not far below
// the norm's epsilon under weights that are not far apart, and costs one product a channel.  Elsewhere hi and lo would lose digits under it:
// a row far below epsilon stays as small as it came, and one may have nothing where the large weights are.  Here the row's digits
// (bfloat16: exactly) are brought to 1 .. 2 first, so that neither they nor their products with the weights vanish on the way, whatever their size.
__device__ __forceinline__ void size_rows(const Seg& g, const Lane& L, uint32_t norm_s, const float (&r)[2], uint32_t (&wa)[2][4], uint32_t (&wb)[2][4],
                                          float2 (&up)[2], float (&back)[2], bool (&fine)[2]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t t = 0u;
#pragma unroll
    for (int m = 0; m < 4; ++m) t = __vmaxu2(t, __vmaxu2(wa[j][m] & 0x7fff7fffu, wb[j][m] & 0x7fff7fffu));
    t = row_max(max(t & 0xffffu, t >> 16));
    if (!g.norm) fine[j] = t < 0x7f80u;
    const int p = min(max(127 - (int)(t >> 7), -126), 126);
    const uint32_t by = (uint32_t)(p + 127) << 7 | (uint32_t)(p + 127) << 23;
    float top = 0.f;
#pragma unroll
    for (int h = 0; h < 4; ++h) {                        // (halves of va, then of vb)
      const uint4 w = lds_v4(norm_s + 256u * (uint32_t)(h & 1) + 16u * (uint32_t)(h < 2 ? L.va : L.vb));
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t& x = h < 2 ? wa[j][2 * (h & 1) + e] : wb[j][2 * (h & 1) + e];
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(x), "r"(by));
        top = fmaxf(top, fmaxf(fabsf(lo16(x) * __uint_as_float(e ? w.z : w.x)), fabsf(hi16(x) * __uint_as_float(e ? w.w : w.y))));
      }
    }
    top = __uint_as_float(row_max(__float_as_uint(top)));
    // y = x 2^-p r w, r = u 2^e with u in 1 .. 2: rows take u 2^k and are taken back by 2^(e - p - k).  No weight overflows under it
    // (grow: the largest weight's exponent), nor does what takes the row back vanish
    const int e = (int)(__float_as_uint(r[j]) >> 23) - 127;
    int k = fit_pow2((int)(__float_as_uint(top) >> 23) + 1 + (g.turned ? 1 : 0));
    k = max(min(k, min(125 - g.grow, g.most + e - p)), -126);
    const float u = __uint_as_float((__float_as_uint(r[j]) & 0x007fffffu) | 0x3f800000u) * pow2(k);
    if (r[j] > 0.f) {                                    // (a row that is not finite: no number comes back)
      up[j] = make_float2(u, u);
      back[j] = pow2(min(max(e - p - k, -126), 127)) * g.t_back;
    }
  }
}

// A slot's two rows: hi and lo into the chunk's buffer, the factor that goes with a row beside its destination.
// kW: 0: as they are, 1: norm and weights, 2: weights without a norm, 3: weights, with or without a norm, every row under a power of two
// of its own.
// kSame: the two rows are heads of one token.  Nothing branches, and pairs are the outer loop: the two rows' chains of operations run
// side by side.  True where a row is too small for the power that it took (kW = 1).
template <int kMode, int kW, bool kSame>
__device__ __forceinline__ bool place_words(const RopeParams& P, const Seg& g, const Lane& L, int left, const int (&pos)[2], uint32_t (&wa)[2][4],
                                            uint32_t (&wb)[2][4], uint32_t xb, uint32_t norm_s, uint32_t freq_s, uint32_t fac_s) {
  // the number that brings a row's channels below 2^15, the one that takes it back at the end
  float2 up[2];
  float back[2];
  bool fine[2], small = false;
  if (kW == 1 || kW == 3) {
    // |x| / rms(x) <= sqrt(128): the norm's own factor, and the weights' power of two
    float ss[2], r[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float2 acc[2];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float2 x = make_float2(lo16(wa[j][m]), hi16(wa[j][m])), y = make_float2(lo16(wb[j][m]), hi16(wb[j][m]));
        acc[0] = m ? fma2(x, x, acc[0]) : mul2(x, x);
        acc[1] = m ? fma2(y, y, acc[1]) : mul2(y, y);
      }
      ss[j] = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1)
#pragma unroll
      for (int j = 0; j < 2; ++j) ss[j] += __shfl_xor_sync(0xffffffffu, ss[j], o);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      fine[j] = ss[j] <= 3.4e38f;
      r[j] = kW == 3 && !g.norm ? 1.f : fine[j] ? rsqrtf(fmaf(ss[j], 1.0f / kHeadDim, P.eps)) : __int_as_float(0x7fffffff);
      up[j] = make_float2(r[j] * g.up, r[j] * g.up);
      back[j] = g.back;
    }
    if (kW == 3) size_rows(g, L, norm_s, r, wa, wb, up, back, fine);
    small = ss[0] < g.least || ss[1] < g.least;
  } else {
    uint32_t top[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {                        // (bf16 bits order as integers)
      uint32_t t = 0u;
#pragma unroll
      for (int m = 0; m < 4; ++m) t = __vmaxu2(t, __vmaxu2(wa[j][m] & 0x7fff7fffu, wb[j][m] & 0x7fff7fffu));
      top[j] = max(t & 0xffffu, t >> 16);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1)
#pragma unroll
      for (int j = 0; j < 2; ++j) top[j] = max(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int k = min(fit_pow2((int)(top[j] >> 7) + g.grow), g.most);
      fine[j] = top[j] < 0x7f80u;
      up[j] = make_float2(pow2(k), pow2(k));
      back[j] = pow2(-k) * g.t_back;
    }
  }
  uint32_t ha[2][4], la[2][4], hb[2][4], lb[2][4];
  float any_a[2][8], any_b[2][8];                        // (kAny: before the rotation)
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    // two pairs' members a, b (kHalf and others: channels 2 m, + 1 of va and of vb; kInter: even and odd channels of four)
    float2 ka, kb, c, s;
    if (kW != 0) {
      if (kMode == kInter) {
        const uint4 x = lds_v4(norm_s + (uint32_t)((m & 1) * 256 + (m < 2 ? L.va : L.vb) * 16));
        ka = make_float2(__uint_as_float(x.x), __uint_as_float(x.z));
        kb = make_float2(__uint_as_float(x.y), __uint_as_float(x.w));
      } else {
        const uint32_t at = norm_s + (uint32_t)((m >> 1) * 256 + (m & 1) * 8);
        const uint2 x = lds_v2(at + 16u * L.va), y = lds_v2(at + 16u * L.vb);
        ka = make_float2(__uint_as_float(x.x), __uint_as_float(x.y));
        kb = make_float2(__uint_as_float(y.x), __uint_as_float(y.y));
      }
    }
    const uint32_t f = kMode == kHalf ? L.freq_at + 2u * m * L.freq_step
                                      : freq_s + 8u * (m < 2 ? L.va : L.vb) + 2u * (m & 1) * 128u;     // (freq_slot)
    const uint32_t f_step = kMode == kHalf ? L.freq_step : 128u;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float2 a, b;
      if (kMode == kInter) {
        const uint32_t x = m < 2 ? wa[j][2 * m] : wb[j][2 * m - 4], y = m < 2 ? wa[j][2 * m + 1] : wb[j][2 * m - 3];
        a = make_float2(lo16(x), lo16(y));
        b = make_float2(hi16(x), hi16(y));
      } else {
        a = make_float2(lo16(wa[j][m]), hi16(wa[j][m]));
        b = make_float2(lo16(wb[j][m]), hi16(wb[j][m]));
      }
      a = mul2(a, kW != 0 ? mul2(ka, up[j]) : up[j]);
      b = mul2(b, kW != 0 ? mul2(kb, up[j]) : up[j]);
      if (kMode == kHalf || kMode == kInter) {
        if (j == 0 || !kSame) {
          phase_sincos(f, pos[j], c.x, s.x);
          phase_sincos(f + f_step, pos[j], c.y, s.y);
        }
        const float2 x = fma2(mul2(b, s), make_float2(-1.f, -1.f), mul2(a, c));
        b = fma2(b, c, mul2(a, s));
        a = x;
      }
      if (kMode == kInter) {
        split(a.x, b.x, m < 2 ? ha[j][2 * m] : hb[j][2 * m - 4], m < 2 ? la[j][2 * m] : lb[j][2 * m - 4]);
        split(a.y, b.y, m < 2 ? ha[j][2 * m + 1] : hb[j][2 * m - 3], m < 2 ? la[j][2 * m + 1] : lb[j][2 * m - 3]);
      } else if (kMode == kAny) {
        any_a[j][2 * m] = a.x, any_a[j][2 * m + 1] = a.y;
        any_b[j][2 * m] = b.x, any_b[j][2 * m + 1] = b.y;
      } else {
        split(a.x, a.y, ha[j][m], la[j][m]);
        split(b.x, b.y, hb[j][m], lb[j][m]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int r = L.r0 + j;
    if (kMode == kAny) {
      // pairs that no lane holds: through the row's own place in the buffer, 512 bytes as float32 in four lines
      const uint32_t line = xb + (uint32_t)((r >> 3) * 1024 + (r & 7) * 128);
      auto at = [&](int ch) {
        return line + (uint32_t)(((ch >> 5) & 1) * 8192 + (ch >> 6) * kHalfBuf + (ch & 31) * 4);
      };
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        sts_v2(at(8 * L.va + e), __float_as_uint(any_a[j][e]), __float_as_uint(any_a[j][e + 1]));
        sts_v2(at(8 * L.vb + e), __float_as_uint(any_b[j][e]), __float_as_uint(any_b[j][e + 1]));
      }
      __syncwarp();
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        float* d = v ? any_b[j] : any_a[j];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int ch = 8 * (v ? L.vb : L.va) + e, h = P.half_rot;
          const int i = ch < h ? ch : ch - h, other = ch < h ? ch + h : ch - h;
          if (ch < 2 * h) {
            float cs, sn;
            phase_sincos(freq_s + 8u * (uint32_t)freq_slot(false, i), j && !kSame ? pos[1] : pos[0], cs, sn);
            uint32_t o;
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(o) : "r"(at(other)) : "memory");
            d[e] = fmaf(d[e], cs, (ch < h ? -sn : sn) * __uint_as_float(o));
          }
        }
      }
      __syncwarp();
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        split(any_a[j][2 * m], any_a[j][2 * m + 1], ha[j][m], la[j][m]);
        split(any_b[j][2 * m], any_b[j][2 * m + 1], hb[j][m], lb[j][m]);
      }
    }
    const uint32_t to_a = xb + (L.at_a ^ (16u * j)) + 128u * j, to_b = xb + (L.at_b ^ (16u * j)) + 128u * j;
    sts_v4(to_a, ha[j]);
    sts_v4(to_a + kHalfBuf, la[j]);
    sts_v4(to_b, hb[j]);
    sts_v4(to_b + kHalfBuf, lb[j]);
    if (L.sub == 0) {
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(fac_s + 4u * (uint32_t)r), "f"(back[j]) : "memory");
      if (!fine[j] && left > j) set_status(P.r.status, KVQ_ERR_NONFINITE);
    }
  }
  return kW == 1 && small;
}
// A slot's two rows from where they came from, each under a power of two of its own.
template <int kMode>
__device__ __noinline__ void place_apart(const RopeParams& P, const Seg& g, Lane L, Place w, int left, int pos0, int pos1, uint32_t xb, uint32_t norm_s,
                                         uint32_t freq_s, uint32_t fac_s) {
  const RotTensor& T = P.r.t[w.tt];
  const int pos[2] = {pos0, pos1};
  uint32_t wa[2][4], wb[2][4];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    int row, head;
    tile_row(T, w.mh, min(w.c * kRtRows + L.r0 + j, T.rows * T.head_div - 1), row, head);   // (as ask_rows)
    const uint4* src = reinterpret_cast<const uint4*>(rope_src(P, w.tt, row, head));
    const uint4 x = __ldg(src + L.va), y = __ldg(src + L.vb);
    wa[j][0] = x.x, wa[j][1] = x.y, wa[j][2] = x.z, wa[j][3] = x.w;
    wb[j][0] = y.x, wb[j][1] = y.y, wb[j][2] = y.z, wb[j][3] = y.w;
  }
  __syncwarp();
  place_words<kMode, 3, false>(P, g, L, left, pos, wa, wb, xb, norm_s, freq_s, fac_s);
}
// Places a slot's two rows.
template <int kMode, int kW, bool kSame>
__device__ __forceinline__ void place_rows(const RopeParams& P, const Seg& g, const Lane& L, const Place& w, int left, uint32_t pos_s, uint32_t raw,
                                           uint64_t* bar_read, uint32_t xb, uint32_t norm_s, uint32_t freq_s, uint32_t fac_s) {
  int pos[2] = {0, 0};
  if (kMode != kNone) {
    const uint2 x = lds_v2(pos_s + 4u * L.r0);
    pos[0] = (int)x.x;
    pos[1] = (int)x.y;
  }
  bool apart = kW == 1 && g.wide;                        // (that of weights without a norm comes here too)
  if (!apart) {
    uint32_t wa[2][4], wb[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint4 x = lds_v4(raw + 256u * (L.r0 + j) + 16u * L.va), y = lds_v4(raw + 256u * (L.r0 + j) + 16u * L.vb);
      wa[j][0] = x.x, wa[j][1] = x.y, wa[j][2] = x.z, wa[j][3] = x.w;
      wb[j][0] = y.x, wb[j][1] = y.y, wb[j][2] = y.z, wb[j][3] = y.w;
    }
    rt_arrive(bar_read, threadIdx.x & 31);               // (the next rows but one may come)
    const bool small = place_words<kMode, kW, kSame>(P, g, L, left, pos, wa, wb, xb, norm_s, freq_s, fac_s);
    apart = kW == 1 && __any_sync(0xffffffffu, small);
  } else {
    rt_arrive(bar_read, threadIdx.x & 31);
  }
  // (Behind the products, and from global memory: the buffer that the rows came from may hold others by now, and a branch between the sums of
  // squares and the products kept these from covering those, 219 us for 16 x 2048 tokens instead of 210.  With the weights' choice
  // it is 211; 316 where the weights are far apart, 421 where all rows are small.)
  if (apart) place_apart<kMode>(P, g, L, w, left, pos[0], pos[1], xb, norm_s, freq_s, fac_s);
}
template <int kMode, int kW>
__device__ __forceinline__ void place_rows(const RopeParams& P, const Seg& g, const Lane& L, const Place& w, int left, uint32_t pos_s, uint32_t raw,
                                           uint64_t* bar_read, uint32_t xb, uint32_t norm_s, uint32_t freq_s, uint32_t fac_s) {
  if (kMode == kNone || g.same) place_rows<kMode, kW, true>(P, g, L, w, left, pos_s, raw, bar_read, xb, norm_s, freq_s, fac_s);
  else place_rows<kMode, kW, false>(P, g, L, w, left, pos_s, raw, bar_read, xb, norm_s, freq_s, fac_s);
}
template <int kMode>
__device__ __forceinline__ void place_rows(const RopeParams& P, const Seg& g, const Lane& L, const Place& w, int left, uint32_t pos_s, uint32_t raw,
                                           uint64_t* bar_read, uint32_t xb, uint32_t norm_s, uint32_t freq_s, uint32_t fac_s) {
  if (g.norm || g.wide) place_rows<kMode, 1>(P, g, L, w, left, pos_s, raw, bar_read, xb, norm_s, freq_s, fac_s);
  else if (kMode != kNone && g.weighted) place_rows<kMode, 2>(P, g, L, w, left, pos_s, raw, bar_read, xb, norm_s, freq_s, fac_s);
  else place_rows<kMode, 0>(P, g, L, w, left, pos_s, raw, bar_read, xb, norm_s, freq_s, fac_s);
}

// A matrix on its way to TMEM lies where rows go (64 KB: all of it), 16-byte piece c of row i so that the lanes of a warp,
// a row each, read from different banks.  (Lanes that read their rows from global memory, 16 of each 512 bytes at a time,
// took 10 to 16 K clocks; 5 K so.  3 x 777 tokens: 25.6 us, now 16.5.)
static_assert(kRtXBuf * 2 == kHeadDim * kHeadDim * 4, "a matrix fills the rows' buffers");
__device__ __forceinline__ uint32_t mat_at(int i, int c) { return 512u * (uint32_t)i + 16u * (uint32_t)(c ^ (i & 7)); }
__device__ __forceinline__ void ask_matrix(const float* mat, uint32_t mat_s, int warp, int lane) {
#pragma unroll 4
  for (int j = 0; j < kHeadDim / kRtWarps; ++j) {
    const int i = warp * (kHeadDim / kRtWarps) + j;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(mat_s + mat_at(i, lane)), "l"(mat + (size_t)i * kHeadDim + 4 * lane) : "memory");
  }
}
__device__ __forceinline__ float4 mat_v4(uint32_t mat_s, int i, int c) {
  const uint4 x = lds_v4(mat_s + mat_at(i, c));
  return make_float4(__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w));
}
// Half of row i of the Walsh-Hadamard matrix into TMEM: entry j is -1 where i & j has an odd number of bits (no lo).
__device__ __forceinline__ void put_hadamard(int i, int part, uint32_t taddr) {
  uint32_t odd = 0u;                                     // of j's lowest four bits
#pragma unroll
  for (int e = 0; e < 16; ++e) odd |= (uint32_t)(__popc(i & e) & 1) << e;
#pragma unroll 1
  for (int blk = 0; blk < 4; ++blk) {
    const uint32_t o = __popc(i & (64 * part + 16 * blk)) & 1 ? ~odd : odd;
    uint32_t h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = 0x3c003c00u | ((o >> (2 * j)) & 1u) << 15 | ((o >> (2 * j + 1)) & 1u) << 31;
    tmem_st8(taddr + 32u * (uint32_t)part + 8u * (uint32_t)blk, h);
  }
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Half of row i of a matrix as hi and lo into TMEM.
__device__ __forceinline__ void split_matrix(uint32_t mat_s, int i, int part, float up, uint32_t taddr) {
#pragma unroll 1
  for (int blk = 0; blk < 4; ++blk) {
    uint32_t h[8], l[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 t4 = mat_v4(mat_s, i, 16 * part + 4 * blk + j);
      const float t[4] = {t4.x * up, t4.y * up, t4.z * up, t4.w * up};
      float y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = lead11(t[e]);
      h[2 * j] = half2_bits(y[0], y[1]);
      h[2 * j + 1] = half2_bits(y[2], y[3]);
      l[2 * j] = half2_bits(t[0] - y[0], t[1] - y[1]);
      l[2 * j + 1] = half2_bits(t[2] - y[2], t[3] - y[3]);
    }
    tmem_st8(taddr + 32u * (uint32_t)part + 8u * (uint32_t)blk, h);
    tmem_st8(taddr + kRtLo + 32u * (uint32_t)part + 8u * (uint32_t)blk, l);
  }
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// The largest exponent field of half a row's entries.
__device__ __forceinline__ uint32_t top_exponent(uint32_t mat_s, int i, int part) {
  uint32_t top = 0;
#pragma unroll 4
  for (int j = 0; j < 16; ++j) {
    const float4 t = mat_v4(mat_s, i, 16 * part + j);
    top = max(max(top, __float_as_uint(fabsf(t.x))), max(__float_as_uint(fabsf(t.y)), max(__float_as_uint(fabsf(t.z)), __float_as_uint(fabsf(t.w)))));
  }
  return top >> 23;
}

__global__ void __launch_bounds__(kRtThreads, 2) rope_tc_kernel(const __grid_constant__ RopeParams P) {
  __shared__ uint32_t tbase_sh;
  __shared__ __align__(8) uint64_t bar_mma[2], bar_raw[2], bar_read[2], bar_x[2], bar_free[2];
  __shared__ volatile int abort_sh;
  __shared__ int uneven_sh;
  __shared__ Seg seg_sh;
  extern __shared__ uint8_t um_smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(um_smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sb = um_saddr(sm);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    abort_sh = 0;
    for (int i = 0; i < 2; ++i) {
      um_mbar_init(&bar_mma[i]);
      rt_init(&bar_raw[i], 64);                          // rows are there
      rt_init(&bar_read[i], kRtWarps);                   // rows are in registers
      rt_init(&bar_x[i], kRtWarps + 1);                  // rows are placed, their destinations known
      rt_init(&bar_free[i], kRtOut);                     // results are out
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  const int c_lo = first_chunk(P, blockIdx.x), c_hi = first_chunk(P, blockIdx.x + 1);
  const int total = c_hi - c_lo;
  if (warp < kRtWarps && total > 0) {                    // (matrices do not come from the grid ahead)
    const Place w = place_of(P, c_lo);
    if (P.r.t[w.tt].mode == ROT_DENSE) ask_matrix(P.r.t[w.tt].mat + (size_t)w.mh * kHeadDim * kHeadDim, sb, warp, lane);
  }
  // No TMEM is taken before the grid ahead has ended: its blocks could be waiting for that TMEM, and this one for them.
  pdl_wait();
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(um_saddr(&tbase_sh)), "r"(kRtCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Only now may the next kernel begin: one that takes all of TMEM could otherwise have it before this CTA does, and
  // wait for this grid.
  pdl_trigger();
  const uint32_t tb = tbase_sh;
  const int q = warp & 3;
  const uint32_t tlane = (uint32_t)(32 * q) << 16;       // this warp's TMEM lanes

  if (warp >= kRtMma) {
    rt_regs_dec<kLastRegs>();
    if (warp == kRtMma) {
      // ---- the MMAs of a chunk, once its rows are placed (code that the whole warp runs, one lane issues) ----
      Place w = place_of(P, c_lo);
      for (int n = 0; n < total; ++n) {
        const int s = n & 1;
        const uint32_t d = tb + kRtAcc + 64u * (uint32_t)s;
        const bool dense = P.r.t[w.tt].mode == ROT_DENSE;
        const uint64_t xd = sw128_desc(sb + (uint32_t)(s * kRtXBuf));
        const bool ok = rt_wait_use(bar_x, n, &abort_sh);
        tc_fence_after();
        if (ok && rt_elect()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint64_t hi = xd + (uint64_t)(((kk >> 2) * 8192 + (kk & 3) * 32) >> 4), lo = hi + (kHalfBuf >> 4);
            rt_mma(d, tb + 8u * (uint32_t)kk, lo, kk > 0);
            rt_mma(d, tb + 8u * (uint32_t)kk, hi, 1u);
            if (dense) rt_mma(d, tb + kRtLo + 8u * (uint32_t)kk, hi, 1u);
          }
          umma_commit(&bar_mma[s]);
        }
        __syncwarp();
        if (++w.c == w.cpm && n + 1 < total) w = place_of(P, c_lo + n + 1);
      }
    } else if (warp != kRtDst) {
      // ---- rows, two chunks ahead ----
      Place w = place_of(P, c_lo);
      for (int n = 0; n < total; ++n) {
        const int s = n & 1;
        if (n >= 2) rt_wait_use(bar_read, n - 2, &abort_sh);
        ask_rows(P, w, (warp - kRtLoad) >> 1, sb + (uint32_t)(kRtRaw + s * kRtRawBuf), sb + (uint32_t)(kRtPos + s * kRtRows * 4), &bar_raw[s], lane);
        if (++w.c == w.cpm && n + 1 < total) w = place_of(P, c_lo + n + 1);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
      // ---- where a chunk's rows go, two to a lane ----
      Place w = place_of(P, c_lo);
      for (int n = 0; n < total; ++n) {
        const RotTensor& T = P.r.t[w.tt];
        const int lg = __ffs(T.head_div) - 1, pairs = T.rows << lg;
        const uint32_t meta = sb + (uint32_t)(kRtMeta + (n & (kMetaSets - 1)) * kRtRows * 8);
        unsigned long long dst[2] = {0ull, 0ull};
#pragma unroll 1
        for (int j = 0; j < 2; ++j) {
          const int p = w.c * kRtRows + 32 * j + lane;
          if (p < pairs) {
            const int row = p >> lg, head = (w.mh << lg) + (p & (T.head_div - 1));
            const int b = T.is_query ? 0 : __ldg(P.r.seq_idx + row), at = T.is_query ? 0 : __ldg(P.r.pos + row);
            const unsigned long long d = (unsigned long long)rot_dst(P.r, T, row, head, b, at, true);
            (j ? dst[1] : dst[0]) = d;
          }
        }
        // (once chunk n - 2 is placed, what chunk n - 4 had here has been used)
        if (n >= 2) rt_wait_use(bar_x, n - 2, &abort_sh);
        sts_u64(meta + 8u * (uint32_t)lane, dst[0]);
        sts_u64(meta + 8u * (uint32_t)(32 + lane), dst[1]);
        rt_arrive(&bar_x[n & 1], lane);
        if (++w.c == w.cpm && n + 1 < total) w = place_of(P, c_lo + n + 1);
      }
    }
  } else if (warp >= kRtWarps) {
    // ---- results: four warps, 32 outputs each ----
    rt_regs_dec<kOutRegs>();
    // stmatrix takes 8 x 8 tiles, rows 8 k + lane % 8, 16-byte piece 4 q + lane / 8, and stores them the other way
    // round; a warp then writes rows 16 q .. out, two at a time
    const uint32_t put = out_at(lane & 7, 4 * q + (lane >> 3)), get = out_at(lane >> 4, lane & 15);
    for (int n = 0; n < total; ++n) {
      const int s = n & 1;
      const uint32_t xb = sb + (uint32_t)(s * kRtXBuf), acc_at = tb + tlane + kRtAcc + 64u * (uint32_t)s;
      const uint32_t fac = sb + (uint32_t)(kRtFac + s * kRtRows * 4), meta = sb + (uint32_t)(kRtMeta + (n & (kMetaSets - 1)) * kRtRows * 8);
      if (warp == kRtWarps) rt_wait_use(bar_mma, n, &abort_sh);
      rt_sync(kBarMma, kRtOut);
      const bool ok = !abort_sh;
      if (ok) {
        tc_fence_after();
        const bool uneven = *reinterpret_cast<volatile int*>(&uneven_sh) != 0;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // outputs (lane >> 2) + 8 j of this warp's 32, rows 8 k + 2 (lane & 3) and the next
          uint32_t acc[2][16];
          tmem_ld_tiles(acc_at + 32u * half, acc[0]);
          tmem_ld_tiles(acc_at + (16u << 16) + 32u * half, acc[1]);
          tmem_wait_ld16(acc[0]);
          tmem_wait_ld16(acc[1]);
          if (uneven) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float f = reinterpret_cast<const float*>(sm + kRtRowFac)[32 * q + (lane >> 2) + 8 * j];
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  uint32_t& v = acc[j >> 1][4 * k + 2 * (j & 1) + e];
                  v = __float_as_uint(__uint_as_float(v) * f);
                }
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint2 f = lds_v2(fac + 4u * (uint32_t)(32 * half + 8 * k + 2 * (lane & 3)));
            const float2 f2 = make_float2(__uint_as_float(f.x), __uint_as_float(f.y));
            uint32_t d[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t* v = acc[j >> 1] + 4 * k + 2 * (j & 1);
              const float2 x = mul2(make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])), f2);
              d[j] = pack_digits(x.x, x.y);              // (two bf16, to nearest)
            }
            asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(xb + put + 1024u * (4 * half + k)),
                         "r"(d[0]), "r"(d[1]), "r"(d[2]), "r"(d[3])
                         : "memory");
          }
        }
        tc_fence_before();
      }
      rt_sync(kBarOut, kRtOut);
      if (ok) {
        // (all loads before the first store, which may be left out)
        unsigned long long dst[4];
        uint4 x[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            dst[j] = lds_u64(meta + 8u * (uint32_t)(16 * q + 8 * h + 2 * j + (lane >> 4)));
            x[j] = lds_v4(xb + (uint32_t)(1024 * (2 * q + h) + 256 * j) + (get ^ (32u * j)));
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (dst[j]) __stcg(reinterpret_cast<uint4*>(dst[j]) + (lane & 15), x[j]);
        }
      }
      rt_arrive(&bar_free[s], lane);
    }
    // after a time-out: what was issued ends before TMEM is given back (bounded)
    if (abort_sh && warp == kRtWarps)
      for (int n = max(total - 2, 0); n < total; ++n) rt_wait(&bar_mma[n & 1], (uint32_t)((n >> 1) & 1));
  } else {
    // ---- rows: placed two to a slot of eight lanes ----
    rt_regs_inc<kPlaceRegs>();
    const int part = warp >> 2, i = 32 * q + lane;       // set-up: matrix row i, half of its inputs
    const int slot = lane >> 3, sub = lane & 7, r0 = 8 * warp + 2 * slot;
    const uint32_t norm_s = sb + kRtNorm, freq_s = sb + kRtFreq;
    uint32_t* exch = reinterpret_cast<uint32_t*>(sm + kRtExch);
    const Seg& g = seg_sh;
    int mode = kNone;
    Lane L{r0, sub, sub, sub + 8, 0u, 0u, 0u, 0u};
    if (tid == 64) reinterpret_cast<uint64_t*>(sm + kRtFreq)[64] = 0ull;
    if (tid < 64)
      reinterpret_cast<uint64_t*>(sm + kRtFreq)[freq_slot(P.interleaved, tid)] = tid < P.half_rot ? __ldg(P.freq + tid) : 0ull;

    // ---- a matrix: T hi and lo into TMEM, the channels' weights, the lanes' pairs ----
    auto set_up = [&](const Place& w, bool first) {
      const RotTensor& T = P.r.t[w.tt];
      const bool had = T.mode == ROT_WHT;
      const bool turned = P.rpos[w.tt] != nullptr;
      if (!had && !first) ask_matrix(T.mat + (size_t)w.mh * kHeadDim * kHeadDim, sb, warp, lane);
      // weights: float32, the first halves of all vectors of eight, then the second
      const bool norm = P.norm[w.tt] != nullptr, weighted = norm || (turned && P.scale != 1.f);
      if (part == 0) {
        float x = norm ? __ldg(P.norm[w.tt] + i) : 1.f;
        if (turned && i < 2 * P.half_rot) x *= P.scale;
        reinterpret_cast<float*>(sm + kRtNorm)[((i >> 2) & 1) * 64 + (i >> 3) * 4 + (i & 3)] = x;
      }
      if (!had) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        rt_sync(kBarPlace, kRtWarps);
        exch[128 * part + i] = top_exponent(sb, i, part);
      }
      rt_sync(kBarPlace, kRtWarps);
      // the matrix's power of two; a row's own where it would lose bits under that one
      int k = 0;
      bool uneven = false;
      if (!had) {
        uint32_t low = 255, high = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t e = max(exch[lane + 32 * j], exch[128 + lane + 32 * j]);
          low = e ? min(low, e) : low;                   // (rows of zeros have no say)
          high = max(high, e);
        }
        low = __reduce_min_sync(0xffffffffu, low);
        high = __reduce_max_sync(0xffffffffu, high);
        uneven = low + 8 < high;
        k = fit_pow2((int)(uneven ? max(exch[i], exch[128 + i]) : high));
        if (uneven && part == 0) reinterpret_cast<float*>(sm + kRtRowFac)[i] = pow2(-k);
      }
      if (tid == 0) uneven_sh = uneven;
      const float t_back = had ? kInvSqrtDim : uneven ? 1.f : pow2(-k);
      if (had) put_hadamard(i, part, tb + tlane);
      else split_matrix(sb, i, part, pow2(k), tb + tlane);
      // which channels a lane holds
      mode = !turned ? kNone : P.interleaved ? kInter : P.half_rot % 8 == 0 ? kHalf : kAny;
      L.va = sub;
      L.vb = sub + 8;
      L.freq_at = freq_s + 8u * sub;                     // (freq_slot of pair 8 va; the next eight positions on)
      L.freq_step = 64u;
      if (mode == kHalf) {
        const int h8 = P.half_rot / 8;
        L.va = sub < h8 ? sub : 2 * h8 + 2 * (sub - h8);
        L.vb = sub < h8 ? sub + h8 : L.va + 1;
        if (sub >= h8) {                                 // (two vectors that are no pair: a frequency of 0)
          L.freq_at = freq_s + 8u * 64u;
          L.freq_step = 0u;
        }
      }
      uint32_t wtop = 0, wlow = ~0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t x = __float_as_uint(fabsf(reinterpret_cast<const float*>(sm + kRtNorm)[4 * lane + j]));
        wtop = max(wtop, x);
        wlow = min(wlow, x);
      }
      wtop = __reduce_max_sync(0xffffffffu, wtop);
      wlow = __reduce_min_sync(0xffffffffu, wlow);
      // the largest weight and the rotation's sqrt 2, by exponents, rounded up; after the norm rows are below 2^4
      const int grow = (weighted ? (int)(wtop >> 23) - 126 : 0) + (turned ? 1 : 0), kn = fit_pow2(130 + grow);
      // (rms r < 1/2, r the norm's factor, where the squares sum to less than 128 eps / 3)
      const float least = norm ? P.eps * (kHeadDim / 3.f) : 0.f;
      const int k_t = had ? 4 : uneven ? 0 : k, most = min(126, 149 - k_t);
      // One power of two for all rows (or that of a row's largest channel before its weight) brings a row's largest channel to 2^-2 or more,
      // 2^-22 of which hi and lo keep, where the smallest weight is not 2^10 below the largest, and no product overflows or vanishes where
      // the largest is near 1.
      const int top_at = (int)(wtop >> 23);
      if (tid == 0 && norm && top_at == 255) set_status(P.r.status, KVQ_ERR_NONFINITE);
      const bool wide = weighted && (top_at - (int)(wlow >> 23) > 9 || top_at < 97 || top_at > 187 || kn > most);
      if (tid == 0) seg_sh = Seg{T.head_div > 1, norm, weighted, grow, turned, wide, pow2(kn), pow2(-kn) * t_back, least, most, t_back};
      rt_sync(kBarPlace, kRtWarps);
      L.at_a = (uint32_t)xs_offset(r0, 8 * L.va);
      L.at_b = (uint32_t)xs_offset(r0, 8 * L.vb);
    };

    bool fresh = true;                                   // the chunk begins a matrix (or this CTA's work)
    int freed = 0;                                       // chunks whose buffer is known to be free again
    Place w = place_of(P, c_lo);
    for (int n = 0; n < total; ++n) {
      const int s = n & 1;
      // (at a new matrix the last one's results are out: TMEM and what its set-up left may be overwritten)
      for (const int want = fresh ? n : n - 1; freed < want; ++freed) rt_wait_use(bar_free, freed, &abort_sh);
      if (fresh) {
        tc_fence_after();
        set_up(w, n == 0);
      }
      rt_wait_use(bar_raw, n, &abort_sh);
      const uint32_t xb = sb + (uint32_t)(s * kRtXBuf), raw = sb + (uint32_t)(kRtRaw + s * kRtRawBuf);
      const uint32_t fac = sb + (uint32_t)(kRtFac + s * kRtRows * 4), pos = sb + (uint32_t)(kRtPos + s * kRtRows * 4);
      const int left = P.r.t[w.tt].rows * P.r.t[w.tt].head_div - w.c * kRtRows - r0;
      if (mode == kHalf) place_rows<kHalf>(P, g, L, w, left, pos, raw, bar_read + s, xb, norm_s, freq_s, fac);
      else if (mode == kInter) place_rows<kInter>(P, g, L, w, left, pos, raw, bar_read + s, xb, norm_s, freq_s, fac);
      else if (mode == kAny) place_rows<kAny>(P, g, L, w, left, pos, raw, bar_read + s, xb, norm_s, freq_s, fac);
      else place_rows<kNone>(P, g, L, w, left, pos, raw, bar_read + s, xb, norm_s, freq_s, fac);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      tc_fence_before();
      rt_arrive(&bar_x[s], lane);
      fresh = ++w.c == w.cpm;
      if (fresh && n + 1 < total) w = place_of(P, c_lo + n + 1);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0 && abort_sh) set_status(P.r.status, KVQ_ERR_TIMEOUT);
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tb), "r"(kRtCols) : "memory");
}

}  // namespace

int launch_rope_tc(RopeParams P, cudaStream_t stream) {
  long long total = 0;
  for (int t = 0; t < 3; ++t) {
    P.r.n_dense[t] = 0;
    if (P.r.t[t].mode == ROT_COPY) continue;
    const long long cpm = ((long long)P.r.t[t].rows * P.r.t[t].head_div + kRtRows - 1) / kRtRows;
    const long long here = (P.r.t[t].heads / P.r.t[t].head_div) * cpm;
    P.r.n_dense[t] = (int)here;                          // (fewer than 2^30: the caller has checked rows x heads)
    total += here;
  }
  if (total == 0) return KVQ_OK;
  if (total > 0x7fffffffLL) return KVQ_ERR_UNSUPPORTED;
  P.r.dense_total = (int)total;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KVQ_ERR_CUDA;
  static std::mutex mu;
  static unsigned long long attr_done = 0;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!(attr_done & (1ull << dev))) {
      if (cudaFuncSetAttribute(rope_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRtSmem) != cudaSuccess)
        return KVQ_ERR_CUDA;
      attr_done |= 1ull << dev;
    }
  }
  const int ctas = (int)std::min(total, 2LL * kSms);
  return launch_pdl(rope_tc_kernel, dim3((unsigned)ctas), dim3(kRtThreads), (size_t)kRtSmem, stream, P) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // namespace kvq
