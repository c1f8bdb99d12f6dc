// kv_attn_tree on the tensor cores: the nodes of a drafted tree attend together, so that a
// sequence's cache is read and its codes are expanded once for all of them.
//
// The mathematics.  For the rows n of one (sequence, kv head) -- a row is a (node, query head of
// the kv head) pair -- and its tokens t:  s[t][n] = scale k_t.q_n,  o_n = sum_t 2^(s - m_n) v_t /
// sum_t 2^(s - m_n), one pass over the tokens with a running reference m_n.
//
// Tile and layout.  A tile is 128 tokens (8 INT2 pages, or 128 BF16 window rows) by N = 64 rows.
// Tokens are the tensor core's M: S^T [128 tokens x N] = K [128 x d] Q^T, and
// O^T [128 channels x N] += V^T [128 channels x 128 tokens] P [128 x N], so
//   * the expanded K and V^T are the A operands and live in TMEM: a page's codes are stored in the
//     fragment order of a 16-row MMA, which is the order of tcgen05.st.16x128b -- one 16-byte load
//     and one AND per two codes puts a page's keys into TMEM, without a pass through shared memory;
//   * a lane of S^T is a token, so a token's scale (Delta, norm) is one number per thread, and a
//     warp reads no scale per score;
//   * P [token][row] goes to shared memory as the MN-major B operand, 16 bytes per 8 rows.
// 128 rows a CTA were tried, early on: the expansion is shared by twice the rows, the second score buffer no longer
// fits.  With groups of 128 it took as long; 16 nodes of 8 heads on 4 x 128 K tokens in groups of 32 took 733 us then,
// 862 with 64 rows, and the two have not been compared since.
// Keys.  With one group per row (G = 128) A holds the codes themselves, exact, and the zero point is
// one more K = 16 step (z against -sum q', hi + lo); Delta multiplies the finished sum.  With more
// groups A holds Delta c as an fp16 hi + lo pair (13 bits), scaled by a power of two per token, exact for groups down
// to 2^-25 of the token's largest, and the zero point's step takes Delta z (22 bits, hi + lo).  (Products of the codes as
// they stand, c 4^s 2^-24, lose bits of groups below 2^-4 of the largest, which large queries of that group bring
// out; whole numbers are one more instruction a register: 64 sequences of 6,000 tokens, 16 nodes of 4 heads, groups
// of 64: 385 -> 411 us, groups of 32 and 128 K tokens 782 -> 809.)
// q' is scaled by a power of two of its row, its largest value to 2^13 .. 2^14: exact down to 2^-22 of that value
// (8 bits above fp16's last step 2^-24, in slots that carry 4^-4), below it off by at most 2^-30 of it; with more
// groups to 2^8 .. 2^9 and no slots, exact down to 2^-25, off by at most 2^-33.  Values are dequantized to fp16,
// Delta (c - z) in one rounding (relative 2^-11 of the value and of Delta z: the output's own rounding to bf16 is
// 2^-8).  P is rounded to fp16, the sums l are fp32.  Window rows are bf16 as they are, with P as a bf16 hi + lo pair.
//
// Softmax reference.  m_n moves only when a score passes it by 15 (in log2): P <= 2^15, and fp16 ends at 2^16.
// It is set to the row's maximum, or up to 12 below it, as far as the maxima of the tile's four quarters lie apart
// by more than 8: where one token leads the others by far, they keep up to 36 binades of fp16 below it (a token
// that takes nearly all of the weight may give nearly nothing, and then the others are the output), and elsewhere
// the row can grow by 15 before a move, which takes some 2,000 clocks (4 below throughout: 106 us instead of 103.5
// for 64 nodes on 32 K tokens).  A CTA takes its pages first, then its window rows, whose P is a pair of bf16 and loses
// nothing beside a reference that is far off: a sink never sets the pages' reference.  (Windows first, reference
// at the maximum: a sink with a zero value row that leads by 20 nats left nothing of the pages' output.)  The
// four warps that share a row's tokens agree by one barrier, whose answer is read when the exponentials are
// formed already; a move rescales O in TMEM.
//
// Roles: 16 softmax warps (4 lane quadrants x 4 shares of the rows), 4 warps that expand keys (or load window
// rows), 8 that expand values, a warp each that issues QK and PV, one that streams pages (1-D bulk copies)
// and one that finds the nodes' ancestors; registers are handed from the latter to the softmax.  S has two
// buffers, so QK(i + 1) and the keys of i + 2 run beside softmax(i) and PV(i - 1).
//
// What bounds it: instruction issue, not the tensor pipe or memory.  A tile of 128 tokens takes 10,000 warp
// instructions (G = 128; a CTA's set-up included), more than half of them softmax, 2,300 the values and 1,000 the
// keys, in 2,700 clocks (1.3 us): the schedulers issue in 75% of their clocks, the pipe of logic, maxima and half
// precision (one warp instruction in two clocks) is busy for 50%, the tensor pipe for 16%, DRAM reads each byte
// once.  Groups of 32 take 11,700.  No part stands out: with its exponentials, its stores of P or the values' stores
// to TMEM left out an earlier version took as long within 2%, without the keys' stores 3 to 8% less; 8 softmax
// warps of 32 rows executed 16% fewer instructions, at 58%, and took 2.5% longer.  Measured: 64 nodes of 4 heads on
// 32 K tokens 103.6 us (332 TFLOP/s), 16 nodes of 8 heads on 4 x 128 K tokens, groups of 32, 910 us (227 TFLOP/s).  Of
// those, what keeps results right at the ends of the number range: a power of two a row, not a CTA (a query may
// be of any size beside its neighbours'), 4% of the latter when it came; pages before windows, which cost the latter
// 2.5% and sped the former up by 2%.
// What those figures hang on:
//   * MMAs are issued from code that the whole warp runs, by one elected lane: from a divergent branch each
//     costs 53 clocks at least, whatever N is;
//   * the roles' loops together stay within 32 KB, which is what an SM keeps of its code: a version with the
//     value loop unrolled over its pages ran at half the speed, waiting for instructions;
//   * about 12 us a CTA of set-up, q' operands, first reference and epilogue, which is why short contexts and
//     narrow trees go to the row kernel (see row_kernel).
//
// Several CTAs share a long sequence (splits over tiles); their partial (m, l, o) are merged by a
// second kernel, one warp per output row.
#include "common.cuh"
#include "launch.h"

#include <cstddef>
#include <mutex>

namespace kvq {
namespace {

constexpr int kNodes = KVQ_TREE_MAX_NODES;
constexpr int kNodeWords = kNodes / 32;
constexpr int kTile = 128;                       // tokens of a tile
constexpr int N = 64;                            // rows (node, query head) of a CTA
constexpr int kTilePages = kTile / kPage;
constexpr int kSmWarps = 16;                     // softmax; then 4 warps for keys, 8 for values, 4 more
constexpr int kKeyWarp = 16, kValWarp = 20, kQkWarp = 28, kPageWarp = 29, kPvWarp = 30, kSeenWarp = 31;
constexpr int kShares = kSmWarps / 4;            // shares of the rows, four warps (128 tokens) each
constexpr int kCols = N / kShares;               // rows of a softmax warp
constexpr int kKeyWarps = 4, kValWarps = 8;
constexpr int kThreadsT = 32 * 32;               // (whole warpgroups: registers are handed over by warpgroup)
constexpr int kStages = 4;                       // page tiles in flight
// Registers a thread by role, of the 64 that 1024 threads launch with.
constexpr int kRegsLaunch = 64, kRegsSoftmax = 72, kRegsKeys = 64, kRegsValues = 56, kRegsIssue = 48;
static_assert(32 * kSmWarps * kRegsSoftmax + 128 * kRegsKeys + 256 * kRegsValues + 128 * kRegsIssue <= kThreadsT * kRegsLaunch, "register split");

// log2 of the largest P before a row's reference moves: page tiles (fp16), window tiles (bf16 pairs); a lead that
// is ordinary, and how far below the maximum a reference is set at most
constexpr float kRefSlack = 15.f, kWinSlack = 30.f, kRefLead = 8.f, kRefBelow = 12.f;
constexpr int kMostSplits = 64;
constexpr int kWinCost = 4;                      // a window tile's time in page tiles'
constexpr long long kSmallCall = 1 << 19;        // row_kernel(): rows x kv heads x tokens
constexpr int kRec = 4 + kHeadDim;               // (m, l, -, -, o[d]) of a partial
constexpr int kSpin = 1 << 15, kSuspend = 20000;  // a wait gives up after that many rounds of at most 20 us
constexpr uint32_t kTmem = 512;
constexpr int kSlab = kTile * 128;               // 128 tokens x 64 16-bit values, 128-byte swizzled

struct TreeParams {
  const uint8_t* pages;
  const int32_t* page_table;
  const int32_t* seq_len;
  const int32_t* s_quant;
  const uint16_t* sink_k;
  const uint16_t* sink_v;
  const uint16_t* ring_k;
  const uint16_t* ring_v;
  const uint16_t* q;
  const int32_t* cu_rows;
  const int32_t* parent;
  uint16_t* out;
  float* part;           // [n_rows][Hq][splits][kRec]
  int32_t* status;
  int batch, hkv, gqa, gqa_log2, s_sink, ring_cap, max_pages, num_pages, page_bytes, l2;
  int n_rows, splits, mp;
  float scale_log2;
};

// ---- primitives --------------------------------------------------------------------------
__device__ __forceinline__ uint32_t saddr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint64_t* b, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(b)) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(saddr(b)), "r"(parity), "r"(kSuspend)
      : "memory");
  return ok != 0;
}
// Bounded wait of a whole warp; gives up as well when another warp has.  Inline (a call has no place
// beside setmaxnreg) and small.
__device__ __forceinline__ bool warp_wait(uint64_t* b, int phase, volatile int* gave_up) {
  bool ok = bar_try(b, (uint32_t)(phase & 1));
  if (!ok) {
#pragma unroll 1
    for (int i = 0; i < kSpin && !ok; ++i) {
      ok = bar_try(b, (uint32_t)(phase & 1));
      if (!ok && *gave_up) break;
    }
    if (!ok) *gave_up = 1;
  }
  return __all_sync(0xffffffffu, ok);
}
// ... for what is in flight when a wait was given up (whatever the outcome)
__device__ __forceinline__ void settle(uint64_t* b, int phase) {
#pragma unroll 1
  for (int i = 0; i < kSpin && !bar_try(b, (uint32_t)(phase & 1)); ++i) {
  }
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(saddr(dst)),
      "l"(src), "r"(bytes), "r"(saddr(bar))
      : "memory");
}
__device__ __forceinline__ void async_copy16(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(saddr(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.cta.sync 4, %0;" ::"n"(32 * kSmWarps) : "memory"); }
// one lane of a converged warp: the code around it stays uniform, so descriptors are formed in uniform
// registers (issued from a divergent lane an MMA takes 53 clocks, so 20 .. 33 at N = 32 .. 64 are lost)
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
template <int R>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }

// shared-memory matrix descriptors, 128-byte swizzle (8 rows of 128 bytes, groups 1024 apart)
__device__ __forceinline__ uint64_t desc_k128(uint32_t a) {                 // K-major
  return (uint64_t)((a & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)2 << 61);
}
__device__ __forceinline__ uint64_t desc_mn128(uint32_t a) {                // MN-major, 64-element blocks kSlab apart
  return (uint64_t)((a & 0x3FFFFu) >> 4) | ((uint64_t)(kSlab >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// K-major without swizzle, K = 16: 8 x 16-byte core matrices, 128 apart along the rows and
// `lead` apart along K
__device__ __forceinline__ uint64_t desc_plain(uint32_t a, uint32_t lead) {
  return (uint64_t)((a & 0x3FFFFu) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
               "r"(a), "l"(b), "r"(idesc), "r"(acc)
               : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
               "l"(a), "l"(b), "r"(idesc), "r"(acc)
               : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(saddr(bar)) : "memory");
}
#define KVQ_IO8(c, b) c(v[b]), c(v[b + 1]), c(v[b + 2]), c(v[b + 3]), c(v[b + 4]), c(v[b + 5]), c(v[b + 6]), c(v[b + 7])
// 16 (8) columns of this warp's lanes -> registers
__device__ __forceinline__ void tm_ld16(uint32_t a, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n "
      "tcgen05.wait::ld.sync.aligned;"
      : KVQ_IO8("=f", 0), KVQ_IO8("=f", 8)
      : "r"(a)
      : "memory");
}
__device__ __forceinline__ void tm_ld8(uint32_t a, float (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];" : KVQ_IO8("=f", 0) : "r"(a));
  asm volatile("tcgen05.wait::ld.sync.aligned;" : KVQ_IO8("+f", 0)::"memory");
}
__device__ __forceinline__ void tm_st8(uint32_t a, const float (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::KVQ_IO8("f", 0), "r"(a) : "memory");
}
// 16 lanes x 32 columns: registers 4 s .. 4 s + 3 are the A fragment of k-step s
#define KVQ_R16(c, v) c(v[0]), c(v[1]), c(v[2]), c(v[3]), c(v[4]), c(v[5]), c(v[6]), c(v[7]), c(v[8]), c(v[9]), c(v[10]), \
                      c(v[11]), c(v[12]), c(v[13]), c(v[14]), c(v[15])
__device__ __forceinline__ void tm_st_frag8(uint32_t a, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::KVQ_R16("r", v),
      "r"(a)
      : "memory");
}
// 16 lanes x 16 columns: two k-steps
__device__ __forceinline__ void tm_st_frag4(uint32_t a, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::KVQ_IO8("r", 0), "r"(a) : "memory");
}
// 16 lanes x 8 columns: the A fragment of one k-step
__device__ __forceinline__ void tm_st_frag2(uint32_t a, const uint32_t (&v)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%4], {%0,%1,%2,%3};" ::"r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(a)
               : "memory");
}
// a s f + c for two float32 at once
__device__ __forceinline__ void scale2(float& a, float& b, float s, float fa, float fb, float ca, float cb) {
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %2};\n mul.rn.f32x2 x, x, y;\n mov.b64 y, {%3, %4};\n"
      " mov.b64 z, {%5, %6};\n fma.rn.f32x2 x, x, y, z;\n mov.b64 {%0, %1}, x;\n}\n"
      : "+f"(a), "+f"(b)
      : "f"(s), "f"(fa), "f"(fb), "f"(ca), "f"(cb));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t h2bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits2h(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t pack16(float a, float b) { return h2bits(__floats2half2_rn(a, b)); }
__device__ __forceinline__ uint32_t packb16(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint4 lds16(const void* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void sts16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// a token's (Delta, z) pairs, one a group
template <int NG>
__device__ __forceinline__ void load_scales(const uint8_t* p, uint32_t (&v)[NG]) {
  if constexpr (NG == 4) {
    const uint4 w = lds16(p);
    v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    v[0] = w.x; v[1] = w.y;
  }
}
__device__ __forceinline__ int slot_pow(int s) { return s <= 4 ? s : s - 5; }
__device__ __forceinline__ uint32_t code_pair(uint32_t w, uint32_t w10, int s) {
  return s <= 4 ? (w & (0x00030003u << (2 * s))) : (w10 & (0x00030003u << (2 * (s - 5))));
}
// Reduce 8 values per lane over the warp's lanes; lane j returns value j % 8's result.
template <class F>
__device__ __forceinline__ float reduce_columns(float (&x)[8], int lane, F f) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int j = 0; j < o; ++j) {
      const float mine = up ? x[j + o] : x[j], other = up ? x[j] : x[j + o];
      x[j] = f(mine, __shfl_xor_sync(0xffffffffu, other, o));
    }
  }
  x[0] = f(x[0], __shfl_xor_sync(0xffffffffu, x[0], 8));
  return f(x[0], __shfl_xor_sync(0xffffffffu, x[0], 16));
}

// A sequence's rows as the kernels see them.
struct SeqState {
  int first, n;          // rows first .. first + n - 1
  int len, edge, L0;     // length, INT2 edge, length before the drafts
  bool bad;              // no tree, or its nodes are not in the BF16 windows
};
__device__ __forceinline__ SeqState seq_state(const TreeParams& P, int b) {
  SeqState s;
  s.first = P.cu_rows[b];
  s.n = P.cu_rows[b + 1] - s.first;
  s.len = P.seq_len[b];
  s.edge = P.s_quant[b];
  s.L0 = s.len - s.n;
  s.bad = s.first < 0 || s.n > P.n_rows || s.first > P.n_rows - max(s.n, 0) || s.n > kNodes || s.L0 < 0 ||
          s.edge > max(s.L0, P.s_sink);
  return s;
}

// Row tiles a sequence takes (a bad one: one, which reports it).
__device__ __forceinline__ int row_tiles(const TreeParams& P, int b) {
  const long long n = (long long)P.cu_rows[b + 1] - P.cu_rows[b];
  if (n < 0) set_status(P.status, KVQ_ERR_BOUNDS);         // (the other sequences have their rows)
  if (n <= 0) return 0;
  return n > kNodes ? 1 : (int)((n * P.gqa + N - 1) / N);
}

struct Layout {          // dynamic shared memory, from a 1024-byte boundary
  static constexpr int kQ = 0;                              // q' fp16, K-major: two slabs of N x 128 B
  static constexpr int kQb = kQ + 2 * N * 128;              // q' bf16 likewise
  static constexpr int kP = kQb + 2 * N * 128;              // P, two buffers of N / 64 slabs
  static constexpr int kPBytes = N / 64 * kSlab;
  static constexpr int kZ = kP + 2 * kPBytes;               // zero-point B operand: N x 16 fp16
  static constexpr int kZa = kZ + N * 32;                   // ... and A: 128 tokens x 16 fp16, two buffers
  // window K and V rows, two slabs each; before them, while a CTA has page tiles, the page stages
  static constexpr int kK = (kZa + 2 * kTile * 32 + 1023) / 1024 * 1024;
  static constexpr int kV = kK + 2 * kSlab;
  static constexpr int kPages = kK;
  static constexpr int kEnd = kV + 2 * kSlab;
  static_assert(kStages * kTilePages * 1568 <= 4 * kSlab, "page stages");
};

struct TreeShared {
  __align__(16) uint64_t page_full[kStages], page_free[kStages], q_full, seen_full, vote[kShares], meet[kShares], k_full[2], v_full[2], s_full[2], s_free[2], p_full[2],
      pv_done[2];
  uint32_t tmem;
  int gave_up;
  int pid[kStages][kTilePages];
  float lane_scale[4][kTile];
  __align__(4) uint16_t alive[4][kTilePages];            // tokens of a tile that exist, by lane quadrant
  __align__(16) float neg_m[N];    // minus the reference of every row
  __align__(16) float alpha[N];    // a moved reference: factor of what is summed so far
  float red[kTile / kCols][N];     // per-quadrant maxima; at the end parts of the sums
  uint8_t v_odd[2][kTile];         // window tiles with drafts: whether a token's value row is not finite
  int moves[kShares];              // the last tile (+ 1) in which a share's references have to move
  __align__(16) uint32_t seen[kNodes][kNodeWords];   // ancestors of every node, itself among them
  int jump[kNodes];                // (while they are found: the next one)
  int whole[kStages];              // every page of the tile is there in whole
  int row[N];                      // output rows: global row * Hq + query head
  __align__(16) float mul[2][N];   // scores' factors of every row: page tiles, window tiles
  int sigma[N];                    // q' in fp16 is 2^sigma q'
};

static_assert(kNodeWords == 4 && offsetof(TreeShared, seen) % 16 == 0 && offsetof(TreeShared, neg_m) % 16 == 0 &&
                  offsetof(TreeShared, alpha) % 16 == 0 && offsetof(TreeShared, mul) % 16 == 0 && Layout::kEnd % 1024 == 0,
              "vector loads");
static_assert(Layout::kEnd + sizeof(TreeShared) <= 227 * 1024, "shared memory of an SM");

template <int NG>
__global__ void __launch_bounds__(kThreadsT, 1) attn_tree_kernel(const __grid_constant__ TreeParams P) {
  using L = Layout;
  static_assert(kCols == 16, "a softmax warp's lanes stand for its rows (twice) at times");
  // TMEM columns: O, S twice (the next product runs while the softmax reads the last), the key operand
  // (64, or 128 as pairs) twice and the value operand (64), twice where there is room
  constexpr int kKCols = NG == 1 ? 64 : 128;
  constexpr int kKBufs = 2, kVBufs = NG == 1 ? 2 : 1;
  constexpr uint32_t kColO = 0, kColS = N, kColK = 3 * N, kColV = kColK + kKBufs * kKCols;
  static_assert(kColV + kVBufs * 64 <= 512, "TMEM columns");
  constexpr uint32_t kIdescF16 = (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);
  constexpr uint32_t kIdescPV = kIdescF16 | (1u << 16);
  constexpr uint32_t kIdescB16 = kIdescF16 | (1u << 7) | (1u << 10);
  constexpr uint32_t kIdescB16PV = kIdescB16 | (1u << 15) | (1u << 16);
  extern __shared__ __align__(1024) uint8_t sm[];           // (all of the shared memory: it starts aligned)
  TreeShared& S = *reinterpret_cast<TreeShared*>(sm + L::kEnd);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  volatile int* gave_up = &S.gave_up;
  pdl_trigger();
  pdl_wait();
  if (saddr(sm) & 1023u) {                                  // (the swizzled operands need it)
    if (tid == 0) set_status(P.status, KVQ_ERR_CUDA);
    return;
  }

  // ---- this CTA's row tile: item blockIdx.x counts the sequences' row tiles in order (every warp
  // looks it up for itself)
  const int split = blockIdx.z, h = blockIdx.y;
  int b = -1, rt = 0;
  for (int b0 = 0, before = 0; b0 < P.batch && b < 0; b0 += 32) {
    const int mine = b0 + lane < P.batch ? row_tiles(P, b0 + lane) : 0;
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += t;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + upto > (int)blockIdx.x);
    if (past) {
      const int at = __ffs(past) - 1;
      b = b0 + at;
      rt = (int)blockIdx.x - before - __shfl_sync(0xffffffffu, upto - mine, at);
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  if (tid == 0 && blockIdx.x == 0 && h == 0 && split == 0 && (P.cu_rows[0] != 0 || P.cu_rows[P.batch] != P.n_rows))
    set_status(P.status, KVQ_ERR_BOUNDS);
  if (b < 0) return;
  const SeqState st = seq_state(P, b);
  const int row0 = rt * N;
  const int ncol = min(N, st.n * P.gqa - row0);
  if (st.bad) {                                             // zeros (the merge writes them when there are splits)
    if (tid == 0) set_status(P.status, KVQ_ERR_BOUNDS);
    if (P.splits == 1 && st.first >= 0)
      for (long long i = tid; i < (long long)st.n * P.gqa * kHeadDim; i += kThreadsT) {
        const long long r = i / (P.gqa * kHeadDim);
        if (st.first + r < P.n_rows)
          P.out[((size_t)(st.first + r) * P.hkv * P.gqa + h * P.gqa) * kHeadDim + i % (P.gqa * kHeadDim)] = 0;
      }
    return;
  }

  // ---- tiles: pages first, then window rows (sink, then ring)
  const int edge = min(st.edge, st.len);
  const int n_sink = min(P.s_sink, st.len), ring0 = max(edge, P.s_sink);
  const int n_win = n_sink + max(0, st.len - ring0);
  const int n_tok = max(0, edge - P.s_sink);
  int np = (n_tok + kPage - 1) / kPage;
  if (np > P.mp) {
    if (tid == 0 && split == 0) set_status(P.status, KVQ_ERR_BOUNDS);
    np = P.mp;
  }
  const int nw = (n_win + kTile - 1) / kTile, ni = (np + kTilePages - 1) / kTilePages;
  // equal shares of the work, a window tile taken as kWinCost page tiles (its rows are loaded, not
  // streamed, and its P is a pair)
  auto first_tile = [&](int k) {
    const int at = (int)((long long)(kWinCost * nw + ni) * k / P.splits);
    return at < ni ? at : ni + (at - ni + kWinCost - 1) / kWinCost;
  };
  const int t0 = first_tile(split), t1 = first_tile(split + 1);
  const int nt = t1 - t0;

  // ---- set-up: barriers, TMEM, q' operands, ancestors
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      bar_init(&S.page_full[i], 1);
      bar_init(&S.page_free[i], kKeyWarps + kValWarps);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&S.k_full[i], kKeyWarps);
      bar_init(&S.v_full[i], kValWarps);
      bar_init(&S.s_full[i], 1);
      bar_init(&S.s_free[i], kSmWarps);
      bar_init(&S.p_full[i], kSmWarps);
      bar_init(&S.pv_done[i], 1);
    }
    bar_init(&S.q_full, kSmWarps);
    bar_init(&S.seen_full, 1);
    for (int i = 0; i < kShares; ++i) {
      bar_init(&S.vote[i], 4);
      bar_init(&S.meet[i], 4);
      S.moves[i] = 0;
    }
    S.gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&S.tmem)), "r"(kTmem) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tb = S.tmem;

  const int pb = P.page_bytes;
  const int npt = max(0, min(t1, ni) - t0);                 // this CTA's page tiles: its first ones
  uint8_t* stages = sm + L::kPages;
  if (warp >= kQkWarp) {
    regs_dec<kRegsIssue>();
    if (warp == kPageWarp) {
      // ---- pages
      const int32_t* tab = P.page_table + (size_t)b * P.max_pages;
      int k = 0;                                            // page tiles streamed
      for (; k < npt; ++k) {
        const int stage = k % kStages;
        const int p = (t0 + k) * kTilePages + lane;
        int pid = -1;
        if (lane < kTilePages && p < np) {
          pid = p < P.max_pages ? tab[p] : -1;
          if ((unsigned)pid >= (unsigned)P.num_pages) {
            pid = -1;
            set_status(P.status, KVQ_ERR_BOUNDS);
          }
        }
        if (k >= kStages && !warp_wait(&S.page_free[stage], k / kStages - 1, gave_up)) break;
        if (lane < kTilePages) S.pid[stage][lane] = pid;
        const int live = __popc(__ballot_sync(0xffffffffu, pid >= 0));
        if (lane == 0) S.whole[stage] = live == kTilePages && n_tok >= kPage * ((t0 + k + 1) * kTilePages);
        __syncwarp();
        if (lane == 0) {
          if (live) bar_expect(&S.page_full[stage], (uint32_t)(live * pb));
          else bar_arrive(&S.page_full[stage]);
        }
        __syncwarp();
        if (pid >= 0)
          bulk_load(stages + (size_t)(stage * kTilePages + lane) * pb, P.pages + ((size_t)pid * P.hkv + h) * pb, (uint32_t)pb,
                    &S.page_full[stage]);
      }
      if (*gave_up)                                         // copies in flight land before the CTA can end
#pragma unroll 1
        for (int j = max(0, k - kStages); j < k; ++j) settle(&S.page_full[j % kStages], j / kStages);
    } else if (warp == kSeenWarp) {
      // ---- ancestors of every node by doubling (four nodes a lane); parents checked
      constexpr int kPer = kNodes / 32;
      int up[kPer];
      uint32_t mine[kPer][kNodeWords];
#pragma unroll
      for (int x = 0; x < kPer; ++x) {
        const int i = lane + 32 * x;
        up[x] = -1;
        if (i < st.n) {
          up[x] = P.parent[st.first + i];
          if (up[x] >= i || up[x] < -1) {
            set_status(P.status, KVQ_ERR_BOUNDS);
            up[x] = -1;
          }
        }
#pragma unroll
        for (int w = 0; w < kNodeWords; ++w) mine[x][w] = x == w ? 1u << lane : 0u;
      }
      // after round r: the 2^r nearest ancestors (itself counted), and where the next one is
#pragma unroll 1
      for (int r = 0;; ++r) {
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
          *reinterpret_cast<uint4*>(S.seen[lane + 32 * x]) = make_uint4(mine[x][0], mine[x][1], mine[x][2], mine[x][3]);
          S.jump[lane + 32 * x] = up[x];
        }
        __syncwarp();
        if ((1 << r) >= kNodes) break;
        int next[kPer];
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
          next[x] = -1;
          if (up[x] >= 0) {
            const uint4 v = *reinterpret_cast<const uint4*>(S.seen[up[x]]);
            mine[x][0] |= v.x; mine[x][1] |= v.y; mine[x][2] |= v.z; mine[x][3] |= v.w;
            next[x] = S.jump[up[x]];
          }
        }
        __syncwarp();
#pragma unroll
        for (int x = 0; x < kPer; ++x) up[x] = next[x];
      }
      if (lane == 0) bar_arrive(&S.seen_full);
    } else if (warp == kQkWarp) {
      // ---- S(i) = K(i) q', one buffer after the other.  (The two products are issued by two warps: a
      // wait and eight issues are a few hundred clocks each, which one warp would take in turn)
      const uint64_t q_d = desc_k128(saddr(sm + L::kQ));
      bool ok = warp_wait(&S.q_full, 0, gave_up);
      int i = 0;
#pragma unroll 1
      for (; ok && i < nt; ++i) {
        if (i > 1) ok = warp_wait(&S.s_free[i & 1], (i >> 1) - 1, gave_up);
        ok = ok && warp_wait(&S.k_full[i & 1], i >> 1, gave_up);
        if (!ok) break;
        fence_after();
        const uint32_t ts = tb + kColS + N * (i & 1);
        if (i >= npt) {
          const uint64_t k_d = desc_k128(saddr(sm + L::kK)), qb_d = desc_k128(saddr(sm + L::kQb));
#pragma unroll 1
          for (int s = 0; s < 8; ++s)
            if (elect())
              mma_ss(ts, k_d + (((s >> 2) * kSlab + (s & 3) * 32) >> 4), qb_d + (((s >> 2) * N * 128 + (s & 3) * 32) >> 4),
                     kIdescB16, s > 0);
        } else {
          const uint32_t ka = tb + kColK + kKCols * (i & 1);
          const uint64_t za = desc_plain(saddr(sm + L::kZa + (i & 1) * kTile * 32), kTile * 16);
          if (elect()) {
#pragma unroll 2
            for (int s = 0; s < 8; ++s) {
              const uint64_t qs = q_d + (((s >> 2) * N * 128 + (s & 3) * 32) >> 4);
              mma_ts(ts, ka + 8 * s, qs, kIdescF16, s > 0);
              if (NG > 1) mma_ts(ts, ka + 64 + 8 * s, qs, kIdescF16, 1u);
            }
            mma_ss(ts, za, desc_plain(saddr(sm + L::kZ), N * 16), kIdescF16, 1u);
          }
        }
        __syncwarp();
        if (elect()) mma_commit(&S.s_full[i & 1]);
        __syncwarp();
      }
      if (!ok && i > 0) settle(&S.s_full[(i - 1) & 1], (i - 1) >> 1);   // what was issued ends before TMEM is given back
    } else if (warp == kPvWarp) {
      // ---- O += V(i) P(i)
      const uint64_t p_d = desc_mn128(saddr(sm + L::kP));
      bool ok = true;
      int i = 0;
#pragma unroll 1
      for (; i < nt; ++i) {
        ok = warp_wait(&S.v_full[i & 1], i >> 1, gave_up) && warp_wait(&S.p_full[i & 1], i >> 1, gave_up);
        if (!ok) break;
        fence_after();
        if (i >= npt) {
          const uint64_t v_d = desc_mn128(saddr(sm + L::kV));
#pragma unroll 1
          for (int kk = 0; kk < 8; ++kk)
            if (elect()) {
              mma_ss(tb + kColO, v_d + kk * (2048 >> 4), p_d + kk * (2048 >> 4), kIdescB16PV, i > 0 || kk > 0);
              mma_ss(tb + kColO, v_d + kk * (2048 >> 4), p_d + ((L::kPBytes + kk * 2048) >> 4), kIdescB16PV, 1u);
            }
        } else {
          const uint64_t p = p_d + (uint64_t)((i & 1) * (L::kPBytes >> 4));
          const uint32_t v = tb + kColV + (kVBufs == 2 ? 64 * (i & 1) : 0);
          if (elect()) {
#pragma unroll 2
            for (int kk = 0; kk < 8; ++kk) mma_ts(tb + kColO, v + 8 * kk, p + kk * (2048 >> 4), kIdescPV, i > 0 || kk > 0);
          }
        }
        __syncwarp();
        if (elect()) mma_commit(&S.pv_done[i & 1]);
        __syncwarp();
      }
      if (!ok && i > 0) settle(&S.pv_done[(i - 1) & 1], (i - 1) >> 1);
    }
  } else if (warp >= kKeyWarp) {
    if (warp < kValWarp) regs_dec<kRegsKeys>();
    else regs_dec<kRegsValues>();
    // ---- operands of a tile, lane quadrant q of TMEM.  Window tiles: the threads copy the rows into
    // swizzled shared memory, 16 lanes a row
    const bool keys = warp < kValWarp;
    const int q = warp & 3, t = tid - 32 * (keys ? kKeyWarp : kValWarp);
    const int row = lane >> 2, quad = lane & 3;
    const uint32_t tq = tb + ((uint32_t)(32 * q) << 16);
    bool ok = true;
    // products up to tile `last` are done, QK's for keys, PV's for values; waited for one after the other (a
    // parity alone says nothing about a phase whose predecessor may not be over)
    int seen_products = 0;
    auto products = [&](int last) {
      for (; ok && seen_products <= last; ++seen_products)
        ok = warp_wait(keys ? &S.s_full[seen_products & 1] : &S.pv_done[seen_products & 1], seen_products >> 1, gave_up);
    };
    if (keys) {
      // ---- keys: tokens 32 q .. 32 q + 31 of a tile, pages 2 q and 2 q + 1
      for (int i = 0; i < npt; ++i) {
        const int stage = i % kStages;
        const int page0 = (t0 + i) * kTilePages;
        ok = warp_wait(&S.page_full[stage], i / kStages, gave_up);
        products(i - kKBufs);
        if (!ok) break;
        fence_after();
        const uint8_t* base = stages + (size_t)stage * kTilePages * pb;
        const uint32_t tk = tq + kColK + kKCols * (i & 1);
#pragma unroll 1
        for (int j = 0; j < 2; ++j) {
          const int pg = 2 * q + j;
          const uint8_t* pgp = base + (size_t)pg * pb;
          const int valid = S.pid[stage][pg] < 0 ? 0 : max(0, min(kPage, n_tok - kPage * (page0 + pg)));
          if (lane == 0) S.alive[i & 3][pg] = (uint16_t)((1u << valid) - 1u);
          const uint32_t ta = tk + ((uint32_t)(16 * j) << 16);
          // (a page that is not there leaves whatever the stage holds: its tokens are masked)
          const uint4 w = lds16(pgp + 16 * lane);
          const uint32_t kw[4] = {w.x, w.y, w.z, w.w};
          const uint32_t kw10[4] = {w.x >> 10, w.y >> 10, w.z >> 10, w.w >> 10};
          const uint8_t* sc = pgp + k_scale_off();
          float ls[2];
          // slots 2 quad, 2 quad + 1 and 8 + 2 quad, 9 + 2 quad of tokens row, row + 8 (z[0 .. 1], z[2 .. 3])
          auto put_zero = [&](const uint32_t (&z)[4]) {
            uint8_t* to = sm + L::kZa + (i & 1) * kTile * 32 + 2 * pg * 128 + row * 16 + quad * 4;
#pragma unroll
            for (int x = 0; x < 4; ++x) *reinterpret_cast<uint32_t*>(to + (x & 1) * 128 + (x >> 1) * kTile * 16) = z[x];
          };
          if constexpr (NG == 1) {
            uint32_t z[4];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const __half2 dz = bits2h(*reinterpret_cast<const uint32_t*>(sc + 4 * (row + 8 * x)));
              ls[x] = __low2float(dz);
              const uint32_t zz = quad == 0 ? (uint32_t)__half_as_ushort(__hmul(__high2half(dz), __float2half_rn(0.03125f))) : 0u;
              z[x] = zz;
              z[2 + x] = zz;
            }
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              uint32_t v[16];
#pragma unroll
              for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int r = 0; r < 4; ++r) v[4 * s + r] = code_pair(kw[r], kw10[r], 4 * hf + s);
              tm_st_frag8(ta + 32 * hf, v);
            }
            put_zero(z);
          } else {
            uint32_t d2[2][NG];                             // Delta 2^k of both tokens, twice in a register
            uint32_t z[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint32_t dz[NG];
              load_scales<NG>(sc + 4 * NG * (row + 8 * x), dz);
              // (the quad's lanes have a group each)
              const float2 f = __half22float2(bits2h(*reinterpret_cast<const uint32_t*>(sc + 4 * NG * (row + 8 * x) + 4 * (quad & (NG - 1)))));
              float top = fmaxf(4.f * f.x, fabsf(f.x * f.y));
#pragma unroll
              for (int o = 1; o < NG; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
              // 2^k: the largest of 4 Delta 2^k and |Delta z| 2^k (z16 may be anything up to 65504, in keys far from 0)
              // in [2^14, 2^15).  A pair hi + lo of c Delta 2^k has 13 bits and fp16 ends at 2^-24: it is exact for
              // groups down to 2^-25 of the largest
              const int e = (int)(__float_as_uint(top) >> 23) - 127;
              const int kx = top > 0.f && top < INFINITY ? 14 - e : 0;
              const float up = __int_as_float((kx + 127) << 23);
              ls[x] = __int_as_float((127 - kx) << 23);
#pragma unroll
              for (int g = 0; g < NG; ++g) d2[x][g] = h2bits(__float2half2_rn(__low2float(bits2h(dz[g])) * up));
              const float prod = f.x * up * f.y;            // (11 + 11 bits: exact)
              const float hi = __half2float(__float2half_rn(prod));
              if (quad < NG) {
                z[x] = pack16(hi, prod - hi);
                z[2 + x] = pack16(hi, 0.f);
              }
            }
            put_zero(z);
#pragma unroll
            for (int s0 = 0; s0 < 8; s0 += 2) {
              uint32_t hi[8], lo[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                // 2^(10 - 2 sp) + c, then c, then Delta 2^k c
                const int s = s0 + (k >> 2), r = k & 3, sp = slot_pow(s);
                const uint32_t one = (uint32_t)(25 - 2 * sp) * 0x04000400u, d = d2[r & 1][s * NG / 8];
                const __half2 c = __hsub2(bits2h(code_pair(kw[r], kw10[r], s) | one), bits2h(one));
                hi[k] = h2bits(__hmul2(c, bits2h(d)));
                lo[k] = h2bits(__hfma2(c, bits2h(d), __hneg2(bits2h(hi[k]))));
              }
              tm_st_frag4(ta + 8 * s0, hi);
              tm_st_frag4(ta + 64 + 8 * s0, lo);
            }
          }
          if (P.l2) {
            const __half* nm = reinterpret_cast<const __half*>(pgp + norm_off(NG, 0));
            ls[0] *= __half2float(nm[row]);
            ls[1] *= __half2float(nm[row + 8]);
          }
          if (quad == 0) {
            S.lane_scale[i & 3][16 * pg + row] = ls[0];
            S.lane_scale[i & 3][16 * pg + row + 8] = ls[1];
          }
        }
        wait_st();
        fence_before();
        fence_async();
        __syncwarp();
        if (lane == 0) {
          bar_arrive(&S.k_full[i & 1]);
          bar_arrive(&S.page_free[stage]);
        }
      }
    } else {
      // ---- values: channels 32 q .. 32 q + 31 of four pages; slots m = 2 q, 2 q + 1 of the words
      const int vg = 32 * q / (kHeadDim / NG);              // the group of these channels
      const int pages = (warp - kValWarp) >> 2;             // this warp's pages: 4 of the 8
      // slots m = 2 q, 2 q + 1 of the words
      uint32_t mask[2], one[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int sp = slot_pow(2 * q + j);
        mask[j] = 0x00030003u << (2 * sp);
        one[j] = (uint32_t)(25 - 2 * sp) * 0x04000400u;     // 2^(10 - 2 sp): the code's bits then count ones
      }
#pragma unroll 1
      for (int i = 0; i < npt; ++i) {
        const int stage = i % kStages;
        ok = warp_wait(&S.page_full[stage], i / kStages, gave_up);
        products(i - kVBufs);
        if (!ok) break;
        fence_after();
        const uint8_t* pgp = stages + (size_t)(stage * kTilePages + 4 * pages) * pb;
        uint32_t tv = tq + kColV + (kVBufs == 2 ? 64 * (i & 1) : 0) + 32 * pages;
        const bool whole = S.whole[stage];
        // (rolled: the roles' loops together have to stay in the instruction cache)
#pragma unroll 1
        for (int pg = 0; pg < 4; ++pg, pgp += pb, tv += 8) {
          const uint4 w = lds16(pgp + kCodeBytes + 16 * lane);
          const uint8_t* dp = pgp + v_delta_off(NG, 2 * quad, vg);
          uint32_t d[2], z[2];
          d[0] = *reinterpret_cast<const uint32_t*>(dp);
          d[1] = *reinterpret_cast<const uint32_t*>(dp + 16 * NG);
          z[0] = *reinterpret_cast<const uint32_t*>(dp + 32 * NG);
          z[1] = *reinterpret_cast<const uint32_t*>(dp + 48 * NG);
          uint32_t vw[2][4] = {{w.x, w.y, w.z, w.w}, {w.x, w.y, w.z, w.w}};
          if (q >= 2) {                                     // slots from 5 on stand 10 bits up
#pragma unroll
            for (int r = 0; r < 4; ++r) vw[1][r] >>= 10;
            if (q == 3) {
#pragma unroll
              for (int r = 0; r < 4; ++r) vw[0][r] = vw[1][r];
            }
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) z[y] = h2bits(__hmul2(bits2h(d[y]), bits2h(z[y] ^ 0x80008000u)));
          uint32_t a[2][4];
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              // 2^(10 - 2 sp) + c, then c (exact), then Delta c - Delta z
              const __half2 c = __hsub2(bits2h((vw[j][r] & mask[j]) | one[j]), bits2h(one[j]));
              a[j][r] = h2bits(__hfma2(c, bits2h(d[r >> 1]), bits2h(z[r >> 1])));
            }
          if (!whole) {                                     // dead tokens: zeros, whatever the page holds there
            const int at = 4 * pages + pg;
            const int valid = S.pid[stage][at] < 0 ? 0 : max(0, min(kPage, n_tok - kPage * ((t0 + i) * kTilePages + at)));
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int tk = 2 * quad + 8 * y;
              const uint32_t m2 = (tk < valid ? 0xffffu : 0u) | (tk + 1 < valid ? 0xffff0000u : 0u);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                a[j][2 * y] &= m2;
                a[j][2 * y + 1] &= m2;
              }
            }
          }
          tm_st_frag2(tv, a[0]);
          tm_st_frag2(tv + (16u << 16), a[1]);
        }
        wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) {
          bar_arrive(&S.v_full[i & 1]);
          bar_arrive(&S.page_free[stage]);
        }
      }
    }
    // ---- window tiles: the rows take the page stages' space, once every warp has read the last pages
    for (int k = max(0, npt - kStages); ok && nt > npt && k < npt; ++k) ok = warp_wait(&S.page_free[k % kStages], k / kStages, gave_up);
#pragma unroll 1
    for (int i = npt; ok && i < nt; ++i) {
      const int w0 = (t0 + i - ni) * kTile;
      // keys once QK(i - 1) has read the last window rows, values once PV(i - 1) has
      products(i > npt ? i - 1 : i - 2);
      if (!ok) break;
      const uint16_t* sink = keys ? P.sink_k : P.sink_v;
      const uint16_t* ring = keys ? P.ring_k : P.ring_v;
      uint8_t* dst = sm + (keys ? L::kK : L::kV);
      const int j = t & 15;
#pragma unroll 1
      for (int r = t >> 4; r < kTile; r += 2 * (keys ? kKeyWarps : kValWarps)) {
        const int w = min(w0 + r, n_win - 1);
        const int tok = w < n_sink ? w : ring0 + w - n_sink;
        const uint16_t* src = w < n_sink ? sink + (((size_t)b * P.hkv + h) * P.s_sink + tok) * kHeadDim
                                         : ring + (((size_t)b * P.hkv + h) * P.ring_cap + tok % P.ring_cap) * kHeadDim;
        // (zeros for rows behind the last: 0 bytes are read)
        async_copy16(dst + (j >> 3) * kSlab + (r >> 3) * 1024 + (r & 7) * 128 + (((j & 7) ^ (r & 7)) << 4), src + 8 * j,
                     w0 + r < n_win ? 16 : 0);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (!keys && (n_sink > st.L0 || w0 + kTile > n_win - st.n)) {
        // drafts: a value row that is not finite is taken out here (0 x NaN would reach rows that do not see
        // it) and the softmax makes the rows that see it NaN
#pragma unroll 1
        for (int r = t >> 4; r < kTile; r += 2 * kValWarps) {
          uint4* at = reinterpret_cast<uint4*>(dst + (j >> 3) * kSlab + (r >> 3) * 1024 + (r & 7) * 128 + (((j & 7) ^ (r & 7)) << 4));
          const uint4 v = *at;
          const int tok = w0 + r < n_sink ? w0 + r : ring0 + w0 + r - n_sink;
          const bool inf = tok >= st.L0 && (bf16_pair_odd(v.x) || bf16_pair_odd(v.y) || bf16_pair_odd(v.z) || bf16_pair_odd(v.w));
          const bool any = (__ballot_sync(0xffffffffu, inf) >> (lane & 16)) & 0xffffu;
          if (any) *at = make_uint4(0u, 0u, 0u, 0u);
          if (j == 0) S.v_odd[i & 1][r] = any;
        }
      }
      if (keys) {
        S.lane_scale[i & 3][t] = 1.f;
        const unsigned alive = __ballot_sync(0xffffffffu, w0 + t < n_win);
        if (lane == 0) {
          S.alive[i & 3][2 * q] = (uint16_t)alive;
          S.alive[i & 3][2 * q + 1] = (uint16_t)(alive >> 16);
        }
      }
      fence_async();
      __syncwarp();
      if (lane == 0) bar_arrive(keys ? &S.k_full[i & 1] : &S.v_full[i & 1]);
    }
  } else {
    regs_inc<kRegsSoftmax>();
    // ---- softmax: token 32 q + lane of every tile, rows kCols share ..
    const int q = warp & 3, share = warp >> 2;
    const uint32_t tq = tb + ((uint32_t)(32 * q) << 16);
    const int c0 = share * kCols, tok = 32 * q + lane;
    // q' operands first (these threads): bf16 rows, 16-byte chunk j of row c in slab j / 8, swizzled
    auto at = [&](int c, int j) { return (j >> 3) * N * 128 + (c >> 3) * 1024 + (c & 7) * 128 + (((j & 7) ^ (c & 7)) << 4); };
    {
      if (tid < N) {
        const int r = row0 + tid;
        S.row[tid] = (st.first + (r >> P.gqa_log2)) * (P.hkv * P.gqa) + h * P.gqa + (r & (P.gqa - 1));
        S.neg_m[tid] = 0.f;
      }
      softmax_sync();
      // 16 lanes a row: bf16 as it is, for the windows; fp16 times a power of two of the row, with one group
      // channel slot s by 4^-s too, for the codes that carry 4^s 2^-24
#pragma unroll 1
      for (int i = tid; i < N * 16; i += 32 * kSmWarps) {
        const int c = i >> 4, j = i & 15;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (c < ncol) v = reinterpret_cast<const uint4*>(P.q + (size_t)S.row[c] * kHeadDim)[j];
        *reinterpret_cast<uint4*>(sm + L::kQb + at(c, j)) = v;
        // (the largest magnitude: bf16 patterns without the sign compare as integers)
        const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
        uint32_t top = max(m << 16, m & 0xffff0000u);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        // amax 2^sigma < 2^14, or 2^9, so that sums of groups stay in range (a row that is not finite stays so)
        const int sigma = top > 0u && top < 0x7f800000u ? min(100, (NG == 1 ? 14 : 9) - ((int)(top >> 23) - 126)) : 0;
        if (j == 0) {
          S.sigma[c] = sigma;
          S.mul[0][c] = P.scale_log2 * ldexpf(1.f, (NG == 1 ? 24 : 0) - sigma);
          S.mul[1][c] = P.scale_log2;
        }
        const float f = __int_as_float((sigma - (NG == 1 ? 2 * slot_pow(j >> 1) : 0) + 127) << 23);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = pack16(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xffff0000u) * f);
        *reinterpret_cast<uint4*>(sm + L::kQ + at(c, j)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
      softmax_sync();
      // zero-point operand, row c: slots 2 g, 2 g + 1: -sum of group g (hi), slot 8 + 2 g: its lo.  Four
      // threads a row, 32 channels each
      if (tid < 4 * N) {
        const int c = tid >> 2, part = tid & 3, sigma = S.sigma[c];
        float acc = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 v = lds16(sm + L::kQb + at(c, 4 * part + j));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) acc += __uint_as_float(w[k] << 16) + __uint_as_float(w[k] & 0xffff0000u);
        }
        if (NG <= 2) acc += __shfl_xor_sync(0xffffffffu, acc, 1);
        if (NG == 1) acc += __shfl_xor_sync(0xffffffffu, acc, 2);
        const float from = __shfl_sync(0xffffffffu, acc, (lane & ~3) + (part * (4 / NG) & 3));   // slot pair `part`: group part
        const float v = part < NG ? -from * ldexpf(1.f, NG == 1 ? sigma - 19 : sigma) : 0.f;
        const float hi = __half2float(__float2half_rn(v));
        uint8_t* to = sm + L::kZ + (c >> 3) * 128 + (c & 7) * 16 + 4 * part;
        *reinterpret_cast<uint32_t*>(to) = pack16(hi, hi);
        *reinterpret_cast<uint32_t*>(to + N * 16) = pack16(v - hi, 0.f);
      }
      fence_async();
      __syncwarp();
      if (lane == 0) bar_arrive(&S.q_full);
    }
    float l[kCols];
#pragma unroll
    for (int j = 0; j < kCols; ++j) l[j] = 0.f;
    bool lost = false;
    bool unseen = true;                                     // row c0 + lane % kCols has seen no token yet
    bool force = true;                                      // ... there are such rows (all four warps agree)
    int meets = 0, pv_seen = 0;
    auto pv_until = [&](int last) {                         // products with V up to tile `last` are done
      for (; pv_seen <= last; ++pv_seen)
        if (!warp_wait(&S.pv_done[pv_seen & 1], pv_seen >> 1, gave_up)) lost = true;
    };
    // the share's four warps meet (bounded, so that a warp that gave up leaves nobody behind)
    auto meet = [&]() {
      __syncwarp();
      if (lane == 0) bar_arrive(&S.meet[share]);
      if (!warp_wait(&S.meet[share], meets++, gave_up)) lost = true;
    };
#pragma unroll 1
    for (int i = 0; i < nt && !lost; ++i) {
      if (!warp_wait(&S.s_full[i & 1], i >> 1, gave_up)) {
        lost = true;
        break;
      }
      fence_after();
      const uint32_t ts = tq + kColS + N * (i & 1);
      const bool win = i >= npt;
      float ls = S.lane_scale[i & 3][tok];
      const float* mul = S.mul[win] + c0;                   // the rows' factors
      const uint32_t alive = *reinterpret_cast<const uint32_t*>(&S.alive[i & 3][2 * q]);
      // window tiles that reach into the drafts: else every row sees every token
      const bool drafts = win && (n_sink > st.L0 || (t0 + i - ni + 1) * kTile > n_win - st.n);
      const bool masked = drafts || alive != 0xffffffffu;
      uint32_t see = 0xffffffffu;                           // rows that see this token
      if (masked) {
        if (drafts) {
          pv_until(i - 2);                                  // (and so V(i - 2) has been there: see products())
          if (!warp_wait(&S.seen_full, 0, gave_up) || !warp_wait(&S.v_full[i & 1], i >> 1, gave_up)) lost = true;
          if (S.v_odd[i & 1][tok]) ls = __int_as_float(0x7fffffff);   // (see where the values are loaded)
        }
        const int w = (t0 + i - ni) * kTile + tok;
        const int node = win ? (w < n_sink ? w : ring0 + w - n_sink) - st.L0 : -1;
        see = (alive >> lane) & 1u ? 0xffffffffu : 0u;
        if (see && drafts && node >= 0) {
          see = 0u;
          const int wd = (node >> 5) & (kNodeWords - 1);
#pragma unroll 1
          for (int j = 0; j < kCols; ++j)
            see |= ((S.seen[min((row0 + c0 + j) >> P.gqa_log2, kNodes - 1)][wd] >> (node & 31)) & 1u) << j;
        }
      }
      float x[kCols];
      bool moved = false;
#pragma unroll 1
      for (;;) {
        tm_ld16(ts + c0, x);
        // scores less the reference
#pragma unroll
        for (int j = 0; j < kCols; j += 4) {
          const float4 m = *reinterpret_cast<const float4*>(&S.neg_m[c0 + j]), f = *reinterpret_cast<const float4*>(mul + j);
          scale2(x[j], x[j + 1], ls, f.x, f.y, m.x, m.y);
          scale2(x[j + 2], x[j + 3], ls, f.z, f.w, m.z, m.w);
        }
        if (masked) {
#pragma unroll
          for (int j = 0; j < kCols; ++j) x[j] = (see >> j) & 1u ? x[j] : -INFINITY;
        }
        if (!moved) {
          float mx[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = max3(x[e], x[4 + e], x[8 + e]);
#pragma unroll
          for (int j = 12; j + 8 <= kCols; j += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], x[j + e], x[j + 4 + e]);
          // (kCols is 4 past a multiple of 8 from 12 on: the last four)
          const bool over = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], x[kCols - 4], x[kCols - 3]),
                                 fmaxf(x[kCols - 2], x[kCols - 1])) > (win ? kWinSlack : kRefSlack);
          // one vote of the four warps, taken while the exponentials are already formed
          const bool any = __any_sync(0xffffffffu, over) || force;
          if (lane == 0) {
            if (any) *(volatile int*)&S.moves[share] = i + 1;
            bar_arrive(&S.vote[share]);
          }
        }
#pragma unroll
        for (int j = 0; j < kCols / 2; ++j) x[j] = ex2(x[j]);
        if (moved) break;
        if (!warp_wait(&S.vote[share], i, gave_up)) {
          lost = true;
          break;
        }
        if (*(volatile int*)&S.moves[share] != i + 1) break;
        // ---- the references move to the rows' maxima so far
        moved = true;
#pragma unroll 1
        for (int j = 0; j < kCols; j += 8) {
          float y[8];
          tm_ld8(ts + c0 + j, y);
          const uint32_t bits = see >> j;
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = (bits >> e) & 1u ? y[e] * ls * mul[j + e] : -INFINITY;
          const float top = reduce_columns(y, lane, [](float a, float b2) { return fmaxf(a, b2); });
          if (lane < 8) S.red[q][c0 + j + lane] = top;
        }
        meet();
        const int c = c0 + lane % kCols;
        const float up = fmaxf(fmaxf(S.red[0][c], S.red[1][c]), fmaxf(S.red[2][c], S.red[3][c]));
        const float low = fminf(fminf(S.red[0][c], S.red[1][c]), fminf(S.red[2][c], S.red[3][c]));
        // a first token sets the reference, later ones only raise it; how far below the maximum: see the
        // head of this file
        const bool any = up > -INFINITY;
        const float ref = up - fminf(fmaxf(up - low - kRefLead, 0.f), kRefBelow);
        const float old = -S.neg_m[c], now = unseen ? (any ? ref : 0.f) : fmaxf(old, ref);
        if (q == 0) S.alpha[c] = unseen ? 0.f : ex2(old - now);
        if (any) unseen = false;
        force = __any_sync(0xffffffffu, unseen);
        meet();                                             // (everyone has read the old references)
        if (q == 0) S.neg_m[c] = -now;
#pragma unroll
        for (int j = 0; j < kCols; j += 4) {
          const float4 al = *reinterpret_cast<const float4*>(&S.alpha[c0 + j]);
          l[j] *= al.x;
          l[j + 1] *= al.y;
          l[j + 2] *= al.z;
          l[j + 3] *= al.w;
        }
        if (i > 0) {                                        // O so far, once PV(i - 1) is done
          if (!warp_wait(&S.pv_done[(i - 1) & 1], (i - 1) >> 1, gave_up)) lost = true;
          fence_after();
#pragma unroll 1
          for (int j = 0; j < kCols; j += 8) {
            float o[8];
            tm_ld8(tq + kColO + c0 + j, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] *= S.alpha[c0 + j + e];
            tm_st8(tq + kColO + c0 + j, o);
          }
          wait_st();
        }
        meet();                                             // (the new references are there)
      }
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&S.s_free[i & 1]);
      // P buffer free: PV(i - 2), or PV(i - 1) for window tiles (which use both buffers)
      pv_until(win ? i - 1 : i - 2);
      // P[token][row], 8 rows a chunk of 16 bytes: a lane's chunks are 16 (j ^ (token % 8)) apart
      const uint32_t p_s = saddr(sm + L::kP) + (c0 >> 6) * kSlab + (tok >> 3) * 1024 + (tok & 7) * 128;
      const uint32_t sw = (uint32_t)(((c0 & 63) >> 3) ^ (tok & 7)) << 4;
#pragma unroll
      for (int j = kCols / 2; j < kCols; ++j) x[j] = ex2(x[j]);
#pragma unroll
      for (int j = 0; j < kCols; ++j) l[j] += x[j];
      if (!win) {
        const uint32_t to = p_s + (i & 1) * L::kPBytes;
#pragma unroll
        for (int j = 0; j < kCols / 8; ++j)
          sts16(to + (sw ^ (16u * j)), pack16(x[8 * j], x[8 * j + 1]), pack16(x[8 * j + 2], x[8 * j + 3]),
                pack16(x[8 * j + 4], x[8 * j + 5]), pack16(x[8 * j + 6], x[8 * j + 7]));
      } else {
#pragma unroll
        for (int j = 0; j < kCols / 8; ++j) {               // bf16 hi, and what it leaves
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float a0 = x[8 * j + 2 * e], a1 = x[8 * j + 2 * e + 1];
            hi[e] = packb16(a0, a1);
            lo[e] = packb16(a0 - __uint_as_float(hi[e] << 16), a1 - __uint_as_float(hi[e] & 0xffff0000u));
          }
          sts16(p_s + (sw ^ (16u * j)), hi[0], hi[1], hi[2], hi[3]);
          sts16(p_s + L::kPBytes + (sw ^ (16u * j)), lo[0], lo[1], lo[2], lo[3]);
        }
      }
      fence_async();
      __syncwarp();
      if (lane == 0) bar_arrive(&S.p_full[i & 1]);
    }
    // ---- sums over the tokens: every lane's through shared memory (where P was), 16-byte chunks
    // permuted by token; then the rows' results
    if (!lost && nt > 0 && !warp_wait(&S.pv_done[(nt - 1) & 1], (nt - 1) >> 1, gave_up)) lost = true;
    fence_after();
    float* scratch = reinterpret_cast<float*>(sm + L::kP);  // [128 tokens][N]
    constexpr int kChunks = kCols / 4;
#pragma unroll
    for (int j = 0; j < kChunks; ++j)
      *reinterpret_cast<float4*>(scratch + tok * N + c0 + 4 * (j ^ (tok & (kChunks - 1)))) =
          make_float4(l[4 * j], l[4 * j + 1], l[4 * j + 2], l[4 * j + 3]);
    meet();
    {
      const int c = tok & (kCols - 1), part = tok / kCols;  // kCols tokens each
      float sum = 0.f;
#pragma unroll 2
      for (int t = part * kCols; t < (part + 1) * kCols; ++t)
        sum += scratch[t * N + c0 + 4 * ((c >> 2) ^ (t & (kChunks - 1))) + (c & 3)];
      S.red[part][c0 + c] = sum;
    }
    meet();
    if (!lost) {
      // every thread: one channel of the share's rows, 8 rows at a time
      const int c = c0 + lane % kCols;
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < kTile / kCols; ++k) sum += S.red[k][c];
      // 1 / l; a row that saw nothing gives 0, one whose sum is no number that
      const float by = P.splits > 1 ? 1.f : sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;
      const float top = sum != 0.f ? -S.neg_m[c] : -1e30f;
      if (P.splits > 1 && q == 0 && lane < kCols && c < ncol)
        *reinterpret_cast<float2*>(P.part + ((size_t)S.row[c] * P.splits + split) * kRec) = make_float2(top, sum);
      const unsigned finite = __ballot_sync(0xffffffffu, fabsf(sum) < INFINITY);
      bool beyond = false;                                  // weights that are numbers, and a sum that is none
#pragma unroll 1
      for (int j = 0; j < kCols && c0 + j < ncol; j += 8) {
        float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (nt > 0) tm_ld8(tq + kColO + c0 + j, o);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = o[e] * __shfl_sync(0xffffffffu, by, j + e);
          const size_t r = (size_t)S.row[c0 + j + e];
          if (c0 + j + e < ncol) {
            beyond |= ((finite >> (j + e)) & 1u) && !(fabsf(o[e]) < INFINITY);
            if (P.splits == 1) P.out[r * kHeadDim + tok] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
            else P.part[(r * P.splits + split) * kRec + 4 + tok] = v;
          }
        }
      }
      if (beyond) set_status(P.status, KVQ_ERR_NONFINITE);  // (a value beyond fp16's 65504, or not finite)
    }
  }
  fence_before();
  __syncthreads();
  if (tid == 0 && *gave_up) set_status(P.status, KVQ_ERR_TIMEOUT);
  if (warp == 0) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tb), "r"(kTmem));
  }
}

// One warp per (row, query head): the splits' partials into the output.
constexpr int kMThreads = 256;
__global__ void __launch_bounds__(kMThreads) attn_tree_merge_kernel(const __grid_constant__ TreeParams P) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int hq = P.hkv * P.gqa;
  const long long r = (long long)blockIdx.x * (kMThreads / 32) + (threadIdx.x >> 5);
  if (r >= (long long)P.n_rows * hq) return;
  const int row = (int)(r / hq);
  if (row < P.cu_rows[0] || row >= P.cu_rows[P.batch]) return;         // a row that no sequence has
  int lo = 0, hi = P.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (P.cu_rows[mid] <= row) lo = mid;
    else hi = mid - 1;
  }
  const SeqState st = seq_state(P, lo);
  float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
  if (!st.bad) {
    const float* rec = P.part + (size_t)r * P.splits * kRec;
    float M = -INFINITY;
    for (int s = lane; s < P.splits; s += 32) M = fmaxf(M, __ldcg(rec + (size_t)s * kRec));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float sum = 0.f;
    for (int s0 = 0; s0 < P.splits; s0 += 8) {
      float m[8], l[8];
      float4 o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (s0 + i < P.splits) {
          const float* p = rec + (size_t)(s0 + i) * kRec;
          m[i] = __ldcg(p);
          l[i] = __ldcg(p + 1);
          o[i] = __ldcg(reinterpret_cast<const float4*>(p + 4) + lane);
        }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (s0 + i < P.splits) {
          const float f = exp2f(m[i] - M);
          sum += l[i] * f;
          O.x += o[i].x * f; O.y += o[i].y * f; O.z += o[i].z * f; O.w += o[i].w * f;
        }
    }
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
    O.x *= inv; O.y *= inv; O.z *= inv; O.w *= inv;
  }
  reinterpret_cast<uint2*>(P.out + (size_t)r * kHeadDim)[lane] = make_uint2(packb16(O.x, O.y), packb16(O.z, O.w));
}

// Row tiles and splits of a call, from its sizes alone.
struct Shape {
  int splits, items;
};
// Tiles of the longest sequence there may be, and CTAs of one split: about as many as the row tiles there will be
// (a sequence's last one is half empty on average).  Both grow with n_rows and max_ctx.
long long tree_tiles(const kvq_config* cfg, int32_t max_ctx) {
  const long long pages = max(0LL, min((long long)cfg->max_pages_per_seq, ((long long)max_ctx - cfg->s_sink + kPage - 1) / kPage));
  const long long win = min((long long)cfg->s_sink + cfg->s_keep + cfg->s_flush + kNodes, (long long)max_ctx);
  return max(1LL, (pages + kTilePages - 1) / kTilePages + (win + kTile - 1) / kTile);
}
int tree_items(const kvq_config* cfg, int32_t n_rows) {
  const long long g = cfg->n_q_heads / cfg->n_kv_heads;
  return (int)min((long long)n_rows, n_rows * g / N + cfg->batch);
}
long long tree_units(const kvq_config* cfg, int32_t n_rows) {
  const long long g = cfg->n_q_heads / cfg->n_kv_heads, per_seq = (n_rows * g + cfg->batch - 1) / cfg->batch;
  return max(1LL, min((long long)tree_items(cfg, n_rows), (per_seq + N - 1) / N * min((long long)cfg->batch, (long long)n_rows))) *
         cfg->n_kv_heads;
}
// CTAs that splits may make of so many: 12 waves, or 24 of more than one wave.  (So that the workspace has a bound.
// Without it 2% of the sizes would take other splits, estimated to be up to 6% faster.)
long long most_ctas(long long units) { return (long long)kSms * (units <= kSms ? 12 : 24); }
Shape tree_shape(const kvq_config* cfg, int32_t n_rows, int32_t max_ctx) {
  Shape s;
  s.items = tree_items(cfg, n_rows);
  const long long tiles = tree_tiles(cfg, max_ctx), units = tree_units(cfg, n_rows);
  // a wave of 152 CTAs takes tiles / splits, and about 6 tiles' time for set-up and merge
  double best = 1e300;
  s.splits = 1;
  for (int k = 1; k <= kMostSplits && k <= tiles && (k == 1 || units * k <= most_ctas(units)); ++k) {
    const double waves = (double)((units * k + kSms - 1) / kSms);
    const double cost = waves * ((double)((tiles + k - 1) / k) + 5.0) + (k > 1 ? 3.0 : 0.0);
    if (cost < best * 0.98) {
      best = cost;
      s.splits = k;
    }
  }
  return s;
}
// Bytes of partials that a call of up to n_rows rows and max_ctx tokens can need.  A split CTA has at most N rows, so
// there are no more partials than N for each of most_ctas(), nor than splits of all rows.
size_t tree_part_bytes(const kvq_config* cfg, int32_t n_rows, int32_t max_ctx) {
  const long long tiles = tree_tiles(cfg, max_ctx), k = min((long long)kMostSplits, tiles);
  if (k <= 1) return 0;
  return (size_t)min((long long)n_rows * cfg->n_q_heads * k, N * most_ctas(tree_units(cfg, n_rows))) * kRec * sizeof(float);
}

}  // namespace
}  // namespace kvq

using namespace kvq;

// Which kernel a call takes, from its sizes alone.  The row kernel (attn.cu) streams a sequence's cache once
// for every 8 (node, head) columns, this one once for every 64 at four to five times the time.  So the row
// kernel has trees of up to 4 groups a tile, the batch's average taken: 64 sequences of 6,000 tokens (groups of 64 /
// 128) take 393 / 373 us there and 409 / 335 us here with 4, 506 / 481 against 410 / 336 with 5.  On short contexts,
// where its windows weigh more, up to 3: 64 sequences of 1,000 tokens take 125 against 130 us with 3, 158 against
// 131 with 4.  It has small calls as well: 16 nodes on 8 kv heads take 15.1 us there and 22.8 us here on 2,000
// tokens, 20.3 and 22.7 on 4,000; 32 nodes 18.8 and 18.7 on 500, 30.7 and 21.7 on 4,000.  Between those it can be off:
// one sequence of 100,000 tokens with 8 nodes of 4 heads takes 93 us there and 71 here with 8 kv heads, 26 and
// 35 with one.  Per-channel keys are the row kernel's alone.
static bool row_kernel(const kvq_config* cfg, int32_t n_rows, int32_t max_ctx) {
  if (cfg->key_axis != KVQ_KEY_PER_TOKEN) return true;
  const long long per_seq = ((long long)n_rows * (cfg->n_q_heads / cfg->n_kv_heads) + cfg->batch - 1) / cfg->batch;
  const long long groups = (per_seq + 7) / 8, tiles = (per_seq + N - 1) / N;
  const long long units = (long long)n_rows * cfg->n_kv_heads;
  return groups <= (max_ctx < 2048 ? 3 : 4) * tiles || (units <= 128 && units * max_ctx <= kSmallCall);
}

// Enough for every call of up to n_rows rows and max_ctx tokens, whichever kernel it takes.
extern "C" size_t kvq_attn_tree_ws_bytes(const kvq_config* cfg, int32_t n_rows, int32_t max_ctx) {
  const size_t rows = kvq_attn_tree_rows_part_bytes(cfg, n_rows, max_ctx);
  const size_t tiles = cfg->key_axis == KVQ_KEY_PER_TOKEN ? tree_part_bytes(cfg, n_rows, max_ctx) : 0;
  return kvq_attn_tree_head_bytes(cfg) + max(rows, tiles);
}

extern "C" int kvq_launch_attn_tree(const kvq_config* cfg, const kvq_cache* cache, const uint16_t* q_rot,
                                    const int32_t* cu_rows, const int32_t* parent, int32_t n_rows, uint16_t* out,
                                    float sm_scale, int32_t max_ctx, void* ws, int32_t* d_status, cudaStream_t stream) {
  if (row_kernel(cfg, n_rows, max_ctx))
    return kvq_launch_attn_tree_rows(cfg, cache, q_rot, cu_rows, parent, n_rows, out, sm_scale, max_ctx, ws, d_status,
                                     stream);
  const Shape s = tree_shape(cfg, n_rows, max_ctx);
  TreeParams P{};
  P.pages = (const uint8_t*)cache->pages;
  P.page_table = cache->page_table;
  P.seq_len = cache->seq_len;
  P.s_quant = cache->s_quant;
  P.sink_k = cache->sink_k;
  P.sink_v = cache->sink_v;
  P.ring_k = cache->ring_k;
  P.ring_v = cache->ring_v;
  P.q = q_rot;
  P.cu_rows = cu_rows;
  P.parent = parent;
  P.out = out;
  P.part = (float*)((char*)ws + kvq_attn_tree_head_bytes(cfg));    // (behind the row kernel's tickets)
  P.status = d_status;
  P.batch = cfg->batch;
  P.hkv = cfg->n_kv_heads;
  P.gqa = cfg->n_q_heads / cfg->n_kv_heads;
  P.gqa_log2 = P.gqa == 8 ? 3 : P.gqa == 4 ? 2 : P.gqa == 2 ? 1 : 0;
  P.s_sink = cfg->s_sink;
  P.ring_cap = cfg->ring_cap;
  P.max_pages = cfg->max_pages_per_seq;
  P.num_pages = cfg->num_pages;
  P.page_bytes = page_head_bytes(cfg->group_size, cfg->key_l2norm, cfg->key_axis);
  P.l2 = cfg->key_l2norm;
  P.n_rows = n_rows;
  P.splits = s.splits;
  P.mp = (int)max(0LL, min((long long)cfg->max_pages_per_seq, ((long long)max_ctx - cfg->s_sink + kPage - 1) / kPage));
  P.scale_log2 = sm_scale * 1.4426950408889634f;
  if (cfg->n_kv_heads > 65535) return KVQ_ERR_UNSUPPORTED;
  const int ng = kHeadDim / cfg->group_size;
  void (*kern)(const TreeParams) = ng == 1 ? attn_tree_kernel<1> : ng == 2 ? attn_tree_kernel<2> : attn_tree_kernel<4>;
  constexpr size_t smem = Layout::kEnd + sizeof(TreeShared);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return KVQ_ERR_CUDA;
  static std::mutex mu;
  static unsigned long long done[3] = {};
  {
    std::lock_guard<std::mutex> lock(mu);
    const int vi = ng == 1 ? 0 : ng == 2 ? 1 : 2;
    if (!(done[vi] & (1ull << dev))) {
      // (the register split counts on what the kernel launches with: a warpgroup would wait for ever)
      cudaFuncAttributes fa;
      if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess || fa.numRegs < kRegsLaunch) return KVQ_ERR_CUDA;
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return KVQ_ERR_CUDA;
      done[vi] |= 1ull << dev;
    }
  }
  if (launch_pdl(kern, dim3(s.items, cfg->n_kv_heads, s.splits), dim3(kThreadsT), smem, stream, P) != cudaSuccess)
    return KVQ_ERR_CUDA;
  if (s.splits > 1) {
    const long long warps = (long long)n_rows * cfg->n_q_heads, per = kMThreads / 32;
    if (launch_pdl(attn_tree_merge_kernel, dim3((unsigned)((warps + per - 1) / per)), dim3(kMThreads), 0, stream, P) != cudaSuccess)
      return KVQ_ERR_CUDA;
  }
  return KVQ_OK;
}
