// What the masked-attention kernels share: the tensor-core forms with an operand in tensor memory, tiles of heads
// loaded by tensor copies, key intervals, and the score function.
#pragma once

#include <cmath>
#include <type_traits>

#include "device_common.cuh"

namespace tpmlp {

constexpr int kTile = 128;                 // query rows and key rows of a tile
constexpr int kBoxBytes = kTile * 128;     // 128 rows x 64 bf16 columns, one 128-byte-swizzled box

// ------------------------------------------------------------------ tcgen05

// Products are issued by a whole warp that stays converged, each instruction under the predicate of one elected lane:
// the descriptors then live in uniform registers and step by constants. (Issued from a branch that only one lane
// takes, with descriptors built per step, a product of 128 x 128 x 16 took 80-125 cycles to issue and 64 to run.)
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t is;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(is));
  return is;
}

__device__ __forceinline__ void umma_bf16_by(uint32_t leader, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]: A's 128 rows are the lanes, two bf16 of K per 32-bit column.
__device__ __forceinline__ void umma_bf16_ta_by(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                                uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}

__device__ __forceinline__ void umma_commit_by(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(leader)
      : "memory");
}

// Whether the phase with this parity has completed. A wait that passes at once still costs a warp 100 cycles; asked this
// way ahead of time, between other work, and then only if the answer was no, it costs next to none.
__device__ __forceinline__ bool mbar_done(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// mbar_wait by polling: for the issuing warp, whose reaction the tensor core waits for. (In the working warps it gained
// nothing over try_wait: 66.0 and 66.4 us when the causal forward took that long.)
__device__ __forceinline__ bool mbar_poll(uint64_t* bar, uint32_t parity, unsigned int* status, unsigned int where) {
  auto done = [&] { return mbar_done(bar, parity); };
  if (done()) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 1024; ++i)
      if (done()) return true;
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      record_timeout(status, where);
      return false;
    }
  }
}

// mbar_wait for the end of work whose length has no bound, as that of a piece with many key tiles: the limit counts from
// the last phase that `stage`, a barrier of the ring through which the work goes, was seen to change to.
__device__ __forceinline__ bool mbar_wait_moving(uint64_t* bar, uint32_t parity, uint64_t* stage, unsigned int* status,
                                                 unsigned int where) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait(a, parity)) return true;
  bool seen = false;
  uint64_t t0 = global_timer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(a, parity)) return true;
    const bool now = mbar_done(stage, 0);
    const uint64_t t = global_timer_ns();
    if (now != seen) {
      seen = now;
      t0 = t;
    } else if (t - t0 > kWaitLimitNs) {
      record_timeout(status, where);
      return false;
    }
  }
}

#define TPMLP_R8(r, o) "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), "r"(r[o + 5]), "r"(r[o + 6]), "r"(r[o + 7])

// 32 lanes x 32 consecutive 32-bit columns: thread i of the warp writes lane (base + i).
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      TPMLP_R8(r, 0), TPMLP_R8(r, 8), TPMLP_R8(r, 16), TPMLP_R8(r, 24)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Moves a warpgroup's share of the block's registers (every warp of the warpgroup calls it; the shares of all
// warpgroups together stay within what the block was launched with).
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// ------------------------------------------------------------------ work

// A kernel's grid has a CTA for every piece of work, but a running CTA takes over the pieces of CTAs that have not
// started (cluster launch control) until none is left, so that a piece's loads begin while the one before it is being
// finished and tensor memory is set up once. One thread asks, for its CTA: returns the piece (a blockIdx.x) or -1, and
// must not ask again after -1. `response` is 16-byte aligned, `bar` an mbarrier of count 1 for this alone.
__device__ __forceinline__ int take_work(uint4* response, uint64_t* bar, uint32_t parity, unsigned int* status,
                                         unsigned int where) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          smem_u32(response)),
      "r"(smem_u32(bar))
      : "memory");
  if (!mbar_wait(bar, parity, status, where)) return -1;
  uint32_t taken, first;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, h;\n\t}"
      : "=r"(taken), "=r"(first)
      : "r"(smem_u32(response))
      : "memory");
  fence_proxy_async_smem();  // the response is read before the next one may be written
  return taken ? static_cast<int>(first) : -1;
}

// ------------------------------------------------------------------ tiles of heads

// Tensor map of one tensor of heads, with the coordinate slots of token, head and sequence.
struct HeadMap {
  CUtensorMap map;
  int row, head, seq;
};

// rows: a copy's, kTile to load tiles, 32 to store a warp's share of one.
inline cudaError_t make_head_map(HeadMap* m, const HeadView& v, int64_t b, int64_t s, int heads, int head_dim,
                                 int rows = kTile) {
  int slots[3];
  const cudaError_t e = make_batched_map(&m->map, BatchedOperand{v.ptr, s, head_dim, v.ld, v.hs, s * v.ld, false}, heads, b,
                                         64, static_cast<uint32_t>(rows), slots);
  m->row = slots[0];
  m->head = slots[1];
  m->seq = slots[2];
  return e;
}

// Loads rows [row, row + 128) of one head (columns [0, 64 * boxes)) into consecutive boxes; rows past the sequence and
// columns past the head are filled with zeros. One thread; completes boxes * kBoxBytes on bar.
__device__ __forceinline__ void load_head_tile(void* dst, const HeadMap& m, uint64_t* bar, int boxes, int row, int head,
                                               int seq) {
  const int c1 = m.row == 1 ? row : (m.head == 1 ? head : seq);
  const int c2 = m.row == 2 ? row : (m.head == 2 ? head : seq);
  const int c3 = m.row == 3 ? row : (m.head == 3 ? head : seq);
  for (int x = 0; x < boxes; ++x)
    tma_load_4d(static_cast<uint8_t*>(dst) + x * kBoxBytes, &m.map, bar, x * 64, c1, c2, c3);
}

// The 16 bytes of columns 8 c .. 8 c + 7 (c < 8) of row r in a box.
__device__ __forceinline__ uint4* box_chunk(uint8_t* box, int r, int c) {
  return reinterpret_cast<uint4*>(box + r * 128 + ((c ^ (r & 7)) << 4));
}
__device__ __forceinline__ const uint4* box_chunk(const uint8_t* box, int r, int c) {
  return reinterpret_cast<const uint4*>(box + r * 128 + ((c ^ (r & 7)) << 4));
}

// Writes 32 rows of an accumulator to a tensor of heads: warp `w` of a tile's four takes lanes 32 w .. 32 w + 31, row
// row0 + 32 w + lane, the columns of boxes [box0, box1), scaled by f (per row) and rounded to bf16; zeros if not live.
// They leave box by box through the warp's own 4 KB at `stage` by tensor copies, which cut rows past the sequence and
// columns past the head: written from the threads that hold the rows, 16 bytes here and there, a tile took 6500 to 8200
// cycles. Returns once the accumulator has been read; the copies may still read `stage` (a later call waits, and so must
// the warp's lane 0 before it gives the place away: bulk_wait_group_read<0>).
__device__ __forceinline__ void store_head_rows(uint8_t* stage, const HeadMap& m, uint32_t acc, float f, bool live,
                                                int w, int lane, int box0, int box1, int row0, int head, int seq,
                                                       int s, int head_dim) {
  const int row = row0 + w * 32;
  for (int x = box0; x < box1 && x * 64 < head_dim; ++x) {
    uint32_t v[64], u[32];
    tmem_ld_32x32b_x32(acc + x * 64, *reinterpret_cast<uint32_t(*)[32]>(v));
    tmem_ld_32x32b_x32(acc + x * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const float a = __uint_as_float(v[2 * e]) * f, b = __uint_as_float(v[2 * e + 1]) * f;
      u[e] = live ? pack_bf16x2(a, b) : 0u;
    }
    if (lane == 0) bulk_wait_group_read<0>();
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 8; ++e) *box_chunk(stage, lane, e) = make_uint4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && row < s) {
      const int c1 = m.row == 1 ? row : (m.head == 1 ? head : seq);
      const int c2 = m.row == 2 ? row : (m.head == 2 ? head : seq);
      const int c3 = m.row == 3 ? row : (m.head == 3 ? head : seq);
      tma_store_4d(&m.map, stage, x * 64, c1, c2, c3);
      bulk_commit_group();
    }
  }
}

// Descriptors of a tile's first K-step, and what each further step adds (the address field counts 16 bytes and a
// shared-memory address never carries out of it). K-major, the rows being M or N: a step is 16 columns, 32 bytes, four
// to a box. MN-major, the head's columns being N: a step is 16 rows.
__device__ __forceinline__ uint64_t desc_rows(uint32_t tile) { return smem_desc_sw128(tile, 16, 1024); }
__device__ __forceinline__ uint64_t desc_cols(uint32_t tile) { return smem_desc_sw128(tile, kBoxBytes, 1024); }
__host__ __device__ constexpr uint64_t step_rows(int kk) { return ((kk >> 2) * kBoxBytes + (kk & 3) * 32) >> 4; }
__host__ __device__ constexpr uint64_t step_cols(int kk) { return (kk * 2048) >> 4; }

// D = A B^T over the heads' columns (ksteps of the HD / 16 steps; the rest are zeros), both tiles K-major.
template <int HD>
__device__ __forceinline__ void issue_rows(uint32_t leader, uint32_t d_tmem, uint32_t a_tile, uint32_t b_tile, int ksteps) {
  constexpr uint32_t kIdesc = idesc_bf16_f32(kTile, kTile, false, false);
  const uint64_t a = desc_rows(a_tile), b = desc_rows(b_tile);
#pragma unroll
  for (int kk = 0; kk < HD / 16; ++kk)
    if (kk < ksteps) umma_bf16_by(leader, d_tmem, a + step_rows(kk), b + step_rows(kk), kIdesc, kk != 0);
}

// The same with A's columns packed in tensor memory from a_tmem.
template <int HD>
__device__ __forceinline__ void issue_rows_ta(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint32_t b_tile, int ksteps) {
  constexpr uint32_t kIdesc = idesc_bf16_f32(kTile, kTile, false, false);
  const uint64_t b = desc_rows(b_tile);
#pragma unroll
  for (int kk = 0; kk < HD / 16; ++kk)
    if (kk < ksteps) umma_bf16_ta_by(leader, d_tmem, a_tmem + kk * 8, b + step_rows(kk), kIdesc, kk != 0);
}

// D (+)= A B over rows 16 * kFrom .. 16 * kTo - 1 of the tile B, which is used MN-major, with A's columns packed in
// tensor memory from a_tmem (kSplit: columns 64.. from a_tmem + 64, else in a row).
template <bool kSplit, int kFrom = 0, int kTo = kTile / 16>
__device__ __forceinline__ void issue_cols(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint32_t b_tile,
                                           uint32_t idesc, uint32_t accumulate) {
  const uint64_t b = desc_cols(b_tile);
#pragma unroll
  for (int kk = kFrom; kk < kTo; ++kk)
    umma_bf16_ta_by(leader, d_tmem, a_tmem + (kSplit ? (kk >> 2) * 64 + (kk & 3) * 8 : kk * 8), b + step_cols(kk), idesc,
                    kk == 0 ? accumulate : 1u);
}

// ------------------------------------------------------------------ long sums

// The tensor core cuts each product off some 25 bits below its accumulator: sums over many rows of like weight drift towards
// zero (means of uniform values over 2^16 keys by 5e-4, 2^17 by 1e-3, 2^20 by 7e-3, 2^23 by 5e-2 of themselves; a bf16
// rounding is 4e-3). Where a sum can have more than kLongSum steps, the kernels are the LONG ones: after every kPart steps
// the warps that will write an accumulator out add it to rows of their own in local memory, and the next product overwrites
// it. The rows take some 2000 cycles every 256 steps of as many, but the code around them would cost shorter sums 1 to 4 %
// (in one kernel: causal forward 65.4 -> 66.4 us, step with window and bias 381 -> 398 us), hence two.
constexpr int kPart = 256, kLongSum = 512;
__device__ __forceinline__ bool part_begins(int step) { return (step & (kPart - 1)) == 0; }

// part[c] = part[c] f + accumulator's column c (the latter alone if it is the first), a row per thread; the tile's lanes.
template <int COLS>
__device__ __forceinline__ void take_part(float* part, uint32_t acc, bool first, float f) {
#pragma unroll 1
  for (int c = 0; c < COLS; c += 32) {
    uint32_t o[32];
    tmem_ld_32x32b_x32(acc + c, o);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 32; ++e)
      part[c + e] = first ? __uint_as_float(o[e]) : fmaf(part[c + e], f, __uint_as_float(o[e]));
  }
}

// The accumulator += part f.
template <int COLS>
__device__ __forceinline__ void give_part(const float* part, uint32_t acc, float f) {
#pragma unroll 1
  for (int c = 0; c < COLS; c += 32) {
    uint32_t o[32];
    tmem_ld_32x32b_x32(acc + c, o);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(fmaf(part[c + e], f, __uint_as_float(o[e])));
    tmem_st_32x32b_x32(acc + c, o);
  }
  tmem_st_wait();
}

// What `use` returns for a call's kernels, which it gets as constants: the columns of a tile (64 or 128), whether scores are
// capped, whether they have a bias.
template <typename Use>
cudaError_t pick_kernel(bool wide, bool cap, bool bias, Use use) {
  using N64 = std::integral_constant<int, 64>;
  using N128 = std::integral_constant<int, 128>;
  auto width = [&](auto hd) {
    return cap ? (bias ? use(hd, std::true_type{}, std::true_type{}) : use(hd, std::true_type{}, std::false_type{}))
               : (bias ? use(hd, std::false_type{}, std::true_type{}) : use(hd, std::false_type{}, std::false_type{}));
  };
  return wide ? width(N128{}) : width(N64{});
}

// ------------------------------------------------------------------ masks and scores

// The key interval of a query row cut to the sequence; {0, 0} when nothing is left.
__device__ __forceinline__ int2 clip_range(int2 r, int s) {
  r.x = max(r.x, 0);
  r.y = min(r.y, s);
  return r.x < r.y ? r : make_int2(0, 0);
}

// What makes a score of q.k, in base 2 (y log2(e)).
struct ScoreParams {
  float scale2;          // scale * log2(e)
  float in_cap2;         // 2 log2(e) scale / cap: e^(2x) = 2^(q.k in_cap2)
  float cap2;            // cap * log2(e)
  float poly2[3], poly3[4];  // tanh(x) = q.k times a polynomial of (q.k)^2, for |x| <= 0.25 and |x| <= 0.48
  float small2, small3;      // |q.k| up to which they hold
};

inline ScoreParams score_params(float scale, float softcap) {
  const double log2e = 1.4426950408889634;
  ScoreParams p{};
  p.scale2 = static_cast<float>(scale * log2e);
  if (softcap > 0.f) {
    p.in_cap2 = static_cast<float>(2.0 * scale * log2e / softcap);
    p.cap2 = static_cast<float>(softcap * log2e);
    // Fits of tanh(x) / x - 1 in powers of x^2 up to 0.068, 0.25 and 0.48.
    const double fit1 = -0.3328233848, fit2[2] = {-0.3332457116, 0.1287641663};
    const double fit3[3] = {-0.3332922397, 0.1322320644, -0.0453897898};
    const double in = static_cast<double>(scale) / softcap;
    auto fits = [&](int power) { return std::pow(in, power) > 1e-35 && std::pow(in, power) < 1e37; };
    // Where a coefficient would leave fp32, the next shorter polynomial on its own range, down to x itself up to 0.0097,
    // where what it leaves out (x^2 / 3) is what the other form is off by.
    const bool one = fits(3), two = fits(5), three = fits(7);
    p.poly2[0] = p.poly3[0] = static_cast<float>(in);
    for (int i = 1; i < 3; ++i)
      p.poly2[i] = two ? static_cast<float>(std::pow(in, 2 * i + 1) * fit2[i - 1])
                       : one && i == 1 ? static_cast<float>(std::pow(in, 3) * fit1) : 0.f;
    p.small2 = static_cast<float>(std::fmin((two ? 0.25 : one ? 0.068 : 0.0097) / in, 1e18));
    for (int i = 1; i < 4; ++i)
      p.poly3[i] = three ? static_cast<float>(std::pow(in, 2 * i + 1) * fit3[i - 1]) : i < 3 ? p.poly2[i] : 0.f;
    p.small3 = three ? static_cast<float>(0.48 / in) : p.small2;
  }
  return p;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(x) of the cap's argument x = q.k scale / cap in two ways (tanh.approx's 2^-11 would not do: the cap multiplies the
// error into the exponent). Any x: 1 - 2 / (1 + e^(2x)), two special-function operations, off by up to 2.7e-7 = 4.5 * 2^-24
// in absolute terms, so taken only where some score of the warp's tile is not small. Small x: x times a polynomial of x^2
// with x's factor in the coefficients. Its first coefficient is x's factor itself and the others are fitted for the smallest
// largest relative error, so that a cap far above the scores leaves them what they are: degree 2 up to 0.25 and 3 up to
// 0.48, either off by 4.9e-7 = 8 * 2^-24 at worst (with the first coefficient fitted too, for the absolute error, small
// scores were off by 4e-6 of themselves: 4e-4 at 100 under a cap of 1e5). On pairs, four and five operations of the FMA
// pipe for two scores.
__device__ __forceinline__ float cap_tanh(float qk, const ScoreParams& p) {
  return fmaf(-2.0f, rcp_approx(1.0f + ex2_approx(qk * p.in_cap2)), 1.0f);
}
// The first way of a pair with the derivative: with E = e^(2x) and r = 1 / (1 + E) it is 4 E r^2, right relative to itself
// where 1 - tanh^2 would leave nothing of it. 4 E stops at 2^120, lest it meets r as infinity.
__device__ __forceinline__ F2 cap_tanh(F2 qk, const ScoreParams& p, F2& d) {
  auto both = [](float v) { return f2_make(v, v); };
  const float2 x = f2_split(f2_fma(qk, both(p.in_cap2), both(2.0f)));
  const F2 e4 = f2_make(ex2_approx(fminf(x.x, 120.0f)), ex2_approx(fminf(x.y, 120.0f)));
  const float2 n = f2_split(f2_fma(e4, both(0.25f), both(1.0f)));
  const F2 r = f2_make(rcp_approx(n.x), rcp_approx(n.y));
  d = f2_mul(r, f2_mul(r, e4));
  return f2_fma(both(-2.0f), r, both(1.0f));
}
template <int N>
__device__ __forceinline__ F2 cap_tanh_small(F2 qk, const float (&poly)[N]) {
  auto both = [](float v) { return f2_make(v, v); };
  const F2 z = f2_mul(qk, qk);
  F2 r = both(poly[N - 1]);
#pragma unroll
  for (int i = N - 2; i >= 0; --i) r = f2_fma(r, z, both(poly[i]));
  return f2_mul(qk, r);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The largest |q.k| of a warp's N scores in every lane.
template <int N>
__device__ __forceinline__ float largest(const float (&y)[N]) {
  float m[4] = {};
#pragma unroll
  for (int c = 0; c < N; c += 8)
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = max3(m[e], fabsf(y[c + 2 * e]), fabsf(y[c + 2 * e + 1]));
  // as numbers of one sign their bits have their order
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(max3(fmaxf(m[0], m[1]), m[2], m[3]))));
}

// tanh of N capped scores in place, by the cheapest form that all of a warp's allow. Causal forward of b2 s4096, 32 heads
// of 128 on 8, cap 50 on scores of deviation 1, 30 on 2.6 and 30 on 16: 251, 298 and 391 us. Against 264, 303 and 398 us in an
// earlier state: without degree 2 299, 304 and 394 us, and the first way alone as long as the last everywhere; taken together
// with the exponents, in copies of that loop, the polynomials cost more than they save (248, 368 and 411 us; one loop for
// all 273, 276 and 483 us).
template <int N>
__device__ __forceinline__ void cap_tanh_all(float (&y)[N], const ScoreParams& p) {
  auto all = [&](const auto& poly) {
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      const float2 v = f2_split(cap_tanh_small(f2_make(y[c], y[c + 1]), poly));
      y[c] = v.x;
      y[c + 1] = v.y;
    }
  };
  const float most = largest(y);
  if (most <= p.small2) {
    all(p.poly2);
  } else if (most <= p.small3) {
    all(p.poly3);
  } else {
#pragma unroll
    for (int c = 0; c < N; ++c) y[c] = cap_tanh(y[c], p);
  }
}

// y <- a y - slope2 |d0 + c| for N columns c, d0 the first column's place less the row's (or the other way round). A
// warp whose rows all lie on one side of its columns takes the bias as a line.
template <int N>
__device__ __forceinline__ void add_bias(float (&y)[N], float a, float slope2, float d0, int side) {
  if (side != 0) {
    const float k = side > 0 ? -slope2 : slope2, off = k * d0;
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      // c stands in the instruction; as a pair it would be two moves (forward with window and bias 112 -> 106 us)
      const F2 b = f2_make(fmaf(k, static_cast<float>(c), off), fmaf(k, static_cast<float>(c + 1), off));
      const float2 v = f2_split(f2_fma(f2_make(y[c], y[c + 1]), f2_make(a, a), b));
      y[c] = v.x;
      y[c + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int c = 0; c < N; ++c) y[c] = fmaf(-slope2, fabsf(d0 + static_cast<float>(c)), y[c] * a);
  }
}

// 1 if columns [col0, col0 + n) all lie at or behind the warp's rows [row0, row0 + 32), -1 if at or before them, else 0.
__device__ __forceinline__ int side_of(int col0, int n, int row0) {
  return col0 >= row0 + 31 ? 1 : col0 + n - 1 <= row0 ? -1 : 0;
}

// Bits [lo, hi) of a word, cut to 0..32.
__device__ __forceinline__ unsigned bit_range(int lo, int hi) {
  const int from = min(max(lo, 0), 32), to = min(max(hi, 0), 32);
  return from < to ? (0xffffffffu >> (32 - (to - from))) << from : 0u;
}

// Bit b of the result in lane i is bit i of lane b's word.
__device__ __forceinline__ unsigned transpose_bits(unsigned x) {
  const int lane = threadIdx.x & 31;
  constexpr unsigned kKeep[5] = {0x0000ffffu, 0x00ff00ffu, 0x0f0f0f0fu, 0x33333333u, 0x55555555u};
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    const int o = 16 >> i;
    const unsigned y = __shfl_xor_sync(0xffffffffu, x, o);
    x = lane & o ? (x & ~kKeep[i]) | ((y & ~kKeep[i]) >> o) : (x & kKeep[i]) | ((y & kKeep[i]) << o);
  }
  return x;
}

}  // namespace tpmlp
