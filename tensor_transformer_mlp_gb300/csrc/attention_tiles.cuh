// What the masked-attention kernels share: the tensor-core forms with an operand in tensor memory, tiles of heads
// loaded by tensor copies, key intervals, and the score function.
#pragma once

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

// mbar_wait by polling: for the issuing warp, whose reaction the tensor core waits for. (try_wait suspends the thread;
// it was seen to return up to 400 cycles after the phase had completed.)
__device__ __forceinline__ bool mbar_poll(uint64_t* bar, uint32_t parity, unsigned int* status, unsigned int where) {
  const uint32_t a = smem_u32(bar);
  auto done = [&] {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(a), "r"(parity)
        : "memory");
    return ok != 0;
  };
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

// The same with 16 columns.
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      TPMLP_R8(r, 0), TPMLP_R8(r, 8)
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

// Writes 32 rows of an accumulator to a tensor of heads: warp `w` of a tile's four takes lanes 32 w .. 32 w + 31, row
// row0 + 32 w + lane, the columns of boxes [box0, box1), scaled by f (per row) and rounded to bf16; zeros if not live.
// They leave through the warp's part of `tile` (shared memory that nothing else uses any more) by tensor copies, which
// cut rows past the sequence and columns past the head: written from the threads that hold the rows, 16 bytes here and
// there, a tile took 6500 to 8200 cycles. Returns when shared memory has been read.
__device__ __forceinline__ void store_head_rows(uint8_t* tile, const HeadMap& m, uint32_t acc, float f, bool live, int w,
                                                int lane, int box0, int box1, int row0, int head, int seq, int s,
                                                int head_dim) {
  for (int x = box0; x < box1 && x * 64 < head_dim; ++x) {
    uint8_t* box = tile + x * kBoxBytes + w * 32 * 128;
#pragma unroll
    for (int c = 0; c < 64; c += 32) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(acc + x * 64 + c, v);
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = __uint_as_float(v[8 * e + 2 * i]) * f, b = __uint_as_float(v[8 * e + 2 * i + 1]) * f;
          u[i] = live ? pack_bf16x2(a, b) : 0u;
        }
        *box_chunk(box, lane, c / 8 + e) = make_uint4(u[0], u[1], u[2], u[3]);
      }
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
  const int row = row0 + w * 32;
  if (lane == 0 && row < s) {
    const int c1 = m.row == 1 ? row : (m.head == 1 ? head : seq);
    const int c2 = m.row == 2 ? row : (m.head == 2 ? head : seq);
    const int c3 = m.row == 3 ? row : (m.head == 3 ? head : seq);
    for (int x = box0; x < box1 && x * 64 < head_dim; ++x)
      tma_store_4d(&m.map, tile + x * kBoxBytes + w * 32 * 128, x * 64, c1, c2, c3);
    bulk_commit_group();
    bulk_wait_group_read<0>();
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

// ------------------------------------------------------------------ masks and scores

// The key interval of a query row cut to the sequence; {0, 0} when nothing is left.
__device__ __forceinline__ int2 clip_range(int2 r, int s) {
  r.x = max(r.x, 0);
  r.y = min(r.y, s);
  return r.x < r.y ? r : make_int2(0, 0);
}

// Scores in base 2: y log2(e) as a function of q.k. With a cap, cap tanh(x / cap) = cap (1 - 2 / (1 + e^(2x/cap))),
// whose absolute error, a few 2^-24 of the cap, is what the exponent sees (tanh.approx's 2^-11 would not do).
struct ScoreParams {
  float scale2;   // scale * log2(e); with a cap: 2 scale log2(e) / cap
  float cap2;     // cap * log2(e)
};

inline ScoreParams score_params(float scale, float softcap) {
  const double log2e = 1.4426950408889634;
  return softcap > 0.f ? ScoreParams{static_cast<float>(2.0 * scale * log2e / softcap), static_cast<float>(softcap * log2e)}
                       : ScoreParams{static_cast<float>(scale * log2e), 0.f};
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / (1 + e^(2x/cap)) = (1 - tanh(x / cap)) / 2 of a raw score.
__device__ __forceinline__ float cap_sigma(float qk, const ScoreParams& p) {
  return rcp_approx(1.0f + ex2_approx(qk * p.scale2));
}

}  // namespace tpmlp
