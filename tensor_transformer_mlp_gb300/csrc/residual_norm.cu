// The norms before and after a block with its gate and residual scale in one pass, and the backward
// (tpmlp_residual_norm, tpmlp_residual_norm_backward). Per token, over the h columns:
//
//   y_hat = y ry, ry = 1 / sqrt(mean(y^2) + eps);   r = alpha x + gate gamma_post y_hat;   u = r rr gamma_pre
//   g = dr + rr (du gamma_pre - r_hat c), c = mean(du gamma_pre r_hat);   dx = alpha g
//   dy = ry (w g - y_hat mean(w g y_hat)), w = gate gamma_post
//   dgamma_pre = sum du r_hat;   dgate = gamma_post S, dgamma_post = gate S summed over the sequences, where
//   S = sum over a sequence's tokens of g y_hat
//
// Without gamma_post y_hat is y (and dy = w g), without a gate or gamma_pre they are one or their half of the work is
// left out. Both directions are bound by memory: 4 values of T a column forward, 6 backward; the backward also by its
// arithmetic, some 19 fp32 operations a value. A row's statistics are one barrier each; the backward has one in all, since
// mean(w g y_hat) is a sum of three products that need no other sum.
// Measured, share of the copy rate: b2 s4096 h4096 with gates of two sequences, bf16 forward 45 to 47 us (0.84 to 0.88), backward
// 73 us with 5 us of sums over CTAs (0.81); fp32 94 (0.84) and 130 us (0.92). 4096 rows of 8192 45 (0.87) and 77 (0.77), 16384 of
// 2048 47 (0.84) and 73 (0.81), 65536 of 512 44 (0.89) and 71 (0.83), of 256 23 (0.86) and 48 (0.62); b40 s512 h640 21 (0.75) and 45
// (0.52). Four single tokens 3.2 and 7.4 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "abi_checks.h"
#include "device_common.cuh"

namespace tpmlp {
namespace {

constexpr int kMaxH = 8192;
constexpr int kSmallH = 512;        // up to here a lane group takes a row, above a CTA does
constexpr int kSmallThreads = 256;
constexpr int kMaxCtas = 1024;      // of the backward, each with a row of partial sums

// Eight columns as they lie in memory, and as four fp32 pairs.
template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  // Keeps the compiler from holding unpacked values (twice the registers) from one use to the next.
  __device__ __forceinline__ void stay_packed() { asm volatile("" : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)); }
  __device__ __forceinline__ void unpack(F2 (&f)[4]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2_make(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const F2 (&f)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = f2_split(f[i]);
      w[i] = pack_bf16x2(t.x, t.y);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void stay_packed() {}
  __device__ __forceinline__ void unpack(F2 (&f)[4]) const {
    f[0] = f2_make(a.x, a.y);
    f[1] = f2_make(a.z, a.w);
    f[2] = f2_make(b.x, b.y);
    f[3] = f2_make(b.z, b.w);
  }
  static __device__ __forceinline__ void store(float* p, const F2 (&f)[4]) {
    const float2 t0 = f2_split(f[0]), t1 = f2_split(f[1]), t2 = f2_split(f[2]), t3 = f2_split(f[3]);
    reinterpret_cast<float4*>(p)[0] = make_float4(t0.x, t0.y, t1.x, t1.y);
    reinterpret_cast<float4*>(p)[1] = make_float4(t2.x, t2.y, t3.x, t3.y);
  }
};

__device__ __forceinline__ float sum2(F2 a) {
  const float2 t = f2_split(a);
  return t.x + t.y;
}
// Eight fp32 gains from column col on; ones where there are none, zeros past h.
__device__ __forceinline__ void load_gain(F2 (&f)[4], const float* gain, int col, int h) {
  if (col >= h || !gain) {
    const float v = col >= h ? 0.f : 1.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = f2_make(v, v);
  } else {
    Vec8<float> t;
    t.load(gain + col);
    t.unpack(f);
  }
}

struct Forward {
  const void *x, *y;
  const float *post, *gate, *pre;
  void *r, *u;
  float alpha, eps, inv_h;
  int64_t rows, s;
  int h;
  bool run_of_rows;  // a CTA's rows lie behind one another
};

struct Backward {
  const void *y, *r, *dr, *du;
  const float *post, *gate, *pre;
  void *dx, *dy;
  float* dgate;
  // partials [gridDim.x][2][h]: the CTA's shares of dgamma_post and dgamma_pre; slots [gridDim.x][2][h] (with a gate): S of
  // the CTA's rows of a sequence that starts before them, and of one that starts in them and ends behind them
  float *partials, *slots;
  float alpha, eps, inv_h;
  int64_t rows, s;
  int h;
};

// CTA c's rows.
__host__ __device__ __forceinline__ int64_t first_row(int64_t rows, int64_t c, int64_t ctas) {
  return rows / ctas * c + min(c, rows % ctas);
}

// ------------------------------------------------------------------ a CTA for a row

// A ring of bulk copies: stage st holds one row of each of the kernel's tensors. Thread 0 issues.
template <int NTEN>
struct RowRing {
  uint8_t* smem;
  uint64_t* full;
  uint32_t row_bytes;
  int64_t step;  // bytes between the CTA's rows
  int stages;
  const uint8_t* src[NTEN];  // the CTA's first row of each tensor; null: none
  __device__ __forceinline__ uint32_t stage_bytes() const { return NTEN * row_bytes; }
  __device__ __forceinline__ void init() const {
    for (int st = 0; st < stages; ++st) mbar_init(&full[st], 1);
    fence_mbar_init();
  }
  // Row i of the CTA into stage st.
  __device__ __forceinline__ void issue(int64_t i, int st) const {
    uint8_t* dst = smem + static_cast<size_t>(st) * stage_bytes();
    uint32_t n = 0;
#pragma unroll
    for (int k = 0; k < NTEN; ++k) n += src[k] ? row_bytes : 0;
    mbar_arrive_expect_tx(&full[st], n);
#pragma unroll
    for (int k = 0; k < NTEN; ++k)
      if (src[k]) bulk_load(dst + k * row_bytes, src[k] + i * step, row_bytes, &full[st]);
  }
  template <typename T>
  __device__ __forceinline__ const T* at(int st, int k) const {
    return reinterpret_cast<const T*>(smem + st * stage_bytes() + k * row_bytes);
  }
  // Waits (bounded) for the copies of rows [from, to), which are all in flight or there.
  __device__ __forceinline__ void drain(int64_t from, int64_t to, unsigned int* status, unsigned int where) const {
    for (int64_t k = from; k < to; ++k) mbar_wait(&full[k % stages], static_cast<uint32_t>((k / stages) & 1), status, where);
  }
};

// A row's stage and its barrier's phase, counted along instead of divided out (a 64-bit division a row and thread costs
// the backward 15 %).
struct RowStage {
  int st = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++st == stages) {
      st = 0;
      phase ^= 1;
    }
  }
};

template <int N>
__device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Rows go through the ring; a row's two sums each meet behind one barrier, every warp adding the
// warps' shares in the same order. A wait that runs out ends the CTA at the next barrier.
template <typename T, int NT, int CH>
__global__ void __launch_bounds__(NT) residual_norm_row_kernel(const __grid_constant__ Forward p, int stages,
                                                               unsigned int* status) {
  constexpr int NW = NT / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float red[2][2][NW];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, nt = blockDim.x;  // at most NT, what the row needs
  const int wl = lane & (NW - 1);  // the warp whose share this lane adds
  // Every gridDim.x-th row, so that all CTAs are at neighbouring rows (b2 s4096 h4096: 46.8 us, with a run of rows each
  // 49.1); but a run of rows where that would bring another sequence's gate with nearly every row (b40 s512 h640 20.0, 25.1).
  const int64_t by = p.run_of_rows ? 1 : gridDim.x, first = p.run_of_rows ? first_row(p.rows, blockIdx.x, gridDim.x) : blockIdx.x;
  const int64_t n = p.run_of_rows ? first_row(p.rows, blockIdx.x + 1, gridDim.x) - first : (p.rows - first + by - 1) / by;
  RowRing<2> ring;
  ring.smem = smem;
  ring.row_bytes = static_cast<uint32_t>(p.h) * sizeof(T);
  ring.step = by * ring.row_bytes;
  ring.stages = stages;
  ring.full = reinterpret_cast<uint64_t*>(smem + static_cast<size_t>(stages) * ring.stage_bytes());
  ring.src[0] = static_cast<const uint8_t*>(p.x) + first * ring.row_bytes;
  ring.src[1] = static_cast<const uint8_t*>(p.y) + first * ring.row_bytes;
  if (tid == 0) ring.init();
  __syncthreads();
  int64_t issued = min(n, static_cast<int64_t>(stages));  // meaningful in thread 0
  if (tid == 0)
    for (int64_t i = 0; i < issued; ++i) ring.issue(i, static_cast<int>(i));

  F2 wt[CH][4], pre[CH][4];
  int64_t seq = -1, seq_end = 0;  // the sequence whose gate wt holds, and its last row's successor
#pragma unroll
  for (int c = 0; c < CH; ++c) load_gain(pre[c], p.pre, (tid + c * nt) * 8, p.h);
  const F2 alpha = f2_make(p.alpha, p.alpha), zero = f2_make(0.f, 0.f);
  int64_t i = 0;
  int aborted = 0;
  RowStage at;
  for (; i < n; ++i, at.next(stages)) {
    const int64_t row = first + i * by;
    if (row >= seq_end) {
      seq = row / p.s;
      seq_end = (seq + 1) * p.s;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = (tid + c * nt) * 8;
        F2 g[4];
        load_gain(wt[c], p.post, col, p.h);
        load_gain(g, p.gate ? p.gate + seq * p.h : nullptr, col, p.h);
#pragma unroll
        for (int e = 0; e < 4; ++e) wt[c][e] = f2_mul(wt[c][e], g[e]);
      }
    }
    const bool ok = mbar_wait(&ring.full[at.st], at.phase, status, 61);
    Vec8<T> xv[CH], yv[CH];
    F2 ss = zero;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (tid + c * nt) * 8;
      xv[c].zero();
      yv[c].zero();
      if (col < p.h) {
        xv[c].load(ring.at<T>(at.st, 0) + col);
        yv[c].load(ring.at<T>(at.st, 1) + col);
      }
      F2 f[4];
      yv[c].unpack(f);
#pragma unroll
      for (int e = 0; e < 4; ++e) ss = f2_fma(f[e], f[e], ss);
    }
    const int par = static_cast<int>(i & 1);
    const float ys = lane_sum<32>(sum2(ss));
    if (lane == 0) red[par][0][w] = ys;
    aborted = __syncthreads_or(!ok);  // the row is in registers everywhere
    if (aborted) break;
    if (tid == 0 && i + stages < n) {
      ring.issue(i + stages, at.st);
      issued = i + stages + 1;
    }
    const float ry = p.post ? rsqrtf(fmaf(lane_sum<NW>(wl * 32 < nt ? red[par][0][wl] : 0.f), p.inv_h, p.eps)) : 1.f;
    F2 rf[CH][4];
    ss = zero;
    const F2 ry2 = f2_make(ry, ry);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (tid + c * nt) * 8;
      F2 xf[4], yf[4];
      yv[c].stay_packed();
      xv[c].unpack(xf);
      yv[c].unpack(yf);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        rf[c][e] = f2_fma(f2_mul(yf[e], ry2), wt[c][e], f2_mul(alpha, xf[e]));
        ss = f2_fma(rf[c][e], rf[c][e], ss);
      }
      if (col < p.h) Vec8<T>::store(static_cast<T*>(p.r) + row * p.h + col, rf[c]);
    }
    if (p.pre) {
      const float rs = lane_sum<32>(sum2(ss));
      if (lane == 0) red[par][1][w] = rs;
      __syncthreads();
      const float rr = rsqrtf(fmaf(lane_sum<NW>(wl * 32 < nt ? red[par][1][wl] : 0.f), p.inv_h, p.eps));
      const F2 rr2 = f2_make(rr, rr);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = (tid + c * nt) * 8;
#pragma unroll
        for (int e = 0; e < 4; ++e) rf[c][e] = f2_mul(f2_mul(rf[c][e], rr2), pre[c][e]);
        if (col < p.h) Vec8<T>::store(static_cast<T*>(p.u) + row * p.h + col, rf[c]);
      }
    }
  }
  if (aborted && tid == 0) ring.drain(i, issued, status, 62);  // copies in flight
}

// The backward's six sums of a row; everything that follows from them.
//   sums: r^2, du' r, y^2, (w y) dr, (w y) du', (w y) r with du' = du gamma_pre
// NORMED: with gamma_post. Without it dy = w g whatever y holds: an infinite y times a ky of 0 would be NaN. A template: b2 s4096
// h4096 bf16 73.2 us, chosen at run time for each value 77.2, by a branch for eight columns 79.6.
template <bool NORMED>
struct RowFactors {
  float rr, kr;  // g = dr + rr du' - kr r
  float ry, ky;  // dy = ry w g - ky y
  __device__ __forceinline__ RowFactors(const float (&s)[6], const Backward& p) {
    rr = p.pre ? rsqrtf(fmaf(s[0], p.inv_h, p.eps)) : 0.f;
    // multiplied out from the sums on: the cube of a root of 1e15 or 1e-15 is none that fp32 holds
    kr = rr * (rr * (rr * (s[1] * p.inv_h)));
    ry = NORMED ? rsqrtf(fmaf(s[2], p.inv_h, p.eps)) : 1.f;
    // the sum of w g y needs no pass of its own: g is a sum of three terms
    ky = NORMED ? ry * (ry * (ry * (p.inv_h * (s[3] + (rr * s[4] - kr * s[5]))))) : 0.f;
  }
};

// One thread's eight columns of a row.
template <typename T>
struct GradColumns {
  Vec8<T> y, r, dr, du;
  __device__ __forceinline__ void zero() {
    y.zero();
    r.zero();
    dr.zero();
    du.zero();
  }
  __device__ __forceinline__ void stay_packed() {
    y.stay_packed();
    r.stay_packed();
    dr.stay_packed();
    du.stay_packed();
  }
  __device__ __forceinline__ void sums(const F2 (&wt)[4], const F2 (&pre)[4], F2 (&s)[6]) const {
    F2 yf[4], rf[4], drf[4], duf[4];
    y.unpack(yf);
    r.unpack(rf);
    dr.unpack(drf);
    du.unpack(duf);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const F2 d = f2_mul(duf[e], pre[e]), wy = f2_mul(wt[e], yf[e]);
      s[0] = f2_fma(rf[e], rf[e], s[0]);
      s[1] = f2_fma(d, rf[e], s[1]);
      s[2] = f2_fma(yf[e], yf[e], s[2]);
      s[3] = f2_fma(wy, drf[e], s[3]);
      s[4] = f2_fma(wy, d, s[4]);
      s[5] = f2_fma(wy, rf[e], s[5]);
    }
  }
  // dx and dy into ox, oy; adds to S and dgamma_pre.
  template <bool NORMED>
  __device__ __forceinline__ void grads(const F2 (&wt)[4], const F2 (&pre)[4], const RowFactors<NORMED>& k, float alpha,
                                        F2 (&ox)[4], F2 (&oy)[4], F2 (&acc_s)[4], F2 (&acc_pre)[4]) const {
    F2 yf[4], rf[4], drf[4], duf[4];
    y.unpack(yf);
    r.unpack(rf);
    dr.unpack(drf);
    du.unpack(duf);
    const F2 rr = f2_make(k.rr, k.rr), nkr = f2_make(-k.kr, -k.kr), ry = f2_make(k.ry, k.ry), nky = f2_make(-k.ky, -k.ky),
             a = f2_make(alpha, alpha);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const F2 drr = f2_mul(duf[e], rr);
      const F2 g = f2_add(drf[e], f2_fma(drr, pre[e], f2_mul(nkr, rf[e])));
      acc_pre[e] = f2_fma(drr, rf[e], acc_pre[e]);
      const F2 gy = f2_mul(g, ry);
      acc_s[e] = f2_fma(gy, yf[e], acc_s[e]);
      ox[e] = f2_mul(a, g);
      oy[e] = NORMED ? f2_fma(gy, wt[e], f2_mul(nky, yf[e])) : f2_mul(gy, wt[e]);
    }
  }
};

// A thread's share of what a CTA (rows [first, end)) leaves of a sequence: its gate's gradient, or S to a slot where other CTAs
// have rows of it too; and gate S added to the CTA's dgamma_post.
__device__ __forceinline__ void leave_sequence(const Backward& p, int64_t seq, int64_t first, int64_t end, int col,
                                               const F2 (&acc)[4], bool none_left) {
  F2 g[4];
  load_gain(g, p.gate ? p.gate + seq * p.h : nullptr, col, p.h);
  if (p.gate) {
    const bool starts_here = seq * p.s >= first, ends_here = (seq + 1) * p.s <= end;
    if (starts_here && ends_here) {
      F2 post[4], out[4];
      load_gain(post, p.post, col, p.h);
#pragma unroll
      for (int e = 0; e < 4; ++e) out[e] = f2_mul(post[e], acc[e]);
      Vec8<float>::store(p.dgate + seq * p.h + col, out);
    } else {
      Vec8<float>::store(p.slots + (2 * static_cast<int64_t>(blockIdx.x) + (starts_here ? 1 : 0)) * p.h + col, acc);
    }
  }
  if (p.post) {
    float* out = p.partials + static_cast<int64_t>(blockIdx.x) * 2 * p.h + col;
    F2 old[4] = {f2_make(0.f, 0.f), f2_make(0.f, 0.f), f2_make(0.f, 0.f), f2_make(0.f, 0.f)};
    if (!none_left) {
      Vec8<float> t;
      t.load(out);
      t.unpack(old);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) old[e] = f2_fma(g[e], acc[e], old[e]);
    Vec8<float>::store(out, old);
  }
}

// Sums eight values a lane over the warp; lane l ends with the total of value (l >> 2) & 7 (9 shuffles).
__device__ __forceinline__ float warp_sums8(float (&v)[8], int lane) {
#pragma unroll
  for (int half = 4, o = 16; half > 0; half >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int k = 0; k < half; ++k) {
      const float send = up ? v[k] : v[k + half], keep = up ? v[k + half] : v[k];
      v[k] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

// One barrier a row: all six sums are taken at once. Between two barriers a thread works out a row's gradients and takes
// the next row's sums, both from the ring, so that neither the sums' way through the CTA nor registers for a whole row hold
// anything up.
// HOLD: a row stays in registers from its sums to its gradients instead, and its stage is refilled at once (for fp32, whose
// rows leave no room for a ring of three and more in flight).
// RING: else rows are read where they lie (fp32 rows of more than 4096 columns: 2048 of 8192 105 us, of 5120 74; held in registers
// beside a ring of one or two, with w and gamma_pre in shared memory, 108 and 78).
template <typename T, int NT, int CH, int MINB, bool HOLD, bool RING, bool NORMED>
__global__ void __launch_bounds__(NT, MINB) residual_norm_row_backward_kernel(const __grid_constant__ Backward p, int stages,
                                                                              unsigned int* status) {
  constexpr int NW = NT / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float red[2][NW][8];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, nt = blockDim.x;  // at most NT, what the row needs
  const int64_t first = first_row(p.rows, blockIdx.x, gridDim.x), n = first_row(p.rows, blockIdx.x + 1, gridDim.x) - first;
  RowRing<4> ring;
  ring.smem = smem;
  ring.row_bytes = static_cast<uint32_t>(p.h) * sizeof(T);
  ring.step = ring.row_bytes;
  ring.stages = stages;
  ring.full = reinterpret_cast<uint64_t*>(smem + static_cast<size_t>(stages) * ring.stage_bytes());
  const void* src[4] = {p.y, p.r, p.dr, p.du};
#pragma unroll
  for (int k = 0; k < 4; ++k) ring.src[k] = src[k] ? static_cast<const uint8_t*>(src[k]) + first * ring.row_bytes : nullptr;
  int64_t issued = min(n, static_cast<int64_t>(stages));  // meaningful in thread 0
  if constexpr (RING) {
    if (tid == 0) ring.init();
    __syncthreads();
    if (tid == 0)
      for (int64_t i = 0; i < issued; ++i) ring.issue(i, static_cast<int>(i));
  }

  const F2 zero = f2_make(0.f, 0.f);
  F2 wt[CH][4], pre[CH][4], acc_s[CH][4], acc_pre[CH][4];
  GradColumns<T> held[HOLD ? CH : 1];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    load_gain(pre[c], p.pre, (tid + c * nt) * 8, p.h);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc_s[c][e] = acc_pre[c][e] = zero;
  }
  int64_t seq = -1, seq_end = first;
  bool none_left = true;  // no sequence of the CTA has ended yet
  auto columns = [&](int64_t i, int st, int col) {
    auto row_of = [&](int k) {
      if constexpr (RING) return ring.template at<T>(st, k) + col;
      return reinterpret_cast<const T*>(ring.src[k] + i * ring.row_bytes) + col;
    };
    GradColumns<T> v;
    v.zero();
    if (col < p.h) {
      if (p.y) v.y.load(row_of(0));
      if (p.r) v.r.load(row_of(1));
      if (p.dr) v.dr.load(row_of(2));
      if (p.du) v.du.load(row_of(3));
    }
    return v;
  };
  // Row i's sums, behind the end of the sequence before it if there is one.
  auto take_sums = [&](int64_t i, const RowStage& at) {
    const int64_t row = first + i;
    if (row >= seq_end) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = (tid + c * nt) * 8;
        if (seq >= 0 && col < p.h) leave_sequence(p, seq, first, first + n, col, acc_s[c], none_left);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc_s[c][e] = zero;
      }
      none_left = seq < 0;
      seq = row / p.s;
      seq_end = (seq + 1) * p.s;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = (tid + c * nt) * 8;
        F2 g[4];
        load_gain(wt[c], p.post, col, p.h);
        load_gain(g, p.gate ? p.gate + seq * p.h : nullptr, col, p.h);
#pragma unroll
        for (int e = 0; e < 4; ++e) wt[c][e] = f2_mul(wt[c][e], g[e]);
      }
    }
    const bool ok = !RING || mbar_wait(&ring.full[at.st], at.phase, status, 63);
    F2 s2[6] = {zero, zero, zero, zero, zero, zero};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const GradColumns<T> v = columns(i, at.st, (tid + c * nt) * 8);
      if constexpr (HOLD) held[c] = v;
      v.sums(wt[c], pre[c], s2);
    }
    float s8[8] = {sum2(s2[0]), sum2(s2[1]), sum2(s2[2]), sum2(s2[3]), sum2(s2[4]), sum2(s2[5]), 0.f, 0.f};
    const float mine = warp_sums8(s8, lane);
    if ((lane & 3) == 0) red[i & 1][w][lane >> 2] = mine;
    return ok;
  };
  RowStage before, here, next;  // of rows i - 1, i and i + 1
  bool ok = take_sums(0, next);
  int64_t i = 0;
  int aborted = 0;
  for (; i < n; ++i) {
    before = here;
    here = next;
    next.next(stages);
    aborted = __syncthreads_or(!ok);  // row i's sums are out, and nobody reads row i - 1 any more
    if (aborted) break;
    if (RING && tid == 0) {  // the stage that nobody reads any more: this row's where it is in registers, else the last one's
      const int64_t done = HOLD ? i : i - 1;
      if (done >= 0 && done + stages < n) {
        ring.issue(done + stages, HOLD ? here.st : before.st);
        issued = done + stages + 1;
      }
    }
    // lane l adds value l & 7 of the warps l >> 3, + 4, ..: the same order in every warp
    float part = 0.f;
#pragma unroll
    for (int k = 0; k < (NW + 3) / 4; ++k) {
      const int warp = (lane >> 3) + 4 * k;
      if (warp * 32 < nt) part += red[i & 1][warp][lane & 7];
    }
    part += __shfl_xor_sync(0xffffffffu, part, 8);
    part += __shfl_xor_sync(0xffffffffu, part, 16);
    float total[6];
#pragma unroll
    for (int k = 0; k < 6; ++k) total[k] = __shfl_sync(0xffffffffu, part, k);
    const RowFactors<NORMED> f(total, p);
    const int64_t row = first + i;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (tid + c * nt) * 8;
      F2 ox[4], oy[4];
      if constexpr (HOLD) {
        held[c].stay_packed();
        held[c].grads(wt[c], pre[c], f, p.alpha, ox, oy, acc_s[c], acc_pre[c]);
      } else {
        columns(i, here.st, col).grads(wt[c], pre[c], f, p.alpha, ox, oy, acc_s[c], acc_pre[c]);
      }
      if (col < p.h) {
        Vec8<T>::store(static_cast<T*>(p.dx) + row * p.h + col, ox);
        Vec8<T>::store(static_cast<T*>(p.dy) + row * p.h + col, oy);
      }
    }
    if (i + 1 < n) ok = take_sums(i + 1, next);
  }
  grid_dependents_may_start();  // the sums below may be scheduled; they wait for this grid's end
  if (RING && aborted && tid == 0) ring.drain(i, issued, status, 64);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int col = (tid + c * nt) * 8;
    if (col < p.h) {
      leave_sequence(p, seq, first, first + n, col, acc_s[c], none_left);
      Vec8<float>::store(p.partials + (static_cast<int64_t>(blockIdx.x) * 2 + 1) * p.h + col, acc_pre[c]);
    }
  }
}

// ------------------------------------------------------------------ a lane group for a row

// Up to 512 columns: `group` lanes (a power of two) take a row, CH vectors of 8 columns each.
__device__ __forceinline__ float group_sum(float v, int group) {
  for (int o = group >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A group's rows are `groups` apart; the next one's values are on their way while one is worked on (65536 rows of 256 and
// 512: 23.3 and 44.6 us; 32.3 and 51.3 without).
template <typename T, int CH>
__global__ void __launch_bounds__(kSmallThreads) residual_norm_small_kernel(const __grid_constant__ Forward p, int group) {
  const int gl = threadIdx.x & (group - 1);
  const int64_t groups = static_cast<int64_t>(gridDim.x) * (kSmallThreads / group);
  const F2 alpha = f2_make(p.alpha, p.alpha), zero = f2_make(0.f, 0.f);
  // all lanes of a warp make the same number of rounds: the shuffles need them
  int64_t row = static_cast<int64_t>(blockIdx.x) * (kSmallThreads / group) + threadIdx.x / group;
  int64_t warp_row = row - (threadIdx.x & 31) / group;
  F2 wt[CH][4], pre[CH][4];
  int64_t seq_end = 0;  // of the sequence whose gate wt holds
#pragma unroll
  for (int c = 0; c < CH; ++c) load_gain(pre[c], p.pre, (gl + c * group) * 8, p.h);
  Vec8<T> xv[CH], yv[CH];
  auto load = [&](int64_t r) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (gl + c * group) * 8;
      xv[c].zero();
      yv[c].zero();
      if (r < p.rows && col < p.h) {
        xv[c].load(static_cast<const T*>(p.x) + r * p.h + col);
        yv[c].load(static_cast<const T*>(p.y) + r * p.h + col);
      }
    }
  };
  load(row);
  for (; warp_row < p.rows; row += groups, warp_row += groups) {
    const bool live = row < p.rows;
    if (live && row >= seq_end) {
      const int64_t seq = row / p.s;
      seq_end = (seq + 1) * p.s;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = (gl + c * group) * 8;
        F2 g[4];
        load_gain(wt[c], p.post, col, p.h);
        load_gain(g, p.gate ? p.gate + seq * p.h : nullptr, col, p.h);
#pragma unroll
        for (int e = 0; e < 4; ++e) wt[c][e] = f2_mul(wt[c][e], g[e]);
      }
    }
    F2 xf[CH][4], yf[CH][4], ss = zero;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      xv[c].unpack(xf[c]);
      yv[c].unpack(yf[c]);
#pragma unroll
      for (int e = 0; e < 4; ++e) ss = f2_fma(yf[c][e], yf[c][e], ss);
    }
    load(row + groups);
    float sum = group_sum(sum2(ss), group);
    const float ry = p.post ? rsqrtf(fmaf(sum, p.inv_h, p.eps)) : 1.f;
    const F2 ry2 = f2_make(ry, ry);
    ss = zero;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        xf[c][e] = f2_fma(f2_mul(yf[c][e], ry2), wt[c][e], f2_mul(alpha, xf[c][e]));  // r
        ss = f2_fma(xf[c][e], xf[c][e], ss);
      }
    sum = group_sum(sum2(ss), group);
    const float rr = rsqrtf(fmaf(sum, p.inv_h, p.eps));
    const F2 rr2 = f2_make(rr, rr);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (gl + c * group) * 8;
      if (!live || col >= p.h) continue;
      Vec8<T>::store(static_cast<T*>(p.r) + row * p.h + col, xf[c]);
      if (p.pre) {
#pragma unroll
        for (int e = 0; e < 4; ++e) xf[c][e] = f2_mul(f2_mul(xf[c][e], rr2), pre[c][e]);
        Vec8<T>::store(static_cast<T*>(p.u) + row * p.h + col, xf[c]);
      }
    }
  }
}

// The CTA's sum of acc, groups of `group` lanes holding the same columns: columns 8 tid .. 8 tid + 7 end in thread tid's `out`.
// red: [NW][cols / 4] of shared memory.
template <int NW, int CH>
__device__ __forceinline__ void cta_sum(float4* red, int cols, int h, int group, F2 (&acc)[CH][4], F2 (&out)[4]) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, gl = tid & (group - 1);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    float v[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 t = f2_split(acc[c][e]);
      v[2 * e] = t.x;
      v[2 * e + 1] = t.y;
    }
    for (int o = 16; o >= group; o >>= 1)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += __shfl_xor_sync(0xffffffffu, v[e], o);
    const int col = (gl + c * group) * 8;
    if (lane < group && col < h) {
      red[w * cols / 4 + col / 4] = make_float4(v[0], v[1], v[2], v[3]);
      red[w * cols / 4 + col / 4 + 1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 4; ++e) out[e] = f2_make(0.f, 0.f);
  if (tid * 8 < h)
    for (int k = 0; k < NW; ++k) {
      const float4 a = red[k * cols / 4 + 2 * tid], b = red[k * cols / 4 + 2 * tid + 1];
      out[0] = f2_add(out[0], f2_make(a.x, a.y));
      out[1] = f2_add(out[1], f2_make(a.z, a.w));
      out[2] = f2_add(out[2], f2_make(b.x, b.y));
      out[3] = f2_add(out[3], f2_make(b.z, b.w));
    }
  __syncthreads();
}

// A CTA's rows are worked on sequence by sequence, each group taking every (256 / group)-th row; what the groups have
// added up meets in shared memory when the sequence, or the CTA's part of it, ends.
template <typename T, int CH, bool NORMED>
__global__ void __launch_bounds__(kSmallThreads, 2)
    residual_norm_small_backward_kernel(const __grid_constant__ Backward p, int group) {
  constexpr int NW = kSmallThreads / 32;
  __shared__ float4 red[NW * kSmallH / 4];
  const int tid = threadIdx.x, gl = tid & (group - 1), ngroups = kSmallThreads / group;
  const int64_t first = first_row(p.rows, blockIdx.x, gridDim.x), last = first_row(p.rows, blockIdx.x + 1, gridDim.x);
  const F2 zero = f2_make(0.f, 0.f);
  F2 wt[CH][4], pre[CH][4], acc_s[CH][4], acc_pre[CH][4];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    load_gain(pre[c], p.pre, (gl + c * group) * 8, p.h);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc_pre[c][e] = zero;
  }
  bool none_left = true;
  for (int64_t at = first; at < last;) {
    const int64_t seq = at / p.s, end = min(last, (seq + 1) * p.s);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (gl + c * group) * 8;
      F2 g[4];
      load_gain(wt[c], p.post, col, p.h);
      load_gain(g, p.gate ? p.gate + seq * p.h : nullptr, col, p.h);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        wt[c][e] = f2_mul(wt[c][e], g[e]);
        acc_s[c][e] = zero;
      }
    }
    GradColumns<T> v[CH];
    auto load = [&](int64_t row) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = (gl + c * group) * 8;
        v[c].zero();
        if (row < end && col < p.h) {
          if (p.y) v[c].y.load(static_cast<const T*>(p.y) + row * p.h + col);
          if (p.r) v[c].r.load(static_cast<const T*>(p.r) + row * p.h + col);
          if (p.dr) v[c].dr.load(static_cast<const T*>(p.dr) + row * p.h + col);
          if (p.du) v[c].du.load(static_cast<const T*>(p.du) + row * p.h + col);
        }
      }
    };
    load(at + tid / group);
    for (; at < end; at += ngroups) {  // the same for every thread
      const int64_t row = at + tid / group;
      const bool live = row < end;
      F2 s2[6] = {zero, zero, zero, zero, zero, zero};
      GradColumns<T> now[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        now[c] = v[c];
        now[c].sums(wt[c], pre[c], s2);
      }
      if constexpr (sizeof(T) == 2 || CH == 1) load(row + ngroups);  // (no registers for it in the others)
      float total[6];
#pragma unroll
      for (int k = 0; k < 6; ++k) total[k] = group_sum(sum2(s2[k]), group);
      const RowFactors<NORMED> f(total, p);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = (gl + c * group) * 8;
        F2 ox[4], oy[4];
        now[c].stay_packed();
        now[c].grads(wt[c], pre[c], f, p.alpha, ox, oy, acc_s[c], acc_pre[c]);
        if (live && col < p.h) {
          Vec8<T>::store(static_cast<T*>(p.dx) + row * p.h + col, ox);
          Vec8<T>::store(static_cast<T*>(p.dy) + row * p.h + col, oy);
        }
      }
      if constexpr (sizeof(T) == 4 && CH == 2) load(row + ngroups);
    }
    at = end;
    if (p.gate || p.post) {
      F2 sum[4];
      cta_sum<NW>(red, kSmallH, p.h, group, acc_s, sum);
      if (tid * 8 < p.h) leave_sequence(p, seq, first, last, tid * 8, sum, none_left);
    }
    none_left = false;
  }
  grid_dependents_may_start();
  F2 sum[4];
  cta_sum<NW>(red, kSmallH, p.h, group, acc_pre, sum);
  if (tid * 8 < p.h) Vec8<float>::store(p.partials + (static_cast<int64_t>(blockIdx.x) * 2 + 1) * p.h + tid * 8, sum);
}

// ------------------------------------------------------------------ a warp for a row

// The backward of rows of 257 to 512 columns, and of bf16 rows of up to 1024, where sequences are long: a warp takes a row, every
// NW-th of its CTA's part of a sequence, from a ring of bulk copies of its own, so that no barrier stands between two rows.
// NW: a multiple of the SM's four schedulers (10 and 14 warps are slower than 8 and 12), as many as registers (CH vectors of 8
// columns a lane) allow. Against a lane group's or a CTA's rows: bf16, 65536 rows of 512 71 us for 86, 384 70 for 81; 32768 of 768
// 59 for 80, 640 59 for 80, 1024 72 for 93 (0.82 of the copy rate); fp32, 32768 of 512 70 for 79, 264 47 for 60.
template <typename T, int NW, int CH, bool NORMED>
__global__ void __launch_bounds__(NW * 32, 1)
    residual_norm_warp_backward_kernel(const __grid_constant__ Backward p, int stages, unsigned int* status) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int64_t first = first_row(p.rows, blockIdx.x, gridDim.x), last = first_row(p.rows, blockIdx.x + 1, gridDim.x);
  RowRing<4> ring;  // the warp's, of rows counted from the tensors' first
  ring.row_bytes = static_cast<uint32_t>(p.h) * sizeof(T);
  ring.step = ring.row_bytes;
  ring.stages = stages;
  const size_t ring_bytes = static_cast<size_t>(stages) * ring.stage_bytes();
  ring.smem = smem + w * ring_bytes;
  float4* red = reinterpret_cast<float4*>(smem + NW * ring_bytes);  // [NW][h / 4]
  ring.full = reinterpret_cast<uint64_t*>(red + NW * p.h / 4) + w * stages;
  const void* src[4] = {p.y, p.r, p.dr, p.du};
#pragma unroll
  for (int k = 0; k < 4; ++k) ring.src[k] = static_cast<const uint8_t*>(src[k]);

  // The warp's rows in order, as far as they have been asked for (lane 0).
  int64_t ask_end = min(last, (first / p.s + 1) * p.s), ask = first + w;
  RowStage into;
  auto ask_next = [&](int64_t& count) {
    while (ask >= ask_end && ask_end < last) {
      ask = ask_end + w;
      ask_end = min(last, ask_end + p.s);
    }
    if (ask >= ask_end) return;
    ring.issue(ask, into.st);
    into.next(stages);
    ask += NW;
    ++count;
  };
  int64_t asked = 0, used = 0;
  if (lane == 0) {
    ring.init();
    for (int i = 0; i < stages; ++i) ask_next(asked);
  }
  __syncthreads();

  const F2 zero = f2_make(0.f, 0.f);
  F2 wt[CH][4], pre[CH][4], acc_s[CH][4], acc_pre[CH][4];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    load_gain(pre[c], p.pre, (lane + c * 32) * 8, p.h);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc_pre[c][e] = zero;
  }
  RowStage at;
  bool ok = true, none_left = true;
  for (int64_t begin = first; begin < last;) {
    const int64_t seq = begin / p.s, end = min(last, (seq + 1) * p.s);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (lane + c * 32) * 8;
      F2 g[4];
      load_gain(wt[c], p.post, col, p.h);
      load_gain(g, p.gate ? p.gate + seq * p.h : nullptr, col, p.h);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        wt[c][e] = f2_mul(wt[c][e], g[e]);
        acc_s[c][e] = zero;
      }
    }
    // A row's sums go through the warp while the row before it has its gradients worked out.
    auto columns = [&](int c, int st) {
      const int col = (lane + c * 32) * 8;
      GradColumns<T> v;
      v.zero();
      if (col < p.h) {
        if (p.y) v.y.load(ring.template at<T>(st, 0) + col);
        if (p.r) v.r.load(ring.template at<T>(st, 1) + col);
        if (p.dr) v.dr.load(ring.template at<T>(st, 2) + col);
        if (p.du) v.du.load(ring.template at<T>(st, 3) + col);
      }
      return v;
    };
    RowStage here;
    float total[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int64_t row = begin + w - NW; row < end && ok; row += NW) {
      const bool next = row + NW < end, now = row >= begin;
      F2 s2[6] = {zero, zero, zero, zero, zero, zero};
      if (next) {
        ok = __all_sync(0xffffffffu, mbar_wait(&ring.full[at.st], at.phase, status, 65));
        if (!ok) break;
        ++used;
#pragma unroll
        for (int c = 0; c < CH; ++c) columns(c, at.st).sums(wt[c], pre[c], s2);
      }
      const RowFactors<NORMED> f(total, p);
      float s8[8] = {sum2(s2[0]), sum2(s2[1]), sum2(s2[2]), sum2(s2[3]), sum2(s2[4]), sum2(s2[5]), 0.f, 0.f};
      const float mine = warp_sums8(s8, lane);
#pragma unroll
      for (int k = 0; k < 6; ++k) total[k] = __shfl_sync(0xffffffffu, mine, 4 * k);
      if (now) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int col = (lane + c * 32) * 8;
          F2 ox[4], oy[4];
          columns(c, here.st).grads(wt[c], pre[c], f, p.alpha, ox, oy, acc_s[c], acc_pre[c]);
          if (col < p.h) {
            Vec8<T>::store(static_cast<T*>(p.dx) + row * p.h + col, ox);
            Vec8<T>::store(static_cast<T*>(p.dy) + row * p.h + col, oy);
          }
        }
        __syncwarp();  // nobody reads the stage any more
        if (lane == 0) ask_next(asked);
      }
      here = at;
      if (next) at.next(stages);
    }
    begin = end;
    if (p.gate || p.post) {
      F2 sum[4];
      cta_sum<NW>(red, p.h, p.h, 32, acc_s, sum);
      if (tid * 8 < p.h) leave_sequence(p, seq, first, last, tid * 8, sum, none_left);
    }
    none_left = false;
  }
  grid_dependents_may_start();
  if (!ok && lane == 0) ring.drain(used, asked, status, 66);
  F2 sum[4];
  cta_sum<NW>(red, p.h, p.h, 32, acc_pre, sum);
  if (tid * 8 < p.h) Vec8<float>::store(p.partials + (static_cast<int64_t>(blockIdx.x) * 2 + 1) * p.h + tid * 8, sum);
}

// ------------------------------------------------------------------ the sums over CTAs

// 32 columns a CTA. Groups of 8 threads each add every 32nd row of partials, then the groups' sums are added by a fixed
// tree. CTAs [0, slices) sum dgamma_post, [slices, 2 slices) dgamma_pre, the others dgate of the sequences that several CTAs
// had rows of: found by sequence, or by the ends of CTAs' rows where there are fewer of those. Launched as a programmatic
// dependent of the backward kernel.
constexpr int kFinishThreads = 256;
struct Finish {
  const float *partials, *slots, *post;
  float *dpost, *dpre, *dgate;
  int64_t rows, s;
  int h, slices, ctas;
  bool by_cta;
};
__global__ void __launch_bounds__(kFinishThreads) residual_norm_finish_kernel(const __grid_constant__ Finish p) {
  grid_wait_for_previous();
  constexpr int kQuads = 8, kGroups = kFinishThreads / kQuads;
  __shared__ float4 grp[kGroups][kQuads];
  const int q = threadIdx.x % kQuads, g = threadIdx.x / kQuads;
  const int part = blockIdx.x / p.slices;
  const int col = (blockIdx.x % p.slices) * 32 + q * 4;
  const bool in = col < p.h;
  const float* src;
  int64_t n, stride = 2 * static_cast<int64_t>(p.h);
  float* out;
  if (part < 2) {
    src = p.partials + part * p.h;
    n = p.ctas;
    out = part == 0 ? p.dpost : p.dpre;
    if (!out) return;
  } else {
    auto cta_of = [&](int64_t row) {
      const int64_t each = p.rows / p.ctas, more = p.rows % p.ctas;
      return row < more * (each + 1) ? row / (each + 1) : more + (row - more * (each + 1)) / each;
    };
    const int64_t seq = p.by_cta ? (first_row(p.rows, part - 1, p.ctas) - 1) / p.s : part - 2;
    const int64_t c0 = cta_of(seq * p.s), c1 = cta_of((seq + 1) * p.s - 1);
    if (c0 == c1 || (p.by_cta && c0 != part - 2)) return;  // written by its CTA; found at an earlier end too
    src = p.slots + (2 * c0 + 1) * p.h;  // then slots 2 c0 + 2, 2 c0 + 4, ..
    n = c1 - c0 + 1;
    out = p.dgate + seq * p.h;
  }
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (in) {
#pragma unroll 8
    for (int64_t k = g; k < n; k += kGroups) {
      const float* from = part < 2 || k == 0 ? src + k * stride : src + k * stride - p.h;
      const float4 v = *reinterpret_cast<const float4*>(from + col);
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
    }
  }
  grp[g][q] = acc;
#pragma unroll
  for (int half = kGroups / 2; half > 0; half >>= 1) {
    __syncthreads();
    if (g < half) {
      const float4 o = grp[g + half][q];
      acc.x += o.x;
      acc.y += o.y;
      acc.z += o.z;
      acc.w += o.w;
      grp[g][q] = acc;
    }
  }
  if (g == 0 && in) {
    if (part >= 2 && p.post) {
      const float4 w = *reinterpret_cast<const float4*>(p.post + col);
      acc = make_float4(acc.x * w.x, acc.y * w.y, acc.z * w.z, acc.w * w.w);
    }
    *reinterpret_cast<float4*>(out + col) = acc;
  }
}

// ------------------------------------------------------------------ host side

int small_group(int h) {
  int group = 4;
  while (group < 32 && group * 8 < h) group *= 2;
  return group;
}

// CTAs of one resident wave of `kernel`, at most `most`.
template <typename K>
cudaError_t wave(int64_t* ctas, K kernel, int threads, size_t smem, int64_t most, const DeviceCtx& ctx) {
  if (most <= ctx.num_sms) {  // nothing to ask
    *ctas = most;
    return cudaSuccess;
  }
  int per_sm = 0;
  const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem);
  if (e != cudaSuccess) return e;
  *ctas = std::max<int64_t>(1, std::min<int64_t>(most, static_cast<int64_t>(std::max(per_sm, 1)) * ctx.num_sms));
  return cudaSuccess;
}

size_t ring_smem(int tensors, int h, size_t size, int stages) {
  return stages * (static_cast<size_t>(tensors) * h * size + sizeof(uint64_t));
}

// Threads of a CTA: a row's vectors of 8 columns, CH a thread, in whole warps.
int row_threads(int h, int ch) { return ((h + 8 * ch - 1) / (8 * ch) + 31) / 32 * 32; }

template <typename T, int NT, int CH>
cudaError_t forward_rows(Forward p, cudaStream_t stream, const DeviceCtx& ctx) {
  static SmemLimit limit;
  const int stages = std::min<int>(4, static_cast<int>(100 * 1024 / ring_smem(2, p.h, sizeof(T), 1)));
  auto kernel = residual_norm_row_kernel<T, NT, CH>;
  const size_t smem = ring_smem(2, p.h, sizeof(T), std::max(stages, 2));
  cudaError_t e = allow_smem(&limit, kernel, 200 * 1024, ctx);
  if (e != cudaSuccess) return e;
  int64_t ctas;
  const int threads = row_threads(p.h, CH);
  if ((e = wave(&ctas, kernel, threads, smem, p.rows, ctx)) != cudaSuccess) return e;
  p.run_of_rows = p.gate && p.s < 4 * ctas && p.s < p.rows;
  kernel<<<static_cast<unsigned>(ctas), threads, smem, stream>>>(p, std::max(stages, 2), ctx.status);
  return cudaGetLastError();
}

template <typename T>
cudaError_t forward_for(const Forward& p, cudaStream_t stream, const DeviceCtx& ctx) {
  if (p.h <= kSmallH) {
    const int group = small_group(p.h);
    const int64_t need = (p.rows * group + kSmallThreads - 1) / kSmallThreads;
    const unsigned ctas = static_cast<unsigned>(std::min<int64_t>(need, static_cast<int64_t>(ctx.num_sms) * 4));
    if (p.h <= 256)
      residual_norm_small_kernel<T, 1><<<ctas, kSmallThreads, 0, stream>>>(p, group);
    else
      residual_norm_small_kernel<T, 2><<<ctas, kSmallThreads, 0, stream>>>(p, group);
    return cudaGetLastError();
  }
  if (p.h <= 1024) return forward_rows<T, 64, 2>(p, stream, ctx);
  if (p.h <= 2048) return forward_rows<T, 128, 2>(p, stream, ctx);
  if (p.h <= 4096) return forward_rows<T, 256, 2>(p, stream, ctx);
  return forward_rows<T, 512, 2>(p, stream, ctx);
}

template <typename T, bool NORMED, int NT, int CH, int MINB, bool HOLD, bool RING = true>
cudaError_t backward_rows(const Backward& p, int64_t* ctas, cudaStream_t stream, const DeviceCtx& ctx) {
  static SmemLimit limit;
  // the row whose gradients are worked out, the next one, and one on its way
  const int stages = RING ? std::min<int>(3, static_cast<int>(200 * 1024 / ring_smem(4, p.h, sizeof(T), 1))) : 0;
  auto kernel = residual_norm_row_backward_kernel<T, NT, CH, MINB, HOLD, RING, NORMED>;
  const size_t smem = ring_smem(4, p.h, sizeof(T), stages);
  cudaError_t e = allow_smem(&limit, kernel, 200 * 1024, ctx);
  if (e != cudaSuccess) return e;
  const int threads = row_threads(p.h, CH);
  if ((e = wave(ctas, kernel, threads, smem, std::min<int64_t>(p.rows, kMaxCtas), ctx)) != cudaSuccess) return e;
  kernel<<<static_cast<unsigned>(*ctas), threads, smem, stream>>>(p, stages, ctx.status);
  return cudaGetLastError();
}

template <typename T, bool NORMED, int NW, int CH>
cudaError_t backward_warps(const Backward& p, int64_t* ctas, cudaStream_t stream, const DeviceCtx& ctx) {
  static SmemLimit limit;
  constexpr size_t kSmem = 226 * 1024;
  const size_t sums = static_cast<size_t>(NW) * p.h * sizeof(float);
  const int stages = std::min<int>(6, static_cast<int>((kSmem - sums) / NW / ring_smem(4, p.h, sizeof(T), 1)));
  // a row whose gradients are worked out and the next one, at the widest rows too
  static_assert((kSmem - NW * CH * 1024) / NW / (4 * CH * 256 * sizeof(T) + sizeof(uint64_t)) >= 2, "two stages a warp");
  auto kernel = residual_norm_warp_backward_kernel<T, NW, CH, NORMED>;
  const cudaError_t e = allow_smem(&limit, kernel, kSmem, ctx);
  if (e != cudaSuccess) return e;
  *ctas = std::min<int64_t>((p.rows + NW - 1) / NW, ctx.num_sms);
  kernel<<<static_cast<unsigned>(*ctas), NW * 32, NW * ring_smem(4, p.h, sizeof(T), stages) + sums, stream>>>(p, stages, ctx.status);
  return cudaGetLastError();
}

template <typename T, bool NORMED>
cudaError_t backward_for(const Backward& p, int64_t* ctas, cudaStream_t stream, const DeviceCtx& ctx) {
  // Each sequence costs a CTA the sums over its warps, and a warp wants rows to have the next one's loads under way (bf16 rows of
  // 1000 or so: 1400 in all 13.7 us against a CTA's 11.3, 8192 26 against 29; sequences of 64, 8320 rows 40.4 and 41.5).
  const bool warps = p.s >= 64 && p.rows >= 4800;
  if (warps && p.h > 256 && p.h <= kSmallH) return backward_warps<T, NORMED, 12, 2>(p, ctas, stream, ctx);
  if (p.h <= kSmallH) {
    const int group = small_group(p.h);
    const int64_t need = (p.rows * group + kSmallThreads - 1) / kSmallThreads;
    *ctas = std::min<int64_t>(need, std::min<int64_t>(static_cast<int64_t>(ctx.num_sms) * 2, kMaxCtas));
    if (p.h <= 256)
      residual_norm_small_backward_kernel<T, 1, NORMED><<<static_cast<unsigned>(*ctas), kSmallThreads, 0, stream>>>(p, group);
    else
      residual_norm_small_backward_kernel<T, 2, NORMED><<<static_cast<unsigned>(*ctas), kSmallThreads, 0, stream>>>(p, group);
    return cudaGetLastError();
  }
  constexpr bool kHold = sizeof(T) == 4;
  if constexpr (!kHold) {
    if (warps && p.h <= 768) return backward_warps<T, NORMED, 8, 3>(p, ctas, stream, ctx);
    if (warps && p.h <= 1024) return backward_warps<T, NORMED, 8, 4>(p, ctas, stream, ctx);
  }
  if (p.h <= 1024) return backward_rows<T, NORMED, 128, 1, 4, kHold>(p, ctas, stream, ctx);
  if constexpr (!kHold) {
    if (p.h <= 2048) return backward_rows<T, NORMED, 128, 2, 4, kHold>(p, ctas, stream, ctx);
    if (p.h <= 4096) return backward_rows<T, NORMED, 256, 2, 2, kHold>(p, ctas, stream, ctx);
    return backward_rows<T, NORMED, 512, 2, 1, kHold>(p, ctas, stream, ctx);
  } else {
    if (p.h <= 2048) return backward_rows<T, NORMED, 256, 1, 2, kHold>(p, ctas, stream, ctx);
    if (p.h <= 4096) return backward_rows<T, NORMED, 512, 1, 1, kHold>(p, ctas, stream, ctx);
    return backward_rows<T, NORMED, 512, 2, 1, false, false>(p, ctas, stream, ctx);  // no ring of two rows, nor registers for one
  }
}

template <typename T>
cudaError_t backward_for(const Backward& p, int64_t* ctas, cudaStream_t stream, const DeviceCtx& ctx) {
  return p.post ? backward_for<T, true>(p, ctas, stream, ctx) : backward_for<T, false>(p, ctas, stream, ctx);
}

tpmlp_status check_norm_shape(float alpha, float eps, int64_t b, int64_t s, int64_t h, tpmlp_dtype dt) {
  if (dt != TPMLP_BF16 && dt != TPMLP_F32) return err(TPMLP_ERR_DTYPE, "unsupported dtype");
  if (b < 0 || s < 0) return err(TPMLP_ERR_SHAPE, "need b, s >= 0");
  if (b > 0 && s > INT32_MAX / b) return err(TPMLP_ERR_SHAPE, "b * s exceeds 2^31-1");
  if (h < 8 || h % 8 != 0 || h > kMaxH) return err(TPMLP_ERR_SHAPE, "h must be a multiple of 8, 8 <= h <= 8192");
  if (!(eps > 0.0f) || !std::isfinite(eps)) return err(TPMLP_ERR_INVALID, "eps must be positive and finite");
  if (!std::isfinite(alpha)) return err(TPMLP_ERR_INVALID, "alpha must be finite");
  return TPMLP_OK;
}

constexpr const char* kAlign = "pointers must be 16-byte aligned";

size_t partials_bytes(int64_t b, int64_t s, int64_t h, bool gate) {
  const int64_t rows = std::min<int64_t>(b * s, kMaxCtas);
  return static_cast<size_t>(gate ? 4 : 2) * rows * h * sizeof(float);
}

}  // namespace
}  // namespace tpmlp

using namespace tpmlp;

extern "C" {

tpmlp_status tpmlp_residual_norm(const void* x, const void* y, const float* gamma_post, const float* gate,
                                 const float* gamma_pre, float alpha, float eps, void* r, void* u, int64_t b, int64_t s,
                                 int64_t h, tpmlp_dtype dt, void* stream) {
  TPMLP_PASS(check_norm_shape(alpha, eps, b, s, h, dt));
  if (b * s == 0) return TPMLP_OK;
  if (!gamma_pre != !u) return err(TPMLP_ERR_INVALID, "gamma_pre and u go together");
  TPMLP_PASS(check_ptrs({x, y, r}, 16, kAlign));
  for (const void* p : {static_cast<const void*>(gamma_post), static_cast<const void*>(gate),
                        static_cast<const void*>(gamma_pre), static_cast<const void*>(u)})
    if (!aligned(p, 16)) return err(TPMLP_ERR_ALIGN, kAlign);
  const int64_t rows = b * s, size = dt == TPMLP_BF16 ? 2 : 4;
  auto of = [&](const void* p) { return flat_region(p, rows * h, size); };
  auto meets = [&](const void* out, const void* in) { return out && out != in && overlap(of(out), of(in)); };
  if (any_overlap({of(r), of(u)}, {flat_region(gamma_post, h, 4), flat_region(gate, b * h, 4), flat_region(gamma_pre, h, 4)}) ||
      meets(r, x) || meets(r, y) || meets(u, x) || meets(u, y))
    return err(TPMLP_ERR_INVALID, "r or u overlaps another tensor of the call (they may be x or y)");
  DeviceCtx ctx;
  TPMLP_PASS_CUDA(get_device_ctx(&ctx), "device context");
  const Forward p{x, y, gamma_post, gate, gamma_pre, r, u, alpha, eps, 1.0f / static_cast<float>(h), rows, s, static_cast<int>(h), false};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  TPMLP_PASS_CUDA(dt == TPMLP_BF16 ? forward_for<__nv_bfloat16>(p, st, ctx) : forward_for<float>(p, st, ctx), "residual norm");
  return TPMLP_OK;
}

size_t tpmlp_residual_norm_backward_workspace_size(int64_t b, int64_t s, int64_t h, int gate) {
  if (b <= 0 || s <= 0 || h <= 0) return 0;
  return partials_bytes(b, s, h, gate != 0);
}

tpmlp_status tpmlp_residual_norm_backward(const void* y, const void* r, const void* dr, const void* du,
                                          const float* gamma_post, const float* gate, const float* gamma_pre, float alpha,
                                          float eps, void* dx, void* dy, float* dgamma_post, float* dgate, float* dgamma_pre,
                                          int64_t b, int64_t s, int64_t h, tpmlp_dtype dt, void* workspace, size_t ws_bytes,
                                          void* stream) {
  TPMLP_PASS(check_norm_shape(alpha, eps, b, s, h, dt));
  if (!gamma_post != !dgamma_post || !gate != !dgate || !gamma_pre != !dgamma_pre)
    return err(TPMLP_ERR_INVALID, "gamma_post, gate and gamma_pre go with their gradients");
  for (const void* p : {static_cast<const void*>(dgamma_post), static_cast<const void*>(dgate),
                        static_cast<const void*>(dgamma_pre)})
    if (!aligned(p, 16)) return err(TPMLP_ERR_ALIGN, kAlign);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (b * s == 0) {
    if (dgamma_post) TPMLP_PASS_CUDA(cudaMemsetAsync(dgamma_post, 0, h * sizeof(float), st), "zero dgamma_post");
    if (dgamma_pre) TPMLP_PASS_CUDA(cudaMemsetAsync(dgamma_pre, 0, h * sizeof(float), st), "zero dgamma_pre");
    if (dgate && b > 0) TPMLP_PASS_CUDA(cudaMemsetAsync(dgate, 0, b * h * sizeof(float), st), "zero dgate");
    return TPMLP_OK;
  }
  if (!gamma_pre != !du) return err(TPMLP_ERR_INVALID, "gamma_pre and du go together");
  if (!dr && !du) return err(TPMLP_ERR_INVALID, "dr may be NULL only beside du");
  TPMLP_PASS(check_ptrs({dx, dy}, 16, kAlign));
  if (gamma_post || gate) TPMLP_PASS(check_ptrs({y}, 16, kAlign));
  if (gamma_pre) TPMLP_PASS(check_ptrs({r}, 16, kAlign));
  if (!gamma_post && !gate) y = nullptr;  // not read
  if (!gamma_pre) r = nullptr;
  for (const void* p : {static_cast<const void*>(gamma_post), static_cast<const void*>(gate),
                        static_cast<const void*>(gamma_pre), dr, du})
    if (!aligned(p, 16)) return err(TPMLP_ERR_ALIGN, kAlign);
  const size_t need = partials_bytes(b, s, h, gate != nullptr);
  if (!workspace || ws_bytes < need) return err(TPMLP_ERR_WORKSPACE, "residual norm backward workspace too small");
  if (!aligned(workspace, 256)) return err(TPMLP_ERR_ALIGN, "workspace not 256-byte aligned");
  const int64_t rows = b * s, size = dt == TPMLP_BF16 ? 2 : 4;
  auto of = [&](const void* p) { return flat_region(p, rows * h, size); };
  const Region gains[] = {flat_region(gamma_post, h, 4), flat_region(gate, b * h, 4), flat_region(gamma_pre, h, 4)};
  bool bad = any_overlap({of(dx), of(dy), flat_region(dgamma_post, h, 4), flat_region(dgate, b * h, 4),
                          flat_region(dgamma_pre, h, 4), flat_region(workspace, static_cast<int64_t>(need), 1)},
                         {gains[0], gains[1], gains[2]}) ||
             any_overlap({flat_region(dgamma_post, h, 4), flat_region(dgate, b * h, 4), flat_region(dgamma_pre, h, 4),
                          flat_region(workspace, static_cast<int64_t>(need), 1)},
                         {of(y), of(r), of(dr), of(du)});
  for (const void* in : {y, r, dr, du})
    for (const void* out : {static_cast<const void*>(dx), static_cast<const void*>(dy)})
      bad = bad || (in && in != out && overlap(of(out), of(in)));
  if (bad) return err(TPMLP_ERR_INVALID, "an output or the workspace overlaps another tensor of the call (dx and dy may be y, r, dr or du)");
  DeviceCtx ctx;
  TPMLP_PASS_CUDA(get_device_ctx(&ctx), "device context");
  if (!gate) {  // one run of tokens
    s = rows;
    b = 1;
  }
  float* partials = static_cast<float*>(workspace);
  float* slots = gate ? partials + 2 * std::min<int64_t>(rows, kMaxCtas) * h : nullptr;
  const Backward p{y, r, dr, du, gamma_post, gate, gamma_pre, dx, dy, dgate, partials, slots, alpha, eps,
                   1.0f / static_cast<float>(h), rows, s, static_cast<int>(h)};
  int64_t ctas = 0;
  TPMLP_PASS_CUDA(dt == TPMLP_BF16 ? backward_for<__nv_bfloat16>(p, &ctas, st, ctx) : backward_for<float>(p, &ctas, st, ctx),
                  "residual norm backward");
  if (!dgamma_post && !dgamma_pre && !dgate) return TPMLP_OK;
  const int slices = static_cast<int>((h + 31) / 32);
  const bool by_cta = b > ctas - 1;
  const Finish f{partials, slots, gamma_post, dgamma_post, dgamma_pre, dgate, rows, s, static_cast<int>(h), slices,
                 static_cast<int>(ctas), by_cta};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((2 + (!gate ? 0 : by_cta ? ctas - 1 : b)) * slices), 1, 1);
  cfg.blockDim = dim3(kFinishThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  TPMLP_PASS_CUDA(cudaLaunchKernelEx(&cfg, residual_norm_finish_kernel, f), "residual norm sums");
  return TPMLP_OK;
}

}  // extern "C"
