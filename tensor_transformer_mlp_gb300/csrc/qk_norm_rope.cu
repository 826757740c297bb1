// RMSNorm of every query and key head and the rotation by position in one pass, and its backward
// (tpmlp_qk_norm_rope, tpmlp_qk_norm_rope_backward).
//
//   u = x r gamma, r = 1 / sqrt(mean(x^2) + eps) over one head's columns;  y = R(pos) u
//   du = R(pos)^T dy, g = du gamma;  dx = r (g - x_hat mean(g x_hat));  dgamma = sum du x_hat
//
// Both are bound by memory (about 4 flops a byte): q and k are read once and written once. A head's
// columns lie eight to a lane on a group of G lanes (the power of two that covers head_dim / 8), so one
// 16-byte load fetches a lane's bf16 share and the row sums are log2(G) shuffles. A group takes up to
// kHeads heads of one token, all queries or all keys, so that what the position and the gain contribute is
// loaded once for them, and loads some of them ahead of their arithmetic, which runs on fp32 pairs.
// Pairs of the half style are brought together by shuffles of the loaded words, before the norm is known.
// Measured at b2 s2048, 32 + 32 heads of 128, share of the copy rate: bf16 half style forward 29.0 us (0.69), backward with
// the gains' sums 48.0 us (0.63); interleaved 28.0 (0.72) and 49.4 us (0.61); 40 columns turned in halves, which pair up
// through shared memory, 46 (0.44) and 66 us (0.46). fp32: 47.8 (0.84) and 69.8 us (0.86), interleaved 48.5 (0.83) and 68.6 us
// (0.88), 40 columns 63.7 (0.63) and 84.8 us (0.71). In bf16 what is left is latency at the ends of the grid's waves and 54
// to 58 % of the issue slots.
// The inverse root is rsqrtf (2 units in the last place at most) and the gains' gradients are summed in fp32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "abi_checks.h"
#include "device_common.cuh"

namespace tpmlp {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxHeadDim = 256;
constexpr int kBwdMaxCtas = 1024;
constexpr int kHeads = 8;
// Heads of a group loaded before the first is worked on: forward 128 bytes a thread (with three CTAs an SM 29.9 us at the
// size of a GPT layer, b2 s2048, 32 heads of 128; 64 bytes and four CTAs 30.4, and single tokens 4.6 us for 4.0),
// backward 64 of each of its two tensors. The fp32 forwards do not quite fit three CTAs' registers (36 to 124 bytes a thread
// go through the L1) and run at 0.83 of the copy rate all the same.
template <typename T>
constexpr int kForwardBatch = 16 / sizeof(T);
template <typename T>
constexpr int kBatch = 8 / sizeof(T);

// Queries and keys go through the same code as parts 0 and 1.
struct RopePart {
  HeadView x, y, dx;    // forward: input, output; backward: input, dy, dx
  const float* gamma;
  int heads, chunks;    // chunks = ceil(heads / kHeads)
};

struct RopeParams {
  RopePart part[2];
  const float *cos_t, *sin_t;
  const int* pos;
  int64_t table_len;
  int64_t tokens, s;
  int hd, rot, group, ctas0;  // CTAs [0, ctas0) work on the queries, the others on the keys
  int table_vec;              // the tables can be read 16 bytes at a time
  float eps, inv_hd;
};

// Eight columns as they lie in memory, and as four fp32 pairs.
template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void unpack(F2 (&f)[4]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2_make(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  __device__ __forceinline__ Vec8 from_lane(int src) const {
    Vec8 o;
    o.v = make_uint4(__shfl_sync(0xffffffffu, v.x, src), __shfl_sync(0xffffffffu, v.y, src),
                     __shfl_sync(0xffffffffu, v.z, src), __shfl_sync(0xffffffffu, v.w, src));
    return o;
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
  __device__ __forceinline__ void unpack(F2 (&f)[4]) const {
    f[0] = f2_make(a.x, a.y);
    f[1] = f2_make(a.z, a.w);
    f[2] = f2_make(b.x, b.y);
    f[3] = f2_make(b.z, b.w);
  }
  __device__ __forceinline__ Vec8 from_lane(int src) const {
    Vec8 o;
    o.a = make_float4(__shfl_sync(0xffffffffu, a.x, src), __shfl_sync(0xffffffffu, a.y, src),
                      __shfl_sync(0xffffffffu, a.z, src), __shfl_sync(0xffffffffu, a.w, src));
    o.b = make_float4(__shfl_sync(0xffffffffu, b.x, src), __shfl_sync(0xffffffffu, b.y, src),
                      __shfl_sync(0xffffffffu, b.z, src), __shfl_sync(0xffffffffu, b.w, src));
    return o;
  }
  static __device__ __forceinline__ void store(float* p, const F2 (&f)[4]) {
    const float2 t0 = f2_split(f[0]), t1 = f2_split(f[1]), t2 = f2_split(f[2]), t3 = f2_split(f[3]);
    reinterpret_cast<float4*>(p)[0] = make_float4(t0.x, t0.y, t1.x, t1.y);
    reinterpret_cast<float4*>(p)[1] = make_float4(t2.x, t2.y, t3.x, t3.y);
  }
};

__device__ __forceinline__ float group_sum(float v, int group) {
  for (int o = group >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float sum4(const F2 (&f)[4]) {
  const float2 t = f2_split(f2_add(f2_add(f[0], f[1]), f2_add(f[2], f[3])));
  return t.x + t.y;
}

// How a column finds the other column of its pair: in its own lane (interleaved); in one other lane of the
// group, rot / 16 further or back (half style with rot / 2 a multiple of 8); or through shared memory.
enum Pairing { kOwnLane, kOtherLane, kAnyLane };

// One lane's share of the work: columns c0 .. c0 + 7, what turns them, and where their partners are. Column e
// of the turned head is f[e] * cs[e] + partner(e) * sn[e]; sn carries the sign of the forward turn or of its
// transpose (`back`), and columns past rot have 1 and 0.
template <int PAIRING>
struct LaneTurn {
  int lane, gl, c0, src;
  float* xch;  // the warp's 32 x 8 floats
  __device__ __forceinline__ LaneTurn(const RopeParams& p, float* xch_all) {
    lane = threadIdx.x & 31;
    gl = lane & (p.group - 1);
    c0 = gl * 8;
    xch = xch_all + (PAIRING == kAnyLane ? (threadIdx.x & ~31) * 8 : 0);
    const int step = p.rot >> 4;
    src = PAIRING != kOtherLane ? lane : gl < step ? lane + step : gl < 2 * step ? lane - step : lane;
  }
  __device__ __forceinline__ int partner_column(const RopeParams& p, int c) const {
    const int half = p.rot >> 1;
    return c >= p.rot ? c : PAIRING == kOwnLane ? c ^ 1 : c < half ? c + half : c - half;
  }
  __device__ __forceinline__ void angles(const RopeParams& p, int64_t pos, bool back, float (&cs)[8], float (&sn)[8]) const {
    const int half = p.rot >> 1;
    const float* ct = p.cos_t + pos * half;
    const float* st = p.sin_t + pos * half;
    if (pos >= p.table_len) {  // not covered: the rotated columns are no numbers
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        cs[e] = c0 + e < p.rot ? __int_as_float(0x7fffffff) : 1.f;
        sn[e] = 0.f;
      }
    } else if (PAIRING == kOtherLane && p.table_vec) {  // eight columns lie on one side of the pairs
      if (c0 < p.rot) {
        const int i = c0 < half ? c0 : c0 - half;
        const bool minus = (c0 < half) != back;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const float4 c = *reinterpret_cast<const float4*>(ct + i + 4 * v), s = *reinterpret_cast<const float4*>(st + i + 4 * v);
          cs[4 * v] = c.x; cs[4 * v + 1] = c.y; cs[4 * v + 2] = c.z; cs[4 * v + 3] = c.w;
          sn[4 * v] = minus ? -s.x : s.x; sn[4 * v + 1] = minus ? -s.y : s.y;
          sn[4 * v + 2] = minus ? -s.z : s.z; sn[4 * v + 3] = minus ? -s.w : s.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          cs[e] = 1.f;
          sn[e] = 0.f;
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = c0 + e;
        cs[e] = 1.f;
        sn[e] = 0.f;
        if (c < p.rot) {
          const int i = PAIRING == kOwnLane ? c >> 1 : (c < half ? c : c - half);
          const bool first = PAIRING == kOwnLane ? (c & 1) == 0 : c < half;
          cs[e] = ct[i];
          sn[e] = first != back ? -st[i] : st[i];
        }
      }
    }
  }
  // Every lane of the warp calls this.
  template <typename T>
  __device__ __forceinline__ void partners(const RopeParams& p, const Vec8<T>& x, const F2 (&f)[4], F2 (&other)[4]) const {
    if constexpr (PAIRING == kOwnLane) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 t = f2_split(f[e]);
        other[e] = f2_make(t.y, t.x);
      }
    } else if constexpr (PAIRING == kOtherLane) {
      x.from_lane(src).unpack(other);
    } else {
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 t = f2_split(f[e]);
        xch[lane * 8 + 2 * e] = t.x;
        xch[lane * 8 + 2 * e + 1] = t.y;
      }
      __syncwarp();
      const float* head = xch + (lane - gl) * 8;
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = head[partner_column(p, c0 + e)];
#pragma unroll
      for (int e = 0; e < 4; ++e) other[e] = f2_make(o[2 * e], o[2 * e + 1]);
    }
  }
};

__device__ __forceinline__ int64_t position_of(const RopeParams& p, int64_t token) {
  return p.pos ? static_cast<int64_t>(p.pos[token]) : token % p.s;
}

template <typename T, int PAIRING>
__global__ void __launch_bounds__(kThreads, 3) qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ float xch_all[PAIRING == kAnyLane ? kThreads * 8 : 1];
  const LaneTurn<PAIRING> t(p, xch_all);
  const bool keys = static_cast<int>(blockIdx.x) >= p.ctas0;
  const RopePart& a = p.part[keys ? 1 : 0];
  const int ngroups = kThreads / p.group;
  const int64_t item = static_cast<int64_t>(blockIdx.x - (keys ? p.ctas0 : 0)) * ngroups + threadIdx.x / p.group;
  int64_t token = item / a.chunks;
  const int h0 = static_cast<int>(item - token * a.chunks) * kHeads;
  const bool act = t.c0 < p.hd && token < p.tokens;
  if (token >= p.tokens) token = p.tokens - 1;  // idle, but it takes the shuffles
  const int64_t pos = position_of(p, token);
  const bool live = act && pos >= 0;
  const T* x = static_cast<const T*>(a.x.ptr) + token * a.x.ld + h0 * a.x.hs + t.c0;
  T* y = static_cast<T*>(a.y.ptr) + token * a.y.ld + h0 * a.y.hs + t.c0;
  F2 ca[4], cb[4];
#pragma unroll 1
  for (int hb = 0; hb < kHeads; hb += kForwardBatch<T>) {
    Vec8<T> v[kForwardBatch<T>];
#pragma unroll
    for (int u = 0; u < kForwardBatch<T>; ++u) {
      v[u].zero();
      if (live && h0 + hb + u < a.heads) v[u].load(x + (hb + u) * a.x.hs);
    }
    if (hb == 0) {  // y = r (f ca + partner cb)
      float cs[8], sn[8];
      t.angles(p, pos < 0 ? 0 : pos, false, cs, sn);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = min(t.c0 + e, p.hd - 1);
        cs[e] *= a.gamma[c];
        sn[e] *= a.gamma[t.partner_column(p, c)];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ca[e] = f2_make(cs[2 * e], cs[2 * e + 1]);
        cb[e] = f2_make(sn[2 * e], sn[2 * e + 1]);
      }
    }
#pragma unroll
    for (int u = 0; u < kForwardBatch<T>; ++u) {
      F2 f[4], other[4], sq[4];
      v[u].unpack(f);
      t.partners(p, v[u], f, other);
#pragma unroll
      for (int e = 0; e < 4; ++e) sq[e] = f2_mul(f[e], f[e]);
      const float ss = group_sum(sum4(sq), p.group);
      const float r = pos < 0 ? 0.f : rsqrtf(fmaf(ss, p.inv_hd, p.eps));
      const F2 r2 = f2_make(r, r);
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = f2_mul(r2, f2_fma(f[e], ca[e], f2_mul(other[e], cb[e])));
      if (act && h0 + hb + u < a.heads) Vec8<T>::store(y + (hb + u) * a.y.hs, f);
    }
  }
}

// partials: [gridDim.x][hd], the gain's gradient from the CTA's items (its groups added in order).
template <typename T, int PAIRING>
__global__ void __launch_bounds__(kThreads, 2)
    qk_norm_rope_backward_kernel(const __grid_constant__ RopeParams p, float* partials) {
  __shared__ float xch_all[kThreads * 8];
  const LaneTurn<PAIRING> t(p, xch_all);
  const bool keys = static_cast<int>(blockIdx.x) >= p.ctas0;
  const RopePart& a = p.part[keys ? 1 : 0];
  const int ngroups = kThreads / p.group;
  const int cta = blockIdx.x - (keys ? p.ctas0 : 0), ctas = keys ? gridDim.x - p.ctas0 : p.ctas0;
  const int64_t items = p.tokens * a.chunks;
  F2 acc[4], gain[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    acc[e] = f2_make(0.f, 0.f);
    gain[e] = f2_make(a.gamma[min(t.c0 + 2 * e, p.hd - 1)], a.gamma[min(t.c0 + 2 * e + 1, p.hd - 1)]);
  }
  // every group of the CTA makes the same number of rounds, so that all lanes take the shuffles
  for (int64_t first = static_cast<int64_t>(cta) * ngroups; first < items; first += static_cast<int64_t>(ctas) * ngroups) {
    const int64_t item = min(first + threadIdx.x / p.group, items - 1);
    const bool act = t.c0 < p.hd && first + threadIdx.x / p.group < items;
    const int64_t token = item / a.chunks;
    const int h0 = static_cast<int>(item - token * a.chunks) * kHeads;
    const int64_t pos = position_of(p, token);
    const bool live = act && pos >= 0;
    const T* x = static_cast<const T*>(a.x.ptr) + token * a.x.ld + h0 * a.x.hs + t.c0;
    const T* y = static_cast<const T*>(a.y.ptr) + token * a.y.ld + h0 * a.y.hs + t.c0;
    T* dx = static_cast<T*>(a.dx.ptr) + token * a.dx.ld + h0 * a.dx.hs + t.c0;
    F2 cs[4], sn[4];
#pragma unroll 1
    for (int hb = 0; hb < kHeads; hb += kBatch<T>) {
      Vec8<T> vx[kBatch<T>], vy[kBatch<T>];
#pragma unroll
      for (int u = 0; u < kBatch<T>; ++u) {
        vx[u].zero();
        vy[u].zero();
        if (live && h0 + hb + u < a.heads) {
          vx[u].load(x + (hb + u) * a.x.hs);
          vy[u].load(y + (hb + u) * a.y.hs);
        }
      }
      if (hb == 0) {
        float c8[8], s8[8];
        t.angles(p, pos < 0 ? 0 : pos, true, c8, s8);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          cs[e] = f2_make(c8[2 * e], c8[2 * e + 1]);
          sn[e] = f2_make(s8[2 * e], s8[2 * e + 1]);
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch<T>; ++u) {
        F2 f[4], d[4], other[4], s1[4], s2[4];
        vx[u].unpack(f);
        vy[u].unpack(d);
        t.partners(p, vy[u], d, other);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          d[e] = f2_fma(d[e], cs[e], f2_mul(other[e], sn[e]));  // du
          other[e] = f2_mul(d[e], f[e]);
          d[e] = f2_mul(d[e], gain[e]);                         // g
          s1[e] = f2_mul(f[e], f[e]);
          s2[e] = f2_mul(d[e], f[e]);
        }
        const float ss = group_sum(sum4(s1), p.group);
        const float gx = group_sum(sum4(s2), p.group);
        const float r = rsqrtf(fmaf(ss, p.inv_hd, p.eps));
        const float m = -gx * p.inv_hd * r * r;  // dx = r (g - x r^2 mean(g x)); r^3 would overflow from eps = 1e-26 down
        const bool on = act && h0 + hb + u < a.heads;
        const float ra = pos < 0 || !on ? 0.f : r;
        const F2 r2 = f2_make(pos < 0 ? 0.f : r, pos < 0 ? 0.f : r), m2 = f2_make(m, m), ra2 = f2_make(ra, ra);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[e] = f2_fma(other[e], ra2, acc[e]);
          d[e] = f2_mul(r2, f2_fma(f[e], m2, d[e]));
        }
        if (on) Vec8<T>::store(dx + (hb + u) * a.dx.hs, d);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 v = f2_split(acc[e]);
    xch_all[threadIdx.x * 8 + 2 * e] = v.x;
    xch_all[threadIdx.x * 8 + 2 * e + 1] = v.y;
  }
  __syncthreads();
  for (int c = threadIdx.x; c < p.hd; c += kThreads) {
    float sum = 0.f;
    for (int g = 0; g < ngroups; ++g) sum += xch_all[g * p.group * 8 + c];
    partials[static_cast<int64_t>(blockIdx.x) * p.hd + c] = sum;
  }
}

// Adds the CTAs' partials in a fixed order: 32 columns of one gain to a CTA, 32 threads for each, which add
// every 32nd partial and are joined by a tree. Launched as the backward's programmatic dependent.
__global__ void __launch_bounds__(1024)
    rope_gain_sum_kernel(const float* __restrict__ partials, int ctas0, int ctas, int hd, float* __restrict__ dgamma_q,
                         float* __restrict__ dgamma_k) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float red[32][33];
  const int col = threadIdx.x & 31, row = threadIdx.x >> 5, c = blockIdx.x * 32 + col;
  const int first = blockIdx.y ? ctas0 : 0, last = blockIdx.y ? ctas : ctas0;
  float sum = 0.f;
  if (c < hd) {
#pragma unroll 8
    for (int i = first + row; i < last; i += 32) sum += partials[static_cast<int64_t>(i) * hd + c];
  }
  red[row][col] = sum;
  for (int o = 16; o > 0; o >>= 1) {
    __syncthreads();
    if (row < o) red[row][col] += red[row + o][col];
  }
  if (row == 0 && c < hd) (blockIdx.y ? dgamma_k : dgamma_q)[c] = red[0][col];
}

tpmlp_status check_strides(int64_t b, int64_t s, int heads, int kv_heads, int hd, std::initializer_list<HeadView> inputs,
                           const HeadView& q_out, const HeadView& k_out) {
  for (const HeadView& v : inputs)
    if (!good_head_strides(v, s)) return err(TPMLP_ERR_SHAPE, "strides must be positive multiples of 8");
  if (!good_head_strides(q_out, s) || !good_head_strides(k_out, s))
    return err(TPMLP_ERR_SHAPE, "strides must be positive multiples of 8");
  if (!heads_apart(q_out, b * s, heads, hd) || !heads_apart(k_out, b * s, kv_heads, hd))
    return err(TPMLP_ERR_SHAPE, "an output's heads overlap");
  return TPMLP_OK;
}

tpmlp_status check(float eps, int64_t table_len, int rot, int style, int64_t b, int64_t s, int heads, int kv_heads,
                   int hd, tpmlp_dtype dt) {
  if (dt != TPMLP_BF16 && dt != TPMLP_F32) return err(TPMLP_ERR_DTYPE, "unsupported dtype");
  if (b < 0 || s < 0 || heads < 1 || kv_heads < 1)
    return err(TPMLP_ERR_SHAPE, "need b, s >= 0 and heads, kv_heads >= 1");
  if (b > 0 && s > INT32_MAX / b) return err(TPMLP_ERR_SHAPE, "b * s exceeds 2^31-1");
  if (heads > 65536 || kv_heads > 65536) return err(TPMLP_ERR_SHAPE, "at most 65536 heads");
  if (hd < 8 || hd % 8 != 0 || hd > kMaxHeadDim)
    return err(TPMLP_ERR_SHAPE, "head_dim must be a multiple of 8, 8 <= head_dim <= 256");
  if (rot < 2 || rot % 2 != 0 || rot > hd) return err(TPMLP_ERR_SHAPE, "rot_dim must be even, 2 <= rot_dim <= head_dim");
  if (table_len < 1) return err(TPMLP_ERR_SHAPE, "table_len must be >= 1");
  if (style != TPMLP_ROPE_HALF && style != TPMLP_ROPE_INTERLEAVED) return err(TPMLP_ERR_INVALID, "unknown rope style");
  if (!(eps > 0.0f)) return err(TPMLP_ERR_INVALID, "eps must be > 0");
  return TPMLP_OK;
}

RopeParams make_params(const RopePart& q, const RopePart& k, const float* cos_table, const float* sin_table,
                       const void* positions, int64_t table_len, int rot, int64_t b, int64_t s, int hd, float eps) {
  RopeParams p{};
  p.part[0] = q;
  p.part[1] = k;
  for (RopePart& a : p.part) a.chunks = (a.heads + kHeads - 1) / kHeads;
  p.cos_t = cos_table;
  p.sin_t = sin_table;
  p.pos = static_cast<const int*>(positions);
  p.table_len = table_len;
  p.tokens = b * s;
  p.s = s;
  p.hd = hd;
  p.rot = rot;
  for (p.group = 1; p.group * 8 < hd;) p.group *= 2;
  p.table_vec = aligned(cos_table, 16) && aligned(sin_table, 16) && (rot / 2) % 4 == 0;
  p.eps = eps;
  p.inv_hd = 1.0f / static_cast<float>(hd);
  return p;
}

// The kernel of a type and a pairing out of K<T, PAIRING>.
#define ROPE_PICK(K, dt, pairing)                                                                                  \
  ((dt) == TPMLP_BF16 ? ((pairing) == kOwnLane     ? K<__nv_bfloat16, kOwnLane>                                    \
                         : (pairing) == kOtherLane ? K<__nv_bfloat16, kOtherLane>                                  \
                                                   : K<__nv_bfloat16, kAnyLane>)                                   \
                      : ((pairing) == kOwnLane     ? K<float, kOwnLane>                                            \
                         : (pairing) == kOtherLane ? K<float, kOtherLane>                                          \
                                                   : K<float, kAnyLane>))

int pairing_of(int style, int rot) {
  return style == TPMLP_ROPE_INTERLEAVED ? kOwnLane : rot % 16 == 0 ? kOtherLane : kAnyLane;
}

}  // namespace
}  // namespace tpmlp

using namespace tpmlp;

extern "C" {

tpmlp_status tpmlp_qk_norm_rope(const void* q, const void* k, const float* gamma_q, const float* gamma_k, float eps,
                                const float* cos_table, const float* sin_table, const void* positions,
                                int64_t table_len, int rot_dim, int style, void* q_out, void* k_out, int64_t b,
                                int64_t s, int heads, int kv_heads, int head_dim, int64_t ld_q, int64_t hs_q,
                                int64_t ld_k, int64_t hs_k, int64_t ld_qo, int64_t hs_qo, int64_t ld_ko,
                                int64_t hs_ko, tpmlp_dtype dt, void* stream) {
  TPMLP_PASS(check(eps, table_len, rot_dim, style, b, s, heads, kv_heads, head_dim, dt));
  TPMLP_PASS(check_strides(b, s, heads, kv_heads, head_dim, {{nullptr, ld_q, hs_q}, {nullptr, ld_k, hs_k}},
                         {q_out, ld_qo, hs_qo}, {k_out, ld_ko, hs_ko}));
  if (b * s == 0) return TPMLP_OK;
  TPMLP_PASS(check_ptrs({q, k, q_out, k_out}, 16, "pointer not 16-byte aligned"));
  TPMLP_PASS(check_ptrs({gamma_q, gamma_k, cos_table, sin_table}, 4, "pointer not 4-byte aligned"));
  if (!aligned(positions, 4)) return err(TPMLP_ERR_ALIGN, "positions not 4-byte aligned");
  const int64_t tokens = b * s, size = dt == TPMLP_BF16 ? 2 : 4;
  auto of = [&](const void* p, int64_t ld, int64_t hs, int n) {
    return heads_region({const_cast<void*>(p), ld, hs}, tokens, n, head_dim, size);
  };
  const Region rq = of(q, ld_q, hs_q, heads), rk = of(k, ld_k, hs_k, kv_heads);
  const Region rqo = of(q_out, ld_qo, hs_qo, heads), rko = of(k_out, ld_ko, hs_ko, kv_heads);
  if (any_overlap({rqo, rko}, {flat_region(gamma_q, head_dim, 4), flat_region(gamma_k, head_dim, 4),
                               flat_region(cos_table, table_len, 2 * rot_dim), flat_region(sin_table, table_len, 2 * rot_dim),
                               flat_region(positions, tokens, 4)}) ||
      overlap(rqo, rk) || overlap(rko, rq) || (!same_region(rqo, rq) && overlap(rqo, rq)) ||
      (!same_region(rko, rk) && overlap(rko, rk)))
    return err(TPMLP_ERR_INVALID,
               "an output overlaps another tensor of the call (in place q_out is q and k_out is k, with the same strides)");
  RopeParams p = make_params({{const_cast<void*>(q), ld_q, hs_q}, {q_out, ld_qo, hs_qo}, {}, gamma_q, heads, 0},
                             {{const_cast<void*>(k), ld_k, hs_k}, {k_out, ld_ko, hs_ko}, {}, gamma_k, kv_heads, 0},
                             cos_table, sin_table, positions, table_len, rot_dim, b, s, head_dim, eps);
  const int64_t ngroups = kThreads / p.group;
  const int64_t ctas0 = (p.tokens * p.part[0].chunks + ngroups - 1) / ngroups;
  const int64_t ctas = ctas0 + (p.tokens * p.part[1].chunks + ngroups - 1) / ngroups;
  if (ctas > INT32_MAX) return err(TPMLP_ERR_SHAPE, "too many heads in all (b * s * heads)");
  p.ctas0 = static_cast<int>(ctas0);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto kernel = ROPE_PICK(qk_norm_rope_kernel, dt, pairing_of(style, rot_dim));
  kernel<<<static_cast<unsigned>(ctas), kThreads, 0, st>>>(p);
  TPMLP_PASS_CUDA(cudaGetLastError(), "qk_norm_rope");
  return TPMLP_OK;
}

size_t tpmlp_qk_norm_rope_backward_workspace_size(int64_t b, int64_t s, int head_dim) {
  if (b <= 0 || s <= 0 || head_dim <= 0) return 0;
  return static_cast<size_t>(kBwdMaxCtas) * static_cast<size_t>(head_dim) * sizeof(float);
}

tpmlp_status tpmlp_qk_norm_rope_backward(const void* q, const void* k, const float* gamma_q, const float* gamma_k,
                                         float eps, const float* cos_table, const float* sin_table,
                                         const void* positions, int64_t table_len, int rot_dim, int style,
                                         const void* dq_out, const void* dk_out, void* dq, void* dk, float* dgamma_q,
                                         float* dgamma_k, int64_t b, int64_t s, int heads, int kv_heads, int head_dim,
                                         int64_t ld_q, int64_t hs_q, int64_t ld_k, int64_t hs_k, int64_t ld_qo,
                                         int64_t hs_qo, int64_t ld_ko, int64_t hs_ko, int64_t ld_dq, int64_t hs_dq,
                                         int64_t ld_dk, int64_t hs_dk, tpmlp_dtype dt, void* workspace,
                                         size_t ws_bytes, void* stream) {
  TPMLP_PASS(check(eps, table_len, rot_dim, style, b, s, heads, kv_heads, head_dim, dt));
  TPMLP_PASS(check_strides(b, s, heads, kv_heads, head_dim,
                         {{nullptr, ld_q, hs_q}, {nullptr, ld_k, hs_k}, {nullptr, ld_qo, hs_qo}, {nullptr, ld_ko, hs_ko}},
                         {dq, ld_dq, hs_dq}, {dk, ld_dk, hs_dk}));
  TPMLP_PASS(check_ptrs({dgamma_q, dgamma_k}, 4, "pointer not 4-byte aligned"));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (b * s == 0) {  // no tokens: the gains' gradients are empty sums
    TPMLP_PASS_CUDA(cudaMemsetAsync(dgamma_q, 0, static_cast<size_t>(head_dim) * sizeof(float), st), "zero dgamma_q");
    TPMLP_PASS_CUDA(cudaMemsetAsync(dgamma_k, 0, static_cast<size_t>(head_dim) * sizeof(float), st), "zero dgamma_k");
    return TPMLP_OK;
  }
  TPMLP_PASS(check_ptrs({q, k, dq_out, dk_out, dq, dk}, 16, "pointer not 16-byte aligned"));
  TPMLP_PASS(check_ptrs({gamma_q, gamma_k, cos_table, sin_table}, 4, "pointer not 4-byte aligned"));
  if (!aligned(positions, 4)) return err(TPMLP_ERR_ALIGN, "positions not 4-byte aligned");
  const size_t need = tpmlp_qk_norm_rope_backward_workspace_size(b, s, head_dim);
  if (!workspace || ws_bytes < need) return err(TPMLP_ERR_WORKSPACE, "qk_norm_rope backward workspace too small");
  if (!aligned(workspace, 16)) return err(TPMLP_ERR_ALIGN, "workspace not 16-byte aligned");
  const int64_t tokens = b * s, size = dt == TPMLP_BF16 ? 2 : 4;
  auto of = [&](const void* p, int64_t ld, int64_t hs, int n) {
    return heads_region({const_cast<void*>(p), ld, hs}, tokens, n, head_dim, size);
  };
  const Region rq = of(q, ld_q, hs_q, heads), rk = of(k, ld_k, hs_k, kv_heads), rqo = of(dq_out, ld_qo, hs_qo, heads),
               rko = of(dk_out, ld_ko, hs_ko, kv_heads), rdq = of(dq, ld_dq, hs_dq, heads), rdk = of(dk, ld_dk, hs_dk, kv_heads);
  const Region rgq = flat_region(dgamma_q, head_dim, 4), rgk = flat_region(dgamma_k, head_dim, 4),
               rws = flat_region(workspace, static_cast<int64_t>(need), 1);
  auto beside = [](const Region& out, const Region& in) { return !same_region(out, in) && overlap(out, in); };
  if (any_overlap({rdq, rdk, rgq, rgk, rws}, {flat_region(gamma_q, head_dim, 4), flat_region(gamma_k, head_dim, 4),
                                              flat_region(cos_table, table_len, 2 * rot_dim), flat_region(sin_table, table_len, 2 * rot_dim),
                                              flat_region(positions, tokens, 4)}) ||
      any_overlap({rgq, rgk, rws}, {rq, rk, rqo, rko}) || overlap(rdq, rk) || overlap(rdq, rko) || overlap(rdk, rq) ||
      overlap(rdk, rqo) || beside(rdq, rq) || beside(rdq, rqo) || beside(rdk, rk) || beside(rdk, rko))
    return err(TPMLP_ERR_INVALID, "an output overlaps another tensor of the call (in place dq is q or dq_out and dk is k or "
                                  "dk_out, with the same strides)");
  DeviceCtx ctx;
  TPMLP_PASS_CUDA(get_device_ctx(&ctx), "device context");
  RopeParams p = make_params(
      {{const_cast<void*>(q), ld_q, hs_q}, {const_cast<void*>(dq_out), ld_qo, hs_qo}, {dq, ld_dq, hs_dq}, gamma_q, heads, 0},
      {{const_cast<void*>(k), ld_k, hs_k}, {const_cast<void*>(dk_out), ld_ko, hs_ko}, {dk, ld_dk, hs_dk}, gamma_k, kv_heads, 0},
      cos_table, sin_table, positions, table_len, rot_dim, b, s, head_dim, eps);
  // Two CTAs a SM, shared out between queries and keys as their heads are.
  const int64_t ngroups = kThreads / p.group;
  const int64_t want0 = (p.tokens * p.part[0].chunks + ngroups - 1) / ngroups;
  const int64_t want1 = (p.tokens * p.part[1].chunks + ngroups - 1) / ngroups;
  const int64_t room = std::min<int64_t>(static_cast<int64_t>(ctx.num_sms) * 2, kBwdMaxCtas);
  const int64_t share0 = std::max<int64_t>(1, std::min<int64_t>(room - 1, room * p.part[0].chunks / (p.part[0].chunks + p.part[1].chunks)));
  p.ctas0 = static_cast<int>(std::min(want0, share0));
  const int grid = p.ctas0 + static_cast<int>(std::min(want1, room - share0));
  float* partials = static_cast<float*>(workspace);
  auto kernel = ROPE_PICK(qk_norm_rope_backward_kernel, dt, pairing_of(style, rot_dim));
  kernel<<<grid, kThreads, 0, st>>>(p, partials);
  TPMLP_PASS_CUDA(cudaGetLastError(), "qk_norm_rope backward");
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((head_dim + 31) / 32), 2);
  cfg.blockDim = dim3(1024);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  TPMLP_PASS_CUDA(cudaLaunchKernelEx(&cfg, rope_gain_sum_kernel, static_cast<const float*>(partials), p.ctas0, grid, head_dim, dgamma_q,
                               dgamma_k),
            "qk_norm_rope gain sums");
  return TPMLP_OK;
}

}  // extern "C"
