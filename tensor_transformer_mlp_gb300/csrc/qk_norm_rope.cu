// RMSNorm of every query and key head and the rotation by position in one pass, and its backward
// (tpmlp_qk_norm_rope, tpmlp_qk_norm_rope_backward).
//
//   u = x r gamma, r = 1 / sqrt(mean(x^2) + eps) over one head's columns;  y = R(pos) u
//   du = R(pos)^T dy, g = du gamma;  dx = r (g - x_hat mean(g x_hat));  dgamma = sum du x_hat
//
// Both are bound by memory (about 4 flops a byte): q and k are read once and written once. A head's
// columns lie eight to a lane on a group of G lanes (the power of two that covers head_dim / 8), so one
// 16-byte load fetches a lane's bf16 share and the row sums are log2(G) shuffles. A CTA takes one token
// at a time and its groups stride over the token's heads: the token's cosines and sines and the gains
// stay in registers for all of them.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdio>

#include "../../include/tpmlp.h"
#include "device_common.cuh"

namespace tpmlp {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxHeadDim = 256;
constexpr int kBwdMaxCtas = 1024;

struct RopeParams {
  HeadView q, k, qo, ko;    // forward: inputs, outputs; backward: x, dy
  HeadView dq, dk;          // backward: dx
  const float *gamma_q, *gamma_k;
  const float *cos_t, *sin_t;
  const int* pos;
  int64_t table_len;
  int64_t tokens, s;
  int heads, kv_heads, hd, rot, interleaved, group;
  float eps, inv_hd;
};

template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = unpack_bf16x2(w[i]);
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                              pack_bf16x2(f[6], f[7]));
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
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

__device__ __forceinline__ float group_sum(float v, int group) {
  for (int o = group >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One lane's share of a head: columns c0 .. c0 + 7 (active lanes), and what turns them. For column e
// the turned value is f[e] * cs[e] + partner(e) * sn[e], where partner(e) is the pair's other column and
// sn carries the sign of the forward turn (columns past rot: 1 and 0).
struct LaneTurn {
  float cs[8], sn[8];
  __device__ __forceinline__ void load(const RopeParams& p, int c0, int64_t pos) {
    const int half = p.rot >> 1;
    const bool in_table = pos < p.table_len;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = c0 + e;
      cs[e] = 1.f;
      sn[e] = 0.f;
      if (c < p.rot) {
        const int i = p.interleaved ? c >> 1 : (c < half ? c : c - half);
        const bool first = p.interleaved ? (c & 1) == 0 : c < half;
        const float nan = __int_as_float(0x7fffffff);
        const float co = in_table ? p.cos_t[pos * half + i] : nan, si = in_table ? p.sin_t[pos * half + i] : nan;
        cs[e] = co;
        sn[e] = first ? -si : si;
      }
    }
  }
};

// f -> R f (back: R^T f) within each group. xch: the warp's 32 x 8 floats for pairs that do not fall on
// whole lanes (rot / 2 no multiple of 8, half style); otherwise the partner columns sit in one lane
// rot / 16 further and a shuffle brings them. Every lane of the warp calls this.
__device__ __forceinline__ void turn(float (&f)[8], const LaneTurn& t, const RopeParams& p, int lane, int gl, int c0,
                                     bool back, float* xch) {
  const float sg = back ? -1.f : 1.f;
  float other[8];
  if (p.interleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) other[e] = f[e ^ 1];
  } else if ((p.rot & 15) == 0) {
    const int step = p.rot >> 4;
    const int src = gl < step ? lane + step : (gl < 2 * step ? lane - step : lane);
#pragma unroll
    for (int e = 0; e < 8; ++e) other[e] = __shfl_sync(0xffffffffu, f[e], src);
  } else {
    float* mine = xch + lane * 8;
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 8; ++e) mine[e] = f[e];
    __syncwarp();
    const float* head = xch + (lane - gl) * 8;
    const int half = p.rot >> 1;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = c0 + e;
      other[e] = c < p.rot ? head[c < half ? c + half : c - half] : 0.f;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = c0 + e < p.rot ? f[e] * t.cs[e] + other[e] * (sg * t.sn[e]) : f[e];
}

__device__ __forceinline__ int64_t position_of(const RopeParams& p, int64_t token) {
  return p.pos ? static_cast<int64_t>(p.pos[token]) : token % p.s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeParams p) {
  __shared__ float xch_all[kThreads * 8];
  const int lane = threadIdx.x & 31, gl = lane & (p.group - 1), c0 = gl * 8;
  float* xch = xch_all + (threadIdx.x & ~31) * 8;
  const bool act = c0 < p.hd;
  const int ngroups = kThreads / p.group, g0 = threadIdx.x / p.group;
  const int all = p.heads + p.kv_heads;
  float gq[8], gk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    gq[e] = act ? p.gamma_q[c0 + e] : 0.f;
    gk[e] = act ? p.gamma_k[c0 + e] : 0.f;
  }
  for (int64_t token = blockIdx.x; token < p.tokens; token += gridDim.x) {
    const int64_t pos = position_of(p, token);
    LaneTurn t;
    t.load(p, c0, pos < 0 ? 0 : pos);
    for (int hb = 0; hb < all; hb += ngroups) {  // uniform over the CTA, so every lane takes the shuffles
      const int h = hb + g0;
      const bool is_q = h < p.heads, on = act && h < all;
      const HeadView& in = is_q ? p.q : p.k;
      const HeadView& out = is_q ? p.qo : p.ko;
      const int64_t hh = is_q ? h : h - p.heads;
      Vec8<T> x;
      x.zero();
      if (on && pos >= 0) x.load(static_cast<const T*>(in.ptr) + token * in.ld + hh * in.hs + c0);
      float f[8];
      x.unpack(f);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
      ss = group_sum(ss, p.group);
      const float r = rsqrtf(fmaf(ss, p.inv_hd, p.eps));
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= r * (is_q ? gq[e] : gk[e]);
      turn(f, t, p, lane, gl, c0, false, xch);
      if (pos < 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = 0.f;
      }
      if (on) Vec8<T>::store(static_cast<T*>(out.ptr) + token * out.ld + hh * out.hs + c0, f);
    }
  }
}

// partials: [gridDim.x][2][hd] (dgamma_q, dgamma_k of the CTA's tokens, its groups added in order).
template <typename T>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_backward_kernel(const RopeParams p, float* partials) {
  __shared__ float xch_all[kThreads * 8];
  const int lane = threadIdx.x & 31, gl = lane & (p.group - 1), c0 = gl * 8;
  float* xch = xch_all + (threadIdx.x & ~31) * 8;
  const bool act = c0 < p.hd;
  const int ngroups = kThreads / p.group, g0 = threadIdx.x / p.group;
  const int all = p.heads + p.kv_heads;
  float gq[8], gk[8], aq[8], ak[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    gq[e] = act ? p.gamma_q[c0 + e] : 0.f;
    gk[e] = act ? p.gamma_k[c0 + e] : 0.f;
    aq[e] = ak[e] = 0.f;
  }
  for (int64_t token = blockIdx.x; token < p.tokens; token += gridDim.x) {
    const int64_t pos = position_of(p, token);
    LaneTurn t;
    t.load(p, c0, pos < 0 ? 0 : pos);
    for (int hb = 0; hb < all; hb += ngroups) {
      const int h = hb + g0;
      const bool is_q = h < p.heads, on = act && h < all;
      const int64_t hh = is_q ? h : h - p.heads;
      const HeadView& in = is_q ? p.q : p.k;
      const HeadView& dyv = is_q ? p.qo : p.ko;
      const HeadView& out = is_q ? p.dq : p.dk;
      Vec8<T> x, dy;
      x.zero();
      dy.zero();
      if (on && pos >= 0) {
        x.load(static_cast<const T*>(in.ptr) + token * in.ld + hh * in.hs + c0);
        dy.load(static_cast<const T*>(dyv.ptr) + token * dyv.ld + hh * dyv.hs + c0);
      }
      float f[8], d[8];
      x.unpack(f);
      dy.unpack(d);
      turn(d, t, p, lane, gl, c0, true, xch);
      float ss = 0.f, gx = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss = fmaf(f[e], f[e], ss);
        gx = fmaf(d[e] * (is_q ? gq[e] : gk[e]), f[e], gx);
      }
      ss = group_sum(ss, p.group);
      gx = group_sum(gx, p.group);
      const float r = rsqrtf(fmaf(ss, p.inv_hd, p.eps));
      const float m = gx * r * p.inv_hd;  // mean(g x_hat)
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xh = f[e] * r;
        o[e] = pos < 0 ? 0.f : r * (d[e] * (is_q ? gq[e] : gk[e]) - xh * m);
        const float dg = on && pos >= 0 ? d[e] * xh : 0.f;
        if (is_q) aq[e] += dg; else ak[e] += dg;
      }
      if (on) Vec8<T>::store(static_cast<T*>(out.ptr) + token * out.ld + hh * out.hs + c0, o);
    }
  }
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) xch_all[threadIdx.x * 8 + e] = part ? ak[e] : aq[e];
    __syncthreads();
    for (int c = threadIdx.x; c < p.hd; c += kThreads) {
      float sum = 0.f;
      for (int g = 0; g < ngroups; ++g) sum += xch_all[g * p.group * 8 + c];
      partials[(static_cast<int64_t>(blockIdx.x) * 2 + part) * p.hd + c] = sum;
    }
  }
}

// Adds the CTAs' partials in a fixed order: each CTA takes one column of 2 * hd, its 128 threads add every
// 128th partial in order and a tree joins them.
__global__ void __launch_bounds__(128)
    rope_gain_sum_kernel(const float* __restrict__ partials, int nparts, int hd, float* __restrict__ dgamma_q,
                         float* __restrict__ dgamma_k) {
  __shared__ float red[128];
  const int c = blockIdx.x;
  float sum = 0.f;
  for (int i = threadIdx.x; i < nparts; i += 128) sum += partials[static_cast<int64_t>(i) * 2 * hd + c];
  red[threadIdx.x] = sum;
  for (int o = 64; o > 0; o >>= 1) {
    __syncthreads();
    if (threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
  }
  if (threadIdx.x == 0) (c < hd ? dgamma_q[c] : dgamma_k[c - hd]) = red[0];
}

tpmlp_status err(tpmlp_status st, const char* msg) { return static_cast<tpmlp_status>(report_error(st, msg)); }

tpmlp_status cuda_err(cudaError_t e, const char* what) {
  char msg[256];
  snprintf(msg, sizeof(msg), "%s: %s", what, cudaGetErrorString(e));
  return err(TPMLP_ERR_CUDA, msg);
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

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

tpmlp_status check_ptrs(std::initializer_list<const void*> ptrs, size_t a) {
  for (const void* p : ptrs) {
    if (!p) return err(TPMLP_ERR_INVALID, "null pointer");
    if (!aligned(p, a)) return err(TPMLP_ERR_ALIGN, a == 16 ? "pointer not 16-byte aligned" : "pointer not 4-byte aligned");
  }
  return TPMLP_OK;
}

int group_of(int hd) {
  int g = 1;
  while (g * 8 < hd) g *= 2;
  return g;
}

}  // namespace
}  // namespace tpmlp

using namespace tpmlp;

#define ROPE_TRY(expr)                  \
  do {                                  \
    tpmlp_status _s = (expr);           \
    if (_s != TPMLP_OK) return _s;      \
  } while (0)
#define ROPE_CUDA(expr, what)                       \
  do {                                              \
    cudaError_t _e = (expr);                        \
    if (_e != cudaSuccess) return cuda_err(_e, what); \
  } while (0)

extern "C" {

tpmlp_status tpmlp_qk_norm_rope(const void* q, const void* k, const float* gamma_q, const float* gamma_k, float eps,
                                const float* cos_table, const float* sin_table, const void* positions,
                                int64_t table_len, int rot_dim, int style, void* q_out, void* k_out, int64_t b,
                                int64_t s, int heads, int kv_heads, int head_dim, int64_t ld_q, int64_t hs_q,
                                int64_t ld_k, int64_t hs_k, int64_t ld_qo, int64_t hs_qo, int64_t ld_ko,
                                int64_t hs_ko, tpmlp_dtype dt, void* stream) {
  ROPE_TRY(check(eps, table_len, rot_dim, style, b, s, heads, kv_heads, head_dim, dt));
  ROPE_TRY(check_strides(b, s, heads, kv_heads, head_dim, {{nullptr, ld_q, hs_q}, {nullptr, ld_k, hs_k}},
                         {q_out, ld_qo, hs_qo}, {k_out, ld_ko, hs_ko}));
  if (b * s == 0) return TPMLP_OK;
  ROPE_TRY(check_ptrs({q, k, q_out, k_out}, 16));
  ROPE_TRY(check_ptrs({gamma_q, gamma_k, cos_table, sin_table}, 4));
  if (!aligned(positions, 4)) return err(TPMLP_ERR_ALIGN, "positions not 4-byte aligned");
  DeviceCtx ctx;
  ROPE_CUDA(get_device_ctx(&ctx), "device context");
  RopeParams p{};
  p.q = {const_cast<void*>(q), ld_q, hs_q};
  p.k = {const_cast<void*>(k), ld_k, hs_k};
  p.qo = {q_out, ld_qo, hs_qo};
  p.ko = {k_out, ld_ko, hs_ko};
  p.gamma_q = gamma_q; p.gamma_k = gamma_k;
  p.cos_t = cos_table; p.sin_t = sin_table;
  p.pos = static_cast<const int*>(positions);
  p.table_len = table_len;
  p.tokens = b * s; p.s = s;
  p.heads = heads; p.kv_heads = kv_heads; p.hd = head_dim; p.rot = rot_dim; p.interleaved = style;
  p.group = group_of(head_dim);
  p.eps = eps; p.inv_hd = 1.0f / static_cast<float>(head_dim);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int grid = static_cast<int>(std::min<int64_t>(p.tokens, static_cast<int64_t>(ctx.num_sms) * 8));
  if (dt == TPMLP_BF16) qk_norm_rope_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(p);
  else qk_norm_rope_kernel<float><<<grid, kThreads, 0, st>>>(p);
  ROPE_CUDA(cudaGetLastError(), "qk_norm_rope");
  return TPMLP_OK;
}

size_t tpmlp_qk_norm_rope_backward_workspace_size(int64_t b, int64_t s, int head_dim) {
  if (b <= 0 || s <= 0 || head_dim <= 0) return 0;
  const int64_t ctas = s > kBwdMaxCtas / b ? kBwdMaxCtas : std::min<int64_t>(b * s, kBwdMaxCtas);
  return static_cast<size_t>(ctas) * 2 * static_cast<size_t>(head_dim) * sizeof(float);
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
  ROPE_TRY(check(eps, table_len, rot_dim, style, b, s, heads, kv_heads, head_dim, dt));
  ROPE_TRY(check_strides(b, s, heads, kv_heads, head_dim,
                         {{nullptr, ld_q, hs_q}, {nullptr, ld_k, hs_k}, {nullptr, ld_qo, hs_qo}, {nullptr, ld_ko, hs_ko}},
                         {dq, ld_dq, hs_dq}, {dk, ld_dk, hs_dk}));
  ROPE_TRY(check_ptrs({dgamma_q, dgamma_k}, 4));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (b * s == 0) {  // no tokens: the gains' gradients are empty sums
    ROPE_CUDA(cudaMemsetAsync(dgamma_q, 0, static_cast<size_t>(head_dim) * sizeof(float), st), "zero dgamma_q");
    ROPE_CUDA(cudaMemsetAsync(dgamma_k, 0, static_cast<size_t>(head_dim) * sizeof(float), st), "zero dgamma_k");
    return TPMLP_OK;
  }
  ROPE_TRY(check_ptrs({q, k, dq_out, dk_out, dq, dk}, 16));
  ROPE_TRY(check_ptrs({gamma_q, gamma_k, cos_table, sin_table}, 4));
  if (!aligned(positions, 4)) return err(TPMLP_ERR_ALIGN, "positions not 4-byte aligned");
  const size_t need = tpmlp_qk_norm_rope_backward_workspace_size(b, s, head_dim);
  if (!workspace || ws_bytes < need) return err(TPMLP_ERR_WORKSPACE, "qk_norm_rope backward workspace too small");
  if (!aligned(workspace, 16)) return err(TPMLP_ERR_ALIGN, "workspace not 16-byte aligned");
  DeviceCtx ctx;
  ROPE_CUDA(get_device_ctx(&ctx), "device context");
  RopeParams p{};
  p.q = {const_cast<void*>(q), ld_q, hs_q};
  p.k = {const_cast<void*>(k), ld_k, hs_k};
  p.qo = {const_cast<void*>(dq_out), ld_qo, hs_qo};
  p.ko = {const_cast<void*>(dk_out), ld_ko, hs_ko};
  p.dq = {dq, ld_dq, hs_dq};
  p.dk = {dk, ld_dk, hs_dk};
  p.gamma_q = gamma_q; p.gamma_k = gamma_k;
  p.cos_t = cos_table; p.sin_t = sin_table;
  p.pos = static_cast<const int*>(positions);
  p.table_len = table_len;
  p.tokens = b * s; p.s = s;
  p.heads = heads; p.kv_heads = kv_heads; p.hd = head_dim; p.rot = rot_dim; p.interleaved = style;
  p.group = group_of(head_dim);
  p.eps = eps; p.inv_hd = 1.0f / static_cast<float>(head_dim);
  const int grid = static_cast<int>(
      std::min<int64_t>(p.tokens, std::min<int64_t>(static_cast<int64_t>(ctx.num_sms) * 4, kBwdMaxCtas)));
  float* partials = static_cast<float*>(workspace);
  if (dt == TPMLP_BF16) qk_norm_rope_backward_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(p, partials);
  else qk_norm_rope_backward_kernel<float><<<grid, kThreads, 0, st>>>(p, partials);
  ROPE_CUDA(cudaGetLastError(), "qk_norm_rope backward");
  rope_gain_sum_kernel<<<2 * head_dim, 128, 0, st>>>(partials, grid, head_dim, dgamma_q, dgamma_k);
  ROPE_CUDA(cudaGetLastError(), "qk_norm_rope gain sums");
  return TPMLP_OK;
}

}  // extern "C"
