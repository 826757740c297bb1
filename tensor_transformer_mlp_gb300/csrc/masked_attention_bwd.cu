// Masked attention, forward and backward, on CUDA cores: one warp per query row (forward, dQ) or per key
// row (dK, dV), 32 keys or queries at a time.
//
//   y_ij = c(scale q_i.k_j) - slope |i - j|,  lse_i = log sum_j exp(y_ij),  P_ij = exp(y_ij - lse_i)
//   o_i = sum_j P_ij v_j;  D_i = d_o_i.o_i,  dX_ij = scale c' P_ij (d_o_i.v_j - D_i)
//   dQ_i = sum_j dX_ij k_j,  dK_j = sum_i dX_ij q_i,  dV_j = sum_i P_ij d_o_i
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "device_common.cuh"

namespace tpmlp {
namespace {

constexpr int kWarps = 4;
constexpr int kCols = 128 / 32;  // columns of a head per lane

using bf16 = __nv_bfloat16;

__device__ __forceinline__ const bf16* row_of(const HeadView& v, int64_t token, int head) {
  return static_cast<const bf16*>(v.ptr) + token * v.ld + head * v.hs;
}

__device__ __forceinline__ float dot(const bf16* a, const bf16* b, int hd) {
  float acc = 0.f;
  for (int c = 0; c < hd; c += 8) {
    const uint4 x = *reinterpret_cast<const uint4*>(a + c), y = *reinterpret_cast<const uint4*>(b + c);
    const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 u = unpack_bf16x2(xw[i]), w = unpack_bf16x2(yw[i]);
      acc = fmaf(u.x, w.x, acc);
      acc = fmaf(u.y, w.y, acc);
    }
  }
  return acc;
}

// y_ij, and the cap's derivative
__device__ __forceinline__ float score(const MaskedAttention& a, float qk, int head, int64_t i, int64_t j, float* dcap) {
  float y = qk * a.scale;
  *dcap = 1.f;
  if (a.softcap > 0.f) {
    const float t = tanhf(y / a.softcap);
    y = a.softcap * t;
    *dcap = 1.f - t * t;
  }
  if (a.slopes) y -= a.slopes[head] * fabsf(static_cast<float>(i - j));
  return y;
}

__device__ __forceinline__ int2 clipped(const MaskedAttention& a, int64_t token) {
  int2 r = a.range[token];
  r.x = max(r.x, 0);
  r.y = min(static_cast<int64_t>(r.y), a.s);
  return r.x < r.y ? r : make_int2(0, 0);
}

__global__ void __launch_bounds__(kWarps * 32) dq_rows_kernel(const MaskedAttention a, const HeadView d_o,
                                                              const HeadView dq, float* dsum) {
  const int lane = threadIdx.x & 31, hd = a.head_dim;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int head = blockIdx.y, kvh = head / (a.heads / a.kv_heads);
  if (i >= a.s) return;
  const int64_t base = blockIdx.z * a.s, token = base + i;
  const int64_t at = (blockIdx.z * static_cast<int64_t>(a.heads) + head) * a.s + i;
  const int2 r = clipped(a, token);
  const bf16 *q = row_of(a.q, token, head), *g = row_of(d_o, token, head);
  const float D = dot(g, row_of(a.o, token, head), hd), lse = a.lse[at];
  if (lane == 0) dsum[at] = D;
  float acc[kCols] = {};
  for (int j0 = r.x; j0 < r.y; j0 += 32) {
    const int j = j0 + lane;
    float dx = 0.f, dcap;
    if (j < r.y) {
      const float y = score(a, dot(q, row_of(a.k, base + j, kvh), hd), head, i, j, &dcap);
      dx = expf(y - lse) * (dot(g, row_of(a.v, base + j, kvh), hd) - D) * dcap * a.scale;
    }
    for (int e = 0; e < min(32, r.y - j0); ++e) {
      const float de = __shfl_sync(0xffffffffu, dx, e);
      const bf16* k = row_of(a.k, base + j0 + e, kvh);
#pragma unroll
      for (int c = 0; c < kCols; ++c)
        if (lane + 32 * c < hd) acc[c] = fmaf(de, __bfloat162float(k[lane + 32 * c]), acc[c]);
    }
  }
  bf16* out = const_cast<bf16*>(row_of(dq, token, head));
#pragma unroll
  for (int c = 0; c < kCols; ++c)
    if (lane + 32 * c < hd) out[lane + 32 * c] = __float2bfloat16(acc[c]);
}

__global__ void __launch_bounds__(kWarps * 32) dkv_rows_kernel(const MaskedAttention a, const HeadView d_o,
                                                               const HeadView dk, const HeadView dv, const float* dsum) {
  const int lane = threadIdx.x & 31, hd = a.head_dim, group = a.heads / a.kv_heads;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int kvh = blockIdx.y;
  if (j >= a.s) return;
  const int64_t base = blockIdx.z * a.s, token = base + j;
  const bf16 *k = row_of(a.k, token, kvh), *v = row_of(a.v, token, kvh);
  float acck[kCols] = {}, accv[kCols] = {};
  for (int head = kvh * group; head < (kvh + 1) * group; ++head) {
    const int64_t at = (blockIdx.z * static_cast<int64_t>(a.heads) + head) * a.s;
    for (int64_t i0 = 0; i0 < a.s; i0 += 32) {
      const int64_t i = i0 + lane;
      bool sees = false;
      if (i < a.s) {
        const int2 r = clipped(a, base + i);
        sees = r.x <= j && j < r.y;
      }
      unsigned left = __ballot_sync(0xffffffffu, sees);
      if (!left) continue;
      float p = 0.f, dx = 0.f, dcap;
      if (sees) {
        const bf16* g = row_of(d_o, base + i, head);
        p = expf(score(a, dot(row_of(a.q, base + i, head), k, hd), head, i, j, &dcap) - a.lse[at + i]);
        dx = p * (dot(g, v, hd) - dsum[at + i]) * dcap * a.scale;
      }
      for (; left; left &= left - 1) {
        const int e = __ffs(left) - 1;
        const float pe = __shfl_sync(0xffffffffu, p, e), de = __shfl_sync(0xffffffffu, dx, e);
        const bf16 *q = row_of(a.q, base + i0 + e, head), *g = row_of(d_o, base + i0 + e, head);
#pragma unroll
        for (int c = 0; c < kCols; ++c)
          if (lane + 32 * c < hd) {
            acck[c] = fmaf(de, __bfloat162float(q[lane + 32 * c]), acck[c]);
            accv[c] = fmaf(pe, __bfloat162float(g[lane + 32 * c]), accv[c]);
          }
      }
    }
  }
  bf16 *ok = const_cast<bf16*>(row_of(dk, token, kvh)), *ov = const_cast<bf16*>(row_of(dv, token, kvh));
#pragma unroll
  for (int c = 0; c < kCols; ++c)
    if (lane + 32 * c < hd) {
      ok[lane + 32 * c] = __float2bfloat16(acck[c]);
      ov[lane + 32 * c] = __float2bfloat16(accv[c]);
    }
}

dim3 rows_grid(const MaskedAttention& a, int heads) {
  return dim3(static_cast<unsigned>((a.s + kWarps - 1) / kWarps), static_cast<unsigned>(heads),
              static_cast<unsigned>(a.b));
}

}  // namespace

cudaError_t launch_masked_attention_backward(const MaskedAttention& a, const HeadView& d_o, const HeadView& dq,
                                             const HeadView& dk, const HeadView& dv, float* dsum, cudaStream_t stream,
                                             const DeviceCtx&) {
  dq_rows_kernel<<<rows_grid(a, a.heads), kWarps * 32, 0, stream>>>(a, d_o, dq, dsum);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  dkv_rows_kernel<<<rows_grid(a, a.kv_heads), kWarps * 32, 0, stream>>>(a, d_o, dk, dv, dsum);
  return cudaGetLastError();
}

}  // namespace tpmlp
