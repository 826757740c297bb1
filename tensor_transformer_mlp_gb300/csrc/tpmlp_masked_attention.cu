// C ABI of masked attention (tpmlp_attention_key_ranges, tpmlp_masked_attention_forward / _backward):
// the checks of the arguments, and the small kernel that turns a batch's documents, prefixes, causality
// and window into one key interval per query. The attention kernels are in
// masked_attention_fwd.cu and masked_attention_bwd.cu.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "abi_checks.h"

namespace tpmlp {
namespace {

constexpr int kRangeThreads = 1024;

// The interval of query i, whose document (or sequence) is [start, end).
__device__ __forceinline__ int2 query_range(int64_t i, int64_t start, int64_t end, int causal, int64_t prefix,
                                            int64_t window) {
  int64_t lo = start, hi = end;
  if (causal) {
    hi = min(hi, max(i + 1, prefix));
  } else if (window > 0) {
    hi = min(hi, i + window);
  }
  if (window > 0) lo = max(lo, i - window + 1);
  return lo < hi ? make_int2(static_cast<int>(lo), static_cast<int>(hi)) : make_int2(0, 0);
}

__global__ void __launch_bounds__(256)
    key_range_kernel(const int* __restrict__ prefix, int causal, int64_t window, int2* __restrict__ out, int64_t b,
                     int64_t s) {
  for (int64_t t = blockIdx.x * 256ll + threadIdx.x; t < b * s; t += gridDim.x * 256ll) {
    const int64_t bi = t / s, i = t - bi * s;
    out[t] = query_range(i, 0, s, causal, prefix ? prefix[bi] : 0, window);
  }
}

// The same with documents, one CTA per sequence. A document is a run of equal ids: token i's starts at the
// last j <= i whose id differs from its left neighbour's and ends at the first such j > i. A warp turns 32
// tokens into one word of start bits with a ballot, so a tile of kWords words costs one pass over its ids, and
// the two searches are bit scans within a word and one running maximum (from the left) and minimum (from the
// right) over the words. A row of one tile (32768 tokens) is done in one go; longer rows sweep their tiles from
// the left, parking each start in out[].x, and then from the right, the thread that wrote a start reading it back.
__global__ void __launch_bounds__(kRangeThreads)
    doc_key_range_kernel(const int* __restrict__ ids_all, const int* __restrict__ prefix, int causal, int64_t window,
                         int2* __restrict__ out_all, int s) {
  constexpr int kWords = kRangeThreads, kWarps = kRangeThreads / 32;
  __shared__ unsigned starts[kWords];
  __shared__ int before[kWords], after[kWords];  // last start left of the word, first start right of it
  __shared__ int total[2][kWarps];
  const int64_t bi = blockIdx.x;
  const int* ids = ids_all + bi * s;
  int2* out = out_all + bi * s;
  const int64_t plen = prefix ? prefix[bi] : 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nwords = (s + 31) / 32, ntiles = (nwords + kWords - 1) / kWords;
  const int sweeps = ntiles > 1 ? 2 : 1;
  for (int sweep = 0; sweep < sweeps; ++sweep) {
    int left = 0, right = s;  // last start in the tiles before (first sweep), first start in those behind (last sweep)
    for (int n = 0; n < ntiles; ++n) {
      const int w0 = (sweep == 0 ? n : ntiles - 1 - n) * kWords;  // the tile's first word in the row
      const int words = min(kWords, nwords - w0);
#pragma unroll 8
      for (int w = warp; w < words; w += kWarps) {
        const int i = (w0 + w) * 32 + lane;
        const bool in = i < s;
        const int id = in ? ids[i] : 0;
        int prev = __shfl_up_sync(0xffffffffu, id, 1);
        if (lane == 0 && i > 0) prev = ids[i - 1];
        const unsigned bits = __ballot_sync(0xffffffffu, in && (i == 0 || id != prev));
        if (lane == 0) starts[w] = bits;
      }
      __syncthreads();
      const int base = (w0 + static_cast<int>(threadIdx.x)) * 32;
      const unsigned bits = static_cast<int>(threadIdx.x) < words ? starts[threadIdx.x] : 0u;
      int last = bits ? base + 31 - __clz(bits) : -1, first = bits ? base + __ffs(bits) - 1 : INT32_MAX;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, last, o), d = __shfl_down_sync(0xffffffffu, first, o);
        if (lane >= o) last = max(last, u);
        if (lane + o < 32) first = min(first, d);
      }
      if (lane == 31) total[0][warp] = last;
      if (lane == 0) total[1][warp] = first;
      __syncthreads();
      {
        const int tl = total[0][lane], tf = total[1][lane];
        const int prior = __reduce_max_sync(0xffffffffu, lane < warp ? tl : left);
        const int later = __reduce_min_sync(0xffffffffu, lane > warp ? tf : right);
        const int lu = __shfl_up_sync(0xffffffffu, last, 1), fd = __shfl_down_sync(0xffffffffu, first, 1);
        before[threadIdx.x] = lane > 0 ? max(prior, lu) : prior;
        after[threadIdx.x] = lane < 31 ? min(later, fd) : later;
        left = max(left, __reduce_max_sync(0xffffffffu, tl));
        right = min(right, __reduce_min_sync(0xffffffffu, tf));
      }
      __syncthreads();
      for (int w = warp; w < words; w += kWarps) {
        const int i = (w0 + w) * 32 + lane;
        if (i >= s) continue;
        const unsigned b = starts[w], upto = b & (0xffffffffu >> (31 - lane)), past = b & ~(0xffffffffu >> (31 - lane));
        const int start = upto ? (w0 + w) * 32 + 31 - __clz(upto) : before[w];
        if (sweep < sweeps - 1) {
          out[i].x = start;
          continue;
        }
        const int end = past ? (w0 + w) * 32 + __ffs(past) - 1 : after[w];
        const int2 r = query_range(i, sweeps == 1 ? start : out[i].x, end, causal, plen, window);
        out[i] = ids[i] < 0 ? make_int2(0, 0) : r;
      }
      __syncthreads();
    }
  }
}

tpmlp_status check_shape(float scale, float softcap, int64_t b, int64_t s, int heads, int kv_heads, int hd,
                         tpmlp_dtype dt, std::initializer_list<HeadView> inputs,
                         std::initializer_list<HeadView> q_outputs, std::initializer_list<HeadView> k_outputs) {
  if (dt != TPMLP_BF16) return err(TPMLP_ERR_DTYPE, "masked attention runs on the bf16 tensor-core path only");
  if (b < 0 || s < 0 || heads < 1 || kv_heads < 1)
    return err(TPMLP_ERR_SHAPE, "need b, s >= 0 and heads, kv_heads >= 1");
  if (b > 0 && s > INT32_MAX / b) return err(TPMLP_ERR_SHAPE, "b * s exceeds 2^31-1");
  if (s > (1 << 30)) return err(TPMLP_ERR_SHAPE, "s must be <= 2^30");
  if (b > 65535 || heads > 65535) return err(TPMLP_ERR_SHAPE, "at most 65535 sequences and heads");
  if (heads % kv_heads != 0) return err(TPMLP_ERR_SHAPE, "heads must be a multiple of kv_heads");
  if (hd < 8 || hd % 8 != 0 || hd > 128)
    return err(TPMLP_ERR_SHAPE, "head_dim must be a multiple of 8, 8 <= head_dim <= 128");
  if ((s + 127) / 128 * b * heads > INT32_MAX)
    return err(TPMLP_ERR_SHAPE, "more than 2^31-1 tiles of 128 queries in all heads");
  for (const auto& list : {inputs, q_outputs, k_outputs})
    for (const HeadView& v : list)
      if (!good_head_strides(v, s))
        return err(TPMLP_ERR_SHAPE, "strides must be positive multiples of 8 (row 2^31, head and sequence 2^38 at most)");
  for (const HeadView& v : q_outputs)
    if (!heads_apart(v, b * s, heads, hd)) return err(TPMLP_ERR_SHAPE, "an output's heads overlap");
  for (const HeadView& v : k_outputs)
    if (!heads_apart(v, b * s, kv_heads, hd)) return err(TPMLP_ERR_SHAPE, "an output's heads overlap");
  if (!(scale > 0.0f) || !std::isfinite(scale)) return err(TPMLP_ERR_INVALID, "scale must be positive and finite");
  if (!(softcap >= 0.0f) || !std::isfinite(softcap)) return err(TPMLP_ERR_INVALID, "softcap must be >= 0 and finite");
  if (scale > 1e30f || softcap > 1e30f || (softcap > 0.0f && scale / softcap > 1e30f))
    return err(TPMLP_ERR_INVALID, "scale, softcap and scale / softcap must be at most 1e30");
  return TPMLP_OK;
}

}  // namespace
}  // namespace tpmlp

using namespace tpmlp;

extern "C" {

tpmlp_status tpmlp_attention_key_ranges(const void* doc_ids, const void* prefix_len, int causal, int64_t window,
                                        void* key_range, int64_t b, int64_t s, void* stream) {
  if (b < 0 || s < 0) return err(TPMLP_ERR_SHAPE, "need b, s >= 0");
  if (b > 0 && s > INT32_MAX / b) return err(TPMLP_ERR_SHAPE, "b * s exceeds 2^31-1");
  if (s > (1 << 30)) return err(TPMLP_ERR_SHAPE, "s must be <= 2^30");
  if (causal != 0 && causal != 1) return err(TPMLP_ERR_INVALID, "causal is 0 or 1");
  if (window < 0) return err(TPMLP_ERR_INVALID, "window must be >= 0");
  if (prefix_len && !causal) return err(TPMLP_ERR_INVALID, "a prefix needs a causal mask");
  if (b * s == 0) return TPMLP_OK;
  TPMLP_PASS(check_ptrs({key_range}, 8, "key_range not 8-byte aligned"));
  if (!aligned(doc_ids, 4) || !aligned(prefix_len, 4))
    return err(TPMLP_ERR_ALIGN, "doc_ids and prefix_len must be 4-byte aligned");
  if (any_overlap({flat_region(key_range, b * s, 8)}, {flat_region(doc_ids, b * s, 4), flat_region(prefix_len, b, 4)}))
    return err(TPMLP_ERR_INVALID, "key_range overlaps doc_ids or prefix_len");
  if (window > s) window = 0;  // reaches past both ends
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int* prefix = static_cast<const int*>(prefix_len);
  int2* out = static_cast<int2*>(key_range);
  if (doc_ids) {
    doc_key_range_kernel<<<static_cast<unsigned>(b), kRangeThreads, 0, st>>>(static_cast<const int*>(doc_ids), prefix,
                                                                             causal, window, out, static_cast<int>(s));
  } else {
    const int64_t ctas = (b * s + 255) / 256;
    key_range_kernel<<<static_cast<unsigned>(ctas < 4096 ? ctas : 4096), 256, 0, st>>>(prefix, causal, window, out, b, s);
  }
  TPMLP_PASS_CUDA(cudaGetLastError(), "key ranges");
  return TPMLP_OK;
}

tpmlp_status tpmlp_masked_attention_forward(const void* q, const void* k, const void* v, const void* key_range,
                                            const float* slopes, float scale, float softcap, void* o, float* lse,
                                            int64_t b, int64_t s, int heads, int kv_heads, int head_dim, int64_t ld_q,
                                            int64_t hs_q, int64_t ld_k, int64_t hs_k, int64_t ld_v, int64_t hs_v,
                                            int64_t ld_o, int64_t hs_o, tpmlp_dtype dt, void* stream) {
  TPMLP_PASS(check_shape(scale, softcap, b, s, heads, kv_heads, head_dim, dt,
                       {{nullptr, ld_q, hs_q}, {nullptr, ld_k, hs_k}, {nullptr, ld_v, hs_v}}, {{o, ld_o, hs_o}}, {}));
  if (b * s == 0) return TPMLP_OK;
  TPMLP_PASS(check_ptrs({q, k, v, o}, 16, "pointers must be 16-byte aligned"));
  TPMLP_PASS(check_ptrs({key_range}, 8, "key_range not 8-byte aligned"));
  TPMLP_PASS(check_ptrs({lse}, 4, "lse not 4-byte aligned"));
  if (!aligned(slopes, 4)) return err(TPMLP_ERR_ALIGN, "slopes not 4-byte aligned");
  MaskedAttention a{{const_cast<void*>(q), ld_q, hs_q}, {const_cast<void*>(k), ld_k, hs_k},
                    {const_cast<void*>(v), ld_v, hs_v}, {o, ld_o, hs_o}, static_cast<const int2*>(key_range), slopes,
                    scale, softcap, lse, b, s, heads, kv_heads, head_dim};
  auto of = [&](const HeadView& view, int n) { return heads_region(view, b * s, n, head_dim, 2); };
  if (any_overlap({of(a.o, heads), flat_region(lse, b * s * heads, 4)},
                  {of(a.q, heads), of(a.k, kv_heads), of(a.v, kv_heads), flat_region(key_range, b * s, 8),
                   flat_region(slopes, heads, 4)}))
    return err(TPMLP_ERR_INVALID, "o or lse overlaps another tensor of the call");
  DeviceCtx ctx;
  TPMLP_PASS_CUDA(get_device_ctx(&ctx), "device context");
  TPMLP_PASS_CUDA(launch_masked_attention_forward(a, static_cast<cudaStream_t>(stream), ctx), "masked attention");
  return TPMLP_OK;
}

size_t tpmlp_masked_attention_backward_workspace_size(int64_t b, int64_t s, int heads) {
  if (b <= 0 || s <= 0 || heads <= 0) return 0;
  return masked_attention_backward_workspace(b, s, heads);
}

tpmlp_status tpmlp_masked_attention_backward(const void* q, const void* k, const void* v, const void* key_range,
                                             const float* slopes, float scale, float softcap, const void* o,
                                             const float* lse, const void* d_o, void* dq, void* dk, void* dv,
                                             int64_t b, int64_t s, int heads, int kv_heads, int head_dim,
                                             int64_t ld_q, int64_t hs_q, int64_t ld_k, int64_t hs_k, int64_t ld_v,
                                             int64_t hs_v, int64_t ld_o, int64_t hs_o, int64_t ld_dq, int64_t hs_dq,
                                             int64_t ld_dk, int64_t hs_dk, int64_t ld_dv, int64_t hs_dv,
                                             tpmlp_dtype dt, void* workspace, size_t ws_bytes, void* stream) {
  TPMLP_PASS(check_shape(scale, softcap, b, s, heads, kv_heads, head_dim, dt,
                       {{nullptr, ld_q, hs_q}, {nullptr, ld_k, hs_k}, {nullptr, ld_v, hs_v}, {nullptr, ld_o, hs_o}},
                       {{dq, ld_dq, hs_dq}}, {{dk, ld_dk, hs_dk}, {dv, ld_dv, hs_dv}}));
  if (b * s == 0) return TPMLP_OK;
  TPMLP_PASS(check_ptrs({q, k, v, o, d_o, dq, dk, dv}, 16, "pointers must be 16-byte aligned"));
  TPMLP_PASS(check_ptrs({key_range}, 8, "key_range not 8-byte aligned"));
  TPMLP_PASS(check_ptrs({lse}, 4, "lse not 4-byte aligned"));
  if (!aligned(slopes, 4)) return err(TPMLP_ERR_ALIGN, "slopes not 4-byte aligned");
  const size_t need = tpmlp_masked_attention_backward_workspace_size(b, s, heads);
  if (!workspace || ws_bytes < need) return err(TPMLP_ERR_WORKSPACE, "masked attention backward workspace too small");
  if (!aligned(workspace, 256)) return err(TPMLP_ERR_ALIGN, "workspace not 256-byte aligned");
  MaskedAttention a{{const_cast<void*>(q), ld_q, hs_q}, {const_cast<void*>(k), ld_k, hs_k},
                    {const_cast<void*>(v), ld_v, hs_v}, {const_cast<void*>(o), ld_o, hs_o},
                    static_cast<const int2*>(key_range), slopes, scale, softcap, const_cast<float*>(lse), b, s, heads,
                    kv_heads, head_dim};
  const HeadView g{const_cast<void*>(d_o), ld_o, hs_o}, gq{dq, ld_dq, hs_dq}, gk{dk, ld_dk, hs_dk}, gv{dv, ld_dv, hs_dv};
  auto of = [&](const HeadView& view, int n) { return heads_region(view, b * s, n, head_dim, 2); };
  if (any_overlap({of(gq, heads), of(gk, kv_heads), of(gv, kv_heads), flat_region(workspace, static_cast<int64_t>(need), 1)},
                  {of(a.q, heads), of(a.k, kv_heads), of(a.v, kv_heads), flat_region(key_range, b * s, 8),
                   flat_region(slopes, heads, 4), of(a.o, heads), flat_region(lse, b * s * heads, 4), of(g, heads)}))
    return err(TPMLP_ERR_INVALID, "dq, dk, dv or the workspace overlaps another tensor of the call");
  DeviceCtx ctx;
  TPMLP_PASS_CUDA(get_device_ctx(&ctx), "device context");
  TPMLP_PASS_CUDA(launch_masked_attention_backward(a, g, gq, gk, gv, workspace, static_cast<cudaStream_t>(stream), ctx),
            "masked attention backward");
  return TPMLP_OK;
}

}  // extern "C"
