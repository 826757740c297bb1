// bf16 products of few rows (tokens) with a large weight matrix, C = T W, on the tensor cores (tcgen05) with the sum over K
// split across CTAs: the gated block's serving form, and its products whose 256 x 256 output tiles would leave most
// SMs idle. Such a product is bound by the weights' bytes (or by K on few SMs), so
//  * the weights' columns take the tensor core's 128 rows and the tokens its columns: a tile is 256 weight columns x up
//    to 256 tokens, two MMAs that share the token tile, and every weight byte is read once a token tile;
//  * a tile's k-blocks are split evenly over `splits` CTAs, chosen by a model of the time (few_rows_plan.h). Neighbouring CTAs
//    take neighbouring tiles of the same k-blocks, so that whole rows of the weights are read at one time. Each streams
//    through a ring of 192 KB (64-deep k-blocks, 32 KB of weights each);
//  * with one split the kernel's epilogue applies the gate and rounds. Otherwise a CTA leaves its fp32 share in a slot of
//    its own and a second kernel adds a tile's shares in order (no atomics). The kernels of a call are programmatic
//    dependents of one another: the second product's ring fills with weights while the first one ends.
// Measured, the SM-pair GEMM in brackets. d4096 m16384 (268 MB of A, 134 MB of B), 4 tokens: FC1 45.5 us, 5.9 TB/s (64); FC2
// 22 us after FC1's end and 3 us of joining (87). 200 tokens: FC2 28 and 7 us (87). n512 d1024 m4096: FC2 12.4 and 5.7 us
// (24), dX 14 and 7 us (43).
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "device_common.cuh"
#include "few_rows_plan.h"

namespace tpmlp {
namespace {

using namespace few_rows;  // the plan: tiles, splits and whether they pay

constexpr int kThreads = 320;  // producer, MMA issuer, eight epilogue warps

__device__ __forceinline__ int tile_token(const Plan& p, int tile) { return tile % p.token_tiles * p.nt; }

// A CTA's way along its items (item = split * tiles + tile) and their k-blocks: the tile's first column and token, and the
// k-block (divisions once an item).
struct Walk {
  int item, col, token, kb, end;
  int rank, gate[2];  // the gated block's gate columns in A of this CTA's two 64-column boxes
  __device__ __forceinline__ void enter(const Plan& p) {
    const int split = item / p.tiles;
    const int tile = item - split * p.tiles;
    col = tile_column(p, tile);
    token = tile_token(p, tile);
    if (p.shard) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int y = col + rank * kBlock + j * 64;
        gate[j] = y + y / p.shard * p.shard;
      }
    }
    kb = static_cast<int>(static_cast<int64_t>(split) * p.num_kb / p.splits);
    end = static_cast<int>(static_cast<int64_t>(split + 1) * p.num_kb / p.splits);
  }
  __device__ __forceinline__ Walk(const Plan& p, int cta_rank)
      : item(blockIdx.x / p.ranks), col(0), token(0), kb(0), end(0), rank(cta_rank), gate{0, 0} {
    enter(p);
  }
  __device__ __forceinline__ bool more(const Plan& p) const { return item < p.items; }
  __device__ __forceinline__ void next_item(const Plan& p) {
    item += p.ctas / p.ranks;
    if (item < p.items) enter(p);
  }
  __device__ __forceinline__ void next(const Plan& p) {
    if (++kb == end) next_item(p);
  }
};

// act(g) u; the forms other than silu out of line, as their code would be there 32 times.
__device__ __noinline__ float gate_other(float g, float u, int act) { return gelu_f<false>(g, act) * u; }
__device__ __forceinline__ float gate_f(float g, float u, int act) {
  return act == kGateSilu ? g * sigmoid_fast(g) * u : gate_other(g, u, act);
}

// What a product leaves: plain: out[n][cols]; gate: out = Y [n][cols], z [n][2 cols] or null. slots (more than one split):
// [items][nt][256] fp32.
struct Outputs {
  __nv_bfloat16 *out, *z;
  float* slots;
  int act;
};

// PAIR: a cluster of two CTAs on two SMs works on a tile (tcgen05 cta_group::2): each has its own 256 weight columns and
// half of the tokens in shared memory, and all tokens in its accumulators, so that a token tile enters an SM only half.
// Barriers as in the SM-pair GEMM (gemm_tc.cu): full and tempty in the even CTA, empty and tfull in both.
template <bool W_MN, bool GATE, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    few_rows_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_t,
                    const __grid_constant__ Plan p, const __grid_constant__ Outputs o, unsigned int* status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int stage_bytes = plan_stage_bytes(p), stages = p.stages;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + stages * stage_bytes);
  uint64_t* empty = full + kMaxStages;
  uint64_t* tfull = empty + kMaxStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const int ntp = (p.nt + 31) & ~31;              // accumulator columns of a block of 128 weight columns
  const int sets = ntp <= 128 ? 2 : 1;            // of two blocks each
  uint32_t tmem_cols = 64;
  while (tmem_cols < static_cast<uint32_t>(2 * ntp * sets)) tmem_cols *= 2;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], PAIR ? 512 : 256);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmap_w);
    tma_prefetch_desc(&tmap_t);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_slot, tmem_cols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, tmem_cols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if constexpr (PAIR)
    cluster_sync_all();
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependents_may_start();

  if (warp == 0) {
    if (lane == 0) {
      auto load = [&](uint8_t* dst, const CUtensorMap* map, int s, int x, int y) {
        if constexpr (PAIR)
          tma_load_2d_pair(dst, map, map_to_cta(&full[s], 0), x, y);
        else
          tma_load_2d(dst, map, &full[s], x, y);
      };
      auto load_weights = [&](const Walk& at, int s) {
        const int col = at.col + rank * cta_columns(p), kb = at.kb;
        uint8_t* dst = smem + s * stage_bytes;
        if (rank == 0) mbar_arrive_expect_tx(&full[s], p.ranks * stage_bytes);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          if constexpr (W_MN) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              int c = col + b * kBlock + j * 64;
              if constexpr (GATE) c = at.gate[j] + b * p.shard;  // block 0: gate columns, block 1: up columns
              load(dst + (2 * b + j) * kBoxBytes, &tmap_w, s, c, kb * kBK);
            }
          } else {
            load(dst + 2 * b * kBoxBytes, &tmap_w, s, kb * kBK, col + b * kBlock);
          }
        }
      };
      auto load_tokens = [&](const Walk& at, int s) {
        load(smem + s * stage_bytes + kWeightBytes, &tmap_t, s, at.kb * kBK, at.token + rank * (p.nt / 2));
      };
      // The weights are there before the kernel in front has ended; the tokens may be what it writes.
      Walk w(p, rank), tok(p, rank);
      int it = 0;
      for (; it < stages && w.more(p); ++it, w.next(p)) load_weights(w, it);
      grid_wait_for_previous();
      for (int i = 0; i < it; ++i, tok.next(p)) load_tokens(tok, i);
      for (; w.more(p); ++it, w.next(p)) {
        const int s = it % stages;
        if (!mbar_wait(&empty[s], ((it / stages) & 1) ^ 1, status, 71)) break;
        load_weights(w, s);
        load_tokens(w, s);
      }
      // The even CTA's full barriers count both CTAs' copies: none is in flight when it leaves (at once on the normal path).
      if (rank == 0 && (PAIR || w.more(p)))
        for (int i = max(0, it - stages); i < it; ++i) mbar_wait(&full[i % stages], (i / stages) & 1, status, 72);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = idesc_bf16_f32(PAIR ? 2 * kBlock : kBlock, p.nt, W_MN, false);
      auto commit = [&](uint64_t* bar) {
        if constexpr (PAIR)
          umma_commit_pair_mc(bar, 0x3);
        else
          umma_commit(bar);
      };
      int it = 0, seg = 0;
      bool ok = true;
      for (Walk at(p, rank); at.more(p) && ok; at.next_item(p), ++seg) {
        const int set = seg % sets;
        if (!mbar_wait(&tempty[set], ((seg / sets) & 1) ^ 1, status, 73)) break;
        tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(set * 2 * ntp);
        for (int first = at.kb; at.kb < at.end; ++at.kb, ++it) {
          const int s = it % stages;
          if (!mbar_wait(&full[s], (it / stages) & 1, status, 74)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t w = smem_u32(smem + s * stage_bytes), t = w + kWeightBytes;
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk) {
            const uint64_t tdesc = smem_desc_sw128(t + kk * 32, 16, 1024);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const uint32_t wb = w + 2 * b * kBoxBytes;
              const uint64_t wdesc = W_MN ? smem_desc_sw128(wb + kk * 2048, kBoxBytes, 1024) : smem_desc_sw128(wb + kk * 32, 16, 1024);
              const uint32_t acc = at.kb != first || kk != 0 ? 1u : 0u;
              if constexpr (PAIR)
                umma_bf16_pair(d + static_cast<uint32_t>(b * ntp), wdesc, tdesc, idesc, acc);
              else
                umma_bf16(d + static_cast<uint32_t>(b * ntp), wdesc, tdesc, idesc, acc);
            }
          }
          commit(&empty[s]);
        }
        if (ok) commit(&tfull[set]);
      }
      if constexpr (PAIR)
        umma_commit_pair(drain);
      else
        umma_commit(drain);
      mbar_wait(drain, 0, status, 75);
    }
  } else {
    // A thread has one weight column of each block and every other 32 tokens: for one token, a warp's 32 lanes write 128
    // bytes of a slot, or 64 of the outputs.
    grid_wait_for_previous();  // what is written may still be read by what ran before
    const int q = warp & 3, t_first = (warp - 2) / 4 * 32;
    // f(i) for the tokens i < n of 32, without a test for each where all are there
    auto each = [](int n, auto&& f) {
      if (n >= 32) {
#pragma unroll
        for (int i = 0; i < 32; ++i) f(i);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i < n) f(i);
      }
    };
    int seg = 0;
    for (Walk at(p, rank); at.more(p); at.next_item(p), ++seg) {
      const int set = seg % sets;
      if (!__all_sync(0xffffffffu, mbar_wait(&tfull[set], (seg / sets) & 1, status, 76))) break;
      tc_fence_after();
      const int token0 = at.token, tokens = min(p.nt, p.n - token0);
      const int tile_col = at.col, col0 = tile_col + rank * cta_columns(p) + q * 32 + lane;
      const uint32_t t_row = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(set * 2 * ntp);
#pragma unroll 1
      for (int t0 = t_first; t0 < tokens; t0 += 64) {
        uint32_t a[32], b[32];
        tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(t0), a);
        tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(ntp + t0), b);
        tmem_ld_wait();
        const int64_t token = token0 + t0;
        if (!PAIR && p.splits > 1) {
          float* out = o.slots + (static_cast<int64_t>(at.item) * p.nt + t0) * kTileCols + q * 32 + lane;
          each(tokens - t0, [&](int i) {
            out[i * kTileCols] = __uint_as_float(a[i]);
            out[i * kTileCols + kBlock] = __uint_as_float(b[i]);
          });
        } else if constexpr (GATE) {
          if (col0 / p.unit == tile_col / p.unit) {
            __nv_bfloat16* out = o.out + token * p.cols + col0;
            if (o.act == kGateSilu) {
              each(tokens - t0, [&](int i) {
                const float g = __uint_as_float(a[i]);
                *out = __float2bfloat16_rn(g * sigmoid_fast(g) * __uint_as_float(b[i]));
                out += p.cols;
              });
            } else {
              each(tokens - t0, [&](int i) {
                *out = __float2bfloat16_rn(gate_other(__uint_as_float(a[i]), __uint_as_float(b[i]), o.act));
                out += p.cols;
              });
            }
            if (o.z) {
              __nv_bfloat16* z = o.z + token * 2 * p.cols + col0 + static_cast<int64_t>(col0 / p.shard) * p.shard;
              each(tokens - t0, [&](int i) {
                z[0] = __float2bfloat16_rn(__uint_as_float(a[i]));
                z[p.shard] = __float2bfloat16_rn(__uint_as_float(b[i]));
                z += 2 * p.cols;
              });
            }
          }
        } else {
          __nv_bfloat16* out = o.out + token * p.cols + col0;
          const bool in0 = col0 < p.cols, in1 = col0 + kBlock < p.cols;
          each(tokens - t0, [&](int i) {
            if (in0) out[0] = __float2bfloat16_rn(__uint_as_float(a[i]));
            if (in1) out[kBlock] = __float2bfloat16_rn(__uint_as_float(b[i]));
            out += p.cols;
          });
        }
      }
      tc_fence_before();
      if constexpr (PAIR)
        mbar_arrive_cluster(map_to_cta(&tempty[set], 0));
      else
        mbar_arrive(&tempty[set]);
    }
  }
  // Neither CTA of a pair leaves while the other may still signal its barriers.
  tc_fence_before();
  __syncwarp();
  if constexpr (PAIR)
    cluster_sync_all();
  else
    __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem, tmem_cols);
    else
      tmem_dealloc(tmem, tmem_cols);
  }
}

// The second kernel: a quad of columns of one token is added up by `subs` threads (a power of two, in warps of their own),
// thread i taking the shares i, i + subs, .. in order; then their sums are added in order. All loads of a thread are
// independent of one another, and few, whatever the splits.
constexpr int kJoinThreads = 256;
// As many as the splits give two shares each, while the CTAs stay one wave (8 an SM).
inline int join_subs(int splits, int64_t threads) {
  int subs = 1;
  while (subs < 8 && 4 * subs <= splits && 2 * subs * threads <= 8ll * kSms * kJoinThreads) subs *= 2;
  return subs;
}

__device__ __forceinline__ void add4(float4& a, const float4& v) {
  a.x += v.x;
  a.y += v.y;
  a.z += v.z;
  a.w += v.w;
}

template <bool GATE>
__global__ void __launch_bounds__(kJoinThreads) few_rows_join_kernel(const __grid_constant__ Plan p, const __grid_constant__ Outputs o,
                                                                     int subs) {
  grid_dependents_may_start();
  grid_wait_for_previous();
  constexpr int kQuads = (GATE ? kBlock : kTileCols) / 4;
  __shared__ float4 sums[GATE ? 2 : 1][kJoinThreads];
  const int here = kJoinThreads / subs, sub = threadIdx.x / here;  // quads of this CTA; 32 or more, so a warp has one sub
  const int64_t item = static_cast<int64_t>(blockIdx.x) * here + threadIdx.x % here;
  const int quad = static_cast<int>(item % kQuads);
  const int64_t rest = item / kQuads;
  const int ct = static_cast<int>(rest / p.n), token = static_cast<int>(rest - static_cast<int64_t>(ct) * p.n);
  const int ti = token / p.nt, tile = ct * p.token_tiles + ti;
  const int col0 = tile_column(p, tile), col = col0 + quad * 4;
  const bool in = ct < p.col_tiles && (GATE ? col / p.unit == col0 / p.unit : col < p.cols);
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f), u = a;
  const int64_t share = static_cast<int64_t>(p.nt) * kTileCols, stride = p.tiles * share;
  const float* src = o.slots + tile * share + (token - ti * p.nt) * kTileCols + quad * 4;
  if (in) {
#pragma unroll 4
    for (int c = sub; c < p.splits; c += subs) {
      add4(a, *reinterpret_cast<const float4*>(src + c * stride));
      if constexpr (GATE) add4(u, *reinterpret_cast<const float4*>(src + c * stride + kBlock));
    }
  }
  // The shares' lines in L2 are given up: dirty, they would be written to HBM when the next product's weights take their place
  // (d4096 m16384, 30 MB of them at 200 tokens: 90 -> 85 us a forward; 128 tokens 85 -> 82; n512 d1024 m4096, where they would
  // stay in L2, 30.8 -> 31.0). A line is read by 8 neighbouring lanes, and by nobody else.
  __syncwarp();
  if (in && (quad & 7) == 0)
    for (int c = sub; c < p.splits; c += subs) {
      l2_discard(src + c * stride);
      if constexpr (GATE) l2_discard(src + c * stride + kBlock);
    }
  if (subs > 1) {
    sums[0][threadIdx.x] = a;
    if constexpr (GATE) sums[1][threadIdx.x] = u;
    __syncthreads();
    if (sub > 0) return;
    for (int i = 1; i < subs; ++i) {
      add4(a, sums[0][threadIdx.x + i * here]);
      if constexpr (GATE) add4(u, sums[1][threadIdx.x + i * here]);
    }
  }
  if (!in) return;
  uint2* out = reinterpret_cast<uint2*>(o.out + static_cast<int64_t>(token) * p.cols + col);
  if constexpr (!GATE) {
    *out = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
  } else {
    *out = make_uint2(pack_bf16x2(gate_f(a.x, u.x, o.act), gate_f(a.y, u.y, o.act)),
                      pack_bf16x2(gate_f(a.z, u.z, o.act), gate_f(a.w, u.w, o.act)));
    if (o.z) {
      __nv_bfloat16* row = o.z + static_cast<int64_t>(token) * 2 * p.cols + col + static_cast<int64_t>(col / p.shard) * p.shard;
      *reinterpret_cast<uint2*>(row) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
      *reinterpret_cast<uint2*>(row + p.shard) = make_uint2(pack_bf16x2(u.x, u.y), pack_bf16x2(u.z, u.w));
    }
  }
}

// ---------------------------------------------------------------------- host side

cudaError_t encode_2d(CUtensorMap* map, const void* ptr, int64_t rows, int64_t cols, uint32_t box_rows) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  if (!encode) return cudaErrorNotSupported;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * 2};
  cuuint32_t box[2] = {64, box_rows}, estr[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), int64_t ctas, int cluster, int threads, int smem, bool dependent,
                         cudaStream_t stream, A... args) {
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (dependent) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <bool W_MN, bool GATE, bool PAIR>
cudaError_t run(Plan p, const void* tokens, int64_t k, const void* w, int64_t w_rows, int64_t w_cols, const Outputs& o,
                bool dependent, cudaStream_t stream, const DeviceCtx& ctx) {
  CUtensorMap tw, tt;
  cudaError_t e = encode_2d(&tw, w, w_rows, w_cols, W_MN ? kBK : kBlock);
  if (e != cudaSuccess) return e;
  if ((e = encode_2d(&tt, tokens, p.n, k, p.nt / p.ranks)) != cudaSuccess) return e;
  static SmemLimit limit;
  auto kernel = few_rows_kernel<W_MN, GATE, PAIR>;
  if ((e = allow_smem(&limit, kernel, kSmemBudget, ctx)) != cudaSuccess) return e;
  p.ctas = std::min(p.items, ctx.num_sms / p.ranks) * p.ranks;
  const int smem = p.stages * plan_stage_bytes(p) + kBarrierBytes + 1024;
  if ((e = launch_after(kernel, p.ctas, p.ranks, kThreads, smem, dependent, stream, tw, tt, p, o, ctx.status)) != cudaSuccess) return e;
  if (p.splits == 1) return cudaSuccess;
  const int64_t threads = static_cast<int64_t>(p.col_tiles) * p.n * ((GATE ? kBlock : kTileCols) / 4);
  const int subs = join_subs(p.splits, threads), here = kJoinThreads / subs;
  return launch_after(few_rows_join_kernel<GATE>, (threads + here - 1) / here, 1, kJoinThreads, 0, true, stream, p, o, subs);
}

}  // namespace

bool gemm_takes_few_rows(int64_t n, int64_t cols, int64_t k) { return few_rows::gemm_pays(n, cols, k); }
bool gated_fc1_takes_few_rows(int64_t n, int64_t d, int64_t m, int t) { return few_rows::gated_fc1_pays(n, d, m, t); }

size_t gated_fc1_few_rows_workspace(int64_t n, int64_t d, int64_t m, int t) { return slot_bytes(make_plan(n, m, d, m, t, true)); }

cudaError_t gated_fc1_few_rows(const void* x, const void* a, void* z, void* y, int64_t n, int64_t d, int64_t m, int t, int act,
                               void* workspace, cudaStream_t stream, const DeviceCtx& ctx) {
  const Outputs o{static_cast<__nv_bfloat16*>(y), static_cast<__nv_bfloat16*>(z), static_cast<float*>(workspace), act};
  const Plan p = make_plan(n, m, d, m, t, true);
  return p.ranks == 2 ? run<true, true, true>(p, x, d, a, d, 2 * m, o, false, stream, ctx)
                      : run<true, true, false>(p, x, d, a, d, 2 * m, o, false, stream, ctx);
}

size_t gemm_few_rows_workspace(int64_t n, int64_t cols, int64_t k) { return slot_bytes(make_plan(n, cols, k, 0, 1, false)); }

cudaError_t gemm_few_rows(const void* tokens, const void* w, bool w_mn, void* out, int64_t n, int64_t cols, int64_t k,
                          void* workspace, bool dependent, cudaStream_t stream, const DeviceCtx& ctx) {
  const Plan p = make_plan(n, cols, k, 0, 1, false);
  const Outputs o{static_cast<__nv_bfloat16*>(out), nullptr, static_cast<float*>(workspace), 0};
  return w_mn ? run<true, false, false>(p, tokens, k, w, k, cols, o, dependent, stream, ctx)
              : run<false, false, false>(p, tokens, k, w, cols, k, o, dependent, stream, ctx);
}

}  // namespace tpmlp
