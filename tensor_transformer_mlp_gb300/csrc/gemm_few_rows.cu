// bf16 products of few rows (tokens) with a large weight matrix, C = T W, on the tensor cores (tcgen05) with the sum over K
// split across CTAs: the gated block's serving form, and its products whose 256 x 256 output tiles would leave most
// SMs idle. Such a product is bound by the weights' bytes (or by K on few SMs), so
//  * the weights' columns take the tensor core's 128 rows and the tokens its columns: a tile is 256 weight columns x up
//    to 256 tokens, two MMAs that share the token tile, and every weight byte is read once a token tile;
//  * a tile's k-blocks are split evenly over `splits` CTAs, chosen by a model of the time (choose_splits). Neighbouring CTAs
//    take neighbouring tiles of the same k-blocks, so that whole rows of the weights are read at one time. Each streams
//    through a ring of 192 KB (64-deep k-blocks, 32 KB of weights each);
//  * with one split the kernel's epilogue applies the gate and rounds. Otherwise a CTA leaves its fp32 share in a slot of
//    its own and a second kernel adds a tile's shares in order (no atomics). The kernels of a call are programmatic
//    dependents of one another: the second product's ring fills with weights while the first one ends.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "device_common.cuh"

namespace tpmlp {
namespace {

constexpr int kTileCols = 256;          // weight columns of a tile: two blocks of 128
constexpr int kBlock = 128;
constexpr int kBK = 64;
constexpr int kMaxTokens = 256;         // tokens of a tile
constexpr int kWeightBytes = kTileCols * kBK * 2;
constexpr int kBoxBytes = 64 * kBK * 2;  // one 64 x 64 box of weights stored [K][cols]
constexpr int kMaxStages = 6;
constexpr int kSmemBudget = 220 * 1024;
constexpr int kBarrierBytes = 256;
constexpr int kThreads = 192;           // producer, MMA issuer, four epilogue warps
constexpr int kSms = 152;               // what splits and workspaces are chosen for, with or without a device
constexpr int kMaxItems = 4 * kSms;

struct Plan {
  int n, cols, num_kb;   // tokens, output columns (of Y for the gate), k-blocks
  int nt, token_tiles;   // tokens of a tile (a multiple of 16) and tiles of them
  int col_tiles, tiles, splits, items, ctas;  // items = tiles * splits
  int shard, unit;       // the gated block's columns (EpiParams), 0: plain
  int stages;
};

__host__ __device__ __forceinline__ int plan_stage_bytes(const Plan& p) { return kWeightBytes + p.nt * kBK * 2; }

// Tile -> its first column and token. Tiles of the same columns are neighbours: their weights meet in L2.
__device__ __forceinline__ int tile_column(const Plan& p, int tile) {
  const int ct = tile / p.token_tiles;
  if (!p.shard) return ct * kTileCols;
  const int per = (p.unit + kBlock - 1) / kBlock;
  return ct / per * p.unit + ct % per * kBlock;
}
__device__ __forceinline__ int tile_token(const Plan& p, int tile) { return tile % p.token_tiles * p.nt; }

// A CTA's way along its items (item = split * tiles + tile) and their k-blocks.
struct Walk {
  int item, tile, kb, end;
  __device__ __forceinline__ void enter(const Plan& p) {
    const int split = item / p.tiles;
    tile = item - split * p.tiles;
    kb = static_cast<int>(static_cast<int64_t>(split) * p.num_kb / p.splits);
    end = static_cast<int>(static_cast<int64_t>(split + 1) * p.num_kb / p.splits);
  }
  __device__ __forceinline__ explicit Walk(const Plan& p) : item(blockIdx.x), tile(0), kb(0), end(0) { enter(p); }
  __device__ __forceinline__ bool more(const Plan& p) const { return item < p.items; }
  __device__ __forceinline__ void next_item(const Plan& p) {
    item += p.ctas;
    if (item < p.items) enter(p);
  }
  __device__ __forceinline__ void next(const Plan& p) {
    if (++kb == end) next_item(p);
  }
};

__device__ __forceinline__ float gate_f(float g, int act) { return act == kGateSilu ? g * sigmoid_fast(g) : gelu_f<false>(g, act); }

// What a product leaves: plain: out[n][cols]; gate: out = Y [n][cols], z [n][2 cols] or null. slots (more than one split):
// [items][nt][256] fp32.
struct Outputs {
  __nv_bfloat16 *out, *z;
  float* slots;
  int act;
};

template <bool W_MN, bool GATE>
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
      mbar_init(&tempty[a], 128);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmap_w);
    tma_prefetch_desc(&tmap_t);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  asm volatile("griddepcontrol.launch_dependents;");

  if (warp == 0) {
    if (lane == 0) {
      auto load_weights = [&](const Walk& at, int s) {
        const int col = tile_column(p, at.tile), kb = at.kb;
        uint8_t* dst = smem + s * stage_bytes;
        mbar_arrive_expect_tx(&full[s], stage_bytes);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          if constexpr (W_MN) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              int c = col + b * kBlock + j * 64;
              if constexpr (GATE) {  // block 0: gate columns, block 1: up columns
                const int y = col + j * 64;
                c = y + (y / p.shard + b) * p.shard;
              }
              tma_load_2d(dst + (2 * b + j) * kBoxBytes, &tmap_w, &full[s], c, kb * kBK);
            }
          } else {
            tma_load_2d(dst + 2 * b * kBoxBytes, &tmap_w, &full[s], kb * kBK, col + b * kBlock);
          }
        }
      };
      auto load_tokens = [&](const Walk& at, int s) {
        tma_load_2d(smem + s * stage_bytes + kWeightBytes, &tmap_t, &full[s], at.kb * kBK, tile_token(p, at.tile));
      };
      // The weights are there before the kernel in front has ended; the tokens may be what it writes.
      Walk w(p), tok(p);
      int it = 0;
      for (; it < stages && w.more(p); ++it, w.next(p)) load_weights(w, it);
      asm volatile("griddepcontrol.wait;" ::: "memory");
      for (int i = 0; i < it; ++i, tok.next(p)) load_tokens(tok, i);
      for (; w.more(p); ++it, w.next(p)) {
        const int s = it % stages;
        if (!mbar_wait(&empty[s], ((it / stages) & 1) ^ 1, status, 71)) break;
        load_weights(w, s);
        load_tokens(w, s);
      }
      if (w.more(p))  // copies still in flight
        for (int i = max(0, it - stages); i < it; ++i) mbar_wait(&full[i % stages], (i / stages) & 1, status, 72);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16_f32(kBlock, p.nt, W_MN, false);
      int it = 0, seg = 0;
      bool ok = true;
      for (Walk at(p); at.more(p) && ok; at.next_item(p), ++seg) {
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
              umma_bf16(d + static_cast<uint32_t>(b * ntp), wdesc, tdesc, idesc, at.kb != first || kk != 0 ? 1u : 0u);
            }
          }
          umma_commit(&empty[s]);
        }
        if (ok) umma_commit(&tfull[set]);
      }
      umma_commit(drain);
      mbar_wait(drain, 0, status, 75);
    }
  } else {
    // A thread has one weight column of each block and all tokens: for one token, a warp's 32 lanes write 128 bytes of
    // a slot, or 64 of the outputs.
    asm volatile("griddepcontrol.wait;" ::: "memory");  // what is written may still be read by what ran before
    const int q = warp & 3;
    int seg = 0;
    for (Walk at(p); at.more(p); at.next_item(p), ++seg) {
      const int set = seg % sets;
      if (!__all_sync(0xffffffffu, mbar_wait(&tfull[set], (seg / sets) & 1, status, 76))) break;
      tc_fence_after();
      const int token0 = tile_token(p, at.tile), tokens = min(p.nt, p.n - token0), col0 = tile_column(p, at.tile);
      const uint32_t t_row = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(set * 2 * ntp);
      if (p.splits > 1) {
        float* out = o.slots + static_cast<int64_t>(at.item) * p.nt * kTileCols + q * 32 + lane;
#pragma unroll 1
        for (int b = 0; b < 2; ++b) {
#pragma unroll 1
          for (int t0 = 0; t0 < tokens; t0 += 32) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(b * ntp + t0), v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (t0 + i < tokens) out[(t0 + i) * kTileCols + b * kBlock] = __uint_as_float(v[i]);
          }
        }
      } else if constexpr (GATE) {
        const int y = col0 + q * 32 + lane;
        const bool in = y / p.unit == col0 / p.unit;
        __nv_bfloat16* out = o.out + static_cast<int64_t>(token0) * p.cols + y;
        __nv_bfloat16* z = o.z ? o.z + static_cast<int64_t>(token0) * 2 * p.cols + y + static_cast<int64_t>(y / p.shard) * p.shard : nullptr;
#pragma unroll 1
        for (int t0 = 0; t0 < tokens; t0 += 32) {
          uint32_t g[32], u[32];
          tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(t0), g);
          tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(ntp + t0), u);
          tmem_ld_wait();
          if (!in) continue;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (t0 + i >= tokens) break;
            const float gi = __uint_as_float(g[i]), ui = __uint_as_float(u[i]);
            out[static_cast<int64_t>(t0 + i) * p.cols] = __float2bfloat16_rn(gate_f(gi, o.act) * ui);
            if (z) {
              z[static_cast<int64_t>(t0 + i) * 2 * p.cols] = __float2bfloat16_rn(gi);
              z[static_cast<int64_t>(t0 + i) * 2 * p.cols + p.shard] = __float2bfloat16_rn(ui);
            }
          }
        }
      } else {
#pragma unroll 1
        for (int b = 0; b < 2; ++b) {
          const int col = col0 + b * kBlock + q * 32 + lane;
          __nv_bfloat16* out = o.out + static_cast<int64_t>(token0) * p.cols + col;
#pragma unroll 1
          for (int t0 = 0; t0 < tokens; t0 += 32) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(b * ntp + t0), v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (t0 + i < tokens && col < p.cols) out[static_cast<int64_t>(t0 + i) * p.cols] = __float2bfloat16_rn(__uint_as_float(v[i]));
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&tempty[set]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, tmem_cols);
  }
}

// The splits' shares of four columns of a tile, added in order: all of a thread's loads are independent.
__device__ __forceinline__ float4 sum_shares(const float* src, int n, int64_t stride) {
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int c = 0; c < n; ++c) {
    const float4 v = *reinterpret_cast<const float4*>(src + c * stride);
    a.x += v.x;
    a.y += v.y;
    a.z += v.z;
    a.w += v.w;
  }
  return a;
}

// A thread 4 columns of one token.
template <bool GATE>
__global__ void __launch_bounds__(256) few_rows_join_kernel(const __grid_constant__ Plan p, const __grid_constant__ Outputs o) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kQuads = (GATE ? kBlock : kTileCols) / 4;
  const int64_t item = blockIdx.x * 256ll + threadIdx.x;
  const int quad = static_cast<int>(item % kQuads);
  const int64_t rest = item / kQuads;
  const int ct = static_cast<int>(rest / p.n), token = static_cast<int>(rest - static_cast<int64_t>(ct) * p.n);
  if (ct >= p.col_tiles) return;
  const int ti = token / p.nt, tile = ct * p.token_tiles + ti;
  const int col0 = tile_column(p, tile), col = col0 + quad * 4;
  if (GATE ? col / p.unit != col0 / p.unit : col >= p.cols) return;
  const int64_t share = static_cast<int64_t>(p.nt) * kTileCols;
  const float* src = o.slots + tile * share + (token - ti * p.nt) * kTileCols + quad * 4;
  const float4 a = sum_shares(src, p.splits, p.tiles * share);
  uint2* out = reinterpret_cast<uint2*>(o.out + static_cast<int64_t>(token) * p.cols + col);
  if constexpr (!GATE) {
    *out = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
  } else {
    const float4 u = sum_shares(src + kBlock, p.splits, p.tiles * share);
    *out = make_uint2(pack_bf16x2(gate_f(a.x, o.act) * u.x, gate_f(a.y, o.act) * u.y),
                      pack_bf16x2(gate_f(a.z, o.act) * u.z, gate_f(a.w, o.act) * u.w));
    if (o.z) {
      __nv_bfloat16* row = o.z + static_cast<int64_t>(token) * 2 * p.cols + col + static_cast<int64_t>(col / p.shard) * p.shard;
      *reinterpret_cast<uint2*>(row) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
      *reinterpret_cast<uint2*>(row + p.shard) = make_uint2(pack_bf16x2(u.x, u.y), pack_bf16x2(u.z, u.w));
    }
  }
}

// ---------------------------------------------------------------------- host side

// Estimated time of a product with `splits` splits, in us: rounds of items, each k-block at the slowest of the weights' share
// of HBM (6.7 TB/s), the tensor core (12.7 TFLOP/s an SM) and what an SM takes in (60 KB a us); the shares' way to L2 and
// back (8 TB/s) and the second kernel.
double split_time(const Plan& p, int splits, int sms) {
  const double items = static_cast<double>(p.tiles) * splits, busy = std::min<double>(items, sms);
  const double kb = std::max({kWeightBytes * busy / 6.7e6, 2.0 * kTileCols * p.nt * kBK / 12.7e6, plan_stage_bytes(p) / 60e3});
  const double rounds = std::ceil(items / sms), blocks = std::ceil(static_cast<double>(p.num_kb) / splits);
  return rounds * (blocks * kb + 1.0) + (splits > 1 ? 3.0 + items * p.nt * kTileCols * 8.0 / 8e6 : 0.0);
}

void choose_splits(Plan* p, int sms) {
  double best = split_time(*p, 1, sms);
  p->splits = 1;
  const int most = std::min(p->num_kb, std::max(1, kMaxItems / p->tiles));
  for (int s = 2; s <= most; ++s) {
    const double t = split_time(*p, s, sms);
    if (t < best) {
      best = t;
      p->splits = s;
    }
  }
}

Plan make_plan(int64_t n, int64_t cols, int64_t k, int64_t m, int t, bool gate) {
  Plan p{};
  p.n = static_cast<int>(n);
  p.cols = static_cast<int>(cols);
  p.num_kb = static_cast<int>((k + kBK - 1) / kBK);
  p.token_tiles = static_cast<int>((n + kMaxTokens - 1) / kMaxTokens);
  p.nt = static_cast<int>(((n + p.token_tiles - 1) / p.token_tiles + 15) / 16 * 16);
  if (gate) {
    p.shard = static_cast<int>(m / t);
    p.unit = p.shard % 64 == 0 ? static_cast<int>(m) : p.shard;
    p.col_tiles = static_cast<int>(m / p.unit * ((p.unit + kBlock - 1) / kBlock));
  } else {
    p.col_tiles = static_cast<int>((cols + kTileCols - 1) / kTileCols);
  }
  p.tiles = p.col_tiles * p.token_tiles;
  choose_splits(&p, kSms);
  p.items = p.tiles * p.splits;
  p.stages = std::min<int>(kMaxStages, (kSmemBudget - kBarrierBytes - 1024) / plan_stage_bytes(p));
  return p;
}

size_t slot_bytes(const Plan& p) {
  return p.splits > 1 ? static_cast<size_t>(p.items) * p.nt * kTileCols * sizeof(float) : 0;
}

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
cudaError_t launch_after(void (*kernel)(P...), int64_t ctas, int threads, int smem, bool dependent, cudaStream_t stream, A... args) {
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <bool W_MN, bool GATE>
cudaError_t run(Plan p, const void* tokens, int64_t k, const void* w, int64_t w_rows, int64_t w_cols, const Outputs& o,
                bool dependent, cudaStream_t stream, const DeviceCtx& ctx) {
  CUtensorMap tw, tt;
  cudaError_t e = encode_2d(&tw, w, w_rows, w_cols, W_MN ? kBK : kBlock);
  if (e != cudaSuccess) return e;
  if ((e = encode_2d(&tt, tokens, p.n, k, p.nt)) != cudaSuccess) return e;
  static SmemLimit limit;
  auto kernel = few_rows_kernel<W_MN, GATE>;
  if ((e = allow_smem(&limit, kernel, kSmemBudget, ctx)) != cudaSuccess) return e;
  p.ctas = std::min(p.items, ctx.num_sms);
  const int smem = p.stages * plan_stage_bytes(p) + kBarrierBytes + 1024;
  if ((e = launch_after(kernel, p.ctas, kThreads, smem, dependent, stream, tw, tt, p, o, ctx.status)) != cudaSuccess) return e;
  if (p.splits == 1) return cudaSuccess;
  const int64_t threads = static_cast<int64_t>(p.col_tiles) * p.n * ((GATE ? kBlock : kTileCols) / 4);
  return launch_after(few_rows_join_kernel<GATE>, (threads + 255) / 256, 256, 0, true, stream, p, o);
}

}  // namespace

bool gated_fc1_takes_few_rows(int64_t n, int64_t d, int64_t m) { return n <= 512; }
bool gemm_takes_few_rows(int64_t n, int64_t cols, int64_t k) { return n <= 512 || ((n + 255) / 256) * ((cols + 255) / 256) <= 38; }

size_t gated_fc1_few_rows_workspace(int64_t n, int64_t d, int64_t m, int t) { return slot_bytes(make_plan(n, m, d, m, t, true)); }

cudaError_t gated_fc1_few_rows(const void* x, const void* a, void* z, void* y, int64_t n, int64_t d, int64_t m, int t, int act,
                               void* workspace, cudaStream_t stream, const DeviceCtx& ctx) {
  const Outputs o{static_cast<__nv_bfloat16*>(y), static_cast<__nv_bfloat16*>(z), static_cast<float*>(workspace), act};
  return run<true, true>(make_plan(n, m, d, m, t, true), x, d, a, d, 2 * m, o, false, stream, ctx);
}

size_t gemm_few_rows_workspace(int64_t n, int64_t cols, int64_t k) { return slot_bytes(make_plan(n, cols, k, 0, 1, false)); }

cudaError_t gemm_few_rows(const void* tokens, const void* w, bool w_mn, void* out, int64_t n, int64_t cols, int64_t k,
                          void* workspace, bool dependent, cudaStream_t stream, const DeviceCtx& ctx) {
  const Plan p = make_plan(n, cols, k, 0, 1, false);
  const Outputs o{static_cast<__nv_bfloat16*>(out), nullptr, static_cast<float*>(workspace), 0};
  return w_mn ? run<true, false>(p, tokens, k, w, k, cols, o, dependent, stream, ctx)
              : run<false, false>(p, tokens, k, w, cols, k, o, dependent, stream, ctx);
}

}  // namespace tpmlp
