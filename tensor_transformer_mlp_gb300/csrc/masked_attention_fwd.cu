// Masked attention, forward, on the tensor cores: o = softmax(y) V and the rows' log-sum-exp, in one pass over the
// keys with running statistics, no score leaving the SM.
//
//   y_ij = c(scale q_i.k_j) - slope |i - j| for lo_i <= j < hi_i;   per key tile, with m the running maximum:
//   P = 2^(y log2 e - m),  l += sum P,  O += P V;   at the end o = O / l,  lse = ln 2 (m + log2 l)
//
// A CTA holds two tiles of 128 queries of one head and walks the key tiles that either of them sees:
//   warps 0-3, 4-7  softmax of query tile 0 and 1, one row per thread (tensor-memory lane)
//   warp 8          one thread loads Q once and K, V tiles through a ring (tensor copies)
//   warp 9          issues the products: S = Q K^T into 128 columns per query tile, and O += P V with P read from
//                   tensor memory (bf16, over the columns of its S)
// The two tiles take turns: while one's softmax runs, the tensor core works on the other's P V and next S. (With an
// issuing warp for each, both softmaxes fell into step and the tensor core waited for them.) S of a tile's next step
// is issued after its P V, and the tensor core runs a thread's products in order, so P is never overwritten
// early and a completed S also says that the P V before it is done: O may then be rescaled. That is done only when the maximum
// grew by more than 2^8 (P then stays below 2^8 and l below 2^8 s, far inside fp32), so almost never: the statistics
// stay those of one common m and the result does not depend on it. With heads of
// more than 64 columns P is handed over in halves of 64 keys, so that its product starts while the second half's
// exponents are still being taken.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attention_tiles.cuh"

namespace tpmlp {
namespace {

constexpr int kSoftmaxWarps = 8;
constexpr int kThreads = (kSoftmaxWarps + 4) * 32;
// Registers: 168 a thread at launch (three warpgroups); the two of the softmax, whose threads hold a row of 128
// scores, take 208 and the third keeps 88 (2 * 208 + 88 = 3 * 168).
constexpr int kRegsSoftmax = 208, kRegsIssue = 88;
constexpr float kRescaleAt = 8.0f;

struct FwdParams {
  HeadMap q, k, v, o;
  const int2* range;
  const float* slopes;
  float* lse;
  ScoreParams sp;
  int s, heads, group, head_dim, nblocks, bheads;  // bheads: heads * b
  unsigned int* status;
};

template <int HD>
struct FwdCfg {
  static constexpr int kBoxes = HD / 64;
  static constexpr int kTileBytes = kBoxes * kBoxBytes;
  static constexpr int kStages = HD == 128 ? 4 : 8;
  static constexpr int kHalves = HD == 128 ? 2 : 1;  // parts in which P is handed over
  static constexpr int kBytes = 1024 + (2 + kStages) * kTileBytes + 512;
};

struct Span {  // key tiles [lo, hi) of a query tile
  int lo, hi;
  __device__ __forceinline__ bool has(int j) const { return lo <= j && j < hi; }
};

template <int HD, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1) masked_attention_forward_kernel(const __grid_constant__ FwdParams p) {
  using L = FwdCfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sq = smem;                                   // two Q tiles
  uint8_t* ring = smem + 2 * L::kTileBytes;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(ring + L::kStages * L::kTileBytes);
  uint64_t* s_full = q_full + 2;
  uint64_t* p_full = s_full + 2;  // [query tile][part of P]
  uint64_t* o_full = p_full + 4;
  uint64_t* kv_full = o_full + 2;
  uint64_t* kv_empty = kv_full + L::kStages;
  uint64_t* drain = kv_empty + L::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int2* warp_span = reinterpret_cast<int2*>(tmem_slot + 2);  // min lo, max hi of each softmax warp's rows

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // query blocks with the most keys (the last, under a causal mask) start first
  const int blk = p.nblocks - 1 - static_cast<int>(blockIdx.x) / p.bheads;
  const int bh = static_cast<int>(blockIdx.x) % p.bheads;
  const int seq = bh / p.heads, head = bh - seq * p.heads, kvh = head / p.group;
  const int q0 = blk * 2 * kTile;
  const int64_t base = static_cast<int64_t>(seq) * p.s;

  int2 r = make_int2(0, 0);
  const int row = q0 + static_cast<int>(threadIdx.x);
  if (warp < kSoftmaxWarps) {
    if (row < p.s) r = clip_range(p.range[base + row], p.s);
    const int lo = __reduce_min_sync(0xffffffffu, r.x < r.y ? r.x : INT32_MAX);
    const int hi = __reduce_max_sync(0xffffffffu, r.y);
    if (lane == 0) warp_span[warp] = make_int2(lo, hi);
  } else if (warp == kSoftmaxWarps) {
    if (lane == 0) {
      for (uint64_t* bar = q_full; bar <= drain; ++bar)
        mbar_init(bar, bar >= p_full && bar < p_full + 4 ? 4 : 1);
      fence_mbar_init();
      for (int i = 0; i < 2; ++i)
        if (q0 + i * kTile < p.s) {  // on their way while the ranges are read; q_full is waited for whatever they are
          mbar_arrive_expect_tx(&q_full[i], L::kTileBytes);
          load_head_tile(sq + i * L::kTileBytes, p.q, &q_full[i], L::kBoxes, q0 + i * kTile, head, seq);
        }
      tma_prefetch_desc(&p.k.map);
      tma_prefetch_desc(&p.v.map);
      tma_prefetch_desc(&p.o.map);
    }
  } else if (warp == kSoftmaxWarps + 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Span span[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int lo = INT32_MAX, hi = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int2 v = warp_span[4 * i + w];
      lo = min(lo, v.x);
      hi = max(hi, v.y);
    }
    span[i] = hi > 0 ? Span{lo / kTile, (hi + kTile - 1) / kTile} : Span{0, 0};
  }
  const bool any0 = span[0].lo < span[0].hi, any1 = span[1].lo < span[1].hi;
  const int j_begin = any0 ? (any1 ? min(span[0].lo, span[1].lo) : span[0].lo) : span[1].lo;
  const int j_end = max(span[0].hi, span[1].hi);
  auto next = [&](int j) {  // the next key tile at or after j that some query tile sees
    while (j < j_end && !span[0].has(j) && !span[1].has(j)) ++j;
    return j;
  };

  if (warp >= kSoftmaxWarps) {
    regs_dec<kRegsIssue>();
    if (warp == kSoftmaxWarps && lane == 0) {
      // ---------------------------------------------------------------- loads
      bool ok = true;
      int n = 0;
      for (int j = next(j_begin); j < j_end && ok; j = next(j + 1)) {
        for (int kv = 0; kv < 2; ++kv, ++n) {
          const int st = n % L::kStages;
          if (!mbar_wait(&kv_empty[st], ((n / L::kStages) & 1) ^ 1, p.status, 0x20)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&kv_full[st], L::kTileBytes);
          load_head_tile(ring + st * L::kTileBytes, kv ? p.v : p.k, &kv_full[st], L::kBoxes, j * kTile, kvh, seq);
        }
      }
      // The copies in flight must land before shared memory goes away (those that the products wait for have).
      if (!ok) {
        for (int k = max(0, n - L::kStages); k < n; ++k)
          mbar_wait(&kv_full[k % L::kStages], (k / L::kStages) & 1, p.status, 0x21);
      }
    } else if (warp == kSoftmaxWarps + 1) {
      // ---------------------------------------------------------------- products
      // A wait that passes and a commit cost 100 to 150 cycles each, which the tensor core must not see: the tiles of
      // the next step are waited for, and tiles released, between products, and S of tile 1 is followed at once by the
      // wait for P of tile 0.
      const uint32_t leader = elect_one();
      const int ksteps = (p.head_dim + 15) / 16;
      const uint32_t idesc_o = idesc_bf16_f32(kTile, ksteps * 16, false, true);
      const uint32_t q_addr = smem_u32(sq), ring_addr = smem_u32(ring);
      bool ok = true;
      auto wait_on = [&](uint64_t* bar, uint32_t parity, unsigned where) {
        if (ok) ok = __all_sync(0xffffffffu, mbar_poll(bar, parity, p.status, where));
      };
      auto commit = [&](uint64_t* bar) { umma_commit_by(leader, bar); };
      auto stage_of = [&](int n) { return ring_addr + (n % L::kStages) * L::kTileBytes; };
      auto wait_tile = [&](int n) { wait_on(&kv_full[n % L::kStages], (n / L::kStages) & 1, 0x22); };
      auto scores = [&](int i, int n) {  // with the K tile of step n
        if (!ok) return;
        issue_rows<HD>(leader, tmem + i * 128, q_addr + i * L::kTileBytes, stage_of(2 * n), ksteps);
        commit(&s_full[i]);
      };
      int j = next(j_begin), jn = next(j + 1), steps[2] = {0, 0};
      if (j < j_end) {
        wait_tile(0);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (i ? any1 : any0) {
            wait_on(&q_full[i], 0, 0x23);
            tc_fence_after();
            if (span[i].has(j)) scores(i, 0);
          }
        wait_tile(1);
      }
      for (int n = 0; j < j_end && ok; ++n) {  // V of step n has arrived
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (span[i].has(j)) {
            const uint32_t to = tmem + 256 + i * 128, tp = tmem + i * 128;
            wait_on(&p_full[2 * i], steps[i] & 1, 0x24);
            tc_fence_after();
            if (!ok) break;
            issue_cols<false, 0, 8 / L::kHalves>(leader, to, tp, stage_of(2 * n + 1), idesc_o, steps[i] != 0);
            if (i == 0) commit(&kv_empty[(2 * n) % L::kStages]);  // K of this step, used before this loop turn
            if constexpr (L::kHalves == 2) {
              wait_on(&p_full[2 * i + 1], steps[i] & 1, 0x24);
              tc_fence_after();
              if (!ok) break;
              issue_cols<false, 4, 8>(leader, to, tp, stage_of(2 * n + 1), idesc_o, 1);
            }
            ++steps[i];
            if (j + 1 == span[i].hi) commit(&o_full[i]);
          } else if (i == 0) {
            commit(&kv_empty[(2 * n) % L::kStages]);
          }
          if (i == 1) {
            commit(&kv_empty[(2 * n + 1) % L::kStages]);
            if (jn < j_end) wait_tile(2 * n + 3);
          } else if (jn < j_end) {
            wait_tile(2 * n + 2);
          }
          if (jn < j_end && span[i].has(jn)) scores(i, n + 1);
        }
        j = jn;
        jn = next(j + 1);
      }
      // every product issued must be done before tensor memory is freed
      commit(drain);
      mbar_wait(drain, 0, p.status, 0x25);
    }
  } else {
    // ------------------------------------------------------------------ softmax
    regs_inc<kRegsSoftmax>();
    const int i = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + i * 128, to = tmem + lanes + 256 + i * 128;
    const float slope2 = BIAS ? p.slopes[head] * kLog2e : 0.f;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    int step = 0;
    const Span mine = i ? span[1] : span[0];
    for (int j = mine.lo; j < mine.hi; ++j, ++step) {
      ok = __all_sync(0xffffffffu, mbar_wait(&s_full[i], step & 1, p.status, 0x26));
      if (!ok) break;
      tc_fence_after();
      auto hand_over = [&](int h) {  // part h of P is in tensor memory
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * i + h]);
      };
      float y[128];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        tmem_ld_32x32b_x32(ts + c * 32, *reinterpret_cast<uint32_t(*)[32]>(reinterpret_cast<uint32_t*>(y) + c * 32));
      tmem_ld_wait();
      const int k0 = j * kTile;
      if constexpr (CAP) cap_tanh_all(y, p.sp);
      if constexpr (BIAS)
        add_bias(y, CAP ? p.sp.cap2 : p.sp.scale2, slope2, static_cast<float>(k0 - row), side_of(k0, kTile, row - lane));
      if (!__all_sync(0xffffffffu, r.x <= k0 && k0 + kTile <= r.y)) {
        const int c0 = r.x - k0;
        const unsigned width = static_cast<unsigned>(r.y - r.x);
#pragma unroll
        for (int c = 0; c < 128; ++c) y[c] = static_cast<unsigned>(c - c0) < width ? y[c] : -INFINITY;
      }
      float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 128; c += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = max3(t[e], y[c + 2 * e], y[c + 2 * e + 1]);
      float top = max3(fmaxf(t[0], t[1]), t[2], t[3]);
      const float unit = BIAS ? 1.0f : CAP ? p.sp.cap2 : p.sp.scale2;  // what brings y to base 2
      top *= unit;
      const bool grow = top > m + kRescaleAt || (m == -INFINITY && top > -INFINITY);
      if (__any_sync(0xffffffffu, grow)) {
        const float m2 = grow ? top : m;
        const float f = m == -INFINITY ? 0.f : ex2_approx(m - m2);
        m = m2;
        l *= f;
        if (step > 0) {  // the first product overwrites O
          for (int c = 0; c < p.head_dim; c += 32) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(to + c, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st_32x32b_x32(to + c, o);
          }
        }
      }
      const float shift = m == -INFINITY ? 0.f : -m;
      const F2 sc = f2_make(unit, unit), sh = f2_make(shift, shift);
      F2 sum0 = f2_make(0.f, 0.f), sum1 = sum0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const F2 v = f2_make(y[h * 64 + 2 * c], y[h * 64 + 2 * c + 1]);
          const float2 z = f2_split(BIAS ? f2_add(v, sh) : f2_fma(v, sc, sh));
          const float a = ex2_approx(z.x), b = ex2_approx(z.y);
          if (c & 1) sum1 = f2_add(sum1, f2_make(a, b));
          else sum0 = f2_add(sum0, f2_make(a, b));
          w[c] = pack_bf16x2(a, b);  // P enters its product in bf16: half a step, 2^-9 of each weight
        }
        tmem_st_32x32b_x32(ts + h * 32, w);
        if (L::kHalves == 2 || h == 1) hand_over(h * (L::kHalves - 1));
      }
      const float2 su = f2_split(f2_add(sum0, sum1));
      l += su.x + su.y;
    }
    if (ok && mine.lo < mine.hi) {
      ok = __all_sync(0xffffffffu, mbar_wait(&o_full[i], 0, p.status, 0x27));
      tc_fence_after();
    }
    // Q's place in shared memory takes the tile's output; Q has been loaded, if only for that.
    if (q0 + i * kTile < p.s && !__all_sync(0xffffffffu, mbar_wait(&q_full[i], 0, p.status, 0x28))) ok = false;
    if (ok) {
      const bool live = l > 0.f;
      store_head_rows(sq + i * L::kTileBytes, p.o, to, live ? 1.0f / l : 0.f, live, warp & 3, lane, 0, L::kBoxes,
                      q0 + i * kTile, head, seq, p.s, p.head_dim);
      if (row < p.s) {
        constexpr float kLn2 = 0.6931471805599453f;
        p.lse[(static_cast<int64_t>(seq) * p.heads + head) * p.s + row] = live ? kLn2 * (m + log2f(l)) : -INFINITY;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftmaxWarps + 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int HD, bool CAP, bool BIAS>
cudaError_t launch(const FwdParams& p, int grid, cudaStream_t stream) {
  auto kernel = masked_attention_forward_kernel<HD, CAP, BIAS>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, FwdCfg<HD>::kBytes);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kThreads, FwdCfg<HD>::kBytes, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_masked_attention_forward(const MaskedAttention& a, cudaStream_t stream, const DeviceCtx& ctx) {
  FwdParams p{};
  const HeadView* views[3] = {&a.q, &a.k, &a.v};
  HeadMap* maps[3] = {&p.q, &p.k, &p.v};
  for (int i = 0; i < 3; ++i) {
    cudaError_t e = make_head_map(maps[i], *views[i], a.b, a.s, i ? a.kv_heads : a.heads, a.head_dim);
    if (e != cudaSuccess) return e;
  }
  cudaError_t e = make_head_map(&p.o, a.o, a.b, a.s, a.heads, a.head_dim, 32);
  if (e != cudaSuccess) return e;
  p.range = a.range;
  p.slopes = a.slopes;
  p.lse = a.lse;
  p.sp = score_params(a.scale, a.softcap);
  p.s = static_cast<int>(a.s);
  p.heads = a.heads;
  p.group = a.heads / a.kv_heads;
  p.head_dim = a.head_dim;
  p.nblocks = static_cast<int>((a.s + 2 * kTile - 1) / (2 * kTile));
  p.bheads = static_cast<int>(a.b) * a.heads;
  p.status = ctx.status;
  const int64_t grid = static_cast<int64_t>(p.nblocks) * p.bheads;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  const int g = static_cast<int>(grid);
  const bool wide = a.head_dim > 64, cap = a.softcap > 0.f, bias = a.slopes != nullptr;
  if (wide)
    return cap ? (bias ? launch<128, true, true>(p, g, stream) : launch<128, true, false>(p, g, stream))
               : (bias ? launch<128, false, true>(p, g, stream) : launch<128, false, false>(p, g, stream));
  return cap ? (bias ? launch<64, true, true>(p, g, stream) : launch<64, true, false>(p, g, stream))
             : (bias ? launch<64, false, true>(p, g, stream) : launch<64, false, false>(p, g, stream));
}

}  // namespace tpmlp
