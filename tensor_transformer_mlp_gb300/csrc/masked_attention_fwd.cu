// Masked attention, forward, on the tensor cores: o = softmax(y) V and the rows' log-sum-exp, in one pass over the
// keys with running statistics, no score leaving the SM.
//
//   y_ij = c(scale q_i.k_j) - slope |i - j| for lo_i <= j < hi_i;   per key tile, with m the running maximum:
//   P = 2^(y log2 e - m),  l += sum P,  O += P V;   at the end o = O / l,  lse = ln 2 (m + log2 l)
//
// A piece of work is two tiles of 128 queries of one head, against the key tiles that either of them sees; a CTA takes one
// after another:
//   warps 0-3, 4-7  softmax of query tile 0 and 1, one row per thread (tensor-memory lane), and its output
//   warp 8          one thread loads Q, and K and V tiles through a ring (tensor copies)
//   warp 9          issues the products: S = Q K^T into 128 columns per query tile, and O += P V with P (bf16) read from
//                   tensor memory
//   warp 10         takes the next piece of work and finds the key tiles that it sees
//   warp 11         heads of up to 64 columns: issues O += P V, and warp 9 only S
// O is rescaled only when the maximum grew by more than 2^8 (P then stays below 2^8 and l below 2^8 s, far inside fp32),
// so almost never: the statistics stay those of one common m and the result does not depend on it.
//
// Heads of more than 64 columns: S and O of two query tiles fill tensor memory, and P goes over its S. The tiles take
// turns: while one's softmax runs, the tensor core works on the other's P V and next S. (With an issuing warp for each
// tile, both softmaxes fell into step and the tensor core waited for them.) S of a tile's next step is issued after its
// P V, and the tensor core runs a thread's products in order, so P is never overwritten early and a completed S also
// says that the P V before it is done. P is handed over in halves of 64 keys, so that its product starts while the second
// half's exponents are still being taken. Bound by shared memory, of which S = Q K^T, with both operands there, wants all
// (2840 cycles a step of two tiles for 2048 of products): full masks, b2 s4096, 32 heads of 128, 356 to 371 us = 1480 to
// 1540 TFLOP/s; causal, b2 s2048, 62 us = 1120 TFLOP/s of the unmasked pairs; causal over 131072 keys 1590 TFLOP/s.
// Heads of up to 64 columns: the products take half of that and the softmax would wait for them, so P has columns of its
// own and S of the next step is issued as soon as this one has been read (b2 s4096, 32 heads of 64: 241 us; as above
// 299 us). Bound by the softmax: 2200 cycles a step, 1024 of them exponents. It is one straight piece of code on purpose:
// a branch around hidden halves of a tile cost more (277 us) than the exponents that it saved.

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
constexpr int kTakeAhead = 2;  // a CTA takes its next piece when this many key tiles are left to load

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
  static constexpr bool kOwnP = HD == 64;       // P has tensor memory of its own, and the two products a warp each
  static constexpr int kHalves = kOwnP ? 1 : 2;  // parts in which P is handed over
  static constexpr int kStageBytes = 32 * 128;   // of output, per softmax warp
  static constexpr int kBytes = (2 + kStages) * kTileBytes + kSoftmaxWarps * kStageBytes + 512;  // 229,888 at HD = 128
  static_assert(kBytes <= 227 * 1024, "shared memory budget");
};

struct Span {  // key tiles [lo, hi) of a query tile
  int lo, hi;
  __device__ __forceinline__ bool has(int j) const { return lo <= j && j < hi; }
};

struct Work {
  int piece;     // -1: none left
  Span span[2];  // key tiles of the two query tiles
  __device__ __forceinline__ bool any(int i) const { return span[i].lo < span[i].hi; }
  __device__ __forceinline__ int begin() const {
    return any(0) ? (any(1) ? min(span[0].lo, span[1].lo) : span[0].lo) : span[1].lo;
  }
  __device__ __forceinline__ int end() const { return max(span[0].hi, span[1].hi); }
  // the next key tile at or after j that some query tile sees
  __device__ __forceinline__ int next(int j) const {
    while (j < end() && !span[0].has(j) && !span[1].has(j)) ++j;
    return j;
  }
};

// Where a piece of work lies. The query blocks with the most keys (the last, under a causal mask) come first.
struct Place {
  int q0, seq, head, kvh;
  int64_t base;
  __device__ __forceinline__ Place(const FwdParams& p, int piece) {
    const int blk = p.nblocks - 1 - piece / p.bheads, bh = piece % p.bheads;
    seq = bh / p.heads;
    head = bh - seq * p.heads;
    kvh = head / p.group;
    q0 = blk * 2 * kTile;
    base = static_cast<int64_t>(seq) * p.s;
  }
};

template <int HD, bool CAP, bool BIAS, bool LONG>
__global__ void __launch_bounds__(kThreads, 1) masked_attention_forward_kernel(const __grid_constant__ FwdParams p) {
  using L = FwdCfg<HD>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sq = smem;  // two Q tiles
  uint8_t* ring = sq + 2 * L::kTileBytes;
  uint8_t* staging = ring + L::kStages * L::kTileBytes;
  uint4* response = reinterpret_cast<uint4*>(staging + kSoftmaxWarps * L::kStageBytes);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(response + 1);
  uint64_t* q_empty = q_full + 2;
  uint64_t* s_full = q_empty + 2;
  uint64_t* p_full = s_full + 2;  // [query tile][part of P]
  uint64_t* o_full = p_full + 4;
  uint64_t* o_empty = o_full + 2;
  uint64_t* work_full = o_empty + 2;
  uint64_t* work_empty = work_full + 2;
  uint64_t* ending = work_empty + 2;
  uint64_t* taken = ending + 1;
  uint64_t* drain = taken + 1;
  uint64_t* s_free = drain + 2;
  uint64_t* kv_full = s_free + 2;
  uint64_t* kv_empty = kv_full + L::kStages;
  Work* works = reinterpret_cast<Work*>(kv_empty + L::kStages);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(works + 2);
  static_assert(16 + (24 + 2 * L::kStages) * 8 + 2 * sizeof(Work) + 4 <= 512, "barrier area");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // With a bias, key tiles are counted from the sequence's end: most rows then meet their nearest keys first, and with
  // them their maximum, where the other way every tile would raise it and have O rescaled.
  const int ktiles = (p.s + kTile - 1) / kTile;
  auto key_of = [&](int j) { return (BIAS ? ktiles - 1 - j : j) * kTile; };  // the first key of tile j
  // A piece's key tiles, by a whole warp; and the keys of this thread's row of a piece.
  auto find_work = [&](int piece) {
    Work w{piece, {}};
    if (piece < 0) return w;
    const Place at(p, piece);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int lo = INT32_MAX, hi = 0;
#pragma unroll
      for (int k = 0; k < kTile; k += 32) {
        const int row = at.q0 + i * kTile + k + lane;
        const int2 r = row < p.s ? clip_range(p.range[at.base + row], p.s) : make_int2(0, 0);
        lo = min(lo, r.x < r.y ? r.x : INT32_MAX);
        hi = max(hi, r.y);
      }
      lo = __reduce_min_sync(0xffffffffu, lo);
      hi = __reduce_max_sync(0xffffffffu, hi);
      if (hi > 0) {
        const int a = lo / kTile, b = (hi + kTile - 1) / kTile;
        w.span[i] = BIAS ? Span{ktiles - b, ktiles - a} : Span{a, b};
      }
    }
    return w;
  };
  auto range_of = [&](int piece) {
    if (piece < 0) return make_int2(0, 0);
    const Place at(p, piece);
    const int row = at.q0 + static_cast<int>(threadIdx.x);
    return row < p.s ? p.range[at.base + row] : make_int2(0, 0);
  };
  Work first{};
  int2 r_next = make_int2(0, 0);
  if (warp < kSoftmaxWarps) {
    r_next = range_of(static_cast<int>(blockIdx.x));
  } else if (warp == kSoftmaxWarps + 2) {
    first = find_work(static_cast<int>(blockIdx.x));
  } else if (warp == kSoftmaxWarps) {
    // a barrier to a lane: one after another they took a fifth of a short prompt (8.2 us against 6.6 in all)
    for (uint64_t* bar = q_full + lane; bar < kv_empty + L::kStages; bar += 32)
      mbar_init(bar, (bar >= p_full && bar < p_full + 4) || (bar >= o_empty && bar < o_empty + 2) ||
                             (bar >= s_free && bar < s_free + 2)
                         ? 4
                     : bar >= work_empty && bar < work_empty + 2 ? kSoftmaxWarps + (L::kOwnP ? 2 : 1)
                                                                 : 1);
    fence_mbar_init();
    if (lane == 0) {
      tma_prefetch_desc(&p.q.map);
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
  auto work_of = [&](int it) {  // the CTA's it-th piece
    Work w{-1, {}};
    if (mbar_wait(&work_full[it & 1], (it >> 1) & 1, p.status, 0x29)) w = works[it & 1];
    return w;
  };

  if (warp >= kSoftmaxWarps) {
    regs_dec<kRegsIssue>();
    if (warp == kSoftmaxWarps && lane == 0) {
      // ---------------------------------------------------------------- loads
      bool ok = true;
      uint32_t n = 0;  // tiles through the ring; it may wrap
      int loaded[2] = {0, 0};
      for (int it = 0; ok; ++it) {
        const Work w = work_of(it);
        if (w.piece < 0) break;
        const Place at(p, w.piece);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (ok && w.any(i)) {
            ok = mbar_wait(&q_empty[i], (loaded[i] & 1) ^ 1, p.status, 0x21);
            if (!ok) break;
            mbar_arrive_expect_tx(&q_full[i], L::kTileBytes);
            load_head_tile(sq + i * L::kTileBytes, p.q, &q_full[i], L::kBoxes, at.q0 + i * kTile, at.head, at.seq);
            ++loaded[i];
          }
        bool told = false;
        for (int j = w.next(w.begin()); j < w.end() && ok; j = w.next(j + 1)) {
          if (!told && w.end() - j <= kTakeAhead) {
            mbar_arrive(ending);
            told = true;
          }
          for (int kv = 0; kv < 2; ++kv, ++n) {
            const uint32_t st = n % L::kStages;
            if (!mbar_wait(&kv_empty[st], ((n / L::kStages) & 1) ^ 1, p.status, 0x20)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&kv_full[st], L::kTileBytes);
            load_head_tile(ring + st * L::kTileBytes, kv ? p.v : p.k, &kv_full[st], L::kBoxes, key_of(j), at.kvh, at.seq);
          }
        }
        if (!told) mbar_arrive(ending);
      }
      // The copies in flight must land before shared memory goes away (those that the products wait for have).
      if (!ok) {
        for (int i = 0; i < 2; ++i)
          if (loaded[i] > 0) mbar_wait(&q_full[i], (loaded[i] - 1) & 1, p.status, 0x21);
        for (uint32_t k = n - min(n, static_cast<uint32_t>(L::kStages)); k != n; ++k)
          mbar_wait(&kv_full[k % L::kStages], (k / L::kStages) & 1, p.status, 0x21);
      }
    } else if (warp == kSoftmaxWarps + 1 || (L::kOwnP && warp == kSoftmaxWarps + 3)) {
      // ---------------------------------------------------------------- products
      const uint32_t leader = elect_one();
      const int ksteps = (p.head_dim + 15) / 16;
      const uint32_t idesc_o = idesc_bf16_f32(kTile, ksteps * 16, false, true);
      const uint32_t q_addr = smem_u32(sq), ring_addr = smem_u32(ring);
      auto commit = [&](uint64_t* bar) { umma_commit_by(leader, bar); };
      if constexpr (L::kOwnP) {
        // One warp issues the scores, the other P V.
        const bool pv = warp == kSoftmaxWarps + 3;
        bool ok = true;
        auto wait_on = [&](uint64_t* bar, uint32_t parity, unsigned where) {
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, p.status, where));
        };
        uint32_t n = 0, steps[2] = {0, 0};  // key tiles, and steps of each query tile, so far; they may wrap
        int pieces[2] = {0, 0};
        for (int it = 0; ok; ++it) {
          const Work w = work_of(it);
          if (__any_sync(0xffffffffu, w.piece < 0)) break;
          const int j_end = w.end();
          for (int j = w.next(w.begin()); j < j_end && ok; j = w.next(j + 1), ++n) {
            const uint32_t t = 2 * n + pv, st = t % L::kStages;
            wait_on(&kv_full[st], (t / L::kStages) & 1, 0x22);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (!ok || !w.span[i].has(j)) continue;
              const bool first = j == w.span[i].lo;
              if (!pv) {
                if (first) wait_on(&q_full[i], pieces[i] & 1, 0x23);
                wait_on(&s_free[i], (steps[i] & 1) ^ 1, 0x2F);
                tc_fence_after();
                if (!ok) break;
                issue_rows<HD>(leader, tmem + i * 128, q_addr + i * L::kTileBytes, ring_addr + st * L::kTileBytes, ksteps);
                commit(&s_full[i]);
                if (j + 1 == w.span[i].hi) commit(&q_empty[i]);
              } else {
                if (first && pieces[i] > 0) wait_on(&o_empty[i], (pieces[i] - 1) & 1, 0x2A);
                wait_on(&p_full[2 * i], steps[i] & 1, 0x24);
                tc_fence_after();
                if (!ok) break;
                issue_cols<false>(leader, tmem + 256 + i * 64, tmem + 384 + i * 64, ring_addr + st * L::kTileBytes, idesc_o,
                                  LONG ? !part_begins(j - w.span[i].lo) : !first);
                commit(&o_full[i]);
              }
              ++steps[i];
            }
            commit(&kv_empty[st]);
          }
          pieces[0] += w.any(0);
          pieces[1] += w.any(1);
          __syncwarp();
          if (lane == 0) mbar_arrive(&work_empty[it & 1]);
        }
        // every product issued must be done before tensor memory is freed
        commit(drain + pv);
        mbar_wait(drain + pv, 0, p.status, 0x25);
      } else {
        // A wait that passes and a commit cost 100 to 150 cycles each, which the tensor core must not see: the tiles of
        // the next step are waited for, and tiles released, between products, and S of tile 1 is followed at once by the
        // wait for P of tile 0.
        bool ok = true;
        auto wait_on = [&](uint64_t* bar, uint32_t parity, unsigned where) {
          if (ok) ok = __all_sync(0xffffffffu, mbar_poll(bar, parity, p.status, where));
        };
        auto stage_of = [&](uint32_t n) { return ring_addr + (n % L::kStages) * L::kTileBytes; };
        auto wait_tile = [&](uint32_t n) { wait_on(&kv_full[n % L::kStages], (n / L::kStages) & 1, 0x22); };
        uint32_t n0 = 0, steps[2] = {0, 0};  // key tiles, and steps of each query tile, so far; they may wrap
        int pieces[2] = {0, 0};
        for (int it = 0; ok; ++it) {
          const Work w = work_of(it);
          if (__any_sync(0xffffffffu, w.piece < 0)) break;
          const int j_end = w.end();
          auto scores = [&](int i, uint32_t n, int j) {  // with the K tile j of step n
            if (!ok) return;
            issue_rows<HD>(leader, tmem + i * 128, q_addr + i * L::kTileBytes, stage_of(2 * n), ksteps);
            commit(&s_full[i]);
            if (j + 1 == w.span[i].hi) commit(&q_empty[i]);
          };
          int j = w.next(w.begin()), jn = w.next(j + 1);
          uint32_t n = n0;
          if (j < j_end) {
            wait_tile(2 * n);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (w.any(i)) {
                wait_on(&q_full[i], pieces[i] & 1, 0x23);
                tc_fence_after();
                if (w.span[i].has(j)) scores(i, n, j);
              }
            wait_tile(2 * n + 1);
          }
          for (; j < j_end && ok; ++n) {  // V of step n has arrived
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (w.span[i].has(j)) {
                const uint32_t to = tmem + 256 + i * 128, tp = tmem + i * 128;
                const bool first = j == w.span[i].lo;
                if (first && pieces[i] > 0) wait_on(&o_empty[i], (pieces[i] - 1) & 1, 0x2A);
                wait_on(&p_full[2 * i], steps[i] & 1, 0x24);
                tc_fence_after();
                if (!ok) break;
                issue_cols<false, 0, 4>(leader, to, tp, stage_of(2 * n + 1), idesc_o,
                                        LONG ? !part_begins(j - w.span[i].lo) : !first);
                if (i == 0) commit(&kv_empty[(2 * n) % L::kStages]);  // K of this step, used before this loop turn
                wait_on(&p_full[2 * i + 1], steps[i] & 1, 0x24);
                tc_fence_after();
                if (!ok) break;
                issue_cols<false, 4, 8>(leader, to, tp, stage_of(2 * n + 1), idesc_o, 1);
                ++steps[i];
                if (j + 1 == w.span[i].hi || (LONG && part_begins(j + 1 - w.span[i].lo))) commit(&o_full[i]);
              } else if (i == 0) {
                commit(&kv_empty[(2 * n) % L::kStages]);
              }
              if (i == 1) {
                commit(&kv_empty[(2 * n + 1) % L::kStages]);
                if (jn < j_end) wait_tile(2 * n + 3);
              } else if (jn < j_end) {
                wait_tile(2 * n + 2);
              }
              if (jn < j_end && w.span[i].has(jn)) scores(i, n + 1, jn);
            }
            j = jn;
            jn = w.next(j + 1);
          }
          n0 = n;
          pieces[0] += w.any(0);
          pieces[1] += w.any(1);
          __syncwarp();
          if (lane == 0) mbar_arrive(&work_empty[it & 1]);
        }
        // every product issued must be done before tensor memory is freed
        commit(drain);
        mbar_wait(drain, 0, p.status, 0x25);
      }
    } else if (warp == kSoftmaxWarps + 2) {
      // ---------------------------------------------------------------- work
      int piece = static_cast<int>(blockIdx.x);
      for (int it = 0;; ++it) {
        const Work w = it == 0 ? first : find_work(piece);
        if (lane == 0) {
          works[it & 1] = w;
          mbar_arrive(&work_full[it & 1]);
        }
        if (piece < 0) break;
        // The next piece is taken when this one nears its end (taken at its start, it would wait behind a long piece
        // while other CTAs ran out of work), in the place in `works` of the one before, which is done with then.
        int next = -1;
        if (lane == 0 && mbar_wait_moving(ending, it & 1, kv_full, p.status, 0x2B) &&
            (it == 0 || mbar_wait(&work_empty[(it - 1) & 1], ((it - 1) >> 1) & 1, p.status, 0x2B)))
          next = take_work(response, taken, it & 1, p.status, 0x2C);
        piece = __shfl_sync(0xffffffffu, next, 0);
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax
    regs_inc<kRegsSoftmax>();
    const int i = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + i * 128, to = tmem + lanes + 256 + i * (L::kOwnP ? 64 : 128);
    const uint32_t tp = L::kOwnP ? tmem + lanes + 384 + i * 64 : ts;
    uint8_t* stage = staging + warp * L::kStageBytes;
    bool ok = true, s_ready = false;  // s_ready: seen ahead of time (kOwnP)
    uint32_t step = 0, parts = 0;  // of this query tile, so far; they may wrap
    [[maybe_unused]] float part[LONG ? HD : 1];           // of a row's O, where there are many key tiles
    Work w = work_of(0);
    for (int it = 0; __all_sync(0xffffffffu, ok && w.piece >= 0); ++it) {
      const Place at(p, w.piece);
      const int row = at.q0 + static_cast<int>(threadIdx.x);
      const int2 r = clip_range(r_next, p.s);
      const float slope2 = BIAS ? p.slopes[at.head] * kLog2e : 0.f;
      float m = -INFINITY, l = 0.f;
      const Span mine = i ? w.span[1] : w.span[0];
      [[maybe_unused]] float part_m = -INFINITY;  // the maximum that part goes by
      [[maybe_unused]] auto part_scale = [&] { return part_m == -INFINITY ? 0.f : ex2_approx(part_m - m); };
      for (int j = mine.lo; j < mine.hi; ++j, ++step) {
        if constexpr (LONG) {
          if (j > mine.lo && part_begins(j - mine.lo)) {
            ok = __all_sync(0xffffffffu, mbar_wait(&o_full[i], (L::kOwnP ? step - 1 : parts) & 1, p.status, 0x27));
            if (!ok) break;
            tc_fence_after();
            ++parts;
            take_part<HD>(part, to, j - mine.lo == kPart, part_scale());
            part_m = m;
          }
        }
        ok = __all_sync(0xffffffffu, s_ready || mbar_wait(&s_full[i], step & 1, p.status, 0x26));
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
        if constexpr (L::kOwnP) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_free[i]);
        }
        const int k0 = key_of(j);
        if constexpr (CAP) cap_tanh_all(y, p.sp);
        if constexpr (BIAS)
          add_bias(y, CAP ? p.sp.cap2 : p.sp.scale2, slope2, static_cast<float>(k0 - row), side_of(k0, kTile, row - lane));
        if (!__all_sync(0xffffffffu, r.x <= k0 && k0 + kTile <= r.y)) {
#pragma unroll
          for (int c = 0; c < 128; c += 32) {
            const unsigned seen = bit_range(r.x - k0 - c, r.y - k0 - c);
#pragma unroll
            for (int e = 0; e < 32; ++e) y[c + e] = (seen >> e) & 1 ? y[c + e] : -INFINITY;
          }
        }
        bool o_ready = false;
        if constexpr (L::kOwnP) o_ready = step > 0 && mbar_done(&o_full[i], (step - 1) & 1);
        float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 128; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) t[e] = max3(t[e], y[c + 2 * e], y[c + 2 * e + 1]);
        float top = max3(fmaxf(t[0], t[1]), t[2], t[3]);
        const float unit = BIAS ? 1.0f : CAP ? p.sp.cap2 : p.sp.scale2;  // what brings y to base 2
        top *= unit;
        const bool grow = top > m + kRescaleAt || (m == -INFINITY && top > -INFINITY);
        if (L::kOwnP && step > 0) {
          ok = __all_sync(0xffffffffu, o_ready || mbar_wait(&o_full[i], (step - 1) & 1, p.status, 0x27));
          if (!ok) break;
          tc_fence_after();
        }
        if (__any_sync(0xffffffffu, grow)) {
          const float m2 = grow ? top : m;
          const float f = m == -INFINITY ? 0.f : ex2_approx(m - m2);
          m = m2;
          l *= f;
          if (LONG ? !part_begins(j - mine.lo) : j > mine.lo) {  // the first product overwrites O
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
          if (L::kOwnP && h == 1) s_ready = mbar_done(&s_full[i], (step + 1) & 1);
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
          tmem_st_32x32b_x32(tp + h * 32, w);
          if (L::kHalves == 2 || h == 1) hand_over(h * (L::kHalves - 1));
        }
        const float2 su = f2_split(f2_add(sum0, sum1));
        l += su.x + su.y;
      }
      if (!ok) break;
      const bool any = mine.lo < mine.hi;
      w = work_of(it + 1);
      r_next = range_of(w.piece);  // on its way during the output
      if (any) {
        ok = __all_sync(0xffffffffu, mbar_wait(&o_full[i], (L::kOwnP ? step - 1 : parts) & 1, p.status, 0x27));
        tc_fence_after();
        ++parts;
      }
      if (ok) {
        if constexpr (LONG) {
          if (mine.hi - mine.lo > kPart) give_part<HD>(part, to, part_scale());
        }
        // Nothing was seen, or scores of -inf alone. A row with NaN or +inf among its scores is not that: its l is NaN, or,
        // where the score overflows only with the scale (the exponents' fma then subtracts infinity from a finite
        // product), 0 beside m = +inf; o and lse get NaN from either.
        const bool live = !(m == -INFINITY && l == 0.f);
        store_head_rows(stage, p.o, to, live ? 1.0f / l : 0.f, live, warp & 3, lane, 0, L::kBoxes, at.q0 + i * kTile,
                               at.head, at.seq, p.s, p.head_dim);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (any) mbar_arrive(&o_empty[i]);
          mbar_arrive(&work_empty[it & 1]);
        }
        if (row < p.s) {
          constexpr float kLn2 = 0.6931471805599453f;
          p.lse[(static_cast<int64_t>(at.seq) * p.heads + at.head) * p.s + row] = live ? kLn2 * (m + log2f(l)) : -INFINITY;
        }
      }
    }
    if (lane == 0) bulk_wait_group_read<0>();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftmaxWarps + 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int HD, bool CAP, bool BIAS, bool LONG>
cudaError_t launch(const FwdParams& p, int grid, cudaStream_t stream, const DeviceCtx& ctx) {
  static SmemLimit done;
  auto kernel = masked_attention_forward_kernel<HD, CAP, BIAS, LONG>;
  const cudaError_t e = allow_smem(&done, kernel, FwdCfg<HD>::kBytes, ctx);
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
  p.bheads = static_cast<int>(a.b * a.heads);
  p.status = ctx.status;
  const int g = p.nblocks * p.bheads;
  const bool wide = a.head_dim > 64, cap = a.softcap > 0.f, bias = a.slopes != nullptr;
  auto by_length = [&](auto hd, auto c, auto bi) {
    constexpr int HD = decltype(hd)::value;
    constexpr bool CAP = decltype(c)::value, BIAS = decltype(bi)::value;
    return (a.s + kTile - 1) / kTile > kLongSum ? launch<HD, CAP, BIAS, true>(p, g, stream, ctx)
                                                : launch<HD, CAP, BIAS, false>(p, g, stream, ctx);
  };
  return pick_kernel(wide, cap, bias, by_length);
}

}  // namespace tpmlp
