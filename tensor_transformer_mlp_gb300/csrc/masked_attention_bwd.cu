// Masked attention, backward, on the tensor cores, in two passes without atomics:
//
//   query pass: per tile of 128 queries, over its key tiles:    dQ_i = sum_j dX_ij k_j
//   key pass:   per tile of 128 keys, over the query tiles that see it and the query heads that share it:
//               dV_j = sum_i P_ij d_o_i,  dK_j = sum_i dX_ij q_i
// with P_ij = exp(y_ij - lse_i) and dX_ij = scale c' P_ij (d_o_i.v_j - D_i) formed again in each (seven products of
// 128 x 128 x head_dim per pair of tiles instead of five). Joining the passes would need dQ summed over key tiles
// across CTAs: fp32 atomics on dQ, in an order that changes from run to run, and a buffer and a pass to round it.
//
// Both passes keep the scores and the gradients of the probabilities in tensor memory, turn them into P and dX there
// (bf16, over the columns of the accumulator that they came from), and feed them to the products from there; shared
// memory only ever holds tiles as they lie in global memory. Warp roles in both:
//   warps 0-7   one row of the accumulators per thread, columns 0-63 (warps 0-3) or 64-127 (warps 4-7)
//   warp 8      tensor copies of the tiles through two rings; in the key pass it takes the CTA's next tile of keys
//   warp 9      issues the products
//   warp 10     query pass: takes the CTA's next tile of queries and finds the key tiles that it sees;
//               key pass: the queries' lse and D, two tiles ahead
// Measured with heads of 128 at b2 s2048, 32 heads, causal: query pass 87 us, key pass 105 us, together 187 us = 920
// TFLOP/s on the five products that a backward cannot do without. A step takes 2070 cycles of the query pass for 1536 of
// products and 2650 of the key pass for 2048: a chain of products, their hand-over (250 cycles each way) and the work on
// P and dX, all eight warps in step. A tile costs some 5000 cycles beside its steps (output, first loads). Heads of 64
// leave room for P and dX beside S and dP, and the products could run ahead of the warps; with an issuing warp each for S
// and dP and for the rest that was no faster (query pass 376 -> 390 us, key pass 536 -> 513 us without a mask, slower
// with a window), nor with half of the warps half a step behind (421, 558 us).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attention_tiles.cuh"

namespace tpmlp {
namespace {

constexpr int kWorkWarps = 8;
constexpr int kThreads = (kWorkWarps + 4) * 32;
constexpr int kTakeAhead = 2;  // a CTA takes its next tile of queries when this many key tiles are left to load
constexpr int kRegsWork = 208, kRegsIssue = 88;  // 2 * 208 + 88 = 3 * 168, the registers at launch

// Summary of a tile of 128 queries: the keys that some row sees lie in [lo, hi), and every row of the tile sees the
// keys of [all_lo, all_hi).
struct TileRange {
  int lo, hi, all_lo, all_hi;
};

struct BwdParams {
  HeadMap q, k, v, o, d_o;    // tiles to load
  HeadMap dq, dk, dv;         // to store by 32 rows
  const int2* range;
  const float* slopes;
  const float* lse;           // [b][heads][s]
  float* dsum;                // [b][heads][s]: D, written by the query pass, read by the key pass
  TileRange* tiles;           // [b][ntiles], likewise
  ScoreParams sp;
  float scale;
  int s, heads, kv_heads, group, head_dim, ntiles, nseq;
  unsigned int* status;
};

// Ring depths. "held" tiles (K of the query pass, Q of the key pass) serve the scores of one step and the product of a
// later one, "passing" tiles (V, d_o) two products in a row. In the query pass the tile's own Q and d_o come through the
// first ring and its o through the second, on their way to tensor memory; the key pass keeps its K and V beside the rings.
template <int HD, bool QUERY_PASS>
struct BwdSmem {
  static constexpr int kBoxes = HD / 64;
  static constexpr int kTileBytes = kBoxes * kBoxBytes;
  static constexpr int kHeld = HD == 128 && !QUERY_PASS ? 3 : 4;
  static constexpr int kPassing = HD == 128 ? 2 : 4;
  static constexpr int kStatBytes = 2 * 2 * kTile * 4;
  // Of output, per working warp; in the key pass with heads of more than 64 columns V's place serves for it.
  static constexpr bool kOwnStage = QUERY_PASS || HD == 64;
  static constexpr int kStageBytes = kOwnStage ? 32 * 128 : 0;
  static constexpr int kTiles = (QUERY_PASS ? 0 : 2) + kHeld + kPassing;
  static constexpr int kBarrierBytes = 320;
  static constexpr int kBytes = kTiles * kTileBytes + kWorkWarps * kStageBytes + kStatBytes + kBarrierBytes;
  static_assert(kBytes <= 227 * 1024, "shared memory budget");  // 231,744 of 232,448 at HD = 128
};

template <bool V>
struct Flag {
  static constexpr bool value = V;
};

// 64 scores q.k to probabilities in place: 2^(y + shift(c, 0)) for columns c, c + 1 (the pair of -lse in base 2; shift(c, x)
// is it with x added to both). done(c, a, b) may change a pair and sees it before the cap's derivative is multiplied in.
// With a bias: side as in side_of, off the bias of the columns' first place where they lie on one side of the row, and
// TILTED if shift has the rest of it already.
template <bool CAP, bool BIAS, bool TILTED, typename Shift, typename Done>
__device__ __forceinline__ void probabilities(float (&w)[64], const ScoreParams& sp, float slope2, int col0, int row,
                                              int side, float off, Shift shift, Done done) {
  const float d0 = static_cast<float>(col0 - row), k = side > 0 ? -slope2 : slope2;
  const float unit = CAP ? sp.cap2 : sp.scale2;
  const F2 u2 = f2_make(unit, unit), one = f2_make(1.0f, 1.0f);
  auto all = [&](auto small, auto line) {
#pragma unroll
    for (int c = 0; c < 64; c += 2) {
      F2 v = f2_make(w[c], w[c + 1]);
      [[maybe_unused]] F2 d = one;  // the cap's derivative
      if constexpr (CAP) {
        if constexpr (decltype(small)::value) {
          v = cap_tanh_small(v, sp.poly3);
          d = f2_sub(one, f2_mul(v, v));  // >= 3/4, so the difference loses nothing
        } else {
          v = cap_tanh(v, sp, d);
        }
      }
      F2 s = shift(c, BIAS && decltype(line)::value ? off : 0.f);
      if constexpr (BIAS) {
        const float c0 = static_cast<float>(c), c1 = static_cast<float>(c + 1);
        if constexpr (decltype(line)::value && !TILTED) {
          const float2 s1 = f2_split(s);
          s = f2_make(fmaf(k, c0, s1.x), fmaf(k, c1, s1.y));
        }
        if constexpr (!decltype(line)::value)
          s = f2_add(s, f2_make(-slope2 * fabsf(d0 + c0), -slope2 * fabsf(d0 + c1)));
      }
      const float2 z = f2_split(f2_fma(v, u2, s));
      float a = ex2_approx(z.x), b = ex2_approx(z.y);
      done(c, a, b);
      if constexpr (CAP) {
        const float2 m = f2_split(f2_mul(f2_make(a, b), d));
        w[c] = m.x;
        w[c + 1] = m.y;
      } else {
        w[c] = a;
        w[c + 1] = b;
      }
    }
  };
  auto both = [&](auto small) {
    if (BIAS && side == 0) all(small, Flag<false>{});
    else all(small, Flag<true>{});
  };
  if (CAP && largest(w) > sp.small3) both(Flag<false>{});
  else both(Flag<true>{});
}

// ------------------------------------------------------------------ query pass

// S and dP take their query-side operand from tensor memory, like dQ its dX: Q and d_o are the same for every key tile,
// and with them in shared memory the two products would read all that it delivers (8 KB per 64 cycles each; 2600 cycles
// a step against 1536 of the products). Tensor memory: S, dP / dX, dQ, 128 columns each, and Q and d_o packed in 64 each.
// S of the next key tile is issued as soon as this one's has been read, so the exponents run beside dP and dQ.
struct QueryWork {
  int piece;      // -1: none left
  int j0, steps;  // its key tiles
};

// Under a causal mask the tiles with the most keys, the last, come first.
struct QueryPlace {
  int tile, q0, seq, head, kvh;
  int64_t base, stat;  // the sequence's first token, and where the head's lse and D start
  __device__ __forceinline__ QueryPlace(const BwdParams& p, int piece) {
    const int bheads = p.heads * p.nseq, bh = piece % bheads;
    tile = p.ntiles - 1 - piece / bheads;
    seq = bh / p.heads;
    head = bh - seq * p.heads;
    kvh = head / p.group;
    q0 = tile * kTile;
    base = static_cast<int64_t>(seq) * p.s;
    stat = (static_cast<int64_t>(seq) * p.heads + head) * p.s;
  }
};

template <int HD, bool CAP, bool BIAS, bool LONG>
__global__ void __launch_bounds__(kThreads, 1) masked_attention_dq_kernel(const __grid_constant__ BwdParams p) {
  using L = BwdSmem<HD, true>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* k_ring = smem;
  uint8_t* v_ring = k_ring + L::kHeld * L::kTileBytes;
  uint8_t* staging = v_ring + L::kPassing * L::kTileBytes;
  float* dsum = reinterpret_cast<float*>(staging + kWorkWarps * L::kStageBytes);  // D of the tile's rows
  uint4* response = reinterpret_cast<uint4*>(dsum + L::kStatBytes / 4);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(response + 1);
  uint64_t* s_full = q_full + 1;
  uint64_t* s_free = s_full + 1;
  uint64_t* dp_full = s_free + 1;
  uint64_t* ds_full = dp_full + 1;
  uint64_t* acc_full = ds_full + 1;
  uint64_t* work_full = acc_full + 1;
  uint64_t* work_empty = work_full + 2;
  uint64_t* ending = work_empty + 2;
  uint64_t* taken = ending + 1;
  uint64_t* drain = taken + 1;
  uint64_t* k_full = drain + 1;
  uint64_t* k_empty = k_full + L::kHeld;
  uint64_t* v_full = k_empty + L::kHeld;
  uint64_t* v_empty = v_full + L::kPassing;
  QueryWork* works = reinterpret_cast<QueryWork*>(v_empty + L::kPassing);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(works + 2);
  static_assert(16 + (13 + 2 * L::kHeld + 2 * L::kPassing) * 8 + 2 * sizeof(QueryWork) + 4 <= L::kBarrierBytes, "barrier area");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == kWorkWarps) {
    for (uint64_t* b = q_full + lane; b < v_empty + L::kPassing; b += 32)
      mbar_init(b, b == q_full || b == s_free || b == ds_full ? kWorkWarps
                   : b >= work_empty && b < work_empty + 2    ? kWorkWarps + 1
                                                              : 1);
    fence_mbar_init();
    if (lane == 0) {
      tma_prefetch_desc(&p.q.map);
      tma_prefetch_desc(&p.k.map);
      tma_prefetch_desc(&p.v.map);
      tma_prefetch_desc(&p.o.map);
      tma_prefetch_desc(&p.d_o.map);
      tma_prefetch_desc(&p.dq.map);
    }
  } else if (warp == kWorkWarps + 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t t_dp = tmem + 128, t_dq = tmem + 256, t_q = tmem + 384, t_g = tmem + 448;
  auto work_of = [&](int it) {  // the CTA's it-th piece
    QueryWork w{-1, 0, 0};
    if (mbar_wait(&work_full[it & 1], (it >> 1) & 1, p.status, 0x2E)) w = works[it & 1];
    return w;
  };

  if (warp >= kWorkWarps) {
    regs_dec<kRegsIssue>();
    if (warp == kWorkWarps && lane == 0) {
      // ---------------------------------------------------------------- loads
      uint32_t kn = 0, vn = 0;  // tiles loaded through the two rings; they may wrap
      bool ok = true;
      auto load = [&](bool held, const HeadMap& m, int row, int head, int seq) {
        const uint32_t st = held ? kn % L::kHeld : vn % L::kPassing;
        uint64_t* full = held ? &k_full[st] : &v_full[st];
        if (ok) ok = held ? mbar_wait(&k_empty[st], ((kn / L::kHeld) & 1) ^ 1, p.status, 0x30)
                          : mbar_wait(&v_empty[st], ((vn / L::kPassing) & 1) ^ 1, p.status, 0x31);
        if (!ok) return;
        mbar_arrive_expect_tx(full, L::kTileBytes);
        load_head_tile((held ? k_ring : v_ring) + st * L::kTileBytes, m, full, L::kBoxes, row, head, seq);
        ++(held ? kn : vn);
      };
      for (int it = 0; ok; ++it) {
        const QueryWork w = work_of(it);
        if (w.piece < 0) break;
        const QueryPlace at(p, w.piece);
        if (w.steps > 0) {
          load(true, p.q, at.q0, at.head, at.seq);
          load(true, p.d_o, at.q0, at.head, at.seq);
          load(false, p.o, at.q0, at.head, at.seq);
        }
        for (int n = 0; n < w.steps && ok; ++n) {
          if (n == max(0, w.steps - kTakeAhead)) mbar_arrive(ending);
          load(true, p.k, (w.j0 + n) * kTile, at.kvh, at.seq);
          load(false, p.v, (w.j0 + n) * kTile, at.kvh, at.seq);
        }
        if (w.steps == 0) mbar_arrive(ending);
      }
      if (!ok) {  // the copies in flight must land before shared memory goes away
        for (uint32_t k = kn - min(kn, static_cast<uint32_t>(L::kHeld)); k != kn; ++k)
          mbar_wait(&k_full[k % L::kHeld], (k / L::kHeld) & 1, p.status, 0x32);
        for (uint32_t k = vn - min(vn, static_cast<uint32_t>(L::kPassing)); k != vn; ++k)
          mbar_wait(&v_full[k % L::kPassing], (k / L::kPassing) & 1, p.status, 0x32);
      }
    } else if (warp == kWorkWarps + 1) {
      // ---------------------------------------------------------------- products
      const uint32_t leader = elect_one();
      const int ksteps = (p.head_dim + 15) / 16;
      const uint32_t idesc_q = idesc_bf16_f32(kTile, ksteps * 16, false, true);
      const uint32_t k_addr = smem_u32(k_ring), v_addr = smem_u32(v_ring);
      bool ok = true;
      auto wait_on = [&](uint64_t* bar, uint32_t parity, unsigned where) {
        if (ok) ok = __all_sync(0xffffffffu, mbar_poll(bar, parity, p.status, where));
        tc_fence_after();
      };
      auto scores = [&](uint32_t k) {  // S = Q K^T with the ring's k-th tile
        wait_on(&k_full[k % L::kHeld], (k / L::kHeld) & 1, 0x34);
        if (!ok) return;
        issue_rows_ta<HD>(leader, tmem, t_q, k_addr + (k % L::kHeld) * L::kTileBytes, ksteps);
        umma_commit_by(leader, s_full);
      };
      auto dprobs = [&](uint32_t v) {  // dP = d_o V^T with the ring's v-th tile
        wait_on(&v_full[v % L::kPassing], (v / L::kPassing) & 1, 0x35);
        if (!ok) return;
        issue_rows_ta<HD>(leader, t_dp, t_g, v_addr + (v % L::kPassing) * L::kTileBytes, ksteps);
        umma_commit_by(leader, dp_full);
        umma_commit_by(leader, &v_empty[v % L::kPassing]);
      };
      uint32_t kn = 0, vn = 0, step = 0, pieces = 0;  // ring tiles, steps and pieces so far; they may wrap
      for (int it = 0; ok; ++it) {
        const QueryWork w = work_of(it);
        if (__any_sync(0xffffffffu, w.piece < 0)) break;
        if (w.steps > 0) {
          kn += 2;  // Q, d_o
          vn += 1;  // o
          wait_on(q_full, pieces & 1, 0x33);
          scores(kn);
          dprobs(vn);
          for (int n = 0; n < w.steps && ok; ++n, ++step) {
            const bool more = n + 1 < w.steps;
            if (more) {
              wait_on(s_free, step & 1, 0x36);
              scores(kn + n + 1);
            }
            wait_on(ds_full, step & 1, 0x36);
            if (!ok) break;
            issue_cols<true>(leader, t_dq, t_dp, k_addr + ((kn + n) % L::kHeld) * L::kTileBytes, idesc_q,
                             LONG ? !part_begins(n) : n != 0);
            if (!more || (LONG && part_begins(n + 1))) umma_commit_by(leader, acc_full);
            if (more) dprobs(vn + n + 1);
            umma_commit_by(leader, &k_empty[(kn + n) % L::kHeld]);
          }
          // the last step's S has been read too, which nobody waits for otherwise
          if (ok) wait_on(s_free, (step - 1) & 1, 0x36);
          kn += w.steps;
          vn += w.steps;
          ++pieces;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&work_empty[it & 1]);
      }
      umma_commit_by(leader, drain);  // every product issued is done before tensor memory is freed
      mbar_wait(drain, 0, p.status, 0x37);
    } else if (warp == kWorkWarps + 2) {
      // ---------------------------------------------------------------- work
      int piece = static_cast<int>(blockIdx.x);
      for (int it = 0;; ++it) {
        QueryWork w{piece, 0, 0};
        if (piece >= 0) {
          const QueryPlace at(p, piece);
          TileRange t{INT32_MAX, 0, 0, INT32_MAX};
#pragma unroll
          for (int k = 0; k < kTile; k += 32) {
            const int row = at.q0 + k + lane;
            const int2 r = row < p.s ? clip_range(p.range[at.base + row], p.s) : make_int2(0, 0);
            const int lo = r.x < r.y ? r.x : INT32_MAX;
            t = TileRange{min(t.lo, lo), max(t.hi, r.y), max(t.all_lo, lo), min(t.all_hi, r.y)};
          }
          t = TileRange{__reduce_min_sync(0xffffffffu, t.lo), __reduce_max_sync(0xffffffffu, t.hi),
                        __reduce_max_sync(0xffffffffu, t.all_lo), __reduce_min_sync(0xffffffffu, t.all_hi)};
          if (t.hi > 0) {
            w.j0 = t.lo / kTile;
            w.steps = (t.hi + kTile - 1) / kTile - w.j0;
          }
          if (at.head == 0 && lane == 0) p.tiles[static_cast<int64_t>(at.seq) * p.ntiles + at.tile] = t;
        }
        if (lane == 0) {
          works[it & 1] = w;
          mbar_arrive(&work_full[it & 1]);
        }
        if (piece < 0) break;
        // The next piece is taken when this one nears its end (taken at its start, it would wait behind a long piece
        // while other CTAs ran out of work), in the place in `works` of the one before, which is done with then.
        int next = -1;
        if (lane == 0 && mbar_wait_moving(ending, it & 1, v_full, p.status, 0x2D) &&
            (it == 0 || mbar_wait(&work_empty[(it - 1) & 1], ((it - 1) >> 1) & 1, p.status, 0x2D)))
          next = take_work(response, taken, it & 1, p.status, 0x2C);
        piece = __shfl_sync(0xffffffffu, next, 0);
      }
    }
  } else {
    // ------------------------------------------------------------------ P, dX
    regs_inc<kRegsWork>();
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int half = warp >> 2, rr = (warp & 3) * 32 + lane;
    uint8_t* stage = staging + warp * L::kStageBytes;
    auto range_of = [&](const QueryWork& w, float* lse2) {  // the row's keys and lse
      *lse2 = 0.f;
      if (w.piece < 0) return make_int2(0, 0);
      const QueryPlace at(p, w.piece);
      if (at.q0 + rr >= p.s) return make_int2(0, 0);
      *lse2 = p.lse[at.stat + at.q0 + rr];
      return p.range[at.base + at.q0 + rr];
    };
    bool ok = true;
    uint32_t kn = 0, vn = 0, step = 0, pieces = 0;  // as the products count them
    uint32_t parts = 0;  // of dQ, so far
    [[maybe_unused]] float part[LONG ? 64 : 1];  // of a row's dQ (warps 4-7: its second 64 columns), for many key tiles
    QueryWork w = work_of(0);
    float lse_next;
    int2 r_next = range_of(w, &lse_next);
    for (int it = 0; __all_sync(0xffffffffu, ok && w.piece >= 0); ++it) {
      const QueryPlace at(p, w.piece);
      const int row = at.q0 + rr, steps = w.steps, j0 = w.j0;
      const int2 r = clip_range(r_next, p.s);
      const bool live = r.x < r.y && lse_next != -INFINITY;  // scores of -inf alone give probabilities of zero
      const float lse2 = live ? lse_next * kLog2e : 0.f;
      const float slope2 = BIAS ? p.slopes[at.head] * kLog2e : 0.f;
      float D = 0.f;
      if (steps > 0) {
        // The row of Q (warps 0-3) or d_o (warps 4-7) goes to tensor memory; each forms half of D = d_o . o.
        const uint32_t os = vn % L::kPassing;
        ok = mbar_wait(&k_full[kn % L::kHeld], (kn / L::kHeld) & 1, p.status, 0x3B) &&
             mbar_wait(&k_full[(kn + 1) % L::kHeld], ((kn + 1) / L::kHeld) & 1, p.status, 0x3B) &&
             mbar_wait(&v_full[os], (vn / L::kPassing) & 1, p.status, 0x3B);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
          const uint8_t* sg = k_ring + ((kn + 1) % L::kHeld) * L::kTileBytes;
          const uint8_t* src = half ? sg : k_ring + (kn % L::kHeld) * L::kTileBytes;
          const uint8_t* so = v_ring + os * L::kTileBytes;
          uint32_t x[HD / 2];
#pragma unroll
          for (int c = 0; c < HD / 8; ++c) {
            const uint4 v = *box_chunk(src + (c >> 3) * kBoxBytes, rr, c & 7);
            x[4 * c] = v.x;
            x[4 * c + 1] = v.y;
            x[4 * c + 2] = v.z;
            x[4 * c + 3] = v.w;
          }
          for (int c = 0; c < HD / 64; ++c)
            tmem_st_32x32b_x32((half ? t_g : t_q) + lanes + c * 32, *reinterpret_cast<uint32_t(*)[32]>(x + c * 32));
          float d[4] = {};
#pragma unroll
          for (int c = 0; c < HD / 16; ++c) {
            const int at = half * (HD / 16) + c, box = (at >> 3) * kBoxBytes;
            const uint4 g = *box_chunk(sg + box, rr, at & 7), u = *box_chunk(so + box, rr, at & 7);
            const uint32_t gw[4] = {g.x, g.y, g.z, g.w}, uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 a = unpack_bf16x2(uw[e]), b = unpack_bf16x2(gw[e]);
              d[e] = fmaf(a.y, b.y, fmaf(a.x, b.x, d[e]));
            }
          }
          dsum[half * kTile + rr] = (d[0] + d[1]) + (d[2] + d[3]);
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(q_full);
        // All rows read and D written, which the working warps wait for like the products (a named barrier has no limit: a
        // warp that gave up in the piece before would leave the others in it).
        ok = ok && __all_sync(0xffffffffu, mbar_wait(q_full, pieces & 1, p.status, 0x3C));
        if (ok && warp == 0 && lane == 0) {
          mbar_arrive(&k_empty[kn % L::kHeld]);
          mbar_arrive(&k_empty[(kn + 1) % L::kHeld]);
          mbar_arrive(&v_empty[os]);
        }
        D = live ? dsum[rr] + dsum[kTile + rr] : 0.f;  // without keys o is zero; d_o may be anything
        if (ok && half && row < p.s) p.dsum[at.stat + row] = D;
        kn += 2 + steps;
        vn += 1 + steps;
      }
      auto wait_for_dq = [&] {  // all products of this part
        ok = __all_sync(0xffffffffu, mbar_wait(acc_full, parts & 1, p.status, 0x3A));
        tc_fence_after();
        ++parts;
      };
      for (int n = 0; n < steps && ok; ++n, ++step) {
        if constexpr (LONG) {
          if (n > 0 && part_begins(n)) {
            wait_for_dq();
            if (!ok) break;
            if (half < L::kBoxes) take_part<64>(part, t_dq + lanes + half * 64, n == kPart, 1.0f);
          }
        }
        ok = __all_sync(0xffffffffu, mbar_wait(s_full, step & 1, p.status, 0x38));
        if (!ok) break;
        tc_fence_after();
        const int k0 = (j0 + n) * kTile + half * 64;
        float w[64];  // P, times the cap's derivative
        const uint32_t ts = tmem + lanes + half * 64;
        tmem_ld_32x32b_x32(ts, *reinterpret_cast<uint32_t(*)[32]>(reinterpret_cast<uint32_t*>(w)));
        tmem_ld_32x32b_x32(ts + 32, *reinterpret_cast<uint32_t(*)[32]>(reinterpret_cast<uint32_t*>(w) + 32));
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_free);
        const int side = BIAS ? side_of(k0, 64, row - lane) : 0;
        probabilities<CAP, BIAS, false>(
            w, p.sp, slope2, k0, row, side, (side > 0 ? -slope2 : slope2) * static_cast<float>(k0 - row),
            [&](int, float add) { return f2_make(add - lse2, add - lse2); }, [](int, float&, float&) {});
        if (!__all_sync(0xffffffffu, r.x <= k0 && k0 + 64 <= r.y)) {
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            const unsigned seen = bit_range(r.x - k0 - c, r.y - k0 - c);
#pragma unroll
            for (int e = 0; e < 32; ++e) w[c + e] = (seen >> e) & 1 ? w[c + e] : 0.f;
          }
        }
        ok = __all_sync(0xffffffffu, mbar_wait(dp_full, step & 1, p.status, 0x39));
        if (!ok) break;
        tc_fence_after();
        uint32_t dp[64], x[32];
        const uint32_t td = t_dp + lanes + half * 64;
        tmem_ld_32x32b_x32(td, *reinterpret_cast<uint32_t(*)[32]>(dp));
        tmem_ld_32x32b_x32(td + 32, *reinterpret_cast<uint32_t(*)[32]>(dp + 32));
        tmem_ld_wait();
        const F2 d2 = f2_make(D, D);
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const F2 g2 = f2_sub(f2_make(__uint_as_float(dp[2 * c]), __uint_as_float(dp[2 * c + 1])), d2);
          const float2 z = f2_split(f2_mul(f2_make(w[2 * c], w[2 * c + 1]), g2));
          x[c] = pack_bf16x2(z.x, z.y);  // dX / scale enters its product in bf16: half a step of each term
        }
        tmem_st_32x32b_x32(td, x);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ds_full);
      }
      if (!ok) break;
      w = work_of(it + 1);
      r_next = range_of(w, &lse_next);  // on its way during the output
      if (steps > 0) {
        wait_for_dq();
        ++pieces;
      }
      if (ok) {
        if constexpr (LONG) {
          if (steps > kPart && half < L::kBoxes) give_part<64>(part, t_dq + lanes + half * 64, 1.0f);
        }
        if (half < L::kBoxes)  // warps 4-7 take the second 64 columns
          store_head_rows(stage, p.dq, t_dq + lanes, p.scale, steps > 0, warp & 3, lane, half, half + 1, at.q0, at.head,
                          at.seq, p.s, p.head_dim);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&work_empty[it & 1]);
      }
    }
    if (lane == 0) bulk_wait_group_read<0>();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWorkWarps + 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ key pass

// Walks the query tiles that see some key of [k0, k1), for each query head of a group in turn; a whole warp calls it.
struct QueryTiles {
  const TileRange* tiles;
  int ntiles, k0, k1, heads_left, base;
  unsigned found;
  int head, tile;
  bool full;  // every row of the tile sees every key
  __device__ __forceinline__ QueryTiles(const TileRange* t, int n, int k0_, int k1_, int first_head, int heads)
      : tiles(t), ntiles(n), k0(k0_), k1(k1_), heads_left(heads), base(-32), found(0), head(first_head), tile(0), full(false) {}
  __device__ __forceinline__ bool next() {
    const int lane = threadIdx.x & 31;
    while (!found) {
      base += 32;
      if (base >= ntiles) {
        base = -32;
        ++head;
        if (--heads_left <= 0) return false;
        continue;
      }
      bool on = false;
      if (base + lane < ntiles) {
        const TileRange t = tiles[base + lane];
        on = t.lo < k1 && t.hi > k0;
      }
      found = __ballot_sync(0xffffffffu, on);
    }
    tile = base + __ffs(found) - 1;
    found &= found - 1;
    const TileRange t = tiles[tile];
    full = t.all_lo <= k0 && t.all_hi >= k1;
    return true;
  }
};

// Under a causal mask the first keys have the most queries and come first.
struct KeyPlace {
  int k0, seq, kvh;
  int64_t base;
  __device__ __forceinline__ KeyPlace(const BwdParams& p, int piece) {
    const int bheads = p.kv_heads * p.nseq, bh = piece % bheads;
    k0 = piece / bheads * kTile;
    seq = bh / p.kv_heads;
    kvh = bh - seq * p.kv_heads;
    base = static_cast<int64_t>(seq) * p.s;
  }
  __device__ __forceinline__ QueryTiles queries(const BwdParams& p) const {
    return QueryTiles(p.tiles + static_cast<int64_t>(seq) * p.ntiles, p.ntiles, k0, min(k0 + kTile, p.s), kvh * p.group,
                      p.group);
  }
};

template <int HD, bool CAP, bool BIAS, bool LONG>
__global__ void __launch_bounds__(kThreads, 1) masked_attention_dkv_kernel(const __grid_constant__ BwdParams p) {
  using L = BwdSmem<HD, false>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sk = smem;
  uint8_t* sv = sk + L::kTileBytes;
  uint8_t* q_ring = sv + L::kTileBytes;
  uint8_t* g_ring = q_ring + L::kHeld * L::kTileBytes;
  uint8_t* staging = L::kOwnStage ? g_ring + L::kPassing * L::kTileBytes : sv;
  // two of {-lse log2(e), with a bias its part within the tile added, [128], D[128]}
  float* stats = reinterpret_cast<float*>(g_ring + L::kPassing * L::kTileBytes + kWorkWarps * L::kStageBytes);
  uint4* response = reinterpret_cast<uint4*>(stats + L::kStatBytes / 4);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(response + 1);
  uint64_t* k_empty = k_full + 1;
  uint64_t* v_full = k_empty + 1;
  uint64_t* v_empty = v_full + 1;
  uint64_t* s_full = v_empty + 1;
  uint64_t* p_full = s_full + 1;
  uint64_t* dp_full = p_full + 1;
  uint64_t* ds_full = dp_full + 1;
  uint64_t* acc_full = ds_full + 1;
  uint64_t* st_full = acc_full + 1;
  uint64_t* st_empty = st_full + 2;
  uint64_t* work_full = st_empty + 2;
  uint64_t* work_empty = work_full + 2;
  uint64_t* taken = work_empty + 2;
  uint64_t* drain = taken + 1;
  uint64_t* q_full = drain + 1;
  uint64_t* q_empty = q_full + L::kHeld;
  uint64_t* g_full = q_empty + L::kHeld;
  uint64_t* g_empty = g_full + L::kPassing;
  int* works = reinterpret_cast<int*>(g_empty + L::kPassing);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(works + 2);
  static_assert(16 + (19 + 2 * L::kHeld + 2 * L::kPassing) * 8 + 8 + 4 <= L::kBarrierBytes, "barrier area");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == kWorkWarps) {
    for (uint64_t* b = k_full + lane; b < g_empty + L::kPassing; b += 32)
      mbar_init(b, (b == v_empty && !L::kOwnStage) || b == p_full || b == ds_full || b == st_empty || b == st_empty + 1
                       ? kWorkWarps
                   : b >= work_empty && b < work_empty + 2 ? kWorkWarps + 2
                                                           : 1);
    fence_mbar_init();
    if (lane == 0) {
      tma_prefetch_desc(&p.q.map);
      tma_prefetch_desc(&p.k.map);
      tma_prefetch_desc(&p.v.map);
      tma_prefetch_desc(&p.d_o.map);
      tma_prefetch_desc(&p.dk.map);
      tma_prefetch_desc(&p.dv.map);
    }
  } else if (warp == kWorkWarps + 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for the query pass's D and tile summaries
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t t_dp = tmem + 128, t_dv = tmem + 256, t_dk = tmem + 384;
  auto work_of = [&](int it) {  // the CTA's it-th piece, -1 past the last; a whole warp calls it
    int piece = -1;
    if (mbar_wait(&work_full[it & 1], (it >> 1) & 1, p.status, 0x4E)) piece = works[it & 1];
    return __all_sync(0xffffffffu, piece >= 0) ? piece : -1;
  };
  auto done_with = [&](int it) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&work_empty[it & 1]);
  };

  if (warp >= kWorkWarps) {
    regs_dec<kRegsIssue>();
    if (warp == kWorkWarps) {
      // ---------------------------------------------------------------- loads
      bool ok = true;
      uint32_t n = 0;  // steps; it may wrap
      int pieces = 0, loaded = 0, loaded_v = 0;  // pieces, and pieces with any steps
      int piece = static_cast<int>(blockIdx.x);
      for (int it = 0;; ++it) {
        if (lane == 0) {
          works[it & 1] = piece;
          mbar_arrive(&work_full[it & 1]);
        }
        if (piece < 0) break;
        const KeyPlace at(p, piece);
        QueryTiles qt = at.queries(p);
        const uint32_t n0 = n;
        for (; ok && qt.next(); ++n) {
          const uint32_t qs = n % L::kHeld, gs = n % L::kPassing;
          ok = __all_sync(0xffffffffu, mbar_wait(&q_empty[qs], ((n / L::kHeld) & 1) ^ 1, p.status, 0x40));
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&q_full[qs], L::kTileBytes);
            load_head_tile(q_ring + qs * L::kTileBytes, p.q, &q_full[qs], L::kBoxes, qt.tile * kTile, qt.head, at.seq);
          }
          if (n == n0) {
            ok = __all_sync(0xffffffffu, mbar_wait(k_empty, (loaded & 1) ^ 1, p.status, 0x42));
            if (!ok) break;
            if (lane == 0) {
              mbar_arrive_expect_tx(k_full, L::kTileBytes);
              load_head_tile(sk, p.k, k_full, L::kBoxes, at.k0, at.kvh, at.seq);
            }
            ++loaded;
          }
          ok = __all_sync(0xffffffffu, mbar_wait(&g_empty[gs], ((n / L::kPassing) & 1) ^ 1, p.status, 0x41));
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&g_full[gs], L::kTileBytes);
            load_head_tile(g_ring + gs * L::kTileBytes, p.d_o, &g_full[gs], L::kBoxes, qt.tile * kTile, qt.head, at.seq);
          }
          if (n == n0) {  // V, perhaps once the outputs that went through its place have left it
            ok = __all_sync(0xffffffffu, mbar_wait(v_empty, ((L::kOwnStage ? loaded - 1 : pieces) & 1) ^ 1, p.status, 0x42));
            if (!ok) break;
            if (lane == 0) {
              mbar_arrive_expect_tx(v_full, L::kTileBytes);
              load_head_tile(sv, p.v, v_full, L::kBoxes, at.k0, at.kvh, at.seq);
            }
            ++loaded_v;
          }
        }
        ++pieces;
        // The next piece, in the place in `works` of the one before this, which is done with then.
        int next = -1;
        if (lane == 0 && ok && (it == 0 || mbar_wait(&work_empty[(it - 1) & 1], ((it - 1) >> 1) & 1, p.status, 0x2D)))
          next = take_work(response, taken, it & 1, p.status, 0x2C);
        piece = __shfl_sync(0xffffffffu, next, 0);
      }
      if (!ok) {  // the copies in flight must land before shared memory goes away
        if (loaded > 0) mbar_wait(k_full, (loaded - 1) & 1, p.status, 0x42);
        if (loaded_v > 0) mbar_wait(v_full, (loaded_v - 1) & 1, p.status, 0x42);
        const uint32_t end = n + 1;  // the step that failed may have begun
        for (uint32_t k = end - min(end, static_cast<uint32_t>(L::kHeld)); k != end; ++k)
          mbar_wait(&q_full[k % L::kHeld], (k / L::kHeld) & 1, p.status, 0x42);
        for (uint32_t k = end - min(end, static_cast<uint32_t>(L::kPassing)); k != end; ++k)
          mbar_wait(&g_full[k % L::kPassing], (k / L::kPassing) & 1, p.status, 0x42);
      }
    } else if (warp == kWorkWarps + 1) {
      // ---------------------------------------------------------------- products
      const uint32_t leader = elect_one();
      const int ksteps = (p.head_dim + 15) / 16;
      const uint32_t idesc_d = idesc_bf16_f32(kTile, ksteps * 16, false, true);
      const uint32_t k_addr = smem_u32(sk), v_addr = smem_u32(sv), q_addr = smem_u32(q_ring), g_addr = smem_u32(g_ring);
      bool ok = true;
      auto wait_on = [&](uint64_t* bar, uint32_t parity, unsigned where) {
        if (ok) ok = __all_sync(0xffffffffu, mbar_poll(bar, parity, p.status, where));
        tc_fence_after();
      };
      auto scores = [&](uint32_t n) {  // S(n)^T = K Q(n)^T
        wait_on(&q_full[n % L::kHeld], (n / L::kHeld) & 1, 0x43);
        if (!ok) return;
        issue_rows<HD>(leader, tmem, k_addr, q_addr + (n % L::kHeld) * L::kTileBytes, ksteps);
        umma_commit_by(leader, s_full);
      };
      auto dprobs = [&](uint32_t n) {  // dP(n)^T = V d_o(n)^T
        wait_on(&g_full[n % L::kPassing], (n / L::kPassing) & 1, 0x44);
        if (!ok) return;
        issue_rows<HD>(leader, t_dp, v_addr, g_addr + (n % L::kPassing) * L::kTileBytes, ksteps);
        umma_commit_by(leader, dp_full);
      };
      uint32_t n = 0, pieces = 0;  // steps, and pieces with any
      for (int it = 0; ok; ++it) {
        const int piece = work_of(it);
        if (piece < 0) break;
        QueryTiles qt = KeyPlace(p, piece).queries(p);
        bool more = qt.next();
        if (more) {
          wait_on(k_full, pieces & 1, 0x45);
          if (ok) scores(n);
          wait_on(v_full, pieces & 1, 0x45);
          if (ok) dprobs(n);
          ++pieces;
        }
        for (int k = 0; more && ok; ++n, ++k) {
          more = qt.next();
          if (!more) {  // S and dP of the last step are on their way: K, and V, may be replaced after them
            umma_commit_by(leader, k_empty);
            if (L::kOwnStage) umma_commit_by(leader, v_empty);
          }
          wait_on(p_full, n & 1, 0x46);
          if (!ok) break;
          issue_cols<true>(leader, t_dv, tmem, g_addr + (n % L::kPassing) * L::kTileBytes, idesc_d,
                           LONG ? !part_begins(k) : k != 0);
          umma_commit_by(leader, &g_empty[n % L::kPassing]);
          if (more) scores(n + 1);
          wait_on(ds_full, n & 1, 0x47);
          if (!ok) break;
          issue_cols<true>(leader, t_dk, t_dp, q_addr + (n % L::kHeld) * L::kTileBytes, idesc_d,
                           LONG ? !part_begins(k) : k != 0);
          umma_commit_by(leader, &q_empty[n % L::kHeld]);
          if (!more || (LONG && part_begins(k + 1))) umma_commit_by(leader, acc_full);
          if (more) dprobs(n + 1);
        }
        done_with(it);
      }
      umma_commit_by(leader, drain);  // every product issued is done before tensor memory is freed
      mbar_wait(drain, 0, p.status, 0x48);
    } else if (warp == kWorkWarps + 2) {
      // ---------------------------------------------------------------- lse and D of the queries
      bool ok = true;
      uint32_t n = 0;
      for (int it = 0; ok; ++it) {
        const int piece = work_of(it);
        if (piece < 0) break;
        const KeyPlace place(p, piece);
        QueryTiles qt = place.queries(p);
        for (; qt.next(); ++n) {
          const int q = qt.tile * kTile + lane * 4;
          const int64_t at = (static_cast<int64_t>(place.seq) * p.heads + qt.head) * p.s + q;
          float l[4], d[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            l[e] = q + e < p.s ? p.lse[at + e] : 0.f;
            l[e] = l[e] == -INFINITY ? 0.f : -l[e] * kLog2e;  // nothing visible, and masked, or scores of -inf alone
            d[e] = q + e < p.s ? p.dsum[at + e] : 0.f;
          }
          // Where queries and keys are different tiles the bias grows with the query: its part within the tile.
          if (BIAS && qt.tile * kTile != place.k0) {
            const float slope2 = p.slopes[qt.head] * kLog2e, k = qt.tile * kTile > place.k0 ? -slope2 : slope2;
#pragma unroll
            for (int e = 0; e < 4; ++e) l[e] = fmaf(k, static_cast<float>(lane * 4 + e), l[e]);
          }
          ok = __all_sync(0xffffffffu, mbar_wait(&st_empty[n & 1], ((n >> 1) & 1) ^ 1, p.status, 0x49));
          if (!ok) break;
          float* st = stats + (n & 1) * 2 * kTile;
          reinterpret_cast<float4*>(st)[lane] = make_float4(l[0], l[1], l[2], l[3]);
          reinterpret_cast<float4*>(st + kTile)[lane] = make_float4(d[0], d[1], d[2], d[3]);
          __syncwarp();
          if (lane == 0) mbar_arrive(&st_full[n & 1]);
        }
        done_with(it);
      }
    }
  } else {
    // ------------------------------------------------------------------ P, dX
    regs_inc<kRegsWork>();
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int half = warp >> 2;
    bool ok = true;
    uint32_t n = 0, parts = 0;  // steps, and parts of dK and dV, so far
    [[maybe_unused]] float part[LONG ? HD : 1];  // of a row's dV (warps 0-3) or dK, where there are many query tiles
    for (int it = 0; ok; ++it) {
      const int piece = work_of(it);
      if (piece < 0) break;
      const KeyPlace at(p, piece);
      const int key = at.k0 + (warp & 3) * 32 + lane;
      QueryTiles qt = at.queries(p);
      const uint32_t acc = (half ? t_dk : t_dv) + lanes;
      auto wait_for_acc = [&] {  // all products of this part
        ok = __all_sync(0xffffffffu, mbar_wait(acc_full, parts & 1, p.status, 0x4D));
        tc_fence_after();
        ++parts;
      };
      int k = 0;  // the piece's steps
      for (; qt.next(); ++n, ++k) {
        if constexpr (LONG) {
          if (k > 0 && part_begins(k)) {
            wait_for_acc();
            if (!ok) break;
            take_part<HD>(part, acc, k == kPart, 1.0f);
          }
        }
        // ranges of the warp's queries, on their way during the waits
        int2 ra = make_int2(0, 0), rb = ra;
        if (!qt.full) {
          const int q = qt.tile * kTile + half * 64 + lane;
          if (q < p.s) ra = p.range[at.base + q];
          if (q + 32 < p.s) rb = p.range[at.base + q + 32];
        }
        ok = __all_sync(0xffffffffu, mbar_wait(&st_full[n & 1], (n >> 1) & 1, p.status, 0x4A));
        // Each lane marks which of the warp's 32 keys two queries see; transposed, which queries see its own key.
        unsigned lo = 0, hi = 0;
        if (!qt.full) {
          auto mark = [&](int2 r) {
            r = clip_range(r, p.s);
            return bit_range(r.x - (key - lane), r.y - (key - lane));
          };
          lo = transpose_bits(mark(ra));
          hi = transpose_bits(mark(rb));
        }
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(s_full, n & 1, p.status, 0x4B));
        if (!ok) break;
        tc_fence_after();
        const float2* lse2 = reinterpret_cast<const float2*>(stats + (n & 1) * 2 * kTile + half * 64);
        const float4* dd = reinterpret_cast<const float4*>(stats + (n & 1) * 2 * kTile + kTile + half * 64);
        const int q0 = qt.tile * kTile + half * 64;
        const float slope2 = BIAS ? p.slopes[qt.head] * kLog2e : 0.f;
        const uint32_t ts = tmem + lanes + half * 64, td = t_dp + lanes + half * 64;
        float w[64];
        tmem_ld_32x32b_x32(ts, *reinterpret_cast<uint32_t(*)[32]>(reinterpret_cast<uint32_t*>(w)));
        tmem_ld_32x32b_x32(ts + 32, *reinterpret_cast<uint32_t(*)[32]>(reinterpret_cast<uint32_t*>(w) + 32));
        tmem_ld_wait();
        // P as it is, packed in x, and times the cap's derivative in w
        uint32_t x[32];
        auto pack_seen = [&](auto masked) {
          const int apart = qt.tile * kTile - at.k0;
          probabilities<CAP, BIAS, true>(
              w, p.sp, slope2, q0, key, apart, (apart > 0 ? -slope2 : slope2) * static_cast<float>(apart + at.k0 - key),
              [&](int c, float add) {
                const float2 l = lse2[c / 2];
                return BIAS ? f2_add(f2_make(l.x, l.y), f2_make(add, add)) : f2_make(l.x, l.y);
              },
              [&](int c, float& a, float& b) {
                if constexpr (decltype(masked)::value) {
                  const unsigned bits = c < 32 ? lo : hi;
                  a = (bits >> (c & 31)) & 1 ? a : 0.f;
                  b = (bits >> ((c & 31) + 1)) & 1 ? b : 0.f;
                }
                x[c / 2] = pack_bf16x2(a, b);  // P enters its product in bf16: half a step of each weight
              });
        };
        if (qt.full) {
          pack_seen(Flag<false>{});
        } else {
          pack_seen(Flag<true>{});
        }
        tmem_st_32x32b_x32(ts, x);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);

        ok = __all_sync(0xffffffffu, mbar_wait(dp_full, n & 1, p.status, 0x4C));
        if (!ok) break;
        tc_fence_after();
        uint32_t dp[64];
        tmem_ld_32x32b_x32(td, *reinterpret_cast<uint32_t(*)[32]>(dp));
        tmem_ld_32x32b_x32(td + 32, *reinterpret_cast<uint32_t(*)[32]>(dp + 32));
        tmem_ld_wait();
#pragma unroll
        for (int c4 = 0; c4 < 16; ++c4) {
          const float4 d4 = dd[c4];
          const F2 a = f2_sub(f2_make(__uint_as_float(dp[4 * c4]), __uint_as_float(dp[4 * c4 + 1])), f2_make(d4.x, d4.y));
          const F2 b = f2_sub(f2_make(__uint_as_float(dp[4 * c4 + 2]), __uint_as_float(dp[4 * c4 + 3])), f2_make(d4.z, d4.w));
          const float2 za = f2_split(f2_mul(f2_make(w[4 * c4], w[4 * c4 + 1]), a));
          const float2 zb = f2_split(f2_mul(f2_make(w[4 * c4 + 2], w[4 * c4 + 3]), b));
          x[2 * c4] = pack_bf16x2(za.x, za.y);
          x[2 * c4 + 1] = pack_bf16x2(zb.x, zb.y);
        }
        tmem_st_32x32b_x32(td, x);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(ds_full);
          mbar_arrive(&st_empty[n & 1]);
        }
      }
      if (ok && k > 0) wait_for_acc();
      if (ok) {
        if constexpr (LONG) {
          if (k > kPart) give_part<HD>(part, acc, 1.0f);
        }
        // warps 0-3 write dV, warps 4-7 dK, a key's row per thread
        store_head_rows(staging + warp * 32 * 128, half ? p.dk : p.dv, acc, half ? p.scale : 1.0f, k > 0, warp & 3, lane, 0,
                        L::kBoxes, at.k0, at.kvh, at.seq, p.s, p.head_dim);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (!L::kOwnStage) {
            bulk_wait_group_read<0>();
            mbar_arrive(v_empty);
          }
          mbar_arrive(&work_empty[it & 1]);
        }
      }
    }
    if (lane == 0) bulk_wait_group_read<0>();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWorkWarps + 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int HD, bool CAP, bool BIAS, bool LONG>
cudaError_t launch_queries(const BwdParams& p, cudaStream_t stream, const DeviceCtx& ctx) {
  static SmemLimit done;
  auto dq = masked_attention_dq_kernel<HD, CAP, BIAS, LONG>;
  const cudaError_t e = allow_smem(&done, dq, BwdSmem<HD, true>::kBytes, ctx);
  if (e != cudaSuccess) return e;
  dq<<<p.ntiles * p.nseq * p.heads, kThreads, BwdSmem<HD, true>::kBytes, stream>>>(p);
  return cudaGetLastError();
}

template <int HD, bool CAP, bool BIAS, bool LONG>
cudaError_t launch_keys(const BwdParams& p, cudaStream_t stream, const DeviceCtx& ctx) {
  static SmemLimit done;
  auto dkv = masked_attention_dkv_kernel<HD, CAP, BIAS, LONG>;
  const cudaError_t e = allow_smem(&done, dkv, BwdSmem<HD, false>::kBytes, ctx);
  if (e != cudaSuccess) return e;
  // the key pass sets itself up while the last CTAs of the query pass finish (programmatic dependent launch)
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.ntiles * p.nseq * p.kv_heads));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = BwdSmem<HD, false>::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, dkv, p);
}

}  // namespace

size_t masked_attention_backward_workspace(int64_t b, int64_t s, int heads) {
  const size_t d = static_cast<size_t>(b) * static_cast<size_t>(s) * static_cast<size_t>(heads) * sizeof(float);
  const size_t t = static_cast<size_t>(b) * static_cast<size_t>((s + kTile - 1) / kTile) * sizeof(TileRange);
  return (d + 255) / 256 * 256 + (t + 255) / 256 * 256;
}

cudaError_t launch_masked_attention_backward(const MaskedAttention& a, const HeadView& d_o, const HeadView& dq,
                                             const HeadView& dk, const HeadView& dv, void* workspace, cudaStream_t stream,
                                             const DeviceCtx& ctx) {
  BwdParams p{};
  const struct {
    HeadMap* map;
    const HeadView* view;
    int heads, rows;
  } maps[] = {{&p.q, &a.q, a.heads, kTile}, {&p.k, &a.k, a.kv_heads, kTile}, {&p.v, &a.v, a.kv_heads, kTile},
              {&p.o, &a.o, a.heads, kTile}, {&p.d_o, &d_o, a.heads, kTile},  {&p.dq, &dq, a.heads, 32},
              {&p.dk, &dk, a.kv_heads, 32}, {&p.dv, &dv, a.kv_heads, 32}};
  for (const auto& m : maps) {
    cudaError_t e = make_head_map(m.map, *m.view, a.b, a.s, m.heads, a.head_dim, m.rows);
    if (e != cudaSuccess) return e;
  }
  p.range = a.range;
  p.slopes = a.slopes;
  p.lse = a.lse;
  p.dsum = static_cast<float*>(workspace);
  const size_t d = static_cast<size_t>(a.b) * static_cast<size_t>(a.s) * static_cast<size_t>(a.heads) * sizeof(float);
  p.tiles = reinterpret_cast<TileRange*>(static_cast<char*>(workspace) + (d + 255) / 256 * 256);
  p.sp = score_params(a.scale, a.softcap);
  p.scale = a.scale;
  p.s = static_cast<int>(a.s);
  p.heads = a.heads;
  p.kv_heads = a.kv_heads;
  p.group = a.heads / a.kv_heads;
  p.head_dim = a.head_dim;
  p.ntiles = static_cast<int>((a.s + kTile - 1) / kTile);
  p.nseq = static_cast<int>(a.b);
  p.status = ctx.status;
  const bool cap = a.softcap > 0.f, bias = a.slopes != nullptr;
  auto both = [&](auto hd, auto c, auto bi) {
    constexpr int HD = decltype(hd)::value;
    constexpr bool CAP = decltype(c)::value, BIAS = decltype(bi)::value;
    const cudaError_t e = p.ntiles > kLongSum ? launch_queries<HD, CAP, BIAS, true>(p, stream, ctx)
                                              : launch_queries<HD, CAP, BIAS, false>(p, stream, ctx);
    if (e != cudaSuccess) return e;
    return static_cast<int64_t>(p.ntiles) * p.group > kLongSum ? launch_keys<HD, CAP, BIAS, true>(p, stream, ctx)
                                                               : launch_keys<HD, CAP, BIAS, false>(p, stream, ctx);
  };
  return pick_kernel(a.head_dim > 64, cap, bias, both);
}

}  // namespace tpmlp
