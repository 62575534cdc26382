// diffragged_fwd at d = 64 (values 128 wide): both maps of a tile of 128 rows in
// one CTA, on tcgen05.
//
// Per key tile S1 = Q1 K1^T, S2 = Q2 K2^T into tensor memory, P_k = 2^(x - m_k)
// as bf16 over S_k, O1 += P1 V, O2 += P2 V: 6 d multiply-adds a pair, and two
// exponentials.  The products and the softmax are those of the dense forward
// (fwd_bf16_sm103.cu): two threads a row and map, exponentials against a running
// reference that sums certify, the exact path where they do not.  What differs:
//   - keys and values come from pages, through warps and rings of their own
//     (three tiles each), so that the next item's tiles are under way while the
//     last one's rows are still being finished;
//   - a warp of its own loads the queries, the heads of a group beside one
//     another ({d, group, tokens} boxes, so that any group up to 64 fills the
//     128 rows as far as whole tokens go); the softmax warps clear what masked
//     rows of a value tile must not spread;
//   - softmax warps whose 16 rows are all past the segment's last one (a single
//     token of four heads fills one warp of eight) only pass the barriers on.
//
// Bound: from a few dozen rows on, the two softmaxes in turn with the products (a
// tile 1.4 us; its products alone 0.75 us, its exponentials 0.5 us); the tensor
// pipe is busy 59 % of the time, the issue slots 47 %.  2048 tokens behind 32768,
// 32 heads over 8: 1146 to 1158 us, 920 to 930 TFLOP/s of the 8 d flop a pair, 1380 to
// 1395 of the 12 d executed (called on end, 1218 us: the GPU then runs at its power
// limit).  A single token a sequence is bound by the keys' and values' bytes, a
// start of 6 us and the join.  A CTA for each map (as at d = 128) took 1272 us, with
// the next tile's logits read ahead into registers 1460; steps of 64 keys, whose
// logits are made while the other half's softmax runs, 1268 (the fixed part of a
// step, 80 of 310 instructions a warp, doubles).
//
// Tensor memory (512 columns): S1 / P1 at 0, S2 / P2 at 128, O1 at 256, O2 at 384;
// shared memory: Q1, Q2 32 KB, three 32 KB tiles of K1, K2 and three of V.
#include <cuda.h>

#include <atomic>
#include <cmath>
#include <cstddef>

#include "ragged_fwd.cuh"
#include "softmax_tile.cuh"

namespace diffattn {
namespace {

constexpr int HD = 64, DV = 128;
constexpr int kSlots = 3;
constexpr int kThreads = 640, kSoftmax = 512, kSoftmaxWarps = kSoftmax / 32;
constexpr int kKeyWarp = 0, kMmaWarp = 1, kValueWarp = 2, kQueryWarp = 3;
constexpr uint32_t kRegsLaunch = 96, kRegsCtrl = 64, kRegsSoftmax = 104;
static_assert(128 * kRegsCtrl + kSoftmax * kRegsSoftmax <= kThreads * kRegsLaunch, "register split");

constexpr uint32_t kBox = kTile * 128;  // 64 bf16 columns of a tile; e4m3 tiles use half of it
constexpr uint32_t kQ = 0, kKeys = 2 * kBox, kValues = kKeys + kSlots * 2 * kBox;
constexpr uint32_t kCtrlAt = kValues + kSlots * 2 * kBox;

struct Ctrl {
  uint64_t k_full[kSlots], k_empty[kSlots], v_full[kSlots], v_empty[kSlots];
  uint64_t q_full, q_empty, s_full[2], p_ready[2], o_done, o_free, drain;
  uint64_t seg_full[kSegRing], seg_empty[kSegRing];
  Segment seg[kSegRing];
  int32_t bad[kSegRing];      // the segment met a page number outside the pool
  int32_t unclean[kSegRing];  // `column` counts
  uint32_t tmem;
  int abort;
  alignas(8) uint8_t column[2][DV];  // fix_each, by segment
  float xch[2 * kTile];
};
static_assert(sizeof(ShareState) <= 2 * kTile * sizeof(float), "the set-up's state lies in xch");
constexpr uint32_t kSmem = kCtrlAt + sizeof(Ctrl) + 1024;
static_assert(kSmem <= 232448, "shared memory");

__host__ __device__ constexpr uint32_t tm_s(int k) { return 128u * k; }
__host__ __device__ constexpr uint32_t tm_o(int k) { return 256u + 128u * k; }

// A piece's O (of one map, in tensor memory), reference and sum with those of the pieces before, which
// are in the part.  (Each thread reads what it has written itself, but for the reference and the sum,
// which a lane of its warp has.)
__device__ __noinline__ float2 merge_piece(const float *part, int key0, uint32_t t_o, bool mine,
                                           float m, float l) {
  tc_fence_after_sync();
  Merge x = {m, l, 0.f, 1.f};
  if (mine) x = merge_states(part[DV * kTile], part[(DV + 1) * kTile], m, l);
#pragma unroll 1
  for (int c0 = 0; c0 < DV / 2; c0 += 32) {
    uint32_t o[32];
    tmem_ld16_x32(t_o + c0, o);
    if (mine) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        o[i] = __float_as_uint(__uint_as_float(o[i]) * x.now +
                               part[(key0 + c0 + i) * kTile] * x.before);
    }
    __syncwarp();
    tmem_st16_x32(t_o + c0, o);
  }
  tmem_st_wait();
  tc_fence_before_sync();
  return make_float2(x.m, x.l);
}

template <bool kFp8>
__global__ void __launch_bounds__(kThreads, 1)
    diffragged_fwd_d64_kernel(const __grid_constant__ CUtensorMap tm_q1,
                              const __grid_constant__ CUtensorMap tm_q2,
                              const __grid_constant__ CUtensorMap tm_k1,
                              const __grid_constant__ CUtensorMap tm_k2,
                              const __grid_constant__ CUtensorMap tm_v,
                              const __grid_constant__ RaggedParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  Ctrl *ctrl = reinterpret_cast<Ctrl *>(smem + kCtrlAt);
  volatile int *abort_flag = &ctrl->abort;
  constexpr uint32_t kRowBytes = kFp8 ? HD : 2 * HD;  // of a query or key row
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int32_t share = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&ctrl->k_full[s], 1);
      mbar_init(&ctrl->k_empty[s], 1);
      mbar_init(&ctrl->v_full[s], 1);
      mbar_init(&ctrl->v_empty[s], 1);
    }
    mbar_init(&ctrl->q_full, 1);
    mbar_init(&ctrl->q_empty, 1);
    for (int k = 0; k < 2; ++k) {
      mbar_init(&ctrl->s_full[k], 1);
      mbar_init(&ctrl->p_ready[k], kSoftmaxWarps / 2);
    }
    mbar_init(&ctrl->o_done, 1);
    mbar_init(&ctrl->o_free, kSoftmaxWarps);
    mbar_init(&ctrl->drain, 1);
    for (int s = 0; s < kSegRing; ++s) {
      mbar_init(&ctrl->seg_full[s], 1);
      mbar_init(&ctrl->seg_empty[s], 3 + kSoftmaxWarps);  // products, values, queries, softmax
    }
    ctrl->abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tm_q1);
    tma_prefetch_desc(&tm_q2);
    tma_prefetch_desc(&tm_k1);
    tma_prefetch_desc(&tm_k2);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&ctrl->tmem, 512);
    tmem_relinquish();
  }
  // Rows past whole tokens are never loaded.
  {
    const uint32_t used = p.tokens * p.group * kRowBytes, all = kTile * kRowBytes;
    for (uint32_t x = used + 16 * threadIdx.x; x < all; x += 16 * kThreads)
      for (int k = 0; k < 2; ++k)
        *reinterpret_cast<uint4 *>(smem + kQ + k * kBox + x) = make_uint4(0, 0, 0, 0);
    if (used < all) fence_async_proxy();
  }
  grid_dependency_wait();
  ShareState *state = reinterpret_cast<ShareState *>(ctrl->xch);
  tc_fence_before_sync();
  Line line;
  if (p.B > kFewSequences)
    line = find_share<kThreads>(p, share, state);
  else
    __syncthreads();
  tc_fence_after_sync();
  grid_dependents_launch();
  const uint32_t tmem = ctrl->tmem;

  // The segments' barriers count segments, those of q and o the ones with keys.
  if (warp < 4) {
    setmaxnreg_dec<kRegsCtrl>();
    if (warp == kKeyWarp) {
      // ------------------------------------------------------------- keys, and the segments
      const int box = lane & 1, piece = lane >> 1, row0 = piece * p.piece_rows;
      const bool piece_ok = row0 < kTile;
      ShareState few;
      if (p.B <= kFewSequences) line = find_share_few(p, share, &few);
      Walk w(p, line, share, p.B <= kFewSequences ? few : *state);
      Ring<kSlots> ring;
      RaggedJoin join = {};
      uint32_t n = 0;
      bool ok = true;
      const auto publish = [&](const Segment &g) {
        const int r = n % kSegRing;
        if (n >= kSegRing)
          ok = mbar_wait_warp(&ctrl->seg_empty[r], (n / kSegRing - 1) & 1, abort_flag, kWaitNs);
        if (ok && lane == 0) {
          ctrl->seg[r] = g;
          ctrl->bad[r] = ctrl->unclean[r] = 0;
          mbar_arrive(&ctrl->seg_full[r]);
        }
        ++n;
      };
      // The end of an item that another share begins comes last where its head has other tiles of
      // rows: their shares then begin at its first keys together, and read them from L2.  (d = 64,
      // 2048 tokens behind 32768: 1194 -> 1151 us; eight times 256 tokens 1085 -> 995 us; a single
      // token has no one to share with: 61 -> 63 us.)
      const bool ends_one = w.more(p) && w.cut && w.tile > 0 && w.s.tiles > 1;
      Segment end_of_one;
      if (ends_one) {
        end_of_one = w.segment(p, share);
        w.next(p);
      }
      for (bool left = ends_one; ok;) {
        const bool walk = w.more(p);
        if (!walk && !left) break;
        const Segment all = walk ? w.segment(p, share) : end_of_one;
        if (!walk) left = false;
        if (all.tile0 == 0 && !(all.flags & kDirect)) join = w.join(line, share, all);
        if ((all.flags & kBadLen) && lane == 0) report_bad_page(p.status);
        int32_t rest = all.tiles;
        while (true) {
          const Segment g = piece_of(walk ? w.segment(p, share) : end_of_one, rest);
          const int r = n % kSegRing;
          publish(g);
          if (!ok || (g.flags & kEmpty)) break;
          int32_t key = g.tile0 * kTile + row0;
          int32_t id = page_of(p, g.b, g.len, key, piece_ok);
          for (int32_t t = 0; t < g.tiles; ++t, key += kTile) {
            const int32_t page = id;
            const bool have = piece_ok && key < g.len;
            const bool bad = have && static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.num_pages);
            if (t + 1 < g.tiles) id = page_of(p, g.b, g.len, key + kTile, piece_ok);
            if (!(ok = ring.wait_empty(ctrl->k_empty, abort_flag))) break;
            const int s = ring.slot();
            if (__any_sync(0xffffffffu, bad)) {
              if (lane == 0) {
                ctrl->bad[r] = 1;
                report_bad_page(p.status);
              }
            }
            if (have && dbg_ok(row0 + p.piece_rows <= kTile, p.status, 100))
              tma_load_4d(smem + kKeys + s * 2 * kBox + box * kBox + row0 * kRowBytes,
                          box ? &tm_k2 : &tm_k1, &ctrl->k_full[s], 0, p.by_page.mod(key), g.hk,
                          bad ? 0 : page);
            const int pieces = __popc(__ballot_sync(0xffffffffu, have));
            if (lane == 0)
              mbar_arrive_expect_tx(&ctrl->k_full[s], pieces * p.piece_rows * kRowBytes);
            ++ring.n;
          }
          rest -= g.tiles;
          if (!ok || rest == 0) break;
        }
        if (!ok) break;
        if (walk) w.next(p);
      }
      if (ok) {
        Segment g = {};
        g.flags = kStop;
        publish(g);
      }
      if (lane == 0) {
        if (p.joins != nullptr) p.joins[share] = join;
        ring.drain(ctrl->k_full);
      }
      __syncwarp();
    } else if (warp == kValueWarp) {
      // ------------------------------------------------------------- values
      const int box = lane & 1, piece = lane >> 1, row0 = piece * p.piece_rows;
      const bool piece_ok = row0 < kTile;
      Ring<kSlots> ring;
      bool ok = true;
      for (uint32_t n = 0; ok; ++n) {
        const int r = n % kSegRing;
        if (!mbar_wait_warp(&ctrl->seg_full[r], (n / kSegRing) & 1, abort_flag, kWaitNs)) break;
        const Segment g = ctrl->seg[r];
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->seg_empty[r]);
        if (g.flags & kStop) break;
        if (g.flags & kEmpty) continue;
        int32_t key = g.tile0 * kTile + row0;
        int32_t id = page_of(p, g.b, g.len, key, piece_ok);
        for (int32_t t = 0; t < g.tiles; ++t, key += kTile) {
          const int32_t page = id;
          const bool have = piece_ok && key < g.len;
          const bool bad = static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.num_pages);
          if (t + 1 < g.tiles) id = page_of(p, g.b, g.len, key + kTile, piece_ok);
          if (!(ok = ring.wait_empty(ctrl->v_empty, abort_flag))) break;
          const int s = ring.slot();
          if (have && dbg_ok(row0 + p.piece_rows <= kTile, p.status, 101))
            tma_load_4d(smem + kValues + s * 2 * kBox + box * kBox + row0 * 128, &tm_v,
                        &ctrl->v_full[s], 64 * box, p.by_page.mod(key), g.hk, bad ? 0 : page);
          const int pieces = __popc(__ballot_sync(0xffffffffu, have));
          if (lane == 0) mbar_arrive_expect_tx(&ctrl->v_full[s], pieces * p.piece_rows * 128);
          ++ring.n;
        }
      }
      if (lane == 0) ring.drain(ctrl->v_full);
      __syncwarp();
    } else if (warp == kQueryWarp) {
      // ------------------------------------------------------------- queries
      uint32_t filled = 0;  // segments with keys
      for (uint32_t n = 0;; ++n) {
        const int r = n % kSegRing;
        if (!mbar_wait_warp(&ctrl->seg_full[r], (n / kSegRing) & 1, abort_flag, kWaitNs)) break;
        const Segment *g = &ctrl->seg[r];
        const int32_t flags = g->flags;
        if (flags & kStop) break;
        if (!(flags & kEmpty)) {
          if (filled > 0 && !mbar_wait_warp(&ctrl->q_empty, (filled - 1) & 1, abort_flag, kWaitNs))
            break;
          if (lane == 0) {
            dbg_ok(g->row >= 0 && g->row + g->tokens <= p.N, p.status, 102);
            mbar_arrive_expect_tx(&ctrl->q_full, 2 * p.tokens * p.group * kRowBytes);
            tma_load_3d(smem + kQ, &tm_q1, &ctrl->q_full, 0, g->hk * p.group, g->row);
            tma_load_3d(smem + kQ + kBox, &tm_q2, &ctrl->q_full, 0, g->hk * p.group, g->row);
          }
          ++filled;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->seg_empty[r]);
      }
      if (lane == 0 && filled > 0) drain_wait(&ctrl->q_full, (filled - 1) & 1);
      __syncwarp();
    } else {
      // ------------------------------------------------------------- products
      constexpr uint32_t kIdescQK = idesc_bf16_f32(kTile, kTile, false);
      constexpr uint32_t kIdescQK8 = idesc_e4m3_f32(kTile, kTile);
      constexpr uint32_t kIdescPV = idesc_bf16_f32(kTile, DV, true);
      auto lo = [](uint64_t d) { return static_cast<uint32_t>(d); };
      const uint32_t dhi =
          static_cast<uint32_t>(smem_desc_sw128(smem_u32(smem + kQ), 16, 1024) >> 32);
      const uint32_t dq = lo(smem_desc_sw128(smem_u32(smem + kQ), 16, 1024));
      const uint32_t dk = lo(smem_desc_sw128(smem_u32(smem + kKeys), 16, 1024));
      const uint32_t dv = lo(smem_desc_sw128(smem_u32(smem + kValues), kBox, 1024));
      auto qk = [&](int k, uint32_t s) {
        if (!dbg_ok(s < kSlots && tmem_cols_ok(tmem + tm_s(k), kTile, tmem, 512), p.status, 103))
          return;
        if (kFp8) {
          const uint64_t a = smem_desc_sw64(smem_u32(smem + kQ + k * kBox));
          const uint64_t b = smem_desc_sw64(smem_u32(smem + kKeys + s * 2 * kBox + k * kBox));
#pragma unroll
          for (int kk = 0; kk < HD / 32; ++kk)
            umma_e4m3_ss_warp(tmem + tm_s(k), a + 2 * kk, b + 2 * kk, kIdescQK8, kk > 0);
        } else {
          const uint32_t a = dq + (k * kBox >> 4), b = dk + ((s * 2 + k) * kBox >> 4);
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk)
            umma_bf16_ss_lo_warp(tmem + tm_s(k), a + 2 * kk, b + 2 * kk, dhi, kIdescQK, kk > 0);
        }
      };
      // P_k's keys 0-63 lie packed over S_k columns 0-31, keys 64-127 over 64-95; 16 keys of V are
      // 2048 bytes.
      auto pv = [&](int k, uint32_t s, bool accumulate) {
        if (!dbg_ok(s < kSlots && tmem_cols_ok(tmem + tm_o(k), DV, tmem, 512), p.status, 104))
          return;
        const uint32_t b = dv + (s * 2 * kBox >> 4);
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          umma_bf16_ts_lo_warp(tmem + tm_o(k), tmem + tm_s(k) + kk * 8 + (kk >= 4 ? 32 : 0),
                               b + 128 * kk, dhi, kIdescPV, (accumulate || kk > 0) ? 1u : 0u);
      };
      auto wait = [&](uint64_t *bar, uint32_t parity) {
        return mbar_wait_warp(bar, parity, abort_flag, kWaitNs);
      };
      bool ok = true;
      uint32_t c = 0, filled = 0;  // key tiles, segments with keys
      for (uint32_t n = 0; ok; ++n) {
        const int r = n % kSegRing;
        if (!(ok = wait(&ctrl->seg_full[r], (n / kSegRing) & 1))) break;
        const int32_t flags = ctrl->seg[r].flags, tiles = ctrl->seg[r].tiles;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->seg_empty[r]);
        if (flags & kStop) break;
        if (flags & kEmpty) continue;
        if (!(ok = wait(&ctrl->q_full, filled & 1))) break;
        for (int32_t t = 0; t < tiles; ++t, ++c) {
          const uint32_t s = c % kSlots, ph = (c / kSlots) & 1;
          if (!(ok = wait(&ctrl->k_full[s], ph))) break;
          tc_fence_after_sync();
          qk(0, s);
          umma_commit_warp(&ctrl->s_full[0]);
          if (t > 0) {
            if (!(ok = wait(&ctrl->p_ready[1], (c - 1) & 1))) break;
            tc_fence_after_sync();
            const uint32_t sp = (c - 1) % kSlots;
            pv(1, sp, t > 1);
            umma_commit_warp(&ctrl->v_empty[sp]);
          }
          qk(1, s);
          umma_commit_warp(&ctrl->s_full[1]);
          umma_commit_warp(&ctrl->k_empty[s]);
          if (t == tiles - 1) umma_commit_warp(&ctrl->q_empty);
          if (!(ok = wait(&ctrl->v_full[s], ph))) break;
          if (!(ok = wait(&ctrl->p_ready[0], c & 1))) break;
          if (t == 0 && filled > 0 && !(ok = wait(&ctrl->o_free, (filled - 1) & 1))) break;
          tc_fence_after_sync();
          pv(0, s, t > 0);
        }
        if (!ok) break;
        if (!(ok = wait(&ctrl->p_ready[1], (c - 1) & 1))) break;
        tc_fence_after_sync();
        pv(1, (c - 1) % kSlots, tiles > 1);
        umma_commit_warp(&ctrl->v_empty[(c - 1) % kSlots]);
        umma_commit_warp(&ctrl->o_done);
        ++filled;
      }
      umma_commit_warp(&ctrl->drain);  // tensor memory is not freed under a running product
      drain_wait(&ctrl->drain, 0);
      __syncwarp();
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    // --------------------------------------------------------------- softmax
    const int sw = warp - 4, k = sw >> 3;        // the map
    const int quarter = warp & 3;                // of tensor memory's lanes
    const int hl = lane & 15, hc = lane >> 4;    // row of the warp's 16; keys 64 hc ..
    const int warp_row = quarter * 32 + ((sw >> 2) & 1) * 16, r = warp_row + hl;
    const int key0 = 64 * hc;
    const uint32_t lane_addr = static_cast<uint32_t>(warp_row) << 16;
    const uint32_t t_s = tmem + lane_addr + tm_s(k), t_o = tmem + lane_addr + tm_o(k);
    const float sl2 = p.scale_log2;
    float *xch = ctrl->xch;
    const int32_t token = p.by_group.div(r), head = r - token * p.group;
    uint32_t c = 0, filled = 0;
    for (uint32_t n = 0;; ++n) {
      const int ring = n % kSegRing;
      // (Every way out of the loop is agreed on: a segment may come after one warp has given up.)
      if (!mbar_wait_warp(&ctrl->seg_full[ring], (n / kSegRing) & 1, abort_flag, kWaitNs)) {
        named_barrier_or(1, kSoftmax, true);
        break;
      }
      const Segment *g = &ctrl->seg[ring];
      const int32_t flags = g->flags;
      if (flags & kStop) {
        named_barrier_or(1, kSoftmax, true);
        break;
      }
      const int32_t tiles = g->tiles, rows = g->tokens * p.group;
      const int32_t pos = g->first + token;
      const int32_t h = g->hk * p.group + head;
      const float lam = r < rows ? p.lambda[h] : 0.f;
      const bool live = warp_row < rows;  // some row of the warp counts
      // The first tile that not all rows see whole (map 2's warps have nothing to do with it).
      const int32_t t_fix = k == 0 ? (seen_by_all(p, *g) + 1) / kTile - g->tile0 : INT32_MAX;
      // Key column x of the segment's tile t is visible to this row iff x <= lim0 - 128 t.  (A row
      // that sees no key, or is none, is computed as one that sees some, and not written.)
      const int32_t lim0 =
          (p.causal ? min(max(pos, 0), g->len - 1) : g->len - 1) - g->tile0 * kTile;
      float m_run = -INFINITY, l_run = 0.f;
      bool ok = true;
      if (!(flags & kEmpty)) {
        for (int32_t t = 0; t < tiles; ++t, ++c) {
          ok = mbar_wait_warp(&ctrl->s_full[k], c & 1, abort_flag, kWaitNs);
          if (!ok) break;
          if (live) {
            tc_fence_after_sync();
            const int lim = lim0 - t * kTile;
            const bool masked = __any_sync(0xffffffffu, lim < kTile - 1);
            if (!dbg_ok_warp(tmem_range_ok(t_s, kTile, tmem, 512, warp, 16) &&
                                 tmem_range_ok(t_o, DV, tmem, 512, warp, 16),
                             p.status, 105)) {
              ok = false;
              break;
            }
            uint32_t pk[kTile / 4];
            float tile_sum = 0.f;
            // As in the dense forward: against the running reference, whose sums certify the tile,
            // or from the maximum.
            if (t == 0) {
              tile_sum = softmax_half_first(t_s, key0, sl2, lim, masked, m_run, pk);
            } else {
              tile_sum = masked ? softmax_half_exp<true>(t_s, key0, m_run, sl2, lim, pk)
                                : softmax_half_exp<false>(t_s, key0, m_run, sl2, lim, pk);
              // (Rows past the segment's last hold whatever lies there, and have no say.)
              if (__any_sync(0xffffffffu, !(tile_sum <= CERT_SUM) && r < rows)) {
                float mt = masked ? softmax_half_max<true>(t_s, key0, lim)
                                  : softmax_half_max<false>(t_s, key0, lim);
                mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
                const float m_new = fmaxf(m_run, mt * sl2 + M_HEADROOM);
                float alpha = 1.f;
                if (m_new > m_run) {  // move m whenever the tile exceeds it
                  alpha = ex2_approx(m_run - m_new);
                  m_run = m_new;
                }
                if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
                  for (int c0 = 0; c0 < DV / 2; c0 += 32) {
                    uint32_t o[32];
                    tmem_ld16_x32(t_o + c0, o);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                      const float2 v = __fmul2_rn(
                          make_float2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])),
                          make_float2(alpha, alpha));
                      o[i] = __float_as_uint(v.x);
                      o[i + 1] = __float_as_uint(v.y);
                    }
                    tmem_st16_x32(t_o + c0, o);
                  }
                }
                l_run *= alpha;
                const float m_use = m_run == -INFINITY ? 0.f : m_run;
                tile_sum = masked ? softmax_half_exp<true>(t_s, key0, m_use, sl2, lim, pk)
                                  : softmax_half_exp<false>(t_s, key0, m_use, sl2, lim, pk);
              }
            }
            l_run += tile_sum;
            tmem_st16_x32(t_s, pk);
            tmem_st_wait();
            tc_fence_before_sync();
          }
          // The first product with the tile's values waits for map 1's warps.
          if (t >= t_fix) {
            uint8_t *values = smem + kValues + (c % kSlots) * 2 * kBox;
            const int32_t key = (g->tile0 + t) * kTile, seen = seen_by_all(p, *g), len = g->len;
            if (!(ok = mbar_wait_warp(&ctrl->v_full[c % kSlots], (c / kSlots) & 1, abort_flag,
                                      kWaitNs)))
              break;
            if (fix_rows<2>(values, 16 * sw, key, seen, len)) {
              uint32_t *columns = reinterpret_cast<uint32_t *>(ctrl->column[n & 1]);
              if (!(ok = open_columns(&ctrl->unclean[ring], columns, DV / 4,
                                      &ctrl->seg_empty[(n - 2) % kSegRing],
                                      ((n - 2) / kSegRing) & 1, n >= 2, abort_flag)))
                break;
              fix_each<2>(values, 16 * sw, key, seen, len, columns);
            }
            fence_async_proxy();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctrl->p_ready[k]);
        }
        if (ok) ok = mbar_wait_warp(&ctrl->o_done, filled & 1, abort_flag, kWaitNs);
        float l_row = l_run + __shfl_xor_sync(0xffffffffu, l_run, 16);
        if ((flags & kAgain) && ok && live) {
          const float2 both = merge_piece(p.part + (g->slot * 2ll + k) * part_floats(DV) + r, key0, t_o,
                                          r < rows, m_run, l_row);
          m_run = both.x;
          l_row = both.y;
        }
        const float inv = 1.f / l_row;
        // (Every thread has read the last segment's exchange: its P of this one came behind it.)
        if (hc == 0) xch[k * kTile + r] = inv;
        if (named_barrier_or(1, kSoftmax, !ok || *abort_flag != 0)) break;
        tc_fence_after_sync();
        ++filled;
        if (!(flags & kDirect)) {
          // A part: O_k column by column, the reference and the sum.
          float *part = p.part + (g->slot * 2ll + k) * part_floats(DV);
          const bool unclean = ctrl->unclean[ring] == 2;
          const int32_t far = pos - seen_by_all(p, *g);
          const bool mine = r < rows;
#pragma unroll 1
          for (int c0 = 0; c0 < DV / 2; c0 += 32) {
            uint32_t v[32];
            tmem_ld16_x32(t_o + c0, v);
            if (mine) {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                float x = __uint_as_float(v[i]);
                if (unclean && ctrl->column[n & 1][key0 + c0 + i] <= far) x = NAN;
                part[(key0 + c0 + i) * kTile + r] = x;
              }
            }
          }
          if (mine && hc == 0) {
            part[DV * kTile + r] = m_run;
            part[(DV + 1) * kTile + r] = ctrl->bad[ring] ? NAN : l_row;
          }
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&ctrl->o_free);
            mbar_arrive(&ctrl->seg_empty[ring]);
          }
          continue;
        }
      }

      // ------------------------------------------------------------- the rows of a whole item
      // This thread's 32 value columns: 64 hc + 32 k ..
      const int col0 = key0 + 32 * k;
      float o[32];
      float ss = 0.f;
      if (flags & kEmpty) {
        const float x = flags & kBadLen ? NAN : 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = x;
      } else {
        const float inv1 = ctrl->bad[ring] ? NAN : xch[r], c2 = lam * xch[kTile + r];
        {
          uint32_t o1[32], o2[32];
          tmem_ld16_x32_nowait(tmem + lane_addr + tm_o(0) + 32 * k, o1);
          tmem_ld16_x32_nowait(tmem + lane_addr + tm_o(1) + 32 * k, o2);
          tmem_ld_wait_x32(o1);
          tmem_ld_wait_x32(o2);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            o[i] = __uint_as_float(o1[i]) * inv1 - __uint_as_float(o2[i]) * c2;
            ss = fmaf(o[i], o[i], ss);
          }
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->o_free);
        if (ctrl->unclean[ring] == 2) {
          const int32_t far = pos - seen_by_all(p, *g);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (ctrl->column[n & 1][col0 + i] <= far) o[i] = ss = NAN;
        }
        if (p.headnorm) {
          named_barrier_sync(1, kSoftmax);  // every thread has read the 1 / l exchange
          if (p.headnorm == 2) {
            float sm = 0.f;
#pragma unroll
            for (int i = 0; i < 32; ++i) sm += o[i];
            sm += __shfl_xor_sync(0xffffffffu, sm, 16);
            if (hc == 0) xch[k * kTile + r] = sm;
            named_barrier_sync(1, kSoftmax);
            const float mu = (xch[r] + xch[kTile + r]) * (1.f / DV);
            named_barrier_sync(1, kSoftmax);
            ss = 0.f;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              o[i] -= mu;
              ss = fmaf(o[i], o[i], ss);
            }
          }
          ss += __shfl_xor_sync(0xffffffffu, ss, 16);
          if (hc == 0) xch[k * kTile + r] = ss;
          named_barrier_sync(1, kSoftmax);
          const float rr = rsqrtf((xch[r] + xch[kTile + r]) * (1.f / DV) + p.eps) * p.out_scale;
          if (p.norm_w != nullptr && r < rows) {
            const float4 *w4 = reinterpret_cast<const float4 *>(p.norm_w + h * DV + col0);
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 w = w4[i / 4];
              o[i] *= rr * w.x;
              o[i + 1] *= rr * w.y;
              o[i + 2] *= rr * w.z;
              o[i + 3] *= rr * w.w;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= rr;
          }
        }
        if (pos < 0) {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.f;
        }
      }
      uint4 pkt[4];
#pragma unroll
      for (int v = 0; v < 4; ++v)
        pkt[v] = make_uint4(pack_bf16x2(o[8 * v], o[8 * v + 1]), pack_bf16x2(o[8 * v + 2], o[8 * v + 3]),
                            pack_bf16x2(o[8 * v + 4], o[8 * v + 5]),
                            pack_bf16x2(o[8 * v + 6], o[8 * v + 7]));
      transpose4_chunks(pkt, lane);
      const int32_t r0 = r - (lane & 3);
      __nv_bfloat16 *out = p.out + g->row * p.out_n + g->hk * p.group * p.out_h + col0 + 8 * (lane & 3);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int32_t i = p.by_group.div(r0 + j);
        if (r0 + j < rows && dbg_ok(g->row + i < p.N, p.status, 106))
          *reinterpret_cast<uint4 *>(out + i * p.out_n + (r0 + j - i * p.group) * p.out_h) = pkt[j];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctrl->seg_empty[ring]);
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && *abort_flag && p.status != nullptr)
    atomicExch(p.status, static_cast<int32_t>(DIFFATTN_ERR_TIMEOUT));
}

}  // namespace

diffattn_status launch_ragged_main_d64(const RaggedParams &p, const CUtensorMap (&maps)[5], bool fp8,
                                       cudaStream_t stream) {
  static std::atomic<bool> ready[2][64];
  return fp8 ? launch_ragged_kernel(diffragged_fwd_d64_kernel<true>, ready[1], p, maps, kThreads,
                                    kSmem, 1, stream)
             : launch_ragged_kernel(diffragged_fwd_d64_kernel<false>, ready[0], p, maps, kThreads,
                                    kSmem, 1, stream);
}

}  // namespace diffattn
