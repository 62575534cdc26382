// diffragged_fwd at d = 128 (values 256 wide): a pair of CTAs takes a tile of 128
// rows, one map each, on tcgen05.
//
// Both maps' accumulators (2 x 256 columns) would fill tensor memory, and two
// passes over the keys with one accumulator (the dense forward's way at this
// width, fwd_d128_sm103.cu) take every product of queries and keys and every
// exponential twice.  One map to a CTA leaves 256 columns for two S in turn, so
// that S of the next tile is made while this one's softmax and product run, and
// is an ordinary softmax attention whose tensor work (6 d^2 multiply-adds a
// row and key tile of both maps, 2 of them for S) hides its exponentials: half
// as many per product as at d = 64.  Values are read by both CTAs of the pair,
// from L2 the second time.
//
// At an item's end CTA m has o_m = (1 or -lambda) O_m / l_m.  Each hands the other
// half of its columns (128 of 256, fp32, through L2: shared memory is full),
// adds what it gets, and finishes those 128 columns; the norm's row sums cross
// through distributed shared memory.  Eight warps of their own do this while the
// softmax warps are at the next item.
//
// Bound: the tensor cores (busy 64 % of a call with seven items to a pair) and the
// items' ends.  2048 tokens behind 16384, 16 heads over 4: 430 to 446 us, 1155 to
// 1199 TFLOP/s of the 8 d flop a pair, 1730 to 1800 of the 12 d executed.  e4m3
// keys, six sequences of 2000 to 5003 of them with 513 to 1025 new tokens: 237 us.
//
// Tensor memory: S / P at 0 and 128 in turn, O at 256; shared memory: Q 32 KB, two
// tiles of K (32 KB each) and two of V (64 KB each).
#include <cuda.h>

#include <atomic>
#include <cmath>
#include <cstddef>

#include "ragged_fwd.cuh"
#include "softmax_tile.cuh"

namespace diffattn {
namespace {

constexpr int HD = 128, DV = 256;
constexpr int kSlots = 2;
constexpr int kThreads = 640, kSoftmax = 256, kSoftmaxWarps = kSoftmax / 32;
constexpr int kFinish = 256, kFinishWarps = kFinish / 32;
constexpr int kKeyWarp = 0, kMmaWarp = 1, kValueWarp = 2, kQueryWarp = 3, kSoftmaxWarp = 4,
              kFinishWarp = 12;
constexpr uint32_t kRegsLaunch = 96, kRegsCtrl = 64, kRegsRest = 104;
static_assert(128 * kRegsCtrl + (kSoftmax + kFinish) * kRegsRest <= kThreads * kRegsLaunch,
              "register split");

constexpr uint32_t kBox = kTile * 128;  // 64 bf16 or 128 e4m3 columns of a tile
constexpr uint32_t kQ = 0, kKeys = 2 * kBox, kValues = kKeys + kSlots * 2 * kBox;
constexpr uint32_t kCtrlAt = kValues + kSlots * 4 * kBox;
constexpr uint32_t kTmO = 256;

struct Ctrl {
  uint64_t k_full[kSlots], k_empty[kSlots], v_full[kSlots], v_empty[kSlots];
  uint64_t q_full, q_empty, s_full[2], p_ready[2], pv_done, o_done, o_free, drain;
  uint64_t l_full[2];  // by segment with keys: the softmax may be done with the next one's as well
  uint64_t peer[2];  // the other CTA's hand-overs, in turn
  uint64_t seg_full[kSegRing], seg_empty[kSegRing];
  Segment seg[kSegRing];
  int32_t bad[kSegRing], unclean[kSegRing];
  uint32_t tmem;
  int abort;
  alignas(8) uint8_t column[2][DV];
  alignas(8) float xch[2][kTile];  // the other CTA's row sums, in turn
  float inv[2][kTile];             // 1 / l of the rows, by segment with keys
};
static_assert(sizeof(ShareState) <= 2 * kTile * sizeof(float), "the set-up's state lies in xch");
constexpr uint32_t kSmem = kCtrlAt + sizeof(Ctrl);
static_assert(kSmem <= 232448, "shared memory");

__device__ __forceinline__ uint32_t peer_address(const void *p, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void peer_store(uint32_t a, float x) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(x) : "memory");
}
__device__ __forceinline__ void peer_arrive(uint32_t bar) {
  asm volatile("fence.acq_rel.cluster;\n\t"
               "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}
// mbar_wait_warp for a barrier that the other CTA arrives on.
__device__ __forceinline__ bool peer_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
  const uint32_t a = smem_u32(bar);
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(a), "r"(parity)
        : "memory");
    if (__all_sync(0xffffffffu, done)) return true;
    if ((it & 63u) == 0) {
      bool stop = *abort != 0;
      if (globaltimer_ns() - t0 > kWaitNs) {
        *abort = 1;
        stop = true;
      }
      if (__any_sync(0xffffffffu, stop)) return false;
    }
  }
}
__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// What a row's O of the pieces before counts times, then that of the piece itself ([2][row], behind
// what the pairs hand over): from a softmax warp to a finishing one, in turn.
__device__ __forceinline__ float *factors_at(const RaggedParams &p, uint32_t turn) {
  return p.swap + (2ll * p.shares * 2 * 128 + (blockIdx.x * 2ll + turn) * 2) * kTile;
}

// A row's reference and sum of a piece with those of the pieces before, which are in the part; leaves
// what either's O counts times.  (These three are functions of their own, so that the short items' code
// keeps its registers.)
__device__ __noinline__ float2 merge_sums(const RaggedParams &p, const Segment &g, int map, int r,
                                          uint32_t turn, float m, float l) {
  const float *part = p.part + (g.slot * 2ll + map) * part_floats(DV) + r;
  const Merge x = merge_states(part[DV * kTile], part[(DV + 1) * kTile], m, l);
  float *factors = factors_at(p, turn) + r;
  factors[0] = x.before;
  factors[kTile] = x.now;
  return make_float2(x.m, x.l);
}

// A piece's O in tensor memory with that of the pieces before, which is in the part.  (Each thread
// reads what it has written itself.)
__device__ __noinline__ void merge_rows(const RaggedParams &p, const Segment &g, int map, int r, int key0,
                                        uint32_t turn, uint32_t t_o) {
  const float *part = p.part + (g.slot * 2ll + map) * part_floats(DV) + r;
  const float *factors = factors_at(p, turn) + r;
  const bool mine = r < g.tokens * p.group;
  const float before = mine ? factors[0] : 0.f, now = mine ? factors[kTile] : 1.f;
#pragma unroll 1
  for (int c0 = 0; c0 < 4; ++c0) {
    const int col = 128 * (c0 >> 1) + 32 * (c0 & 1);
    uint32_t o[32];
    tmem_ld16_x32(t_o + col, o);
    if (mine) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        o[i] = __float_as_uint(__uint_as_float(o[i]) * now + part[(key0 + col + i) * kTile] * before);
    }
    __syncwarp();
    tmem_st16_x32(t_o + col, o);
  }
  tmem_st_wait();
}

// Hands over what this CTA's finishing threads have written for the other, and takes what that one has:
// the `handed`-th time.
__device__ __noinline__ bool exchange_pair(Ctrl *ctrl, uint32_t peer_bar, uint32_t handed) {
  named_barrier_sync(1, kFinish);
  if (threadIdx.x == 32 * kFinishWarp) peer_arrive(peer_bar + 8 * (handed & 1));
  return peer_wait(&ctrl->peer[handed & 1], (handed >> 1) & 1, &ctrl->abort);
}

template <bool kFp8>
__global__ void __launch_bounds__(kThreads, 1)
    diffragged_fwd_d128_kernel(const __grid_constant__ CUtensorMap tm_q1,
                               const __grid_constant__ CUtensorMap tm_q2,
                               const __grid_constant__ CUtensorMap tm_k1,
                               const __grid_constant__ CUtensorMap tm_k2,
                               const __grid_constant__ CUtensorMap tm_v,
                               const __grid_constant__ RaggedParams p) {
  // (No room for slack: the declared alignment is what the swizzled tiles need.)
  extern __shared__ __align__(1024) uint8_t smem[];
  Ctrl *ctrl = reinterpret_cast<Ctrl *>(smem + kCtrlAt);
  volatile int *abort_flag = &ctrl->abort;
  constexpr int kKeyBoxes = kFp8 ? 1 : 2;  // of 128 bytes a row
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int32_t share = blockIdx.x >> 1;
  const int map = blockIdx.x & 1;
  const CUtensorMap *tm_q = map ? &tm_q2 : &tm_q1, *tm_k = map ? &tm_k2 : &tm_k1;

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
      mbar_init(&ctrl->p_ready[k], kSoftmaxWarps);
      mbar_init(&ctrl->peer[k], 1);
      mbar_init(&ctrl->l_full[k], kSoftmaxWarps);
    }
    mbar_init(&ctrl->pv_done, 1);
    mbar_init(&ctrl->o_done, 1);
    mbar_init(&ctrl->o_free, kFinishWarps);
    mbar_init(&ctrl->drain, 1);
    for (int s = 0; s < kSegRing; ++s) {
      mbar_init(&ctrl->seg_full[s], 1);
      mbar_init(&ctrl->seg_empty[s], 3 + kSoftmaxWarps + kFinishWarps);
    }
    ctrl->abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(tm_q);
    tma_prefetch_desc(tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&ctrl->tmem, 512);
    tmem_relinquish();
  }
  {  // rows past whole tokens are never loaded
    const uint32_t used = p.tokens * p.group * 128;
    for (uint32_t x = used + 16 * threadIdx.x; x < kBox; x += 16 * kThreads)
      for (int k = 0; k < kKeyBoxes; ++k)
        *reinterpret_cast<uint4 *>(smem + kQ + k * kBox + x) = make_uint4(0, 0, 0, 0);
    if (used < kBox) fence_async_proxy();
  }
  cluster_barrier();  // both CTAs' barriers are set before either arrives on the other's
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

  // (The register budget of each side's code goes by the branch that it stands in.)
  if (warp < kSoftmaxWarp) {
    setmaxnreg_dec<kRegsCtrl>();
    if (warp == kKeyWarp) {
      // --------------------------------------------------------------- keys, and the segments
      const int box = lane % kKeyBoxes, piece = lane / kKeyBoxes, row0 = piece * p.piece_rows;
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
      // rows: their shares then begin at its first keys together, and read them from L2.  (Measured
      // at d = 64, see ragged_fwd_d64.cu; here it only keeps the two alike.)
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
            if (__any_sync(0xffffffffu, bad) && lane == 0) {
              ctrl->bad[r] = 1;
              report_bad_page(p.status);
            }
            if (have && dbg_ok(row0 + p.piece_rows <= kTile, p.status, 120))
              tma_load_4d(smem + kKeys + s * 2 * kBox + box * kBox + row0 * 128, tm_k,
                          &ctrl->k_full[s], 64 * box, p.by_page.mod(key), g.hk, bad ? 0 : page);
            const int pieces = __popc(__ballot_sync(0xffffffffu, have));
            if (lane == 0) mbar_arrive_expect_tx(&ctrl->k_full[s], pieces * p.piece_rows * 128);
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
        if (p.joins != nullptr && map == 0) p.joins[share] = join;
        ring.drain(ctrl->k_full);
      }
      __syncwarp();
    } else if (warp == kValueWarp) {
      // --------------------------------------------------------------- values
      const int box = lane & 3, piece = lane >> 2, row0 = piece * p.piece_rows;
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
          if (have && dbg_ok(row0 + p.piece_rows <= kTile, p.status, 121))
            tma_load_4d(smem + kValues + s * 4 * kBox + box * kBox + row0 * 128, &tm_v,
                        &ctrl->v_full[s], 64 * box, p.by_page.mod(key), g.hk, bad ? 0 : page);
          const int pieces = __popc(__ballot_sync(0xffffffffu, have));
          if (lane == 0) mbar_arrive_expect_tx(&ctrl->v_full[s], pieces * p.piece_rows * 128);
          ++ring.n;
        }
      }
      if (lane == 0) ring.drain(ctrl->v_full);
      __syncwarp();
    } else if (warp == kQueryWarp) {
      // --------------------------------------------------------------- queries
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
            dbg_ok(g->row >= 0 && g->row + g->tokens <= p.N, p.status, 122);
            mbar_arrive_expect_tx(&ctrl->q_full, kKeyBoxes * p.tokens * p.group * 128);
            for (int k = 0; k < kKeyBoxes; ++k)
              tma_load_3d(smem + kQ + k * kBox, tm_q, &ctrl->q_full, 64 * k, g->hk * p.group,
                          g->row);
          }
          ++filled;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->seg_empty[r]);
      }
      if (lane == 0 && filled > 0) drain_wait(&ctrl->q_full, (filled - 1) & 1);
      __syncwarp();
    } else {
      // --------------------------------------------------------------- products
      constexpr uint32_t kIdescQK = idesc_bf16_f32(kTile, kTile, false);
      constexpr uint32_t kIdescQK8 = idesc_e4m3_f32(kTile, kTile);
      constexpr uint32_t kIdescPV = idesc_bf16_f32(kTile, DV, true);
      const uint64_t q64 = smem_desc_sw128(smem_u32(smem + kQ), 16, 1024);
      const uint64_t k64 = smem_desc_sw128(smem_u32(smem + kKeys), 16, 1024);
      const uint32_t dhi = static_cast<uint32_t>(q64 >> 32);
      const uint32_t dq = static_cast<uint32_t>(q64), dk = static_cast<uint32_t>(k64);
      const uint32_t dv =
          static_cast<uint32_t>(smem_desc_sw128(smem_u32(smem + kValues), kBox, 1024));
      auto qk = [&](uint32_t c) {  // S of key tile c
        const uint32_t s = c % kSlots, to = tmem + 128 * (c & 1);
        if (!dbg_ok(tmem_cols_ok(to, kTile, tmem, 512), p.status, 123)) return;
        if (kFp8) {
          const uint64_t b = k64 + (s * 2 * kBox >> 4);
#pragma unroll
          for (int kk = 0; kk < HD / 32; ++kk)
            umma_e4m3_ss_warp(to, q64 + 2 * kk, b + 2 * kk, kIdescQK8, kk > 0);
        } else {
          const uint32_t b = dk + (s * 2 * kBox >> 4);
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * kBox + 32 * (kk & 3)) >> 4;
            umma_bf16_ss_lo_warp(to, dq + off, b + off, dhi, kIdescQK, kk > 0);
          }
        }
      };
      auto pv = [&](uint32_t c, bool accumulate) {
        const uint32_t b = dv + ((c % kSlots) * 4 * kBox >> 4), from = tmem + 128 * (c & 1);
        if (!dbg_ok(tmem_cols_ok(tmem + kTmO, DV, tmem, 512), p.status, 124)) return;
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          umma_bf16_ts_lo_warp(tmem + kTmO, from + kk * 8 + (kk >= 4 ? 32 : 0), b + 128 * kk, dhi,
                               kIdescPV, (accumulate || kk > 0) ? 1u : 0u);
      };
      auto wait = [&](uint64_t *bar, uint32_t parity) {
        return mbar_wait_warp(bar, parity, abort_flag, kWaitNs);
      };
      bool ok = true;
      uint32_t c = 0, filled = 0;
      for (uint32_t n = 0; ok; ++n) {
        const int r = n % kSegRing;
        if (!(ok = wait(&ctrl->seg_full[r], (n / kSegRing) & 1))) break;
        const int32_t flags = ctrl->seg[r].flags, tiles = ctrl->seg[r].tiles;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->seg_empty[r]);
        if (flags & kStop) break;
        if (flags & kEmpty) continue;
        if (!(ok = wait(&ctrl->q_full, filled & 1))) break;
        // S one tile ahead of P V, into the S that P V before last has read.
        const auto next_s = [&](int32_t t) {
          const uint32_t cc = c + t;
          if (!wait(&ctrl->k_full[cc % kSlots], (cc / kSlots) & 1)) return false;
          tc_fence_after_sync();
          qk(cc);
          umma_commit_warp(&ctrl->s_full[cc & 1]);
          umma_commit_warp(&ctrl->k_empty[cc % kSlots]);
          if (t == tiles - 1) umma_commit_warp(&ctrl->q_empty);
          return true;
        };
        if (!(ok = next_s(0))) break;
        for (int32_t t = 0; t < tiles; ++t) {
          const uint32_t cc = c + t;
          if (t + 1 < tiles && !(ok = next_s(t + 1))) break;
          if (!(ok = wait(&ctrl->v_full[cc % kSlots], (cc / kSlots) & 1))) break;
          if (!(ok = wait(&ctrl->p_ready[cc & 1], (cc >> 1) & 1))) break;
          if (t == 0 && filled > 0 && !(ok = wait(&ctrl->o_free, (filled - 1) & 1))) break;
          tc_fence_after_sync();
          pv(cc, t > 0);
          umma_commit_warp(&ctrl->v_empty[cc % kSlots]);
          umma_commit_warp(&ctrl->pv_done);
        }
        if (!ok) break;
        umma_commit_warp(&ctrl->o_done);
        c += tiles;
        ++filled;
      }
      umma_commit_warp(&ctrl->drain);
      drain_wait(&ctrl->drain, 0);
      __syncwarp();
    }
  } else {
    setmaxnreg_inc<kRegsRest>();
    if (warp < kFinishWarp) {
      // --------------------------------------------------------------- softmax
      const int sw = warp - kSoftmaxWarp;
      const int hl = lane & 15, hc = lane >> 4;
      const int warp_row = (warp & 3) * 32 + (sw >> 2) * 16, r = warp_row + hl;
      const int key0 = 64 * hc;
      const uint32_t lane_addr = static_cast<uint32_t>(warp_row) << 16;
      const uint32_t t_o = tmem + lane_addr + kTmO;
      const float sl2 = p.scale_log2;
      const int32_t token = p.by_group.div(r);
      uint32_t c = 0, filled = 0;
      for (uint32_t n = 0;; ++n) {
        const int ring = n % kSegRing;
        if (!mbar_wait_warp(&ctrl->seg_full[ring], (n / kSegRing) & 1, abort_flag, kWaitNs)) break;
        const Segment *g = &ctrl->seg[ring];
        const int32_t flags = g->flags;
        if (flags & kStop) break;
        if (!(flags & kEmpty)) {
          const int32_t tiles = g->tiles, rows = g->tokens * p.group;
          const bool live = warp_row < rows;
          const int32_t seen = seen_by_all(p, *g), len = g->len;
          const int32_t first_key = g->tile0 * kTile;
          const int32_t lim0 =
              (p.causal ? min(max(g->first + token, 0), g->len - 1) : g->len - 1) - g->tile0 * kTile;
          float m_run = -INFINITY, l_run = 0.f;
          bool ok = true;
          for (int32_t t = 0; t < tiles; ++t, ++c) {
            const uint32_t t_s = tmem + lane_addr + 128 * (c & 1);
            ok = mbar_wait_warp(&ctrl->s_full[c & 1], (c >> 1) & 1, abort_flag, kWaitNs);
            if (!ok) break;
            if (live) {
              tc_fence_after_sync();
              const int lim = lim0 - t * kTile;
              const bool masked = __any_sync(0xffffffffu, lim < kTile - 1);
              if (!dbg_ok_warp(tmem_range_ok(t_s, kTile, tmem, 512, warp, 16) &&
                                   tmem_range_ok(t_o, DV, tmem, 512, warp, 16),
                               p.status, 125)) {
                ok = false;
                break;
              }
              uint32_t pk[kTile / 4];
              float tile_sum = 0.f;
              if (t == 0) {
                tile_sum = softmax_half_first(t_s, key0, sl2, lim, masked, m_run, pk);
              } else {
                tile_sum = masked ? softmax_half_exp<true, true>(t_s, key0, m_run, sl2, lim, pk)
                                  : softmax_half_exp<false, true>(t_s, key0, m_run, sl2, lim, pk);
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
                    // (S of this tile was made behind the product before last; the last one's end is
                    // awaited here.)
                    if (!(ok = mbar_wait_warp(&ctrl->pv_done, (c - 1) & 1, abort_flag, kWaitNs))) break;
                    tc_fence_after_sync();
#pragma unroll 1
                    for (int c0 = 0; c0 < 4; ++c0) {
                      const uint32_t at = t_o + 128 * (c0 >> 1) + 32 * (c0 & 1);
                      uint32_t o[32];
                      tmem_ld16_x32(at, o);
#pragma unroll
                      for (int i = 0; i < 32; i += 2) {
                        const float2 v = __fmul2_rn(
                            make_float2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])),
                            make_float2(alpha, alpha));
                        o[i] = __float_as_uint(v.x);
                        o[i + 1] = __float_as_uint(v.y);
                      }
                      tmem_st16_x32(at, o);
                    }
                  }
                  l_run *= alpha;
                  const float m_use = m_run == -INFINITY ? 0.f : m_run;
                  tile_sum = masked ? softmax_half_exp<true, true>(t_s, key0, m_use, sl2, lim, pk)
                                    : softmax_half_exp<false, true>(t_s, key0, m_use, sl2, lim, pk);
                }
              }
              l_run += tile_sum;
              tmem_st16_x32(t_s, pk);
              tmem_st_wait();
              tc_fence_before_sync();
            }
            if (first_key + (t + 1) * kTile - 1 > seen) {
              uint8_t *values = smem + kValues + (c % kSlots) * 4 * kBox;
              const int32_t key = first_key + t * kTile;
              if (!(ok = mbar_wait_warp(&ctrl->v_full[c % kSlots], (c / kSlots) & 1, abort_flag, kWaitNs)))
                break;
              if (fix_rows<4>(values, 16 * sw, key, seen, len)) {
                uint32_t *columns = reinterpret_cast<uint32_t *>(ctrl->column[n & 1]);
                if (!(ok = open_columns(&ctrl->unclean[ring], columns, DV / 4,
                                        &ctrl->seg_empty[(n - 2) % kSegRing], ((n - 2) / kSegRing) & 1,
                                        n >= 2, abort_flag)))
                  break;
                fix_each<4>(values, 16 * sw, key, seen, len, columns);
              }
              fence_async_proxy();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctrl->p_ready[c & 1]);
          }
          if (!ok) break;
          float l_row = l_run + __shfl_xor_sync(0xffffffffu, l_run, 16);
          if (hc == 0) {
            if ((flags & kAgain) && r < rows) {
              const float2 both = merge_sums(p, *g, map, r, filled & 1, m_run, l_row);
              m_run = both.x;
              l_row = both.y;
            }
            // (The row's last sum but one has been read: the first product behind it awaited that.)
            ctrl->inv[filled & 1][r] = 1.f / l_row;
            if (!(flags & kDirect) && r < rows) {
              float *part = p.part + (g->slot * 2ll + map) * part_floats(DV) + r;
              part[DV * kTile] = m_run;
              part[(DV + 1) * kTile] = ctrl->bad[ring] ? NAN : l_row;
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctrl->l_full[filled & 1]);
          ++filled;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->seg_empty[ring]);
      }
    } else {
      // --------------------------------------------------------------- finished items
      const int fw = warp - kFinishWarp;
      const int hl = lane & 15, hc = lane >> 4;
      const int warp_row = (warp & 3) * 32 + (fw >> 2) * 16, r = warp_row + hl;
      const int key0 = 64 * hc;
      const uint32_t t_o = tmem + (static_cast<uint32_t>(warp_row) << 16) + kTmO;
      const int32_t token = p.by_group.div(r), head = r - token * p.group;
      const uint32_t peer_xch = peer_address(&ctrl->xch[0][0], map ^ 1);
      const uint32_t peer_bar = peer_address(&ctrl->peer[0], map ^ 1);
      uint32_t filled = 0, direct = 0, handed = 0;
      // Hands over what this CTA's threads have written for the other, and takes what that one has.
      const auto exchange = [&]() {
        named_barrier_sync(1, kFinish);
        if (threadIdx.x == 32 * kFinishWarp) peer_arrive(peer_bar + 8 * (handed & 1));
        const bool ok = peer_wait(&ctrl->peer[handed & 1], (handed >> 1) & 1, abort_flag);
        ++handed;
        return ok;
      };
      for (uint32_t n = 0;; ++n) {
        const int ring = n % kSegRing;
        // (Every way out of the loop is agreed on: a segment may come after one warp has given up.)
        const bool got =
            mbar_wait_warp(&ctrl->seg_full[ring], (n / kSegRing) & 1, abort_flag, kWaitNs);
        const Segment *g = &ctrl->seg[ring];
        const int32_t flags = got ? g->flags : kStop;
        if (flags & kStop) {
          named_barrier_or(1, kFinish, true);
          break;
        }
        const int32_t rows = g->tokens * p.group;
        const int32_t pos = g->first + token;
        const int32_t h = g->hk * p.group + head;
        const bool live = warp_row < rows;
        float coef = r < rows ? (map ? -p.lambda[h] : 1.f) : 0.f;
        if (!(flags & kEmpty)) {
          bool ok = mbar_wait_warp(&ctrl->l_full[filled & 1], (filled >> 1) & 1, abort_flag, kWaitNs);
          if (ok) ok = mbar_wait_warp(&ctrl->o_done, filled & 1, abort_flag, kWaitNs);
          if (named_barrier_or(1, kFinish, !ok || *abort_flag != 0)) break;
          tc_fence_after_sync();
          coef *= ctrl->bad[ring] ? NAN : ctrl->inv[filled & 1][r];
          if (flags & kAgain) {
            if (live) merge_rows(p, *g, map, r, key0, filled & 1, t_o);
            // (The CTAs of a pair meet at each piece at least: neither falls behind by more.)
            if (named_barrier_or(1, kFinish, !exchange_pair(ctrl, peer_bar, handed++))) break;
          }
          ++filled;
          if (!(flags & kDirect)) {
            // A part: O column by column.
            float *part = p.part + (g->slot * 2ll + map) * part_floats(DV);
            const bool unclean = ctrl->unclean[ring] == 2;
            const int32_t far = pos - seen_by_all(p, *g);
            const bool mine = r < rows;
#pragma unroll 1
            for (int c0 = 0; c0 < 4; ++c0) {
              const int col = 128 * (c0 >> 1) + 32 * (c0 & 1);
              uint32_t v[32];
              tmem_ld16_x32(t_o + col, v);
              if (mine) {
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  float x = __uint_as_float(v[i]);
                  if (unclean && ctrl->column[n & 1][key0 + col + i] <= far) x = NAN;
                  part[(key0 + col + i) * kTile + r] = x;
                }
              }
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

        // This thread's columns: 128 map + 64 hc .., of its row.
        const int col0 = 128 * map + key0;
        float o[64];
        if (flags & kEmpty) {
          const float x = flags & kBadLen ? NAN : 0.f;
#pragma unroll
          for (int i = 0; i < 64; ++i) o[i] = x;
        } else {
          // [CTA][turn][column of the other's half][row]
          float *give = p.swap + ((blockIdx.x * 2ll + (direct & 1)) * 128 + key0) * kTile + r;
          const float *take =
              p.swap + (((blockIdx.x ^ 1) * 2ll + (direct & 1)) * 128 + key0) * kTile + r;
          ++direct;
#pragma unroll
          for (int c0 = 0; c0 < 64; c0 += 32) {
            uint32_t v[32];
            tmem_ld16_x32(t_o + 128 * (map ^ 1) + c0, v);
            if (live)
#pragma unroll
              for (int i = 0; i < 32; ++i) give[(c0 + i) * kTile] = __uint_as_float(v[i]) * coef;
          }
#pragma unroll
          for (int c0 = 0; c0 < 64; c0 += 32) {
            uint32_t v[32];
            tmem_ld16_x32(t_o + 128 * map + c0, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[c0 + i] = __uint_as_float(v[i]) * coef;
          }
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctrl->o_free);
          bool fine = exchange();
          if (live) {
            // Sixteen on their way at a time: there are no registers for more beside o.
#pragma unroll
            for (int i0 = 0; i0 < 64; i0 += 16) {
              float x[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) x[i] = __ldcg(take + (i0 + i) * kTile);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i0 + i] += x[i];
              asm volatile("" ::: "memory");
            }
          }
          if (ctrl->unclean[ring] == 2) {
            const int32_t far = pos - seen_by_all(p, *g);
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (ctrl->column[n & 1][col0 + i] <= far) o[i] = NAN;
          }
          if (p.headnorm) {
            // The sum over the row of both CTAs' threads.
            const auto row_sum = [&](float x) {
              x += __shfl_xor_sync(0xffffffffu, x, 16);
              const uint32_t turn = handed & 1;
              if (hc == 0) peer_store(peer_xch + 4 * (turn * kTile + r), x);
              fine &= exchange();
              return x + ctrl->xch[turn][r];
            };
            if (p.headnorm == 2) {
              float sm = 0.f;
#pragma unroll
              for (int i = 0; i < 64; ++i) sm += o[i];
              const float mu = row_sum(sm) * (1.f / DV);
#pragma unroll
              for (int i = 0; i < 64; ++i) o[i] -= mu;
            }
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 64; ++i) ss = fmaf(o[i], o[i], ss);
            const float rr = rsqrtf(row_sum(ss) * (1.f / DV) + p.eps) * p.out_scale;
            if (p.norm_w != nullptr && r < rows) {
              const float4 *w4 = reinterpret_cast<const float4 *>(p.norm_w + h * DV + col0);
#pragma unroll
              for (int i = 0; i < 64; i += 4) {
                const float4 w = w4[i / 4];
                o[i] *= rr * w.x;
                o[i + 1] *= rr * w.y;
                o[i + 2] *= rr * w.z;
                o[i + 3] *= rr * w.w;
                if (i % 16 == 12) asm volatile("" ::: "memory");
              }
            } else {
#pragma unroll
              for (int i = 0; i < 64; ++i) o[i] *= rr;
            }
          }
          if (pos < 0) {
#pragma unroll
            for (int i = 0; i < 64; ++i) o[i] = 0.f;
          }
          if (named_barrier_or(1, kFinish, !fine)) break;
        }
        if (live) {
          uint4 pkt[8];
#pragma unroll
          for (int v = 0; v < 8; ++v)
            pkt[v] = make_uint4(
                pack_bf16x2(o[8 * v], o[8 * v + 1]), pack_bf16x2(o[8 * v + 2], o[8 * v + 3]),
                pack_bf16x2(o[8 * v + 4], o[8 * v + 5]), pack_bf16x2(o[8 * v + 6], o[8 * v + 7]));
          transpose8_chunks(pkt, lane);
          const int32_t r0 = r - (lane & 7);
          __nv_bfloat16 *out =
              p.out + g->row * p.out_n + g->hk * p.group * p.out_h + col0 + 8 * (lane & 7);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int32_t i = p.by_group.div(r0 + j);
            if (r0 + j < rows && dbg_ok(g->row + i < p.N, p.status, 126))
              *reinterpret_cast<uint4 *>(out + i * p.out_n + (r0 + j - i * p.group) * p.out_h) = pkt[j];
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctrl->seg_empty[ring]);
      }
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
  cluster_barrier();  // neither leaves while the other may still write to it
}

}  // namespace

size_t ragged_swap_bytes(int shares) {
  return size_t{2} * shares * 2 * (128 + 2) * kTile * sizeof(float);  // with factors_at
}

diffattn_status launch_ragged_main_d128(const RaggedParams &p, const CUtensorMap (&maps)[5],
                                        bool fp8, cudaStream_t stream) {
  static std::atomic<bool> ready[2][64];
  return fp8 ? launch_ragged_kernel(diffragged_fwd_d128_kernel<true>, ready[1], p, maps, kThreads,
                                    kSmem, 2, stream)
             : launch_ragged_kernel(diffragged_fwd_d128_kernel<false>, ready[0], p, maps, kThreads,
                                    kSmem, 2, stream);
}

}  // namespace diffattn
