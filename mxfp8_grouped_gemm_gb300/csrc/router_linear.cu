// Backward of the router's linear layer for dense logit gradients.
//
// mxg_router_bwd takes the gradients of the k chosen logits of a token; a loss
// on the whole softmax (the balance loss) gives every logit one.  With
// G = dlogits [T][E]:
//   dx        = dx_in + G W_r      (bf16, rounded once)
//   dw_router = G^T x              (fp32, fixed-order sums)
// At most 256 experts make both products thin: reading x and dx_in and writing
// dx (6 bytes an element) bounds them, so they run on the tensor cores beside
// the stream of tiles.
//
// Precision.  x and W_r are bf16 already; an fp32 gradient is cut into three
// bf16 parts of eight significant bits each (g = high + mid + low exactly).
// dx takes high and mid (2^-16 of g, far below its own rounding); dW takes all
// three, each into columns of its own.  The tensor cores cut their running sums
// instead of rounding them (measured: 2e-7 of the result after 16 MMAs, 9e-7
// after 64, 4e-6 after 256), so an accumulator is read out every 256 tokens
// and added up in fp32 registers.
//
// One launch: some CTAs compute dW, the others dx, shared out by bytes moved.
//  dW: a unit is 128 hidden columns x up to 64 experts.  D[h][part, e] =
//      x[t][h]^T G[t][part, e], both operands read across the contraction
//      (MN-major), 64 tokens a stage.  The line of all (unit, token block)
//      is cut into equal pieces, one per CTA; a CTA leaves one partial per unit
//      it touches, numbered unit + CTA (unique: along the line one of the two
//      grows at every seam), and the CTA that brings a unit's count of partials
//      to its end adds them up in order.  No CTA waits for another.
//  dx: 128 tokens x 128 hidden columns a tile, K = 64 experts x 2 parts a step
//      (W_r read across).  G stays while the CTA goes along the tokens'
//      columns.  dx_in comes by TMA into the buffer that the result leaves from.
//
// Measured, both launches (T x H x E, with dx_in): 16384 x 4096 x 8 71 us (5.7
// TB/s: HBM), 8191 x 2048 x 64 28.4 us (3.6 TB/s), 8192 x 2048 x 128 39 us,
// without dx_in 5003 x 1024 x 256 28 us.  7 us are the launches and the split;
// beyond 64 experts the products count (a tile's MMAs take 135 cycles each, a
// block of dW 900), and joining the partials of dW about 7 us.
#include <climits>

#include "api_common.h"
#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace mxg {
namespace {

constexpr int kRlTok = 128;                       // tokens of a dx tile
constexpr int kRlStep = 64;                       // tokens of a dW block
constexpr int kRlCols = 128;                      // hidden columns of a unit or tile
constexpr int kRlGroup = 64;                      // most experts of a group
// warp 0 TMA, warp 1 MMA, warp 2 TMA of dx_in, warps 4-19 epilogue (dW: 4-11)
constexpr int kRlThreads = 640;
constexpr int kRlBox = kRlTok * 128;              // 128 rows of 128 bytes
constexpr int kRlSmallBox = kRlStep * 128;        // 64 rows
constexpr int kRlFlush = 4;                       // dW blocks per accumulator (256 tokens)
constexpr int kRlRing = 229376;                   // bytes of all rings
constexpr int kRlG = 2 * kRlBox;                  // dx: high and mid of a group for 128 tokens
constexpr int kRlW = kRlGroup * 256;              // dx: 64 experts x 128 columns of W_r
constexpr int kRlGs = 4;                          // dx: most slots for G
constexpr int kRlIo = 2 * kRlBox;                 // dx: one tile of dx_in / dx
constexpr int kRlIos = 4;                         // most; even: a buffer always serves the same group of epilogue warps
constexpr int kRlMaxStages = 8;
constexpr int kRlSmem = 1024 + kRlRing + 1024;
static_assert(kRlSmem <= 232448, "shared memory budget");
// The two epilogue groups take turns at the tiles.  With an odd number of
// buffers a group would see only every second phase of a buffer's barrier, and
// a parity wait cannot tell the phase it waits for from the one before last.
static_assert(kRlIos % 2 == 0, "each buffer belongs to one epilogue group");

// dx: what shared memory holds.  One group: G of two ranges of tokens, two
// blocks of W_r, four output buffers.  More: G of one range, all groups, two
// output buffers, and as many blocks of W_r as fit.
struct RlDx {
  int gs, ws, ios;
};
__host__ __device__ constexpr RlDx rl_dx_slots(int groups) {
  return groups == 1 ? RlDx{2, 2, 4} : RlDx{groups, (kRlRing - groups * kRlG - 2 * kRlIo) / kRlW, 2};
}
constexpr bool rl_dx_fits(int groups) {
  const RlDx d = rl_dx_slots(groups);
  return d.gs <= kRlGs && d.gs % groups == 0 && d.ws >= 2 && d.ws <= kRlMaxStages && d.ios <= kRlIos && d.ios % 2 == 0 &&
         d.gs * kRlG + d.ws * kRlW + d.ios * kRlIo <= kRlRing;
}
static_assert(rl_dx_fits(1) && rl_dx_fits(2) && rl_dx_fits(3) && rl_dx_fits(4), "dx rings");

struct RlArgs {
  int T, H, E;
  int eg;                                         // experts of a group, padded to 16
  int groups;
  int tb;                                         // dW blocks of tokens
  int tiles_t;                                    // dx tiles of tokens
  int units;                                      // dW: (H / 128) x groups
  int n_dw, n_dx;                                 // CTAs of each kind
  int stages, stage_bytes, g_boxes;               // dW ring
  int has_in;
  float* part;                                    // [units + n_dw][eg][128]
  int32_t* count;                                 // [units], zero: partials left so far
  float* dw;                                      // [E][H]
  int32_t* status;
};

__device__ __forceinline__ int64_t rl_cut(int64_t n, int i, int parts) { return n * i / parts; }

// The CTA of n whose piece of a line of `all` blocks holds block i.
__device__ __forceinline__ int rl_owner(int64_t all, int64_t i, int n) {
  int c = static_cast<int>(i * n / all);          // its piece starts at or before i
  while (rl_cut(all, c + 1, n) <= i) ++c;
  return c;
}

struct RlBars {
  uint64_t *full, *empty, *tfull, *tempty, *io_full, *io_empty, *g_full, *g_empty, *drained, *join;
  volatile int* abort_flag;
  volatile int* never_set;
  volatile int* last;                             // this CTA left a unit's last partial
};

// Joins the eight epilogue warps, bounded like every wait; false: some warp gave up.
__device__ __forceinline__ bool epilogue_sync(const RlBars& B, uint32_t& phase, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(B.join);
  const bool ok = mbar_wait_bounded(B.join, phase, B.abort_flag, kWaitLimitNs);
  phase ^= 1;
  return __all_sync(0xffffffffu, ok);
}

// dW CTA c of n_dw.
__device__ void rl_dw(const RlArgs& P, const CUtensorMap* tmX, const CUtensorMap* tmG, uint8_t* sm, const RlBars& B,
                      uint32_t tmem, int warp, int lane, int c) {
  const int64_t all = static_cast<int64_t>(P.units) * P.tb;
  const int64_t lo = rl_cut(all, c, P.n_dw), hi = rl_cut(all, c + 1, P.n_dw);
  const int N = 3 * P.eg;
  auto fail = [&]() {
    report(P.status, MXG_ERR_TIMEOUT);
    *B.abort_flag = 1;
  };
  if (warp == 0) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 0;
      bool aborted = false;
      int u = static_cast<int>(lo / P.tb), tb = static_cast<int>(lo - static_cast<int64_t>(u) * P.tb);
      int ht = u / P.groups, g = u - ht * P.groups;
      for (int64_t i = lo; i < hi; ++i) {
        const int t0 = tb * kRlStep;
        if (!mbar_wait_bounded(&B.empty[stage], phase ^ 1, B.abort_flag, kWaitLimitNs)) {
          fail();
          aborted = true;
          break;
        }
        uint8_t* s = sm + stage * P.stage_bytes;
        mbar_arrive_expect_tx(&B.full[stage], static_cast<uint32_t>(P.stage_bytes));
        for (int h = 0; h < 2; ++h) tma_load_2d(s + h * kRlSmallBox, tmX, ht * kRlCols + 64 * h, t0, &B.full[stage]);
        for (int h = 0; h < P.g_boxes; ++h)
          tma_load_2d(s + (2 + h) * kRlSmallBox, tmG, g * N + 64 * h, t0, &B.full[stage]);
        if (++tb == P.tb) {
          tb = 0;
          if (++g == P.groups) {
            g = 0;
            ++ht;
          }
        }
        if (++stage == static_cast<uint32_t>(P.stages)) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (aborted) {                              // let copies already in flight land before the CTA exits
        const uint64_t w0 = globaltimer_ns();
        while (globaltimer_ns() - w0 < 1000000ull) __nanosleep(1000);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
      const uint32_t id = idesc_bf16(kRlCols, N) | kIdescAMn | kIdescBMn;
      int64_t i = lo, unit_end = (lo / P.tb + 1) * P.tb;
      bool aborted = false;
      while (i < hi && !aborted) {
        // a run of blocks of one unit that shares an accumulator
        if (i == unit_end) unit_end += P.tb;
        int64_t end = unit_end < hi ? unit_end : hi;
        end = end < i + kRlFlush ? end : i + kRlFlush;
        if (!mbar_wait_bounded(&B.tempty[acc], acc_phase ^ 1, B.abort_flag, kWaitLimitNs)) {
          fail();
          break;
        }
        tc_fence_after();
        bool first = true;
        for (; i < end; ++i) {
          if (!mbar_wait_bounded(&B.full[stage], phase, B.abort_flag, kWaitLimitNs)) {
            fail();
            aborted = true;
            break;
          }
          tc_fence_after();
          const uint32_t s = smem_u32(sm + stage * P.stage_bytes);
          const uint64_t xd = smem_desc(s, kRlSmallBox, 1024, kLayoutSwizzle128B);
          const uint64_t gd = smem_desc(s + 2 * kRlSmallBox, kRlSmallBox, 1024, kLayoutSwizzle128B);
#pragma unroll
          for (int k = 0; k < kRlStep / 16; ++k)   // 16 tokens: 16 rows of 128 bytes
            mma_bf16<1>(tmem + acc * 256, xd + k * (2048 >> 4), gd + k * (2048 >> 4), id, first && k == 0 ? 0u : 1u);
          first = false;
          mma_commit<1>(&B.empty[stage]);
          if (++stage == static_cast<uint32_t>(P.stages)) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (aborted) break;
        mma_commit<1>(&B.tfull[acc]);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      }
      mma_commit<1>(B.drained);
      mbar_wait_bounded(B.drained, 0, B.never_set, kWaitLimitNs);
    }
  } else if (warp >= 4 && warp < 12) {
    // lane = hidden column; warps 4-7 the first half of the group's experts, warps 8-11 the second
    const int q = warp & 3, hf = (warp - 4) >> 2;
    const int half = P.eg / 2;                    // 8, 16, 24 or 32
    const int row = q * 32 + lane;
    float sum[kRlGroup / 2];
#pragma unroll
    for (int e = 0; e < kRlGroup / 2; ++e) sum[e] = 0.f;
    uint32_t acc = 0, acc_phase = 0, join_phase = 0;
    int u = static_cast<int>(lo / P.tb);
    int64_t i = lo, unit_end = static_cast<int64_t>(u + 1) * P.tb;
    while (i < hi) {
      if (i == unit_end) {
        ++u;
        unit_end += P.tb;
      }
      int64_t end = unit_end < hi ? unit_end : hi;
      const int64_t stop = end;
      end = end < i + kRlFlush ? end : i + kRlFlush;
      bool got = mbar_wait_bounded(&B.tfull[acc], acc_phase, B.abort_flag, kWaitLimitNs);
      got = __all_sync(0xffffffffu, got);
      if (!got) {
        if (lane == 0) fail();
        break;
      }
      tc_fence_after();
      const uint32_t ta = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * 256 + hf * half;
#pragma unroll
      for (int j = 0; j < kRlGroup / 16; ++j) {
        if (8 * j < half) {
          uint32_t a[8], b[8], d[8];
          tmem_ld_32x32b_x8(ta + 8 * j, a);
          tmem_ld_32x32b_x8(ta + P.eg + 8 * j, b);
          tmem_ld_32x32b_x8(ta + 2 * P.eg + 8 * j, d);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 8; ++e)
            sum[8 * j + e] += (__uint_as_float(d[e]) + __uint_as_float(b[e])) + __uint_as_float(a[e]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&B.tempty[acc]);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
      if (end == stop) {                          // the unit, or this CTA's share of it, is complete
        const int64_t u0 = unit_end - P.tb;
        const int c0 = rl_owner(all, u0, P.n_dw), c1 = rl_owner(all, unit_end - 1, P.n_dw);
        const int ht = u / P.groups, e0 = (u - ht * P.groups) * P.eg;
        float* part = P.part + (static_cast<int64_t>(u + c) * P.eg + hf * half) * kRlCols + row;
        float* out = P.dw + static_cast<int64_t>(e0 + hf * half) * P.H + ht * kRlCols + row;
#pragma unroll
        for (int e = 0; e < kRlGroup / 2; ++e) {
          if (e < half) {
            if (c0 != c1) part[e * kRlCols] = sum[e];
            else if (e0 + hf * half + e < P.E) out[static_cast<int64_t>(e) * P.H] = sum[e];
          }
          sum[e] = 0.f;
        }
        if (c0 != c1) {
          __threadfence();
          bool ok = epilogue_sync(B, join_phase, lane);
          if (ok && warp == 4 && lane == 0) *B.last = atomicAdd(P.count + u, 1) == c1 - c0;
          ok = ok && epilogue_sync(B, join_phase, lane);
          if (ok && *B.last) {
            __threadfence();
            const float* from = P.part + (static_cast<int64_t>(u) * P.eg + hf * half) * kRlCols + row;
#pragma unroll
            for (int e1 = 0; e1 < kRlGroup / 2; e1 += 16) {
              // two partials requested together, added in order; past the half and the last one the loads
              // repeat a valid value, so that no branch makes them wait for one another
              for (int k = c0; k <= c1; k += 2) {
                float v[2][16];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                  for (int e = 0; e < 16; ++e)
                    v[j][e] = __ldcg(from + (static_cast<int64_t>(min(k + j, c1)) * P.eg + (e1 + e < half ? e1 + e : 0)) * kRlCols);
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                  for (int e = 0; e < 16; ++e) sum[e1 + e] += k + j <= c1 ? v[j][e] : 0.f;
              }
            }
#pragma unroll
            for (int e = 0; e < kRlGroup / 2; ++e) {
              if (e < half && e0 + hf * half + e < P.E) out[static_cast<int64_t>(e) * P.H] = sum[e];
              sum[e] = 0.f;
            }
          }
          ok = ok && epilogue_sync(B, join_phase, lane);         // the flag may be written again
          if (!ok) {
            if (lane == 0) fail();
            break;
          }
        }
      }
      i = end;
    }
  }
}

// dx CTA c of n_dx.
__device__ void rl_dx(const RlArgs& P, const CUtensorMap* tmG, const CUtensorMap* tmW, const CUtensorMap* tmIn,
                      const CUtensorMap* tmOut, uint8_t* sm, const RlBars& B, uint32_t tmem, int warp, int lane,
                      int c) {
  const int hts = P.H / kRlCols;
  const int64_t all = static_cast<int64_t>(P.tiles_t) * hts;
  const int64_t lo = rl_cut(all, c, P.n_dx), hi = rl_cut(all, c + 1, P.n_dx);
  const int t_lo = static_cast<int>(lo / hts) * kRlTok, h_lo = static_cast<int>(lo % hts);
  const RlDx slots = rl_dx_slots(P.groups);
  uint8_t* wr = sm + slots.gs * kRlG;
  uint8_t* io = wr + slots.ws * kRlW;
  const int g_boxes = (2 * P.eg + 63) / 64;       // high and mid of the group
  auto fail = [&]() {
    report(P.status, MXG_ERR_TIMEOUT);
    *B.abort_flag = 1;
  };
  if (warp == 0) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, gs = 0, g_phase = 0;
      bool aborted = false;
      int hi_t = h_lo, t0 = t_lo;
      for (int64_t i = lo; i < hi && !aborted; ++i) {
        const int h0 = hi_t * kRlCols;
        for (int g = 0; g < P.groups; ++g) {
          if (i == lo || hi_t == 0) {             // G serves all tiles of its tokens
            if (!mbar_wait_bounded(&B.g_empty[gs], g_phase ^ 1, B.abort_flag, kWaitLimitNs)) {
              fail();
              aborted = true;
              break;
            }
            mbar_arrive_expect_tx(&B.g_full[gs], static_cast<uint32_t>(g_boxes * kRlBox));
            for (int h = 0; h < g_boxes; ++h)
              tma_load_2d(sm + gs * kRlG + h * kRlBox, tmG, g * 3 * P.eg + 64 * h, t0, &B.g_full[gs]);
            if (++gs == static_cast<uint32_t>(slots.gs)) {
              gs = 0;
              g_phase ^= 1;
            }
          }
          if (!mbar_wait_bounded(&B.empty[stage], phase ^ 1, B.abort_flag, kWaitLimitNs)) {
            fail();
            aborted = true;
            break;
          }
          const int w_box = P.eg * 128;
          mbar_arrive_expect_tx(&B.full[stage], static_cast<uint32_t>(2 * w_box));
          for (int h = 0; h < 2; ++h)
            tma_load_2d(wr + stage * kRlW + h * w_box, tmW, h0 + 64 * h, g * P.eg, &B.full[stage]);
          if (++stage == static_cast<uint32_t>(slots.ws)) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (++hi_t == hts) {
          hi_t = 0;
          t0 += kRlTok;
        }
      }
      if (aborted) {
        const uint64_t w0 = globaltimer_ns();
        while (globaltimer_ns() - w0 < 1000000ull) __nanosleep(1000);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, gs = 0, g_phase = 0, acc = 0, acc_phase = 0;
      const uint32_t id = idesc_bf16(kRlTok, kRlCols) | kIdescBMn;
      bool aborted = false;
      int hi_t = h_lo - 1;
      for (int64_t i = lo; i < hi && !aborted; ++i) {
        if (++hi_t == hts) hi_t = 0;
        if (!mbar_wait_bounded(&B.tempty[acc], acc_phase ^ 1, B.abort_flag, kWaitLimitNs)) {
          fail();
          break;
        }
        uint32_t on = 0;
        for (int g = 0; g < P.groups; ++g) {      // slot gs + g: the slots hold whole sets of groups
          if ((i == lo || hi_t == 0) && !mbar_wait_bounded(&B.g_full[gs + g], g_phase, B.abort_flag, kWaitLimitNs)) {
            fail();
            aborted = true;
            break;
          }
          if (!mbar_wait_bounded(&B.full[stage], phase, B.abort_flag, kWaitLimitNs)) {
            fail();
            aborted = true;
            break;
          }
          tc_fence_after();
          const uint64_t gd = smem_desc(smem_u32(sm + (gs + g) * kRlG), 0, 1024, kLayoutSwizzle128B);
          const uint64_t wd = smem_desc(smem_u32(wr + stage * kRlW), P.eg * 128, 1024, kLayoutSwizzle128B);
          for (int part = 1; part >= 0; --part)
            for (int k = 0; k < P.eg / 16; ++k) {
              const int col = part * P.eg + 16 * k;
              mma_bf16<1>(tmem + acc * 256, gd + (((col >> 6) * kRlBox + (col & 63) * 2) >> 4), wd + k * (2048 >> 4), id, on);
              on = 1;
            }
          mma_commit<1>(&B.empty[stage]);
          if (++stage == static_cast<uint32_t>(slots.ws)) {
            stage = 0;
            phase ^= 1;
          }
          if (hi_t == hts - 1) mma_commit<1>(&B.g_empty[gs + g]);      // the last use of this G
        }
        if (aborted) break;
        if (hi_t == hts - 1) {
          gs += P.groups;
          if (gs == static_cast<uint32_t>(slots.gs)) {
            gs = 0;
            g_phase ^= 1;
          }
        }
        mma_commit<1>(&B.tfull[acc]);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      }
      mma_commit<1>(B.drained);
      mbar_wait_bounded(B.drained, 0, B.never_set, kWaitLimitNs);
    }
  } else if (warp == 2) {
    if (lane == 0 && P.has_in) {                  // dx_in runs ahead of the products by up to four tiles
      uint32_t ib = 0, ib_phase = 0;
      int hi_t = h_lo, t0 = t_lo;
      bool aborted = false;
      for (int64_t i = lo; i < hi; ++i) {
        if (!mbar_wait_bounded(&B.io_empty[ib], ib_phase ^ 1, B.abort_flag, kWaitLimitNs)) {
          fail();
          aborted = true;
          break;
        }
        mbar_arrive_expect_tx(&B.io_full[ib], kRlIo);
        for (int h = 0; h < 2; ++h)
          tma_load_2d(io + ib * kRlIo + h * kRlBox, tmIn, hi_t * kRlCols + 64 * h, t0, &B.io_full[ib]);
        if (++ib == static_cast<uint32_t>(slots.ios)) {
          ib = 0;
          ib_phase ^= 1;
        }
        if (++hi_t == hts) {
          hi_t = 0;
          t0 += kRlTok;
        }
      }
      if (aborted) {
        const uint64_t w0 = globaltimer_ns();
        while (globaltimer_ns() - w0 < 1000000ull) __nanosleep(1000);
      }
    }
  } else if (warp >= 4) {
    // Two groups of eight warps take turns at the tiles (group a: accumulator a).
    // Rows 32 q .., columns 64 hf ..: 32 rows of 128 bytes of an io buffer belong to this warp
    const int q = warp & 3, hf = ((warp - 4) >> 2) & 1, acc = (warp - 4) >> 3;
    uint32_t acc_phase = 0, ib = acc, ib_phase = 0;
    int t0 = t_lo, hi_t = h_lo + acc;
    for (int64_t i = lo + acc; i < hi; i += 2, hi_t += 2) {
      while (hi_t >= hts) {
        hi_t -= hts;
        t0 += kRlTok;
      }
      const int h0 = hi_t * kRlCols;
      uint8_t* buf = io + ib * kRlIo + hf * kRlBox + q * 4096 + lane * 128;
      bool got = mbar_wait_bounded(P.has_in ? &B.io_full[ib] : &B.io_empty[ib], P.has_in ? ib_phase : ib_phase ^ 1,
                                   B.abort_flag, kWaitLimitNs);
      got = mbar_wait_bounded(&B.tfull[acc], acc_phase, B.abort_flag, kWaitLimitNs) && got;
      got = __all_sync(0xffffffffu, got);
      if (!got) {
        if (lane == 0) fail();
        break;
      }
      tc_fence_after();
      const uint32_t ta = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * 256 + hf * 64;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(ta + 32 * half, r);
        tmem_ld_wait();
        if (half == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&B.tempty[acc]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {             // 16-byte piece 4 half + j of the row, 128-byte swizzle
          uint4* p = reinterpret_cast<uint4*>(buf + (((4 * half + j) ^ (lane & 7)) << 4));
          uint32_t v[4] = {0u, 0u, 0u, 0u};
          if (P.has_in) {
            const uint4 d = *p;
            v[0] = d.x;
            v[1] = d.y;
            v[2] = d.z;
            v[3] = d.w;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] = pack_bf16x2(__uint_as_float(v[e] << 16) + __uint_as_float(r[8 * j + 2 * e]),
                               __uint_as_float(v[e] & 0xffff0000u) + __uint_as_float(r[8 * j + 2 * e + 1]));
          *p = make_uint4(v[0], v[1], v[2], v[3]);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (t0 + q * 32 < P.T)
          tma_store_2d(tmOut, io + ib * kRlIo + hf * kRlBox + q * 4096, h0 + 64 * hf, t0 + q * 32);
        bulk_commit_group();
        bulk_wait_group_read<0>();                // the store has left the buffer
        mbar_arrive(&B.io_empty[ib]);
      }
      acc_phase ^= 1;
      ib += 2;
      if (ib >= static_cast<uint32_t>(slots.ios)) {
        ib -= slots.ios;
        ib_phase ^= 1;
      }
    }
    if (lane == 0) bulk_wait_group<0>();          // the stores have completed before the CTA exits
    __syncwarp();
  }
}

__global__ void __launch_bounds__(kRlThreads, 1)
    router_linear_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmGs,
                         const __grid_constant__ CUtensorMap tmG,
                         const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmIn,
                         const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ RlArgs P) {
  extern __shared__ uint8_t raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kRlRing);
  RlBars B;
  B.full = bars;
  B.empty = B.full + kRlMaxStages;
  B.tfull = B.empty + kRlMaxStages;
  B.tempty = B.tfull + 2;
  B.io_full = B.tempty + 2;
  B.io_empty = B.io_full + kRlIos;
  B.g_full = B.io_empty + kRlIos;
  B.g_empty = B.g_full + kRlGs;
  B.drained = B.g_empty + kRlGs;
  B.join = B.drained + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(B.join + 1);
  B.abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  B.never_set = B.abort_flag + 1;
  B.last = B.abort_flag + 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x;
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(c < P.n_dw ? &tmGs : &tmG);
    tma_prefetch_desc(c < P.n_dw ? &tmX : &tmW);
    if (c >= P.n_dw) {
      tma_prefetch_desc(&tmIn);
      tma_prefetch_desc(&tmOut);
    }
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kRlMaxStages; ++s) {
      mbar_init(&B.full[s], 1);
      mbar_init(&B.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&B.tfull[a], 1);
      mbar_init(&B.tempty[a], 8);
    }
    for (int i = 0; i < kRlIos; ++i) {
      mbar_init(&B.io_full[i], 1);
      mbar_init(&B.io_empty[i], 8);
    }
    for (int i = 0; i < kRlGs; ++i) {
      mbar_init(&B.g_full[i], 1);
      mbar_init(&B.g_empty[i], 1);
    }
    mbar_init(B.drained, 1);
    mbar_init(B.join, 8);
    *B.abort_flag = 0;
    *B.never_set = 0;
    fence_barrier_init();
  }
  __syncthreads();
  if (warp == 1) {
    tmem_alloc<1>(tmem_slot, 512);
    tmem_relinquish<1>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  dependency_wait();                              // the parts of G; whatever else the stream did before
  if (c < P.n_dw) rl_dw(P, &tmX, &tmGs, sm, B, tmem, warp, lane, c);
  else rl_dx(P, &tmG, &tmW, &tmIn, &tmOut, sm, B, tmem, warp, lane, c - P.n_dw);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc<1>(tmem, 512);
}

// G in three bf16 parts: parts[t][group][part][eg], zero past E.  Each part
// takes the next eight significant bits (cut, so that the parts add up to g
// exactly and none overflows); an infinity or NaN stays in the first, a NaN with
// the quiet bit set, since the bits that are cut off may be all that it has.
__global__ void __launch_bounds__(256) router_split_kernel(const float* __restrict__ g, int T, int E, int eg,
                                                          int groups, uint16_t* __restrict__ parts, int units,
                                                          int32_t* __restrict__ count) {
  launch_dependents();
  const int quads = groups * eg / 4;              // four experts per thread
  const int tpb = 256 / quads;                    // tokens per block (quads <= 64)
  for (int i = blockIdx.x * 256 + threadIdx.x; i < units; i += gridDim.x * 256) count[i] = 0;
  if (threadIdx.x >= tpb * quads) return;
  const int tl = threadIdx.x / quads, e = 4 * (threadIdx.x - tl * quads);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * tpb + tl;
  if (t >= T) return;
  const float* src = g + t * E + e;
  uint32_t v[4] = {0u, 0u, 0u, 0u};
  if (E % 4 == 0) {
    if (e < E) {
      const float4 f = *reinterpret_cast<const float4*>(src);
      v[0] = __float_as_uint(f.x);
      v[1] = __float_as_uint(f.y);
      v[2] = __float_as_uint(f.z);
      v[3] = __float_as_uint(f.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e + i < E) v[i] = __float_as_uint(src[i]);
  }
  uint32_t p[3][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p[0][i] = v[i] >> 16;
    p[1][i] = p[2][i] = 0u;
    if ((v[i] & 0x7fffffffu) > 0x7f800000u) p[0][i] |= 0x40u;
    if ((v[i] & 0x7f800000u) != 0x7f800000u) {
      const float r = __uint_as_float(v[i]) - __uint_as_float(v[i] & 0xffff0000u);
      const uint32_t b = __float_as_uint(r) & 0xffff0000u;
      p[1][i] = b >> 16;
      p[2][i] = __float_as_uint(r - __uint_as_float(b)) >> 16;
    }
  }
  const int grp = e / eg;
  uint16_t* dst = parts + (t * groups + grp) * 3 * eg + (e - grp * eg);
#pragma unroll
  for (int k = 0; k < 3; ++k)
    *reinterpret_cast<uint2*>(dst + k * eg) = make_uint2(p[k][0] | p[k][1] << 16, p[k][2] | p[k][3] << 16);
}

constexpr int kRlMostDw = 1024;                   // partials are sized for this many dW CTAs at most

// dW CTAs of `sms`: the number that lets both products end together.  In cycles,
// from timings of each product alone and of both with 48 to 112 CTAs for dW: a
// block of tokens takes 500 and its bytes at 100 a cycle, joining a unit's
// partials 14000 (17000 unless the CTAs of one range of tokens go through its
// rows side by side, 3500 where every CTA has whole units), a tile 1000 and 135
// per MMA but at least 1950, its first operands 4000.  The choice is within 7 %
// of the best multiple of eight at eleven shapes; shared out by bytes alone it
// was up to 25 % off (4096 x 4096 x 192: 58.5 us, now 49.6).
int rl_share(int sms, int units, int64_t blocks, int stage_bytes, int64_t tiles, int mmas) {
  const int64_t most = blocks < kRlMostDw ? blocks : kRlMostDw;
  const int64_t block = 500 + stage_bytes / 100, tile = mmas < 8 ? 1950 : 1000 + 135 * mmas;
  int best = 1;
  int64_t best_cost = INT64_MAX;
  for (int n = 1; n <= most && (n < sms || n == 1); n = n < 8 ? 2 * n : n + 8) {
    const int64_t dx = sms > n ? sms - n : 1;
    const int64_t cost_dw = (blocks + n - 1) / n * block + (units % n == 0 ? 3500 : n % units == 0 ? 14000 : 17000);
    const int64_t cost_dx = (tiles + dx - 1) / dx * tile + 4000;
    const int64_t cost = cost_dw > cost_dx ? cost_dw : cost_dx;
    if (cost < best_cost) {
      best_cost = cost;
      best = n;
    }
  }
  return best;
}

struct RlPlan {
  int eg, groups, tb, tiles_t, units;
  int64_t parts, part, count, bytes;
};

RlPlan rl_plan(int T, int H, int E) {
  RlPlan p{};
  p.groups = (E + kRlGroup - 1) / kRlGroup;
  p.eg = p.groups > 1 ? kRlGroup : (E + 15) / 16 * 16;
  p.tb = (T + kRlStep - 1) / kRlStep;
  p.tiles_t = (T + kRlTok - 1) / kRlTok;
  p.units = H / kRlCols * p.groups;
  const int64_t blocks = static_cast<int64_t>(p.units) * p.tb;
  api::Carver w;
  p.parts = w.take(2ll * T * p.groups * p.eg * 3);
  p.part = w.take(4ll * (p.units + (blocks < kRlMostDw ? blocks : kRlMostDw)) * p.eg * kRlCols);
  p.count = w.take(4ll * p.units);
  p.bytes = w.off;
  return p;
}

}  // namespace
}  // namespace mxg

using namespace mxg;

extern "C" size_t mxg_router_linear_bwd_workspace_bytes(int T, int H, int E) {
  if (T <= 0 || H <= 0 || E <= 0 || H % kRlCols != 0 || E > 256) return 0;
  return static_cast<size_t>(rl_plan(T, H, E).bytes);
}

extern "C" int mxg_router_linear_bwd(const uint16_t* x, const uint16_t* w_router, const float* dlogits,
                                     const uint16_t* dx_in, int T, int H, int E, uint16_t* dx, float* dw_router,
                                     void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  if (!x || !w_router || !dlogits || !dx || !dw_router || !workspace || !dev_status) return MXG_ERR_ARG;
  if (T <= 0 || H <= 0 || E <= 0) return MXG_ERR_ARG;
  if (H % kRlCols != 0 || E > 256) return MXG_ERR_SHAPE;
  if (!api::aligned32(x) || !api::aligned32(w_router) || !api::aligned32(dlogits) || !api::aligned32(dx_in) ||
      !api::aligned32(dx) || !api::aligned32(dw_router) || !api::aligned32(workspace))
    return MXG_ERR_ALIGN;
  if (workspace_bytes < mxg_router_linear_bwd_workspace_bytes(T, H, E)) return MXG_ERR_WORKSPACE;
  api::NvtxRange nvtx("mxg.router_linear_bwd");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const RlPlan p = rl_plan(T, H, E);
  uint16_t* parts = api::at<uint16_t>(workspace, p.parts);
  RlArgs a{};
  a.T = T;
  a.H = H;
  a.E = E;
  a.eg = p.eg;
  a.groups = p.groups;
  a.tb = p.tb;
  a.tiles_t = p.tiles_t;
  a.units = p.units;
  a.g_boxes = (3 * p.eg + 63) / 64;
  a.stage_bytes = (2 + a.g_boxes) * kRlSmallBox;
  a.stages = kRlRing / a.stage_bytes < kRlMaxStages ? kRlRing / a.stage_bytes : kRlMaxStages;
  a.has_in = dx_in != nullptr;
  a.part = api::at<float>(workspace, p.part);
  a.status = dev_status;
  a.count = api::at<int32_t>(workspace, p.count);
  a.dw = dw_router;
  const int sms = device_sms();
  const int hts = H / kRlCols;
  const int64_t blocks = static_cast<int64_t>(p.units) * p.tb, tiles = static_cast<int64_t>(p.tiles_t) * hts;
  a.n_dw = rl_share(sms, p.units, blocks, a.stage_bytes, tiles, p.groups * p.eg / 8);
  const int64_t n_dx = sms > a.n_dw ? sms - a.n_dw : 1;
  a.n_dx = static_cast<int>(n_dx < tiles ? n_dx : tiles);

  CUtensorMap mx, mgs, mg, mw, mi, mo;
  if (!tma_map_bf16(&mx, x, H, T, kRlStep) || !tma_map_bf16(&mgs, parts, 3ll * p.groups * p.eg, T, kRlStep) ||
      !tma_map_bf16(&mg, parts, 3ll * p.groups * p.eg, T, kRlTok) ||
      !tma_map_bf16(&mw, w_router, H, E, static_cast<uint32_t>(p.eg)) ||
      !tma_map_bf16(&mi, dx_in ? dx_in : dx, H, T, kRlTok) || !tma_map_bf16(&mo, dx, H, T, 32))
    return MXG_ERR_CUDA;
  const int tpb = 256 / (p.groups * p.eg / 4);
  router_split_kernel<<<static_cast<unsigned>((T + static_cast<int64_t>(tpb) - 1) / tpb), 256, 0, s>>>(
      dlogits, T, E, p.eg, p.groups, parts, p.units, a.count);
  count_launch();
  MXG_TRY(cudaGetLastError());
  MXG_TRY(allow_smem(router_linear_kernel, kRlSmem));
  return api::cuda_status(launch_after(router_linear_kernel, dim3(static_cast<unsigned>(a.n_dw + a.n_dx)),
                                       dim3(kRlThreads), kRlSmem, s, mx, mgs, mg, mw, mi, mo, a));
}
