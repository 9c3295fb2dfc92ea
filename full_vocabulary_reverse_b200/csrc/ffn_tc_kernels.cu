// ffn_tc_kernels.cu -- the gated feed-forward block in bf16 on the tcgen05
// tensor cores.
//
//   g = x Wg^T, u = x Wu^T, a = act(g) u, y = a Wd^T
//   da = dy Wd, dg = da u act'(g), du = da act(g)
//   dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, dWd = dy^T a
//
// ffn_pair_kernel<EPI, ACT>: 256 x 256 tiles on CTA pairs (tcgen05.mma
// cta_group::2), for many rows.  EPI says what a tile goes through:
//   UP     the B tile is 128 rows of Wg (staged by CTA 0) and the same 128 rows
//          of Wu (CTA 1), so one accumulator row holds g in columns 0..127 and
//          u in 128..255: the epilogue rounds a = act(g) u once and stores g
//          and u in fp32 where a backward pass wants them
//   DGATE  da from the accumulator, g and u from memory: a, dg and du, each
//          rounded once as the next products' operands (DGATE_TERMS, for few
//          elements: in two bf16 terms, the second as T rows more; its up to 92
//          bytes of spills at 168 registers do not show beside the launches)
//   GEMM   a list of up to four products in one launch (the backward pass runs
//          dx, dWg, dWu and dWd together, so that one's tail is filled by
//          another's tiles), bf16 results, or fp32 parts of a split K
// Operands are read K-major or MN-major as they lie in memory: nothing is
// transposed or copied.  dx is one product over two segments of K, (dg, Wg)
// and (du, Wu).
//
// ffn_skinny_kernel: for few rows, where reading the weights bounds the time.
// The weights are the M operand (128 rows a tile), the rows of x the N operand;
// every CTA streams an equal share of all (tile, K) steps, whatever tile
// borders lie in it, and leaves fp32 parts that a small kernel joins in a fixed
// order (with the activation between the two halves of the block).  For few
// elements a is two bf16 terms, 2 T rows of the second half.
//
// What bounds them, with T = 8192, H = O = 2048, F = 6144:
//   UP    0.30 ms (1.39 PFLOP/s; the tensor pipe needs 512 SM cycles for a 256 x
//         256 x 64 step), 0.37 with g and u stored beside it (403 MB)
//   DGATE 0.23 ms: 206 GFLOP, but 760 MB through memory, g and u most of it.  In
//         row-major order each lane's 16 bytes lay in a line of their own and the
//         same work took 0.48 ms; hence the blocks of ffn_saved_at
//   GEMM  0.15 ms for y, 0.75 for the four backward products (1.38 PFLOP/s)
// together as much as the power limit leaves (a library product runs at 1.40
// sustained).  ffn_skinny_kernel by HBM where the weights are large: 181 MB
// (H = 4096, F = 11008, 23 rows) in 30 us, and by its start-up, some 5 us, where
// they are small.
#include <cuda_bf16.h>

#include "bounds.cuh"
#include "ffn_act.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace rkl {

RKL_DEFINE_BOUNDS_READER(read_and_clear_bounds_ffn)

namespace {

__device__ int g_ffn_err = 0;

constexpr int kEpiWarps = 8;
constexpr int kPairThreads = 64 + 32 * kEpiWarps;
constexpr int kOperand = 128 * kBK * 2;        // 16 KB: 128 rows (or columns) x 64 deep
constexpr int kHalfStage = 2 * kOperand;       // A and B, 64 deep
constexpr int kPairStage = 2 * kHalfStage;     // 128 deep: eight MMAs a stage keep the issue loop ahead
constexpr int kPairStages = 3;
constexpr int kBox = 4096;                     // one 32-row staging box per epilogue warp
constexpr int kPairTmem = 512;                 // two accumulators of 256 columns
constexpr int kRing = 4;                       // tile-index ring depth
constexpr size_t kPairSmem = 1024 + size_t(kPairStages) * kPairStage + kEpiWarps * kBox + 256;

__device__ __forceinline__ uint8_t* align_1k(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

__device__ __forceinline__ void give_up(volatile int* abort_flag, int bit) {
  atomicOr(&g_ffn_err, bit);
  *abort_flag = 1;
}

// One work item of the launch's list: a tile of a product, over a part of K.
struct Item {
  int q, m, n;       // product; tile row and column
  int lo, hi, part;  // 128-deep steps [lo, hi); index of the part
};

__device__ __forceinline__ Item item_of(const FfnPairArgs& a, int i) {
  Item t;
  t.q = 0;
  while (t.q + 1 < a.n && i >= a.p[t.q + 1].first) ++t.q;
  const FfnPairProduct& p = a.p[t.q];
  const int l = i - p.first;
  const int tiles = p.mt * p.nt;
  t.part = l / tiles;
  const int tile = l - t.part * tiles;
  // The dimension with fewer tiles runs fast: the tiles in flight then share
  // the other operand's slices, which are read from memory once.
  if (p.nt <= p.mt) {
    t.m = tile / p.nt;
    t.n = tile - t.m * p.nt;
  } else {
    t.n = tile / p.mt;
    t.m = tile - t.n * p.mt;
  }
  const int steps = p.segments * p.steps;
  t.lo = static_cast<int>(static_cast<long long>(steps) * t.part / p.parts);
  t.hi = static_cast<int>(static_cast<long long>(steps) * (t.part + 1) / p.parts);
  return t;
}

// What rounding to the packed pair left of two values, rounded too; 0 where the
// rounded value is not finite, which the first term carries alone.
__device__ __forceinline__ uint32_t rest_bf16x2(float v0, float v1, uint32_t rounded) {
  const float h0 = __uint_as_float(rounded << 16), h1 = __uint_as_float(rounded & 0xffff0000u);
  return pack_bf16x2(isfinite(h0) ? v0 - h0 : 0.f, isfinite(h1) ? v1 - h1 : 0.f);
}

// 32 bf16 of each of 32 rows: 16 packed words of a lane's row into one half of
// the warp's staging box (64-byte rows, 64-byte swizzle), then a TMA store.
// The halves alternate, so a store waits only for the one two boxes back.
__device__ __forceinline__ void store_bf16_box(uint8_t* buf, int& flip, int lane, const uint32_t* w,
                                               const CUtensorMap* map, int x, int y, bool inside) {
  uint8_t* half = buf + flip * (kBox / 2);
  flip ^= 1;
  if (lane == 0) bulk_wait_read<1>();
  __syncwarp();
  const uint32_t row = smem_u32(half) + lane * 64;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    st_shared_v4(row + ((i ^ ((lane >> 1) & 3)) << 4), w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (inside && RKL_BOUNDS(x >= 0 && (x & 7) == 0 && y >= 0)) tma_store_2d(map, half, x, y);
    bulk_commit();  // (an empty group where nothing is stored: the count of boxes stays right)
  }
}

// 32 fp32 of each of 32 rows, through the whole box.  A second, empty group
// follows: the next bf16 store leaves one group pending, and this one reads both
// halves.
__device__ __forceinline__ void store_f32_box(uint8_t* buf, int lane, const float* v, const CUtensorMap* map, int x,
                                              int y, bool inside) {
  if (lane == 0) bulk_wait_read<0>();
  __syncwarp();
  const uint32_t row = smem_u32(buf) + lane * 128;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    st_shared_v4(row + ((i ^ (lane & 7)) << 4), __float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                 __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0 && inside && RKL_BOUNDS(x >= 0 && (x & 3) == 0 && y >= 0)) {
    tma_store_2d(map, buf, x, y);
    bulk_commit();
    bulk_commit();
  }
}

}  // namespace

template <int EPI, int ACT>
__global__ void __launch_bounds__(kPairThreads, 1) ffn_pair_kernel(const __grid_constant__ FfnPairArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_1k(smem_raw);
  uint8_t* stg = smem + kPairStages * kPairStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(stg + kEpiWarps * kBox);
  uint64_t* full = bars;
  uint64_t* empty = full + kPairStages;
  uint64_t* acc_full = empty + kPairStages;  // [2]
  uint64_t* acc_empty = acc_full + 2;        // [2]
  uint64_t* tear = acc_empty + 2;
  uint64_t* ring_full = tear + 1;            // [kRing]
  uint64_t* ring_empty = ring_full + kRing;  // [kRing]
  int* ring = reinterpret_cast<int*>(ring_empty + kRing);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(ring + kRing);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kPairStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 2 * kEpiWarps);  // both CTAs' epilogues
    }
    mbar_init(tear, 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&ring_full[i], 1);
      mbar_init(&ring_empty[i], 2 + 2 * kEpiWarps);  // leader's MMA warp, peer's producer, both epilogues
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 2) {
    tmem_alloc_pair(tmem_holder, kPairTmem);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  if (threadIdx.x == 0) let_next_launch_begin();
  wait_for_last_launch();
  // the next launch of this call counts its tiles from zero
  if (a.zero_counter != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *a.zero_counter = 0;

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t full0 = mapa_shared(smem_u32(full), 0);
      int stage = 0;
      uint32_t phase = 0, armed = 0, last_par = 0;
      bool ok = true;
      for (int i = 0; ok; ++i) {
        const int slot = i % kRing;
        const uint32_t rp = (i / kRing) & 1;
        int t;
        if (leader) {
          if (!mbar_wait_cluster(&ring_empty[slot], rp ^ 1, abort_flag)) {
            give_up(abort_flag, ERR_WAIT_AUX);
            break;
          }
          // items of unequal length are claimed, equal ones dealt out
          t = a.counter != nullptr ? atomicAdd(a.counter, 1)
                                   : static_cast<int>(blockIdx.x >> 1) + i * static_cast<int>(gridDim.x >> 1);
          if (t >= a.items) t = -1;
          ring[slot] = t;
          st_cluster_u32(mapa_shared(smem_u32(&ring[slot]), 1), static_cast<uint32_t>(t));
          mbar_arrive(&ring_full[slot]);
          mbar_arrive_cluster(mapa_shared(smem_u32(&ring_full[slot]), 1));
        } else {
          if (!mbar_wait_cluster(&ring_full[slot], rp, abort_flag)) {
            give_up(abort_flag, ERR_WAIT_AUX);
            break;
          }
          t = ring[slot];
          mbar_arrive_cluster(mapa_shared(smem_u32(&ring_empty[slot]), 0));
        }
        if (t < 0) break;
        const Item it = item_of(a, t);
        const FfnPairProduct& p = a.p[it.q];
        const int m0 = it.m * 256 + static_cast<int>(rank) * 128;
        const int n0 = EPI == FFN_UP ? it.n * 128 : it.n * 256 + static_cast<int>(rank) * 128;
        if (!RKL_BOUNDS(t < a.items && it.m < p.mt && it.n < p.nt && it.lo >= 0 && it.hi <= p.segments * p.steps)) {
          give_up(abort_flag, ERR_BOUNDS);
          break;
        }
        for (int s = it.lo; s < it.hi; ++s) {
          if (!mbar_wait_cluster(&empty[stage], phase ^ 1, abort_flag)) {
            give_up(abort_flag, ERR_WAIT_TMA_EMPTY);
            ok = false;
            break;
          }
          const int seg = s >= p.steps ? 1 : 0;
          const int k0 = (s - seg * p.steps) * 2 * kBK;
          const CUtensorMap* ma = &p.a[seg];
          const CUtensorMap* mb = EPI == FFN_UP ? &p.b[rank] : &p.b[seg];
          const uint32_t fb = full0 + stage * 8;
          if (leader) mbar_arrive_expect_tx(&full[stage], 2 * kPairStage);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint8_t* sa = smem + stage * kPairStage + h * kHalfStage;
            uint8_t* sb = sa + kOperand;
            const int k = k0 + h * kBK;
            if (p.a_mn) {
              tma_load_2d_pair(sa, ma, fb, m0, k);
              tma_load_2d_pair(sa + kOperand / 2, ma, fb, m0 + 64, k);
            } else {
              tma_load_2d_pair(sa, ma, fb, k, m0);
            }
            if (p.b_mn) {
              tma_load_2d_pair(sb, mb, fb, n0, k);
              tma_load_2d_pair(sb + kOperand / 2, mb, fb, n0 + 64, k);
            } else {
              tma_load_2d_pair(sb, mb, fb, k, n0);
            }
          }
          armed |= 1u << stage;
          last_par = (last_par & ~(1u << stage)) | (phase << stage);
          if (++stage == kPairStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // The leader's full barriers count both CTAs' loads: drain them there.
      if (leader)
        for (int i = 0; i < kPairStages; ++i)
          if (armed & (1u << i)) {
            volatile int never = 0;
            if (!mbar_wait(&full[i], (last_par >> i) & 1, &never)) atomicOr(&g_ffn_err, ERR_WAIT_TEARDOWN);
          }
    }
  } else if (warp == 1) {
    if (leader) {  // the whole warp runs the loop, one lane issues
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int i = 0; ok; ++i) {
        const int slot = i % kRing;
        if (!__all_sync(0xffffffffu, mbar_wait(&ring_full[slot], (i / kRing) & 1, abort_flag))) {
          give_up(abort_flag, ERR_WAIT_AUX);
          break;
        }
        const int t = __shfl_sync(0xffffffffu, ring[slot], 0);
        if (lane == 0) mbar_arrive(&ring_empty[slot]);
        __syncwarp();
        if (t < 0) break;
        const Item it = item_of(a, t);
        const FfnPairProduct& p = a.p[it.q];
        // The operands' layouts are settled here, once a tile: the issue loop
        // below has no branch.  K-major: a 16-deep slice is 32 B along the
        // swizzled row; MN-major: 16 rows of 128 B, the 64-wide blocks
        // kOperand / 2 apart.
        const uint32_t idesc = idesc_bf16(256, 256, p.a_mn, p.b_mn);
        const uint32_t a_step = p.a_mn ? 2048u >> 4 : 32u >> 4, b_step = p.b_mn ? 2048u >> 4 : 32u >> 4;
        const uint64_t a_desc = sdesc_sw128(smem_u32(smem), p.a_mn ? kOperand / 2 : 16u, 1024);
        const uint64_t b_desc = sdesc_sw128(smem_u32(smem) + kOperand, p.b_mn ? kOperand / 2 : 16u, 1024);
        const int acc = i & 1;
        const uint32_t d = tmem_base + acc * 256;
        if (!__all_sync(0xffffffffu, mbar_wait_cluster(&acc_empty[acc], ((i >> 1) & 1) ^ 1, abort_flag))) {
          give_up(abort_flag, ERR_WAIT_ACC_EMPTY);
          break;
        }
        tc_fence_after();
        uint32_t more = 0;
        for (int s = it.lo; s < it.hi; ++s) {
          ok = __all_sync(0xffffffffu, mbar_wait(&full[stage], phase, abort_flag));
          if (!ok) {
            give_up(abort_flag, ERR_WAIT_TMA_FULL);
            break;
          }
          tc_fence_after();
          const uint32_t at = stage * (kPairStage >> 4);  // of the stage, in the descriptors' 16-byte units
          if (elect_one()) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int k = 0; k < kBK / 16; ++k)
                umma_bf16_pair(d, a_desc + (at + h * (kHalfStage >> 4) + a_step * k),
                               b_desc + (at + h * (kHalfStage >> 4) + b_step * k), idesc, more | h | k);
            umma_commit_pair(&empty[stage], 0x3);
          }
          more = 1;
          if (++stage == kPairStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (ok && elect_one()) umma_commit_pair(&acc_full[acc], 0x3);
      }
      if (elect_one()) {
        umma_commit_pair(tear, 0x1);
        volatile int never = 0;
        if (!mbar_wait(tear, 0, &never)) atomicOr(&g_ffn_err, ERR_WAIT_TEARDOWN);
      }
      __syncwarp();
    }
  } else {
    const int quarter = warp & 3;
    const int half = (warp - 2) >> 2;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t ring_empty0 = mapa_shared(smem_u32(ring_empty), 0);
    const uint32_t acc_empty0 = mapa_shared(smem_u32(acc_empty), 0);
    uint8_t* buf = stg + (warp - 2) * kBox;
    int flip = 0;  // half of the box that the next bf16 store takes
    for (int i = 0;; ++i) {
      const int slot = i % kRing;
      bool ok = mbar_wait_cluster(&ring_full[slot], (i / kRing) & 1, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        if (lane == 0) give_up(abort_flag, ERR_WAIT_AUX);
        break;
      }
      const int t = ring[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(ring_empty0 + slot * 8);
      if (t < 0) break;
      const Item it = item_of(a, t);
      const FfnPairProduct& p = a.p[it.q];
      const int acc = i & 1;
      const int row0 = it.m * 256 + static_cast<int>(rank) * 128 + quarter * 32;
      const bool live = row0 < p.M;  // boxes behind the last row are not stored
      ok = mbar_wait_cluster(&acc_full[acc], (i >> 1) & 1, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        if (lane == 0) give_up(abort_flag, ERR_WAIT_ACC_FULL);
        break;
      }
      tc_fence_after();
      const uint32_t tb = tmem_base + lane_off + acc * 256;
      auto release = [&] {  // the last column of this warp is in registers
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty0 + acc * 8);
      };
      if (EPI == FFN_UP) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int col = half * 64 + c * 32;
          const int x = it.n * 128 + col;
          float g[32], u[32];
          tmem_ld_32x32(tb + col, g);
          tmem_ld_32x32(tb + 128 + col, u);
          tmem_wait_ld();
          if (c == 1) release();
          const bool in = live && x < p.N;
          if (a.saved != nullptr && in) {
            float* sg = a.saved + ffn_saved_at(row0 + lane, x, p.N);
            float* su = sg + ffn_saved_plane(p.M, p.N);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              __stcs(reinterpret_cast<float4*>(sg + e * 128), make_float4(g[4 * e], g[4 * e + 1], g[4 * e + 2], g[4 * e + 3]));
              __stcs(reinterpret_cast<float4*>(su + e * 128), make_float4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]));
            }
          }
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e] = pack_bf16x2(act_only<ACT, true>(g[2 * e]) * u[2 * e],
                               act_only<ACT, true>(g[2 * e + 1]) * u[2 * e + 1]);
          store_bf16_box(buf, flip, lane, w, &p.c, x, row0, in);
        }
      } else if (EPI == FFN_DGATE || EPI == FFN_DGATE_TERMS) {
        const long long plane = ffn_saved_plane(p.M, p.N);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          const int col = half * 128 + c * 32;
          const int x = it.n * 256 + col;
          const bool in = live && x < p.N;
          const float* sg = a.saved + ffn_saved_at(row0 + lane, x, p.N);
          const float* su = sg + plane;
          float g[32], u[32], da[32];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4*>(g + 4 * e) = in ? __ldcs(reinterpret_cast<const float4*>(sg + e * 128)) : z;
            *reinterpret_cast<float4*>(u + 4 * e) = in ? __ldcs(reinterpret_cast<const float4*>(su + e * 128)) : z;
          }
          tmem_ld_32x32(tb + col, da);
          tmem_wait_ld();
          if (c == 3) release();
          uint32_t wa[16], wg[16], wu[16], ra[16], rg[16], ru[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float s0, s1;
            const float h0 = act_with_slope<ACT, true>(g[2 * e], &s0);
            const float h1 = act_with_slope<ACT, true>(g[2 * e + 1], &s1);
            const float d0 = da[2 * e], d1 = da[2 * e + 1], u0 = u[2 * e], u1 = u[2 * e + 1];
            const float a0 = h0 * u0, a1 = h1 * u1, dg0 = d0 * u0 * s0, dg1 = d1 * u1 * s1, du0 = d0 * h0, du1 = d1 * h1;
            wa[e] = pack_bf16x2(a0, a1);
            wg[e] = pack_bf16x2(dg0, dg1);
            wu[e] = pack_bf16x2(du0, du1);
            if (EPI == FFN_DGATE_TERMS) {
              ra[e] = rest_bf16x2(a0, a1, wa[e]);
              rg[e] = rest_bf16x2(dg0, dg1, wg[e]);
              ru[e] = rest_bf16x2(du0, du1, wu[e]);
            }
          }
          store_bf16_box(buf, flip, lane, wa, &p.c, x, row0, in);
          store_bf16_box(buf, flip, lane, wg, &a.c2, x, row0, in);
          store_bf16_box(buf, flip, lane, wu, &a.c3, x, row0, in);
          if (EPI == FFN_DGATE_TERMS) {
            store_bf16_box(buf, flip, lane, ra, &a.rest[0], x, row0, in);
            store_bf16_box(buf, flip, lane, rg, &a.rest[1], x, row0, in);
            store_bf16_box(buf, flip, lane, ru, &a.rest[2], x, row0, in);
          }
        }
      } else {
#pragma unroll 1
        for (int b = 0; b < 2; ++b) {
          const int col = half * 128 + b * 64;
          const int x = it.n * 256 + col;
          float v[64];
          tmem_ld_32x32(tb + col, v);
          tmem_ld_32x32(tb + col + 32, v + 32);
          tmem_wait_ld();
          if (b == 1) release();
          if (p.part_rows > 0) {
            const int y = it.part * p.part_rows + row0;
            store_f32_box(buf, lane, v, &p.c, x, y, live && x < p.N);
            store_f32_box(buf, lane, v + 32, &p.c, x + 32, y, live && x + 32 < p.N);
          } else {
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) w[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
            store_bf16_box(buf, flip, lane, w, &p.c, x, row0, live && x < p.N);
            store_bf16_box(buf, flip, lane, w + 16, &p.c, x + 32, row0, live && x + 32 < p.N);
          }
        }
      }
    }
    if (lane == 0) bulk_wait<0>();
    __syncwarp();
  }

  // Neither CTA may release its TMEM or shared memory while the pair MMAs or
  // the other CTA can still touch them.
  tc_fence_before();
  cluster_sync();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kPairTmem);
  }
}

// ============================================================================
// Few rows
// ============================================================================
namespace {
constexpr int kSkinnyThreads = 64 + 32 * 4;
constexpr int kSkinnyMaxStages = 12;
constexpr size_t kSkinnySmem = 1024 + 221184 + 512;  // stages of up to 216 KB in all, barriers
constexpr int kSkinnyTmem = 2 * kFfnSkinnyRows;      // two accumulators of up to kFfnSkinnyRows columns
}  // namespace

// Steps are numbered tile by tile (128 weight rows each), `steps` 64-deep ones a
// tile; CTA c takes steps [c per, (c + 1) per).  What it has of a tile is that
// tile's part number c - (first CTA of the tile).
__global__ void __launch_bounds__(kSkinnyThreads, 1) ffn_skinny_kernel(const __grid_constant__ FfnSkinnyArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_1k(smem_raw);
  const int b_bytes = a.cols * kBK * 2;  // cols: rows of x, rounded up to 16
  const int stage_bytes = kOperand + b_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + 221184);
  uint64_t* empty = full + kSkinnyMaxStages;
  uint64_t* acc_full = empty + kSkinnyMaxStages;  // [2]
  uint64_t* acc_empty = acc_full + 2;             // [2]
  uint64_t* tear = acc_empty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(tear + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const long long lo = static_cast<long long>(blockIdx.x) * a.per;
  const long long all = static_cast<long long>(a.tiles) * a.steps;
  const long long hi = lo + a.per < all ? lo + a.per : all;

  const int first_tile = static_cast<int>(lo / a.steps), first_k = static_cast<int>(lo % a.steps);
  const int early = hi - lo < a.stages ? static_cast<int>(hi - lo) : a.stages;
  auto load_w = [&](int st, int tile, int k) {
    const bool second = tile >= a.tiles_first;
    mbar_arrive_expect_tx(&full[st], stage_bytes);
    tma_load_2d(smem + st * stage_bytes, second ? &a.w2 : &a.w1, &full[st], k * kBK,
                (second ? tile - a.tiles_first : tile) * 128);
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
    }
    mbar_init(tear, 1);
    *abort_flag = 0;
    fence_barrier_init();
    // The weights do not depend on the launch before this one, x and the parts'
    // memory may: the ring fills with weights at once, up to 216 KB on each SM
    // while that launch ends and this one gets ready.
    for (int i = 0, t = first_tile, k = first_k; i < early; ++i) {
      load_w(i, t, k);
      if (++k == a.steps) {
        k = 0;
        ++t;
      }
    }
  }
  if (warp == 2) {
    tmem_alloc(tmem_holder, kSkinnyTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  if (threadIdx.x == 0) let_next_launch_begin();

  if (warp == 0) {
    if (lane == 0) {
      auto load_x = [&](int st, int k) {
        tma_load_2d(smem + st * stage_bytes + kOperand, &a.x, &full[st], k * kBK, 0);
      };
      int stage = 0;
      uint32_t phase = 0, armed = 0, last_par = 0;
      int tile = first_tile, k = first_k;
      wait_for_last_launch();
      for (long long s = lo; s < hi; ++s) {
        if (!RKL_BOUNDS(tile < a.tiles && k < a.steps)) {
          give_up(abort_flag, ERR_BOUNDS);
          break;
        }
        if (s - lo >= early) {
          if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag)) {
            give_up(abort_flag, ERR_WAIT_TMA_EMPTY);
            break;
          }
          load_w(stage, tile, k);
        }
        load_x(stage, k);
        armed |= 1u << stage;
        last_par = (last_par & ~(1u << stage)) | (phase << stage);
        if (++stage == a.stages) {
          stage = 0;
          phase ^= 1;
        }
        if (++k == a.steps) {
          k = 0;
          ++tile;
        }
      }
      for (int i = 0; i < a.stages; ++i)
        if (armed & (1u << i)) {
          volatile int never = 0;
          if (!mbar_wait(&full[i], (last_par >> i) & 1, &never)) atomicOr(&g_ffn_err, ERR_WAIT_TEARDOWN);
        }
    }
  } else if (warp == 1) {
    // The whole warp runs the loop and one lane issues: the MMAs' operands then
    // live in uniform registers.  What a step costs here besides its bytes is
    // this loop's own latency, so it holds nothing that can be settled outside.
    // A stage's descriptors are the first one's with the address moved, slices
    // of 16 lie 32 B apart.
    const uint32_t idesc = idesc_bf16(128, a.cols, 0, 0);
    const uint64_t first_desc = sdesc_sw128(smem_u32(smem), 16, 1024);
    const int stages = a.stages, steps = a.steps, stage_desc = stage_bytes >> 4;
    int stage = 0;
    uint64_t desc = first_desc;
    uint32_t phase = 0;
    bool ok = true;
    int k = first_k;
    int i = 0;  // accumulators handed over
    for (int left = static_cast<int>(hi - lo); left > 0 && ok; ++i) {
      const int acc = i & 1, n = left < steps - k ? left : steps - k;
      const uint32_t d = tmem_base + acc * kFfnSkinnyRows;
      if (!__all_sync(0xffffffffu, mbar_wait(&acc_empty[acc], ((i >> 1) & 1) ^ 1, abort_flag))) {
        give_up(abort_flag, ERR_WAIT_ACC_EMPTY);
        break;
      }
      tc_fence_after();
      uint32_t more = 0;
      for (int x = 0; x < n; ++x) {
        ok = __all_sync(0xffffffffu, mbar_wait(&full[stage], phase, abort_flag));
        if (!ok) {
          give_up(abort_flag, ERR_WAIT_TMA_FULL);
          break;
        }
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < kBK / 16; ++j)
            umma_bf16(d, desc + 2 * j, desc + (kOperand >> 4) + 2 * j, idesc, more | j);
          umma_commit(&empty[stage]);
        }
        more = 1;
        desc += stage_desc;
        if (++stage == stages) {
          stage = 0;
          desc = first_desc;
          phase ^= 1;
        }
      }
      if (ok && elect_one()) umma_commit(&acc_full[acc]);
      left -= n;
      k = 0;
    }
    if (elect_one()) {
      umma_commit(tear);
      volatile int never = 0;
      if (!mbar_wait(tear, 0, &never)) atomicOr(&g_ffn_err, ERR_WAIT_TEARDOWN);
    }
    __syncwarp();
  } else {
    wait_for_last_launch();
    const int quarter = warp & 3;
    int i = 0;
    for (long long s = lo; s < hi; ++i) {
      const int tile = static_cast<int>(s / a.steps);
      const long long end = static_cast<long long>(tile + 1) * a.steps;
      const int part = static_cast<int>(blockIdx.x - static_cast<long long>(tile) * a.steps / a.per);
      const int acc = i & 1;
      bool ok = mbar_wait(&acc_full[acc], (i >> 1) & 1, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        if (lane == 0) give_up(abort_flag, ERR_WAIT_ACC_FULL);
        break;
      }
      tc_fence_after();
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * kFfnSkinnyRows;
      float* out = a.part + static_cast<long long>(part) * a.T * a.pitch + tile * 128 + quarter * 32 + lane;
      const bool in = RKL_BOUNDS(part >= 0 && part < a.parts && tile < a.tiles);
      for (int c = 0; c < a.cols; c += 16) {
        float v[16];
        tmem_ld_32x16(tb + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (in && c + e < a.T) out[static_cast<long long>(c + e) * a.pitch] = v[e];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[acc]);
      s = end < hi ? end : hi;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kSkinnyTmem);
  }
}

// ============================================================================
// Joining the parts
// ============================================================================
namespace {

// Parts of the column's tile.  per > 0: of ffn_skinny_kernel's numbering.
__device__ __forceinline__ int parts_of(const FfnJoinArgs& a, int col) {
  if (a.per == 0) return a.parts;
  const long long first = static_cast<long long>(col / 128) * a.steps;
  return static_cast<int>((first + a.steps - 1) / a.per - first / a.per) + 1;
}

// The sum of 4 neighbouring columns' parts, in the parts' order.
__device__ __forceinline__ float4 sum_parts(const FfnJoinArgs& a, long long row, int col) {
  const float* p = a.part + row * a.pitch + col;
  float4 s = *reinterpret_cast<const float4*>(p);
  const int n = parts_of(a, col);
  for (int j = 1; j < n; ++j) {
    const float4 v = *reinterpret_cast<const float4*>(p + j * a.slab);
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  }
  return s;
}

}  // namespace

// out [T, N] bf16 = the parts' sum, or (GATED) act(g) u of the sums g at column
// n and u at a.second + n.  TERMS = 2: of the sums of rows t and T + t, or
// (GATED) in two terms, the second at a.rest.
template <bool GATED, int ACT, int TERMS>
__global__ void __launch_bounds__(256) ffn_join_kernel(const __grid_constant__ FfnJoinArgs a) {
  if (threadIdx.x == 0) let_next_launch_begin();
  wait_for_last_launch();
  const int n4 = a.N / 4;  // N is a multiple of 8
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<long long>(a.T) * n4) return;
  const long long row = i / n4;
  const int col = static_cast<int>(i - row * n4) * 4;
  float4 v = sum_parts(a, row, col);
  if (!GATED && TERMS == 2) {
    const float4 r = sum_parts(a, row + a.T, col);
    v.x += r.x;
    v.y += r.y;
    v.z += r.z;
    v.w += r.w;
  }
  const long long at = row * a.N + col;
  if (GATED) {
    const float4 u = sum_parts(a, row, a.second + col);
    if (a.saved != nullptr) {
      float* sg = a.saved + ffn_saved_at(row, col, a.N);
      *reinterpret_cast<float4*>(sg) = v;
      *reinterpret_cast<float4*>(sg + ffn_saved_plane(a.T, a.N)) = u;
    }
    v.x = act_only<ACT, true>(v.x) * u.x;
    v.y = act_only<ACT, true>(v.y) * u.y;
    v.z = act_only<ACT, true>(v.z) * u.z;
    v.w = act_only<ACT, true>(v.w) * u.w;
  }
  const uint2 w = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  *reinterpret_cast<uint2*>(a.out + at) = w;
  if (GATED && TERMS == 2)
    *reinterpret_cast<uint2*>(a.rest + at) = make_uint2(rest_bf16x2(v.x, v.y, w.x), rest_bf16x2(v.z, v.w, w.y));
}

// Matrices whose rows are not whole multiples of 16 bytes, which TMA needs, are
// laid out anew with zeros behind their rows and columns (zero weights give zero
// g, u and gradients there, or NaN in a row that is not finite: the second
// products do not read those columns), and results are brought back: a few bytes an
// element beside the products, which then run on the tensor cores (T = 5999, H =
// 349, F = 699, O = 351, forward and backward: 2.8 ms on the CUDA cores before).
__global__ void __launch_bounds__(256) ffn_pad_kernel(const __grid_constant__ FfnPadArgs a) {
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < a.total;
       i += static_cast<long long>(gridDim.x) * 256) {
    int q = 0;
    while (q + 1 < a.n && i >= a.item[q + 1].first) ++q;
    const FfnPadItem& m = a.item[q];
    const long long at = i - m.first, row = at / m.dst_cols;
    const int col = static_cast<int>(at - row * m.dst_cols);
    m.dst[at] = row < m.rows && col < m.cols ? m.src[row * m.src_pitch + col] : 0;
  }
}

// ============================================================================
// Host launchers
// ============================================================================
cudaError_t launch_ffn_pad(const FfnPadArgs& a, cudaStream_t s) {
  if (a.total == 0) return cudaSuccess;
  LaunchScope scope(K_FFN_PAD, s);
  const long long blocks = (a.total + 1023) / 1024;
  ffn_pad_kernel<<<static_cast<unsigned>(blocks < 148 * 16 ? blocks : 148 * 16), 256, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename K>
static cudaError_t allow_smem(K kernel, size_t bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
}

cudaError_t ffn_tc_setup() {
  cudaError_t e;
#define RKL_FFN_SETUP(...) \
  if ((e = allow_smem(__VA_ARGS__, kPairSmem)) != cudaSuccess) return e
  RKL_FFN_SETUP((ffn_pair_kernel<FFN_UP, ACT_SILU>));
  RKL_FFN_SETUP((ffn_pair_kernel<FFN_UP, ACT_GELU>));
  RKL_FFN_SETUP((ffn_pair_kernel<FFN_UP, ACT_GELU_TANH>));
  RKL_FFN_SETUP((ffn_pair_kernel<FFN_UP, ACT_RELU>));
  RKL_FFN_SETUP((ffn_pair_kernel<FFN_DGATE, ACT_SILU>));
  RKL_FFN_SETUP((ffn_pair_kernel<FFN_DGATE, ACT_GELU>));
  RKL_FFN_SETUP((ffn_pair_kernel<FFN_DGATE, ACT_GELU_TANH>));
  RKL_FFN_SETUP((ffn_pair_kernel<FFN_DGATE, ACT_RELU>));
  RKL_FFN_SETUP((ffn_pair_kernel<FFN_DGATE_TERMS, ACT_SILU>));
  RKL_FFN_SETUP((ffn_pair_kernel<FFN_DGATE_TERMS, ACT_GELU>));
  RKL_FFN_SETUP((ffn_pair_kernel<FFN_DGATE_TERMS, ACT_GELU_TANH>));
  RKL_FFN_SETUP((ffn_pair_kernel<FFN_DGATE_TERMS, ACT_RELU>));
  RKL_FFN_SETUP((ffn_pair_kernel<FFN_GEMM, 0>));
#undef RKL_FFN_SETUP
  return allow_smem(ffn_skinny_kernel, kSkinnySmem);
}

// follows: the launch comes right behind another of the same call and may begin
// while that one ends.
template <typename K, typename A>
static cudaError_t launch_ffn(K kernel, unsigned grid, unsigned threads, size_t smem, bool pairs, bool follows,
                              cudaStream_t s, const A& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if (pairs) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = 2;
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs++].val.clusterDim.z = 1;
  }
  if (follows) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

cudaError_t launch_ffn_pair(int mode, int act, const FfnPairArgs& a, int sms, cudaStream_t s) {
  LaunchScope scope(mode == FFN_UP ? K_FFN_UP_TC : mode == FFN_GEMM ? K_FFN_GEMM_TC : K_FFN_DGATE_TC, s);
  const int grid = (2 * a.items < sms ? 2 * a.items : sms) & ~1;  // whole CTA pairs
  if (mode == FFN_GEMM) return launch_ffn(ffn_pair_kernel<FFN_GEMM, 0>, grid, kPairThreads, kPairSmem, true, a.follows, s, a);
  if (mode == FFN_UP) switch (act) {
      case ACT_SILU: return launch_ffn(ffn_pair_kernel<FFN_UP, ACT_SILU>, grid, kPairThreads, kPairSmem, true, a.follows, s, a);
      case ACT_GELU: return launch_ffn(ffn_pair_kernel<FFN_UP, ACT_GELU>, grid, kPairThreads, kPairSmem, true, a.follows, s, a);
      case ACT_GELU_TANH: return launch_ffn(ffn_pair_kernel<FFN_UP, ACT_GELU_TANH>, grid, kPairThreads, kPairSmem, true, a.follows, s, a);
      default: return launch_ffn(ffn_pair_kernel<FFN_UP, ACT_RELU>, grid, kPairThreads, kPairSmem, true, a.follows, s, a);
    }
  if (mode == FFN_DGATE_TERMS) switch (act) {
      case ACT_SILU: return launch_ffn(ffn_pair_kernel<FFN_DGATE_TERMS, ACT_SILU>, grid, kPairThreads, kPairSmem, true, a.follows, s, a);
      case ACT_GELU: return launch_ffn(ffn_pair_kernel<FFN_DGATE_TERMS, ACT_GELU>, grid, kPairThreads, kPairSmem, true, a.follows, s, a);
      case ACT_GELU_TANH: return launch_ffn(ffn_pair_kernel<FFN_DGATE_TERMS, ACT_GELU_TANH>, grid, kPairThreads, kPairSmem, true, a.follows, s, a);
      default: return launch_ffn(ffn_pair_kernel<FFN_DGATE_TERMS, ACT_RELU>, grid, kPairThreads, kPairSmem, true, a.follows, s, a);
    }
  switch (act) {
    case ACT_SILU: return launch_ffn(ffn_pair_kernel<FFN_DGATE, ACT_SILU>, grid, kPairThreads, kPairSmem, true, a.follows, s, a);
    case ACT_GELU: return launch_ffn(ffn_pair_kernel<FFN_DGATE, ACT_GELU>, grid, kPairThreads, kPairSmem, true, a.follows, s, a);
    case ACT_GELU_TANH: return launch_ffn(ffn_pair_kernel<FFN_DGATE, ACT_GELU_TANH>, grid, kPairThreads, kPairSmem, true, a.follows, s, a);
    default: return launch_ffn(ffn_pair_kernel<FFN_DGATE, ACT_RELU>, grid, kPairThreads, kPairSmem, true, a.follows, s, a);
  }
}

cudaError_t launch_ffn_skinny(FfnSkinnyArgs a, int grid, cudaStream_t s) {
  LaunchScope scope(K_FFN_SKINNY_TC, s);
  const int stage = kOperand + a.cols * kBK * 2;
  a.stages = 221184 / stage < kSkinnyMaxStages ? 221184 / stage : kSkinnyMaxStages;
  return launch_ffn(ffn_skinny_kernel, grid, kSkinnyThreads, kSkinnySmem, false, a.follows, s, a);
}

template <int TERMS>
static cudaError_t join(int act, const FfnJoinArgs& a, cudaStream_t s) {
  const long long blocks = (static_cast<long long>(a.T) * (a.N / 4) + 255) / 256;
  const unsigned grid = static_cast<unsigned>(blocks);
  switch (act) {
    case -1: return launch_ffn(ffn_join_kernel<false, 0, TERMS>, grid, 256, 0, false, true, s, a);
    case ACT_SILU: return launch_ffn(ffn_join_kernel<true, ACT_SILU, TERMS>, grid, 256, 0, false, true, s, a);
    case ACT_GELU: return launch_ffn(ffn_join_kernel<true, ACT_GELU, TERMS>, grid, 256, 0, false, true, s, a);
    case ACT_GELU_TANH: return launch_ffn(ffn_join_kernel<true, ACT_GELU_TANH, TERMS>, grid, 256, 0, false, true, s, a);
    default: return launch_ffn(ffn_join_kernel<true, ACT_RELU, TERMS>, grid, 256, 0, false, true, s, a);
  }
}

cudaError_t launch_ffn_join(int act, const FfnJoinArgs& a, cudaStream_t s) {
  LaunchScope scope(K_FFN_JOIN, s);
  return a.terms > 1 ? join<2>(act, a, s) : join<1>(act, a, s);
}

cudaError_t read_and_clear_ffn_error(int* code) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_ffn_err, sizeof(int));
  if (e != cudaSuccess) return e;
  *code = v;
  if (v != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_ffn_err, &zero, sizeof(int));
  }
  return e;
}

}  // namespace rkl
