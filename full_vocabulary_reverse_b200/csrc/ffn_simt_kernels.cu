// ffn_simt_kernels.cu -- the gated feed-forward block in fp32 on the CUDA cores
// (tcgen05 has no fp32 input kind).
//
//   g = x Wg^T, u = x Wu^T, a = act(g) u, y = a Wd^T
//   da = dy Wd, dg = da u act'(g), du = da act(g)
//   dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, dWd = dy^T a
//
// One tiled product kernel does all of them: C(m, n) = sum_k A(m, k) B(k, n)
// with any strides, BT x BT tiles, the next slice's loads under way while
// the present one is multiplied.  A thread owns 8 x 8 results: rows and
// columns in two groups of 4, BT / 2 apart.  So the up form puts Wg's columns in
// the tile's first half and Wu's in the second, and a thread holds g and u of
// the same elements: the activation, the product and the rounding happen in its
// registers.
//
// Bound by shared memory and the FFMA pipe alike: of a 16-byte read every 8
// lanes take a cycle, so 8 x 8 results need 16 cycles of reads for 16 cycles of
// multiply-adds (4 x 4 results a thread, 8 for 4, ran half as fast).  BT = 128
// where there are many tiles; else 64, whose 64 threads of results are four
// times over, each for a quarter of every slice, and add up at the end: with
// one tile an SM, 2 warps alone took twice as long.  fp32 forward and backward:
// T = 509, H = O = 515, F = 1031 in 0.24 ms (20 TFLOP/s), T = 4096, H = O = 2048,
// F = 4096 in 13.5 (46; a library's fp32 products run at 56).
#include "ffn_act.cuh"
#include "kernels.h"

namespace rkl {
namespace {

constexpr int kResults = 8;  // of a thread, each way
constexpr int kSimtThreads = 256;
template <int BT>
constexpr int kDepth = BT == 64 ? 32 : 16;  // of a slice of K (the small tile has fewer instructions between barriers)
template <int BT>
constexpr int kGroups = kSimtThreads / ((BT / kResults) * (BT / kResults));  // of threads that share a tile's K
template <int BT>
constexpr int kShare = BT * kDepth<BT> / kSimtThreads;  // elements of an operand's slice that a thread moves

__device__ __forceinline__ float act_of(int act, float g, float* slope) {
  switch (act) {
    case ACT_SILU: return act_with_slope<ACT_SILU, false>(g, slope);
    case ACT_GELU: return act_with_slope<ACT_GELU, false>(g, slope);
    case ACT_GELU_TANH: return act_with_slope<ACT_GELU_TANH, false>(g, slope);
    default: return act_with_slope<ACT_RELU, false>(g, slope);
  }
}

// Two fp32 multiply-adds in one instruction: the issue slots that this saves go
// to the shared-memory reads beside them.
__device__ __forceinline__ uint64_t twice(float x) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void fma2(uint64_t& d, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}

// Where element i of this thread's share of a slice lies: BT positions along m
// (or n) x kDepth along k.  Neighbouring threads run along the dimension that is
// contiguous in memory.
template <int BT>
__device__ __forceinline__ void slice_place(bool k_fast, int i, int* mn, int* k) {
  const int e = threadIdx.x + i * kSimtThreads;
  *k = k_fast ? e % kDepth<BT> : e / BT;
  *mn = k_fast ? e / kDepth<BT> : e % BT;
}

// This thread's share of an operand's slices: position `mn` of the tile is row
// mn0 + mn of p, or from position `half` on (half > 0) row mn0 + mn - half of
// p2; rows at mn_end and behind are zero.  Element i of a slice lies offset[i]
// elements behind the slice's start.
template <int BT>
struct Operand {
  const float *p, *p2;  // at (mn0, first k of the next slice)
  long long s_k;
  int offset[kShare<BT>];
  uint32_t rows, upper;  // bits: the element's row is there; it comes from p2
  bool k_fast;

  __device__ __forceinline__ Operand(const float* base, const float* base2, long long s_mn, long long stride_k,
                                     long long mn0, long long mn_end, int half)
      : p(base + mn0 * s_mn), p2(half > 0 ? base2 + mn0 * s_mn : nullptr), s_k(stride_k), rows(0), upper(0),
        k_fast(stride_k == 1) {
#pragma unroll
    for (int i = 0; i < kShare<BT>; ++i) {
      int mn, k;
      slice_place<BT>(k_fast, i, &mn, &k);
      const bool second = half > 0 && mn >= half;
      const int row = second ? mn - half : mn;
      offset[i] = static_cast<int>(row * s_mn + k * s_k);  // strides are at most 2^20, one of them 1: it fits
      rows |= (mn0 + row < mn_end ? 1u : 0u) << i;
      upper |= (second ? 1u : 0u) << i;
    }
  }
  __device__ __forceinline__ void advance() {
    p += kDepth<BT> * s_k;
    p2 += kDepth<BT> * s_k;
  }
  // The slice with `left` positions along k, straight into shared memory, 4
  // bytes at a time (rows need no alignment), zeros where nothing is read.
  __device__ __forceinline__ void fetch(int left, float (*s)[BT + 4]) const {
#pragma unroll
    for (int i = 0; i < kShare<BT>; ++i) {
      int mn, k;
      slice_place<BT>(k_fast, i, &mn, &k);
      const bool in = ((rows >> i) & 1) && k < left;
      const float* from = ((upper >> i) & 1 ? p2 : p) + offset[i];
      const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(&s[k][mn]));
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(in ? from : p), "r"(in ? 4 : 0)
                   : "memory");
    }
  }
};

// What element (m, n) goes through: its sum, and in the up form u's.
template <int MODE>
__device__ __forceinline__ void finish(const FfnSimtArgs& a, const FfnProduct& p, long long m, long long n, float sum,
                                       float u) {
  const long long at = m * p.N + n;
  float* c = p.c + at;
  float slope;
  if (MODE == FFN_UP) {
    *c = act_of(a.act, sum, &slope) * u;
    if (a.saved != nullptr) {
      const long long sv = ffn_saved_at(m, n, p.N);
      a.saved[sv] = sum;
      a.saved[ffn_saved_plane(p.M, p.N) + sv] = u;
    }
  } else if (MODE == FFN_DGATE) {
    const long long sv = ffn_saved_at(m, n, p.N), one = p.M * p.N;
    const float g = a.saved[sv], up = a.saved[ffn_saved_plane(p.M, p.N) + sv];
    const float h = act_of(a.act, g, &slope);
    *c = h * up;                   // a
    c[one] = sum * up * slope;     // dg
    c[2 * one] = sum * h;          // du
  } else {
    *c = sum;
  }
}

}  // namespace

template <int BT, int MODE>
__global__ void __launch_bounds__(kSimtThreads, 2) ffn_simt_kernel(const __grid_constant__ FfnSimtArgs a) {
  constexpr int R = kResults;
  constexpr int STEP = BT / 2;  // between a thread's groups of 4
  constexpr int BN = MODE == FFN_UP ? BT / 2 : BT;  // result columns of a tile
  constexpr int RING = 2;  // one slice is multiplied, the next is on its way
  __shared__ __align__(16) float sa[RING][kDepth<BT>][BT + 4];
  __shared__ __align__(16) float sb[RING][kDepth<BT>][BT + 4];
  static_assert(kGroups<BT> == 1 || sizeof(sa) >= size_t(BT) * BT * 4, "a group's sums fit into sa or sb");

  int q = 0;
  while (q + 1 < a.n && static_cast<int>(blockIdx.x) >= a.p[q + 1].first_tile) ++q;
  const FfnProduct& p = a.p[q];
  const int tile = blockIdx.x - p.first_tile;
  const int n_tiles = static_cast<int>((p.N + BN - 1) / BN);
  const long long m0 = static_cast<long long>(tile / n_tiles) * BT, n0 = static_cast<long long>(tile % n_tiles) * BN;
  const int group = threadIdx.x / (kSimtThreads / kGroups<BT>);
  const int tx = threadIdx.x % (BT / R), ty = threadIdx.x / (BT / R) % (BT / R);

  uint64_t acc2[R][R / 2];  // neighbouring columns in pairs
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < R / 2; ++j) acc2[i][j] = 0;

  Operand<BT> oa(p.a[0], nullptr, p.sam, p.sak, m0, p.M, 0);
  Operand<BT> ob(p.b[0], p.b[1], p.sbn, p.sbk, n0, p.N, MODE == FFN_UP ? BN : 0);
  // Slices of all segments of K, one behind another; the loads run ahead.
  const int per_segment = static_cast<int>((p.K + kDepth<BT> - 1) / kDepth<BT>);
  const int slices = per_segment * p.segments;
  int ahead = 0;                     // next slice to load
  int left = static_cast<int>(p.K);  // positions along k from it to its segment's end
  auto advance = [&] {
    ++ahead;
    left -= kDepth<BT>;
    oa.advance();
    ob.advance();
    if (ahead == per_segment && p.segments == 2) {
      left = static_cast<int>(p.K);
      oa.p = p.a[1] + m0 * p.sam;
      ob.p = p.b[1] + n0 * p.sbn;
    }
  };
  auto multiply = [&](int slot) {
#pragma unroll
    for (int d = 0; d < kDepth<BT> / kGroups<BT>; ++d) {
      const int k = group * (kDepth<BT> / kGroups<BT>) + d;
      float x[R];
      uint64_t w[R / 2];
#pragma unroll
      for (int h = 0; h < R / 4; ++h)
        *reinterpret_cast<float4*>(&x[4 * h]) = *reinterpret_cast<const float4*>(&sa[slot][k][ty * 4 + h * STEP]);
#pragma unroll
      for (int h = 0; h < R / 4; ++h) {
        const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(&sb[slot][k][tx * 4 + h * STEP]);
        w[2 * h] = two.x;
        w[2 * h + 1] = two.y;
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const uint64_t xx = twice(x[i]);
#pragma unroll
        for (int j = 0; j < R / 2; ++j) fma2(acc2[i][j], xx, w[j]);
      }
    }
  };
  auto issue = [&] {  // (a group each time, an empty one at the end)
    if (ahead < slices) {
      oa.fetch(left, sa[ahead % RING]);
      ob.fetch(left, sb[ahead % RING]);
      advance();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int i = 0; i < RING - 1; ++i) issue();
  for (int s = 0; s < slices; ++s) {
    asm volatile("cp.async.wait_group %0;" ::"n"(RING - 2) : "memory");
    __syncthreads();  // slice s is there for all; all are done with slice s - 1, whose slot the next load takes
    issue();
    multiply(s % RING);
  }

  float acc[R][R];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < R / 2; ++j)
      asm("mov.b64 {%0, %1}, %2;" : "=f"(acc[i][2 * j]), "=f"(acc[i][2 * j + 1]) : "l"(acc2[i][j]));
  if constexpr (kGroups<BT> == 4) {
    // The four groups' sums join in shared memory, (0 + 2) + (1 + 3), each
    // thread's 64 values a lane's distance apart.
    constexpr int kLanes = kSimtThreads / 4;
    float* own = &sa[0][0][0] + threadIdx.x % kLanes;
    float* odd = &sb[0][0][0] + threadIdx.x % kLanes;
    auto put_sums = [&](float* to) {
#pragma unroll
      for (int i = 0; i < R * R; ++i) to[i * kLanes] = acc[i / R][i % R];
    };
    auto add_sums = [&](const float* from) {
#pragma unroll
      for (int i = 0; i < R * R; ++i) acc[i / R][i % R] += from[i * kLanes];
    };
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    if (group == 2) put_sums(own);
    if (group == 3) put_sums(odd);
    __syncthreads();
    if (group == 0) add_sums(own);
    if (group == 1) add_sums(odd);
    __syncthreads();
    if (group == 1) put_sums(own);
    __syncthreads();
    // The tile, row by row, for all 256 threads to finish.
    float(*whole)[BT] = reinterpret_cast<float(*)[BT]>(&sb[0][0][0]);
    if (group == 0) {
      add_sums(own);
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float4*>(&whole[ty * 4 + (i / 4) * STEP + i % 4][tx * 4 + h * STEP]) =
              *reinterpret_cast<const float4*>(&acc[i][4 * h]);
    }
    __syncthreads();
#pragma unroll 4
    for (int e = threadIdx.x; e < BT * BN; e += kSimtThreads) {
      const int r = e / BN, c = e % BN;
      if (m0 + r < p.M && n0 + c < p.N) finish<MODE>(a, p, m0 + r, n0 + c, whole[r][c], whole[r][(c + BN) % BT]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const long long m = m0 + ty * 4 + (i / 4) * STEP + i % 4;
      if (m >= p.M) continue;
#pragma unroll
      for (int j = 0; j < (MODE == FFN_UP ? 4 : R); ++j) {
        // up: a thread's first group of columns are gates, its second the ups of the same elements
        const long long n = n0 + tx * 4 + (j / 4) * STEP + j % 4;
        if (n < p.N) finish<MODE>(a, p, m, n, acc[i][j], acc[i][(j + 4) % R]);
      }
    }
  }
}

template <int BT>
static cudaError_t launch_simt_bt(int mode, FfnSimtArgs& a, cudaStream_t s) {
  long long tiles = 0;
  for (int i = 0; i < a.n; ++i) {
    a.p[i].first_tile = static_cast<int>(tiles);
    const int bn = mode == FFN_UP ? BT / 2 : BT;
    tiles += (a.p[i].M + BT - 1) / BT * ((a.p[i].N + bn - 1) / bn);
  }
  if (tiles == 0) return cudaSuccess;
  if (tiles > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  const dim3 grid(static_cast<unsigned>(tiles));
  LaunchScope scope(mode == FFN_UP ? K_FFN_UP_SIMT : mode == FFN_DGATE ? K_FFN_DGATE_SIMT : K_FFN_GEMM_SIMT, s);
  if (mode == FFN_UP)
    ffn_simt_kernel<BT, FFN_UP><<<grid, kSimtThreads, 0, s>>>(a);
  else if (mode == FFN_DGATE)
    ffn_simt_kernel<BT, FFN_DGATE><<<grid, kSimtThreads, 0, s>>>(a);
  else
    ffn_simt_kernel<BT, FFN_GEMM><<<grid, kSimtThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_ffn_simt(int mode, FfnSimtArgs a, int sms, cudaStream_t s) {
  long long big = 0;
  for (int i = 0; i < a.n; ++i) big += (a.p[i].M + 127) / 128 * ((a.p[i].N + (mode == FFN_UP ? 63 : 127)) / (mode == FFN_UP ? 64 : 128));
  // 128-wide tiles do twice the work for each shared load, but take four times
  // as long each, one or two on an SM: they pay from some two waves on (T = 2000, H = O = 1024,
  // F = 2048: 2.06 ms forward and backward against 2.35).
  const bool wide = big >= 2 * sms;
  return wide ? launch_simt_bt<128>(mode, a, s) : launch_simt_bt<64>(mode, a, s);
}

}  // namespace rkl
