// ffn_simt_kernels.cu -- the gated feed-forward block on the CUDA cores: fp32
// (tcgen05 has no fp32 input kind), and bf16 whose sizes or addresses the
// tensor-core path's 16-byte TMA rows rule out.
//
//   g = x Wg^T, u = x Wu^T, a = act(g) u, y = a Wd^T
//   da = dy Wd, dg = da u act'(g), du = da act(g)
//   dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, dWd = dy^T a
//
// One tiled product kernel does all of them: C(m, n) = sum_k A(m, k) B(k, n)
// with any strides, 256 threads on a BT x BT tile, 16 deep, the next slice's
// loads in registers while the present one is multiplied.  A thread owns R x R
// results (R = BT / 16): rows and columns in groups of 4, BT / 2 apart.  So the
// up form puts Wg's columns in the tile's first half and Wu's in the second (its
// groups of columns are R / 2 wide), and a thread holds g and u of the same
// elements: the activation, the product and the rounding happen in its registers.
//
// Bound by the FFMA pipe (128 a clock and SM).  BT = 128 (64 results a thread,
// 4 16-byte shared loads for 64 FFMA) where its tiles fill the SMs; else 64.
#include <cuda_bf16.h>

#include "ffn_act.cuh"
#include "kernels.h"

namespace rkl {
namespace {

constexpr int kDepth = 16;
constexpr int kSimtThreads = 256;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ float act_of(int act, float g, float* slope) {
  switch (act) {
    case ACT_SILU: return act_with_slope<ACT_SILU, false>(g, slope);
    case ACT_GELU: return act_with_slope<ACT_GELU, false>(g, slope);
    case ACT_GELU_TANH: return act_with_slope<ACT_GELU_TANH, false>(g, slope);
    default: return act_with_slope<ACT_RELU, false>(g, slope);
  }
}

// One slice of an operand: BT positions along m (or n) x kDepth along k,
// element i of a thread's BT / 16.  Neighbouring threads run along the
// dimension that is contiguous in memory.
template <typename T, int BT>
struct Slice {
  float v[BT / 16];

  __device__ __forceinline__ static void place(bool k_fast, int i, int* mn, int* k) {
    const int e = threadIdx.x + i * kSimtThreads;
    *k = k_fast ? e % kDepth : e / BT;
    *mn = k_fast ? e / kDepth : e % BT;
  }
  // positions [mn0, mn_end) x [k0, k_end) hold values, the others zero
  __device__ __forceinline__ void load(const T* p, long long s_mn, long long s_k, long long mn0, long long mn_end,
                                       long long k0, long long k_end, int first, int half) {
    const bool k_fast = s_k == 1;
#pragma unroll
    for (int i = 0; i < BT / 16; ++i) {
      int mn, k;
      place(k_fast, i, &mn, &k);
      if (half > 0 && (mn < first || mn >= first + half)) continue;  // the other half's operand fills it
      const long long m = mn0 + mn - first;
      v[i] = m < mn_end && k0 + k < k_end ? to_f32(p[m * s_mn + (k0 + k) * s_k]) : 0.f;
    }
  }
  __device__ __forceinline__ void store(float (*s)[BT + 4], bool k_fast) const {
#pragma unroll
    for (int i = 0; i < BT / 16; ++i) {
      int mn, k;
      place(k_fast, i, &mn, &k);
      s[k][mn] = v[i];
    }
  }
};

}  // namespace

template <typename T, int BT, int MODE>
__global__ void __launch_bounds__(kSimtThreads) ffn_simt_kernel(const __grid_constant__ FfnSimtArgs a) {
  constexpr int R = BT / 16;       // results a thread and dimension
  constexpr int STEP = BT * 4 / R;  // between a thread's groups of 4 rows
  constexpr int CW = MODE == FFN_UP ? R / 2 : 4;  // columns of a group: up needs two groups, gates and ups
  constexpr int CSTEP = BT * CW / R;
  constexpr int BN = MODE == FFN_UP ? BT / 2 : BT;  // result columns of a tile
  __shared__ __align__(16) float sa[2][kDepth][BT + 4];
  __shared__ __align__(16) float sb[2][kDepth][BT + 4];

  int q = 0;
  while (q + 1 < a.n && static_cast<int>(blockIdx.x) >= a.p[q + 1].first_tile) ++q;
  const FfnProduct& p = a.p[q];
  const int tile = blockIdx.x - p.first_tile;
  const int n_tiles = static_cast<int>((p.N + BN - 1) / BN);
  const long long m0 = static_cast<long long>(tile / n_tiles) * BT, n0 = static_cast<long long>(tile % n_tiles) * BN;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;

  float acc[R][R];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < R; ++j) acc[i][j] = 0.f;

  Slice<T, BT> la, lb;
  int buf = 0;
  for (int seg = 0; seg < p.segments; ++seg) {
    const T* A = static_cast<const T*>(p.a[seg]);
    const T* B = static_cast<const T*>(p.b[seg]);
    const T* B2 = static_cast<const T*>(p.b[1]);  // up: Wu
    const bool ak = p.sak == 1, bk = p.sbk == 1;
    auto fetch = [&](long long k0) {
      la.load(A, p.sam, p.sak, m0, p.M, k0, p.K, 0, 0);
      if (MODE == FFN_UP) {
        lb.load(B, p.sbn, p.sbk, n0, p.N, k0, p.K, 0, BN);
        lb.load(B2, p.sbn, p.sbk, n0, p.N, k0, p.K, BN, BN);
      } else {
        lb.load(B, p.sbn, p.sbk, n0, p.N, k0, p.K, 0, 0);
      }
    };
    fetch(0);
    for (long long k0 = 0; k0 < p.K; k0 += kDepth) {
      la.store(sa[buf], ak);
      lb.store(sb[buf], bk);
      __syncthreads();  // (the other buffer's readers are past the barrier before this one)
      if (k0 + kDepth < p.K) fetch(k0 + kDepth);
#pragma unroll
      for (int k = 0; k < kDepth; ++k) {
        float x[R], w[R];
#pragma unroll
        for (int h = 0; h < R / 4; ++h)
          *reinterpret_cast<float4*>(&x[4 * h]) = *reinterpret_cast<const float4*>(&sa[buf][k][ty * 4 + h * STEP]);
#pragma unroll
        for (int h = 0; h < R / CW; ++h) {
          if (CW == 4)
            *reinterpret_cast<float4*>(&w[CW * h]) =
                *reinterpret_cast<const float4*>(&sb[buf][k][tx * CW + h * CSTEP]);
          else
            *reinterpret_cast<float2*>(&w[CW * h]) =
                *reinterpret_cast<const float2*>(&sb[buf][k][tx * CW + h * CSTEP]);
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int j = 0; j < R; ++j) acc[i][j] = fmaf(x[i], w[j], acc[i][j]);
      }
      buf ^= 1;
    }
  }

#pragma unroll
  for (int i = 0; i < R; ++i) {
    const long long m = m0 + ty * 4 + (i / 4) * STEP + i % 4;
    if (m >= p.M) continue;
    if (MODE == FFN_UP) {
      // a thread's first group of columns are gates, its second the ups of the same elements
#pragma unroll
      for (int j = 0; j < CW; ++j) {
        const long long n = n0 + tx * CW + j;
        if (n >= p.N) continue;
        const long long at = m * p.N + n;
        const float g = acc[i][j], u = acc[i][j + CW];
        float slope;
        put(static_cast<T*>(p.c) + at, act_of(a.act, g, &slope) * u);
        if (a.saved != nullptr) {
          const long long sv = ffn_saved_at(m, n, p.N);
          a.saved[sv] = g;
          a.saved[ffn_saved_plane(p.M, p.N) + sv] = u;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const long long n = n0 + tx * CW + (j / CW) * CSTEP + j % CW;
        if (n >= p.N) continue;
        const long long at = m * p.N + n;
        if (MODE == FFN_DGATE) {
          const long long sv = ffn_saved_at(m, n, p.N);
          const float g = a.saved[sv], u = a.saved[ffn_saved_plane(p.M, p.N) + sv], da = acc[i][j];
          float slope;
          const float h = act_of(a.act, g, &slope);
          const long long one = p.M * p.N;
          put(static_cast<T*>(p.c) + at, h * u);               // a
          put(static_cast<T*>(p.c) + one + at, da * u * slope);  // dg
          put(static_cast<T*>(p.c) + 2 * one + at, da * h);      // du
        } else {
          put(static_cast<T*>(p.c) + at, acc[i][j]);
        }
      }
    }
  }
}

template <typename T, int BT>
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
    ffn_simt_kernel<T, BT, FFN_UP><<<grid, kSimtThreads, 0, s>>>(a);
  else if (mode == FFN_DGATE)
    ffn_simt_kernel<T, BT, FFN_DGATE><<<grid, kSimtThreads, 0, s>>>(a);
  else
    ffn_simt_kernel<T, BT, FFN_GEMM><<<grid, kSimtThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_ffn_simt(int mode, bool bf16, FfnSimtArgs a, int sms, cudaStream_t s) {
  long long big = 0;
  for (int i = 0; i < a.n; ++i) big += (a.p[i].M + 127) / 128 * ((a.p[i].N + (mode == FFN_UP ? 63 : 127)) / (mode == FFN_UP ? 64 : 128));
  // 128-wide tiles do twice the work for each shared load; below one tile an SM the 64-wide ones use more SMs
  const bool wide = big >= sms;
  if (bf16)
    return wide ? launch_simt_bt<__nv_bfloat16, 128>(mode, a, s) : launch_simt_bt<__nv_bfloat16, 64>(mode, a, s);
  return wide ? launch_simt_bt<float, 128>(mode, a, s) : launch_simt_bt<float, 64>(mode, a, s);
}

}  // namespace rkl
