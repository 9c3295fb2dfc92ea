// optim_kernels.cu -- the optimizer step behind the loss's backward: the
// global norm of many gradients and an AdamW step over many tensors, with
// first and second moments held in 32 bits or in 8.
//
// AdamW with decoupled weight decay (Loshchilov and Hutter, "Decoupled Weight
// Decay Regularization"), t = steps + 1, c = min(1, max_norm / norm):
//     g = c grad
//     m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2
//     p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// all in fp32 registers, whatever the tensors' types.
//
// The state of all tensors is one flat array per moment.  A tensor's place in
// it starts at a multiple of kOptBlock = 256 elements, so a block of 256
// belongs to one tensor; one warp takes a block at a time, 8 elements a lane.
// The 8-bit form holds a block as 256 e4m3 codes and one fp32 scale (largest
// magnitude / 448), so the warp that updates a block also finds its scale.
//
// Both kernels are bound by memory: they touch every byte once.  The tables of
// tensors travel in the kernel's parameters (up to kOptTensors a launch), so a
// step needs no copy to the device and can be captured in a graph.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "bounds.cuh"
#include "kernels.h"

namespace rkl {

RKL_DEFINE_BOUNDS_READER(read_and_clear_bounds_optim)

namespace {

constexpr int kWarps = kOptWarps;
constexpr unsigned kAll = 0xffffffffu;

// ---- loads and stores of 8 consecutive elements of one lane
// `wide`: 8 elements from a 32-byte boundary in memory, all inside the tensor.
// fp32 moves as one 32-byte access a lane, bf16 as 16, e4m3 as 8.
__device__ __forceinline__ void ld8_f32(const float* p, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "l"(p));
}

__device__ __forceinline__ void st8_f32(float* p, const float* v) {
  const uint32_t* r = reinterpret_cast<const uint32_t*>(v);
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ void bf16x8_to_f32(const uint4& q, float* v) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 8 elements [i, i + 8) of a tensor of n; elements behind its end read as 0.
__device__ __forceinline__ void load8(const void* base, bool bf16, bool wide, long long i, long long n, float* v) {
  if (bf16) {
    const uint16_t* p = static_cast<const uint16_t*>(base) + i;
    if (wide && i + 8 <= n) {
      const uint4 q = __ldcs(reinterpret_cast<const uint4*>(p));
      bf16x8_to_f32(q, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = i + e < n ? __uint_as_float(static_cast<uint32_t>(p[e]) << 16) : 0.f;
    }
  } else {
    const float* p = static_cast<const float*>(base) + i;
    if (wide && i + 8 <= n) {
      ld8_f32(p, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = i + e < n ? p[e] : 0.f;
    }
  }
}

__device__ __forceinline__ void store8(void* base, bool bf16, bool wide, long long i, long long n, const float* v) {
  if (bf16) {
    uint16_t* p = static_cast<uint16_t*>(base) + i;
    if (wide && i + 8 <= n) {
      *reinterpret_cast<uint4*>(p) =
          make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (i + e < n) p[e] = static_cast<uint16_t>(pack_bf16(v[e], 0.f) & 0xffffu);
    }
  } else {
    float* p = static_cast<float*>(base) + i;
    if (wide && i + 8 <= n) {
      st8_f32(p, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (i + e < n) p[e] = v[e];
    }
  }
}

// The tensor that holds `block`: the last one with first[t] <= block.
__device__ __forceinline__ int find_tensor(const int* first, int n, int block) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= block)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// ---- 8-bit states
constexpr float kE4m3Max = 448.f;
constexpr float kTinyBlock = 7.888609e-31f;  // 2^-100: a block no larger than this is held as zeros (its scale's
                                             // reciprocal would leave the range of fp32)

// The final mix of MurmurHash3 (Austin Appleby, public domain).
__device__ __forceinline__ uint32_t mix32(uint32_t h) {
  h ^= h >> 16;
  h *= 0x85EBCA6Bu;
  h ^= h >> 13;
  h *= 0xC2B2AE35u;
  return h ^ (h >> 16);
}

__device__ __forceinline__ float e4m3_to_f32(uint32_t code) {
  __nv_fp8_e4m3 c;
  c.__x = static_cast<__nv_fp8_storage_t>(code);
  return static_cast<float>(c);
}

// Two floats to two e4m3 codes, to nearest (ties to even), saturating.
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void unpack_e4m3x8(uint2 q, float scale, float* v) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = e4m3_to_f32((w[i >> 2] >> (8 * (i & 3))) & 0xffu) * scale;
}

__device__ __forceinline__ uint2 pack_e4m3x8(const float* v) {
  uint2 q;
  q.x = pack_e4m3(v[0], v[1]) | (pack_e4m3(v[2], v[3]) << 16);
  q.y = pack_e4m3(v[4], v[5]) | (pack_e4m3(v[6], v[7]) << 16);
  return q;
}

// Largest magnitude of the warp's 256 values.  Magnitudes are compared as
// integers, which orders them as floats do and puts a NaN above all, so a NaN
// reaches the scale instead of vanishing.
__device__ __forceinline__ float warp_absmax(const float* v) {
  uint32_t b = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) b = max(b, __float_as_uint(v[e]) & 0x7fffffffu);
  return __uint_as_float(__reduce_max_sync(kAll, b));
}

// r in [0, 448] up or down to an e4m3 value: up with the probability of the
// rest, by the 20 random bits of h.  e4m3 keeps 3 of fp32's 23 mantissa bits
// in the normal range, so adding 20 random bits below them and cutting carries
// exactly when rest + random >= 1; below 2^-6 the values are 2^-9 apart.  A
// positive r never becomes 0: a second moment of 0 beside a first moment that
// is not would blow the next update up.
__device__ __forceinline__ float stochastic_e4m3(float r, uint32_t h) {
  const uint32_t rnd = h >> 12;
  float q;
  if (r >= 0.015625f) {
    q = __uint_as_float((__float_as_uint(r) + rnd) & 0xfff00000u);
  } else {
    q = floorf(fmaf(r, 512.f, static_cast<float>(rnd) * 9.5367431640625e-7f)) * 0.001953125f;
    if (r > 0.f) q = fmaxf(q, 0.001953125f);
  }
  return r != r ? r : fminf(q, kE4m3Max);
}

}  // namespace

// ============================================================================
// AdamW
// ============================================================================
template <int BITS>
__global__ void __launch_bounds__(32 * kWarps) adamw_kernel(const __grid_constant__ AdamwArgs a) {
  __shared__ float s_step, s_root, s_clip;
  __shared__ uint32_t s_key;
  __shared__ int s_skip;
  if (threadIdx.x == 0) {
    const int t = *reinterpret_cast<volatile int*>(a.control) + 1;
    float clip = 1.f;
    int skip = 0;
    if (a.norm != nullptr) {
      const float norm = *a.norm;
      clip = fminf(1.f, a.max_norm / norm);
      skip = !(norm <= 3.402823466e38f);  // infinity or NaN: the step leaves everything as it is
      if (norm == 0.f) clip = 1.f;
    }
    const float lr = a.lr_dev != nullptr ? *a.lr_dev : a.lr;
    // 1 - b^t = -expm1(t log b) keeps its digits at the first steps
    s_step = lr / -expm1f(static_cast<float>(t) * a.log_beta1);
    s_root = rsqrtf(-expm1f(static_cast<float>(t) * a.log_beta2));
    s_clip = clip;
    s_skip = skip;
    s_key = mix32(static_cast<uint32_t>(t) * 0x9E3779B1u + a.seed);
    // The step counter moves once, by the block that reads it last: every
    // block has its t before it takes a ticket.
    if (a.advance) {
      __threadfence();
      if (atomicAdd(&a.control[1], 1) == static_cast<int>(gridDim.x) - 1) {
        a.control[1] = 0;
        if (!skip) a.control[0] = t;
      }
    }
  }
  __syncthreads();
  if (s_skip) return;
  const float step = s_step, root = s_root, clip = s_clip;
  const float lr = a.lr_dev != nullptr ? *a.lr_dev : a.lr;
  const int lane = threadIdx.x & 31;
  int t = -1;
  int t_end = 0;
  for (int b = blockIdx.x * kWarps + (threadIdx.x >> 5); b < a.blocks; b += gridDim.x * kWarps) {
    if (t < 0 || b >= t_end) {
      t = find_tensor(a.first, a.n, b);
      t_end = t + 1 < a.n ? a.first[t + 1] : a.blocks;
    }
    const AdamwTensor& x = a.t[t];
    const long long i = static_cast<long long>(b - a.first[t]) * kOptBlock + lane * 8;  // in the tensor
    const long long s = x.at + i;                                                       // in the state
    // (the whole warp's block, so that the warp stays together)
    if (!RKL_BOUNDS(i >= lane * 8 && s - lane * 8 + kOptBlock <= a.total && (x.at & (kOptBlock - 1)) == 0)) continue;
    float g[8], m[8], v[8], p[8];
    load8(x.grad, x.flags & OPT_GRAD_BF16, x.flags & OPT_WIDE_GRAD, i, x.n, g);
    float* master = a.master != nullptr ? a.master + s : nullptr;
    if (master != nullptr)
      ld8_f32(master, p);
    else
      load8(x.param, x.flags & OPT_PARAM_BF16, x.flags & OPT_WIDE_PARAM, i, x.n, p);
    const long long q = s / kOptBlock;  // the block's scale
    if (BITS == 32) {
      ld8_f32(static_cast<const float*>(a.m) + s, m);
      ld8_f32(static_cast<const float*>(a.v) + s, v);
    } else {
      const uint2 cm = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.m) + s));
      const uint2 cv = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.v) + s));
      unpack_e4m3x8(cm, a.m_scale[q], m);
      unpack_e4m3x8(cv, a.v_scale[q], v);
    }
    const float keep = 1.f - lr * x.decay;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float ge = g[e] * clip;
      m[e] = fmaf(a.beta1, m[e], a.omb1 * ge);
      v[e] = fmaf(a.beta2, v[e], a.omb2 * ge * ge);
      // square root and quotient by the hardware's approximations (2^-22): the
      // update is lr times smaller than p's own scale, its last bits are lost in p
      float sq;
      asm("sqrt.approx.f32 %0, %1;" : "=f"(sq) : "f"(v[e]));
      p[e] = fmaf(p[e], keep, -__fdividef(step * m[e], fmaf(sq, root, a.eps)));
    }
    if (master != nullptr) st8_f32(master, p);
    store8(x.param, x.flags & OPT_PARAM_BF16, x.flags & OPT_WIDE_PARAM, i, x.n, p);
    if (BITS == 32) {
      st8_f32(static_cast<float*>(a.m) + s, m);
      st8_f32(static_cast<float*>(a.v) + s, v);
    } else {
      const float mm = warp_absmax(m), vm = warp_absmax(v);
      const bool m_some = !(mm <= kTinyBlock), v_some = !(vm <= kTinyBlock);
      const float mi = m_some ? kE4m3Max / mm : 0.f, vi = v_some ? kE4m3Max / vm : 0.f;
      // First moment to the nearest code: b1 leaves each step a tenth of a new
      // value, above the half step of the code.  Second moment stochastically:
      // with b2 = 0.999 a step moves it by less than half a code's step, and to
      // the nearest it would never move at all.
      const uint32_t hi = mix32(s_key + static_cast<uint32_t>(static_cast<unsigned long long>(s) >> 32));
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        m[e] *= mi;
        v[e] = stochastic_e4m3(fminf(v[e] * vi, kE4m3Max), mix32(static_cast<uint32_t>(s + e) ^ hi));
      }
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.m) + s) = pack_e4m3x8(m);
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.v) + s) = pack_e4m3x8(v);
      if (lane == 0) {
        a.m_scale[q] = m_some ? mm / kE4m3Max : 0.f;
        a.v_scale[q] = v_some ? vm / kE4m3Max : 0.f;
      }
    }
  }
}

// ============================================================================
// Global gradient norm
// ============================================================================
// Sum of the squares of 8 values, in 64 bits.  Squares of values outside
// [2^-40, 2^60] leave fp32's range or digits: a lane that holds one (rare)
// squares in 64 bits, the others add 8 squares in fp32 first.  So the norm is
// right for every finite gradient, and infinity or NaN only where one is.
__device__ __forceinline__ double sum_squares(const float* v) {
  float hi = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) hi = fmaxf(hi, fabsf(v[e]));
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) s = fmaf(v[e], v[e], s);
  if (s == 0.f && hi == 0.f) return 0.0;
  if (hi < 1.152921504606847e18f && hi > 9.094947e-13f) return static_cast<double>(s);
  double d = 0.0;
#pragma unroll
  for (int e = 0; e < 8; ++e) d = fma(static_cast<double>(v[e]), static_cast<double>(v[e]), d);
  return d;
}

__device__ __forceinline__ double block_sum(double d) {
  __shared__ double part[kWarps];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(kAll, d, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = d;
  __syncthreads();
  d = 0.0;
  for (int w = 0; w < kWarps; ++w) d += part[w];
  return d;
}

// Each block sums the squares of every gridDim.x-th chunk of kNormChunk
// elements, in a fixed order, into one partial sum: no atomics, so the same
// gradients give the same norm bit for bit.
__global__ void __launch_bounds__(32 * kWarps) norm_partial_kernel(const __grid_constant__ NormArgs a) {
  const int lane = threadIdx.x & 31;
  double sum = 0.0;
  int t = -1, t_end = 0;
  for (int b = blockIdx.x * kWarps + (threadIdx.x >> 5); b < a.chunks; b += gridDim.x * kWarps) {
    if (t < 0 || b >= t_end) {
      t = find_tensor(a.first, a.n, b);
      t_end = t + 1 < a.n ? a.first[t + 1] : a.chunks;
    }
    const NormTensor& x = a.t[t];
    const long long i = static_cast<long long>(b - a.first[t]) * kNormChunk + lane * 8;
    if (!RKL_BOUNDS(i >= 0 && i < x.n + kNormChunk)) continue;
    float v[4][8];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      load8(x.grad, x.flags & OPT_GRAD_BF16, x.flags & OPT_WIDE_GRAD, i + 256 * j, x.n, v[j]);
#pragma unroll
    for (int j = 0; j < 4; ++j) sum += sum_squares(v[j]);
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) a.partial[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(32 * kWarps) norm_final_kernel(const double* partial, int n, float* norm) {
  double sum = 0.0;
  for (int i = threadIdx.x; i < n; i += 32 * kWarps) sum += partial[i];
  sum = block_sum(sum);
  if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(sum));
}

// ============================================================================
// Host launchers
// ============================================================================
cudaError_t launch_adamw(int bits, const AdamwArgs& a, int grid, cudaStream_t s) {
  LaunchScope scope(bits == 8 ? K_ADAMW8 : K_ADAMW, s);
  if (bits == 8)
    adamw_kernel<8><<<grid, 32 * kWarps, 0, s>>>(a);
  else
    adamw_kernel<32><<<grid, 32 * kWarps, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_norm_partial(const NormArgs& a, int grid, cudaStream_t s) {
  LaunchScope scope(K_NORM_PARTIAL, s);
  norm_partial_kernel<<<grid, 32 * kWarps, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_norm_final(const double* partial, int n, float* norm, cudaStream_t s) {
  LaunchScope scope(K_NORM_FINAL, s);
  norm_final_kernel<<<1, 32 * kWarps, 0, s>>>(partial, n, norm);
  return cudaGetLastError();
}

}  // namespace rkl
