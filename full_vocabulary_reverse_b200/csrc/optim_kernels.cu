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
// Every byte is touched once.  The tables of tensors travel in the kernels'
// parameters (up to kOptTensors a launch), so a step needs no copy to the device
// and can be captured in a graph.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

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
constexpr float kLargeV = 16384.f;
constexpr double kLargest = 3.4028234663852886e38;  // of fp32
constexpr double kInfinity = HUGE_VAL;
constexpr float kUlp = 5.9604645e-8f;        // 2^-24
constexpr uint32_t kVNear = 17u << 4;        // fp32's error of v's place between two codes, in 2^-24 of the way

// The final mix of MurmurHash3 (Austin Appleby, public domain).
__device__ __forceinline__ uint32_t mix32(uint32_t h) {
  h ^= h >> 16;
  h *= 0x85EBCA6Bu;
  h ^= h >> 13;
  h *= 0xC2B2AE35u;
  return h ^ (h >> 16);
}

// e4m3 codes to floats (every value is one of fp16 too).
__device__ __forceinline__ void unpack_e4m3x8(uint2 q, float* v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint16_t two = static_cast<uint16_t>(i < 2 ? q.x >> (16 * i) : q.y >> (16 * (i - 2)));
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Element i of a tensor of n.
__device__ __forceinline__ void prefetch_element(const void* base, bool bf16, long long i, long long n) {
  if (RKL_BOUNDS(i < n)) prefetch_l2(static_cast<const char*>(base) + i * (bf16 ? 2 : 4));
}

// Two fp32 values in one register pair, one instruction for both.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 both(uint64_t p) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
  return f;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// The four words' top bytes.
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

// Two floats to two e4m3 codes, to nearest (ties to even), saturating.
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint2 pack_e4m3x8(const float* v) {
  uint2 q;
  q.x = pack_e4m3(v[0], v[1]) | (pack_e4m3(v[2], v[3]) << 16);
  q.y = pack_e4m3(v[4], v[5]) | (pack_e4m3(v[6], v[7]) << 16);
  return q;
}

// Largest of the warp's magnitudes, whose bits are ordered as integers; a NaN
// is above all, so it reaches the scale instead of vanishing.
__device__ __forceinline__ float warp_max_magnitude(float v) {
  return __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(v)));
}

// One element's moments in 64 bits (a block that holds a value too near the
// border of two codes for fp32 to tell takes these; see below).
__device__ __forceinline__ double e4m3_to_f64(uint32_t code) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(code & 0xffu)));
  return static_cast<double>(__half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xffffu))));
}
// Which of a lane's 8 second moments are above 0 by what they are made of, the
// gradients or (where those count) the old codes: 1 in the byte of each.
__device__ __noinline__ uint2 above_zero(const void* grad, uint32_t flags, long long i, long long n, uint2 old, bool kept) {
  float g[8];
  load8(grad, flags & OPT_GRAD_BF16, flags & OPT_WIDE_GRAD, i, n, g);
  uint32_t one[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const bool was = kept && (((e < 4 ? old.x : old.y) >> (8 * (e & 3))) & 0x7f) != 0;
    if (g[e] != 0.f || was) one[e / 4] |= 1u << (8 * (e & 3));
  }
  return make_uint2(one[0], one[1]);
}
struct Exact {
  double beta1, beta2, clip, m_scale, v_scale;
};
__device__ __noinline__ double exact_m(const Exact& x, uint32_t code, float grad) {
  return x.beta1 * (e4m3_to_f64(code) * x.m_scale) + (1 - x.beta1) * (grad * x.clip);
}
__device__ __noinline__ double exact_v(const Exact& x, uint32_t code, float grad) {
  const double g = grad * x.clip;
  return x.beta2 * (e4m3_to_f64(code) * x.v_scale) + (1 - x.beta2) * g * g;
}
// The step between e4m3 values at r >= 0: 2^(exponent - 3), 2^-9 at least.
__device__ __forceinline__ double e4m3_step(double r) {
  const long long exponent = max(__double_as_longlong(r) & 0x7ff0000000000000ll, 0x3f90000000000000ll);
  return __longlong_as_double(exponent - (3ll << 52));
}
// 1 / x of a power of two.
__device__ __forceinline__ double inverse_of(double x) {
  return __longlong_as_double(0x7fe0000000000000ll - __double_as_longlong(x));
}
__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

}  // namespace

// ============================================================================
// AdamW
// ============================================================================
namespace {

// What every block of a launch needs, found by its first thread.
struct StepConsts {
  float step, root, clip, lr;  // lr / (1 - b1^t), 1 / sqrt(1 - b2^t), gradient scale, learning rate
  double clip64;
  uint32_t key;
  int skip;
};

__device__ __forceinline__ void begin_step(const AdamwArgs& a, StepConsts* c) {
  if (threadIdx.x == 0) {
    const int t = *reinterpret_cast<volatile int*>(a.control) + 1;
    double clip = 1;
    int skip = 0;
    if (a.norm != nullptr) {
      const float norm = *a.norm;
      skip = !(norm <= 3.402823466e38f);  // infinity or NaN: the step leaves everything as it is
      if (norm > 0.f) clip = fmin(1.0, a.max_norm / static_cast<double>(norm));
    }
    c->lr = a.lr_dev != nullptr ? *a.lr_dev : a.lr;
    // 1 - b^t = -expm1(t log b) keeps its digits at the first steps
    c->step = c->lr / -expm1f(static_cast<float>(t) * a.log_beta1);
    c->root = rsqrtf(-expm1f(static_cast<float>(t) * a.log_beta2));
    c->clip = static_cast<float>(clip);
    c->clip64 = clip;
    c->skip = skip;
    c->key = mix32(static_cast<uint32_t>(t) * 0x9E3779B1u + a.seed);
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
}

// p from the new moments: square root and quotient by the hardware's
// approximations (2^-22 each; a v below the normal numbers has its root).  The update is lr times smaller than p's own
// scale, its last bits are lost in p.
__device__ __forceinline__ float new_param(float p, float m, float v, float keep, float step, float root, float eps) {
  float sq, inv;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(sq) : "f"(v));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(fmaf(sq, root, eps)));
  return fmaf(p, keep, -(step * m) * inv);
}

}  // namespace

// 32-bit moments.  Bound by memory: 30 bytes an element with bf16 parameters,
// master copies and fp32 gradients, moved at 6.2 TB/s (349 M elements in 1.68
// ms; a plain copy runs at 6.55).
__global__ void __launch_bounds__(32 * kWarps) adamw_kernel(const __grid_constant__ AdamwArgs a) {
  __shared__ StepConsts k;
  begin_step(a, &k);
  if (k.skip) return;
  const float step = k.step, root = k.root, clip = k.clip, lr = k.lr;
  const int lane = threadIdx.x & 31;
  int t = -1, t_end = 0;
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
    ld8_f32(static_cast<const float*>(a.m) + s, m);
    ld8_f32(static_cast<const float*>(a.v) + s, v);
    const float keep = 1.f - lr * x.decay;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float ge = g[e] * clip;
      m[e] = fmaf(a.beta1, m[e], a.omb1 * ge);
      v[e] = fmaf(a.beta2, v[e], a.omb2 * ge * ge);
      p[e] = new_param(p[e], m[e], v[e], keep, step, root, a.eps);
    }
    st8_f32(static_cast<float*>(a.m) + s, m);
    st8_f32(static_cast<float*>(a.v) + s, v);
    if (master != nullptr) st8_f32(master, p);
    store8(x.param, x.flags & OPT_PARAM_BF16, x.flags & OPT_WIDE_PARAM, i, x.n, p);
  }
}

// 8-bit moments: 10 bytes an element with bf16 parameters and gradients.  The
// arithmetic (about 70 instructions an element, most of them the codes' and the
// random numbers') and the waits of 24 warps an SM set the time, not memory: 349 M
// elements take 1.0 to 1.35 ms, by how many blocks look again in 64 bits (2 in 100
// on changing gradients, about 15 where the gradient stays the same and moments
// stop next to borders).
// Paired fp32 instructions took 10 % of the instructions away; 24 warps an SM
// with the next block's lines on their way to L2 ran faster than 16 or 32 (80
// registers a thread; the second look spills 20 bytes).
//
// Beside the codes, fp32 arithmetic finds the values that lie within its error
// of a border between two codes; their block then looks at those again in 64
// bits.  So a step's codes are the 64-bit formula's of the state that it finds.
// (Its scales are the rounded quotients of the fp32 largest, within 8 u of the
// terms off the formula's: over many steps a few codes next to borders part from
// a computation in 64 bits throughout.)  With u = 2^-24, r = value 448 / largest:
//   m: off by 5 u t, t = |b1 m| + |(1 - b1) g|, whatever cancels in it; the
//      block's largest by 5 u of its own t; r by 2 u more: below
//      t 448 / largest u (7 + 5 W), W the block's largest t over the largest.
//   v: all terms are positive, 7 u; the largest as much, r 2 u more: 16 u of r,
//      and a code's step is r / 16 at least.  Below fp32's normal numbers a term
//      is off by up to 2^-149, that is 2^-40 of r in a block that has a scale (16
//      u of the smallest code's step are 2^-29); whether v is above 0 is then
//      asked of what it is made of: where a code came out as 0, which blocks of
//      moments near each other do not have (blocks that hold moments of 0 beside
//      others take 15 % longer for it; a look at every gradient would take 3 %
//      everywhere).
__global__ void __launch_bounds__(32 * kWarps, 3) adamw8_kernel(const __grid_constant__ AdamwArgs a) {
  __shared__ StepConsts k;
  begin_step(a, &k);
  if (k.skip) return;
  const float step = k.step, root = k.root, clip = k.clip, lr = k.lr;
  const uint32_t key = k.key;
  const int lane = threadIdx.x & 31;
  int t = -1, t_end = 0;
  for (int b = blockIdx.x * kWarps + (threadIdx.x >> 5); b < a.blocks; b += gridDim.x * kWarps) {
    if (t < 0 || b >= t_end) {
      t = find_tensor(a.first, a.n, b);
      t_end = t + 1 < a.n ? a.first[t + 1] : a.blocks;
    }
    const AdamwTensor& x = a.t[t];
    const long long i = static_cast<long long>(b - a.first[t]) * kOptBlock + lane * 8;  // in the tensor
    const long long s = x.at + i;                                                       // in the state
    if (!RKL_BOUNDS(i >= lane * 8 && s - lane * 8 + kOptBlock <= a.total && (x.at & (kOptBlock - 1)) == 0)) continue;
    const long long q = s / kOptBlock;  // the block's scale
    uint2* cm = reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.m) + s);
    uint2* cv = reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.v) + s);
    const uint2 om = __ldcs(cm), ov = __ldcs(cv);
    // The next block's lines start on their way to L2: with 24 warps an SM the
    // wait for memory showed otherwise.  (A lane whose elements lie behind the
    // tensor's end, in its last block, has nothing to fetch.)
    const long long far_on = static_cast<long long>(gridDim.x) * kWarps * kOptBlock;
    if (i + far_on < x.n) {
      prefetch_l2(cm + far_on / 8);
      prefetch_l2(cv + far_on / 8);
      prefetch_element(x.grad, x.flags & OPT_GRAD_BF16, i + far_on, x.n);
      if (a.master != nullptr)
        prefetch_l2(a.master + s + far_on);
      else
        prefetch_element(x.param, x.flags & OPT_PARAM_BF16, i + far_on, x.n);
    }
    const float ms = a.m_scale[q], vs = a.v_scale[q];
    uint64_t m[4], v[4], term[4];  // neighbouring elements in pairs
    float m_top = 0.f, v_top = 0.f, term_top = 0.f;
    {
      float g[8], p[8], mc[8], vc[8];
      load8(x.grad, x.flags & OPT_GRAD_BF16, x.flags & OPT_WIDE_GRAD, i, x.n, g);
      float* master = a.master != nullptr ? a.master + s : nullptr;
      if (master != nullptr)
        ld8_f32(master, p);
      else
        load8(x.param, x.flags & OPT_PARAM_BF16, x.flags & OPT_WIDE_PARAM, i, x.n, p);
      unpack_e4m3x8(om, mc);
      unpack_e4m3x8(ov, vc);
      const float keep = 1.f - lr * x.decay, mk = a.beta1 * ms, vk = a.beta2 * vs;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint64_t ge = mul2(pair(g[2 * e], g[2 * e + 1]), pair(clip, clip));
        const uint64_t m1 = mul2(pair(mc[2 * e], mc[2 * e + 1]), pair(mk, mk)), m2 = mul2(ge, pair(a.omb1, a.omb1));
        m[e] = add2(m1, m2);
        const float2 h1 = both(m1), h2 = both(m2), mf = both(m[e]);
        const float t0 = fabsf(h1.x) + fabsf(h2.x), t1 = fabsf(h1.y) + fabsf(h2.y);
        term[e] = pair(t0, t1);
        v[e] = fma2(mul2(ge, pair(a.omb2, a.omb2)), ge, mul2(pair(vc[2 * e], vc[2 * e + 1]), pair(vk, vk)));
        const float2 vf = both(v[e]);
        // (as new_param does; a v below the normal numbers counts as 0, which eps is above)
        float q0, q1, r0, r1;
        asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(q0) : "f"(vf.x));
        asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(q1) : "f"(vf.y));
        const float2 den = both(fma2(pair(q0, q1), pair(root, root), pair(a.eps, a.eps)));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(den.x));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(den.y));
        const uint64_t change = mul2(mul2(m[e], pair(-step, -step)), pair(r0, r1));
        const float2 pf = both(fma2(pair(p[2 * e], p[2 * e + 1]), pair(keep, keep), change));
        p[2 * e] = pf.x;
        p[2 * e + 1] = pf.y;
        m_top = max3_nan(m_top, fabsf(mf.x), fabsf(mf.y));
        v_top = max3_nan(v_top, vf.x, vf.y);
        term_top = max3_nan(term_top, t0, t1);
      }
      if (master != nullptr) st8_f32(master, p);
      store8(x.param, x.flags & OPT_PARAM_BF16, x.flags & OPT_WIDE_PARAM, i, x.n, p);
    }
    const float mm = warp_max_magnitude(m_top), vm = warp_max_magnitude(v_top), tm = warp_max_magnitude(term_top);
    const bool m_some = !(mm <= kTinyBlock), v_some = !(vm <= kTinyBlock);
    // Both scales (lanes 2 and 3 of every 4) and their reciprocals (0 and 1) in
    // one division: alone, each took 1.4 % of the step.
    const float top = lane & 1 ? vm : mm;
    const float quotient = __fdiv_rn(lane & 2 ? top : kE4m3Max, lane & 2 ? kE4m3Max : top);
    const float mi = m_some ? __shfl_sync(kAll, quotient, 0) : 0.f, vi = v_some ? __shfl_sync(kAll, quotient, 1) : 0.f;
    const bool far = vm > kLargeV;  // vi 2^-120 leaves fp32's normal range: all of v in 64 bits
    const float vi120 = vi * 7.52316384526264e-37f;
    // First moment to the nearest code: b1 leaves each step a tenth of a new
    // value, above the half step of the code.  Second moment stochastically:
    // with b2 = 0.999 a step moves it by less than half a code's step, and to
    // the nearest it would never move at all.
    const float w = tm * mi * (1.f / kE4m3Max);
    const float off = mi * kUlp * fmaf(5.f, w, 7.f);
    const uint32_t place =
        static_cast<uint32_t>(s) ^ mix32(key + static_cast<uint32_t>(static_cast<unsigned long long>(s) >> 32));
    // By how much two |m| lie in fp32's error of the border next to them (above
    // 0: they do): distance to the code plus error less half the code's step.
    // The step is 2^-3 of 2^exponent (that of the smallest normal code at least);
    // adding 1.5 x 2^20 times 2^exponent rounds to a multiple of it.
    auto in_reach = [&](uint64_t me, uint64_t te) {
      const float2 r = both(me);
      const uint64_t top = pair(fmaxf(__uint_as_float(__float_as_uint(r.x) & 0x7f800000u), 0.015625f),
                                fmaxf(__uint_as_float(__float_as_uint(r.y) & 0x7f800000u), 0.015625f));
      const uint64_t code = fma2(top, pair(-1572864.f, -1572864.f), fma2(top, pair(1572864.f, 1572864.f), me));
      const float2 rest = both(fma2(code, pair(-1.f, -1.f), me));
      const float2 room = both(fma2(te, pair(off, off), mul2(top, pair(-0.0625f, -0.0625f))));
      return make_float2(fabsf(rest.x) + room.x, fabsf(rest.y) + room.y);
    };
    // r 2^-120 has e4m3's exponent and mantissa above 20 more bits; 16 times
    // them the code is the top byte, and adding 24 random bits (20 and 4 that
    // cannot matter) carries into it exactly when rest + random >= 1.
    auto raised = [&](float r120, int e) {
      const uint32_t h = mix32(place ^ static_cast<uint32_t>(e));
      return __float_as_uint(r120) * 16u + (h >> 8);
    };
    auto v_window = [](uint32_t y) { return y * 256u + (kVNear << 8); };  // below 2 kVNear << 8: next to a border
    float reach = -1.f;
    uint32_t nearest_v = 0xffffffffu, y[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      m[e] = mul2(m[e], pair(mi, mi));
      const float2 d = in_reach(m[e], term[e]);
      reach = max3_nan(reach, d.x, d.y);
      const float2 r120 = both(mul2(v[e], pair(vi120, vi120)));
      y[2 * e] = raised(r120.x, 2 * e);
      y[2 * e + 1] = raised(r120.y, 2 * e + 1);
      // (the largest value's carry out of the last code is next to a border)
      nearest_v = min(min(nearest_v, v_window(y[2 * e])), v_window(y[2 * e + 1]));
    }
    float mq[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = both(m[e]);
      mq[2 * e] = f.x;
      mq[2 * e + 1] = f.y;
    }
    uint2 code_v = make_uint2(top_bytes(y[0], y[1], y[2], y[3]), top_bytes(y[4], y[5], y[6], y[7]));
    // Codes of 0: bytes are at most 0x7e, adding 0x7f reaches a byte's top bit from 1 on.
    const bool zero = ((code_v.x + 0x7f7f7f7fu) & (code_v.y + 0x7f7f7f7fu) & 0x80808080u) != 0x80808080u && v_some;
    // (one vote where, as mostly, there is nothing to look at again)
    if (far || __any_sync(kAll, (!(reach < 0.f) && m_some) || nearest_v < (kVNear << 9) || zero)) {
      const bool near_m = __any_sync(kAll, !(reach < 0.f)) && m_some;
      const bool near_v = far || __any_sync(kAll, nearest_v < (kVNear << 9));
      if (near_m || near_v) {
        const Exact z{a.beta1_64, a.beta2_64, k.clip64, ms, vs};
        float g[8];
        load8(x.grad, x.flags & OPT_GRAD_BF16, x.flags & OPT_WIDE_GRAD, i, x.n, g);
        if (near_m) {
          double most = 0;  // among those that may be the largest
          const float least_r = kE4m3Max * fmaf(w, -16.f * kUlp, 1.f);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (!(fabsf(mq[e]) < least_r)) most = fmax(most, fabs(exact_m(z, (e < 4 ? om.x : om.y) >> (8 * (e & 3)), g[e])));
          most = warp_max(most);
          const double inv = 448.0 / most;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 d = in_reach(m[e / 2], term[e / 2]);
            if (!((e & 1 ? d.y : d.x) < 0.f)) {
              const double r = exact_m(z, (e < 4 ? om.x : om.y) >> (8 * (e & 3)), g[e]) * inv;
              const double gap = e4m3_step(fabs(r));
              mq[e] = static_cast<float>(rint(r * inverse_of(gap)) * gap);
            }
          }
        }
        if (near_v) {
          double most = 0;
          const float least_v = far ? 0.f : vm * (1.f - 32.f * kUlp);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 vf = both(v[e / 2]);
            if (!((e & 1 ? vf.y : vf.x) < least_v)) most = fmax(most, exact_v(z, (e < 4 ? ov.x : ov.y) >> (8 * (e & 3)), g[e]));
          }
          most = warp_max(most);
          if (far) {  // in 64 bits too: vm may be infinite where the scale is not
            if (most < kInfinity) most = fmin(most, 448.0 * kLargest);
            if (lane == 0) a.v_scale[q] = static_cast<float>(most / 448.0);
          }
          const double inv = v_some ? 448.0 / most : 0.0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 r120 = both(mul2(v[e / 2], pair(vi120, vi120)));
            if (far || v_window(raised(e & 1 ? r120.y : r120.x, e)) < (kVNear << 9)) {
              const double r = exact_v(z, (e < 4 ? ov.x : ov.y) >> (8 * (e & 3)), g[e]) * inv;
              const double gap = e4m3_step(r);
              const double up =
                  floor(r * inverse_of(gap) + (mix32(place ^ static_cast<uint32_t>(e)) >> 12) * 9.5367431640625e-7) * gap;
              const uint32_t code = __float_as_uint(static_cast<float>(up) * 7.52316384526264e-37f) >> 20;
              y[e] = min(max(code, r > 0 ? 1u : 0u), 126u) << 24;
            }
          }
        }
      }
      if (near_v) code_v = make_uint2(top_bytes(y[0], y[1], y[2], y[3]), top_bytes(y[4], y[5], y[6], y[7]));
      // Codes of 0, rare but where a moment is 0: not from above it, in fp32 or
      // not.  A second moment of 0 beside a first moment that is not would blow
      // the next update up.
      if (__any_sync(kAll, zero)) {
        const uint2 one = above_zero(x.grad, x.flags, i, x.n, ov, a.beta2_64 > 0 && vs > 0.f);
        code_v.x |= one.x & ~((code_v.x + 0x7f7f7f7fu) >> 7);
        code_v.y |= one.y & ~((code_v.y + 0x7f7f7f7fu) >> 7);
      }
    }
    *cv = code_v;
    *cm = pack_e4m3x8(mq);
    if (lane == 2) a.m_scale[q] = m_some ? quotient : 0.f;
    if (lane == 3 && !far) a.v_scale[q] = v_some ? quotient : 0.f;
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
// gradients give the same norm bit for bit.  Bound by memory: 349 M bf16
// elements in 105 us, 6.6 TB/s.
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
    // A chunk inside the tensor: all its loads are in flight before the first
    // sum (behind a test each they went one by one, at 3.7 TB/s).
    if ((x.flags & OPT_WIDE_GRAD) && i - lane * 8 + kNormChunk <= x.n) {
      if (x.flags & OPT_GRAD_BF16) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x.grad) + i);
        uint4 q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = __ldcs(p + 32 * j);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float v[8];
          bf16x8_to_f32(q[j], v);
          sum += sum_squares(v);
        }
      } else {
        const float* p = static_cast<const float*>(x.grad) + i;
        float v[4][8];
#pragma unroll
        for (int j = 0; j < 4; ++j) ld8_f32(p + 256 * j, v[j]);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum += sum_squares(v[j]);
      }
      continue;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[8];
      load8(x.grad, x.flags & OPT_GRAD_BF16, x.flags & OPT_WIDE_GRAD, i + 256 * j, x.n, v);
      sum += sum_squares(v);
    }
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
    adamw8_kernel<<<grid, 32 * kWarps, 0, s>>>(a);
  else
    adamw_kernel<<<grid, 32 * kWarps, 0, s>>>(a);
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
