// api.cu -- the C ABI of librkl.so (declared in include/rkl.h).
//
// Argument validation, workspace layout, TMA descriptor encoding, per-device
// one-time setup and the launch sequence of each entry point.  Every numeric
// step runs in the kernels of tc_kernels.cu / small_kernels.cu /
// simt_kernels.cu; nothing here touches tensor data on the host.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>
#include <vector>

#include <nvtx3/nvToolsExt.h>

#include "rkl.h"
#include "ffn_act.cuh"
#include "kernels.h"

namespace rkl {

// An NVTX range over one C-ABI call, named after the entry point.  Profilers
// that listen to NVTX (Nsight Systems, Nsight Compute's range filters) show
// each call with its kernels under it; without one attached a push/pop costs
// a few nanoseconds.
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};
#define RKL_NVTX_RANGE() ::rkl::NvtxRange rkl_nvtx_range_(__func__)

// ------------------------------------------------------------------ errors
static thread_local std::string g_last_error;

static rkl_status fail(rkl_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return s;
}

#define RKL_CUDA(call)                                                                          \
  do {                                                                                          \
    cudaError_t e__ = (call);                                                                   \
    if (e__ != cudaSuccess) return fail(RKL_ERR_CUDA, "%s: %s", #call, cudaGetErrorString(e__)); \
  } while (0)

// ------------------------------------------------------------------ profiling
static const char* const kKernelNames[K_COUNT] = {
    "compact_rows", "gather_rows",   "fwd_dual_tc",  "fwd_single_tc", "teacher_lse", "combine_splits",
    "scatter_loss", "reduce_loss",   "row_weights",  "dz_dual_tc",    "dz_single_tc", "grad_dw_dh_tc",
    "scatter_dh",   "fwd_simt_fp32", "dz_simt_fp32", "grad_simt_fp32", "pair_fwd",   "pair_bwd",
    "count_teachers", "build_slots", "topk_fwd", "topk_bwd", "zw_dual_tc", "dz_topk_tc", "topk_rowk",
    "zw_single_tc", "dz_topk_single_tc", "adamw", "adamw8", "norm_partial", "norm_final",
    "ffn_up_simt", "ffn_dgate_simt", "ffn_gemm_simt", "ffn_up_tc", "ffn_dgate_tc", "ffn_gemm_tc", "ffn_skinny_tc",
    "ffn_join", "ffn_pad"};

const char* kernel_name(int id) { return (id >= 0 && id < K_COUNT) ? kKernelNames[id] : nullptr; }

struct ProfRec {
  int id;
  cudaEvent_t a, b;
};
static std::mutex g_prof_mu;
static std::atomic<bool> g_profile{false};
static std::atomic<long long> g_launches{0};
static std::vector<ProfRec> g_prof_pending;
static double g_prof_ms[K_COUNT];
static long long g_prof_n[K_COUNT];

LaunchScope::LaunchScope(int id_, cudaStream_t s) : id(id_), stream(s) {
  g_launches.fetch_add(1);
  if (g_profile.load()) {
    if (cudaEventCreate(&ev0) == cudaSuccess && cudaEventCreate(&ev1) == cudaSuccess) {
      cudaEventRecord(ev0, s);
    } else {
      ev0 = ev1 = nullptr;
    }
  }
}

LaunchScope::~LaunchScope() {
  if (ev0 && ev1) {
    cudaEventRecord(ev1, stream);
    std::lock_guard<std::mutex> lk(g_prof_mu);
    g_prof_pending.push_back({id, ev0, ev1});
  }
}

// ------------------------------------------------------------------ devices
struct DevState {
  int sms = 0;
  unsigned long long ready[8] = {};  // the last contexts that the kernels' attributes were set in (0: none)
  int next = 0;
};
static std::mutex g_dev_mu;
static DevState g_devs[64];

// A function of the driver by its name; nullptr where there is none.
static void* driver_entry(const char* name) {
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  const bool found = cudaGetDriverEntryPoint(name, &p, cudaEnableDefault, &q) == cudaSuccess;
  return found && q == cudaDriverEntryPointSuccess ? p : nullptr;
}

// The current context's number.  A thread that has made no runtime call yet
// (autograd's backward thread) has no current context, which encoding a tensor
// map needs: it gets the device's own.  Another one that the caller has made
// current stays so.
static cudaError_t need_context(int dev, unsigned long long* id) {
  typedef CUresult (*GetCurrentFn)(CUcontext*);
  typedef CUresult (*GetIdFn)(CUcontext, unsigned long long*);
  static const GetCurrentFn get = reinterpret_cast<GetCurrentFn>(driver_entry("cuCtxGetCurrent"));
  static const GetIdFn number = reinterpret_cast<GetIdFn>(driver_entry("cuCtxGetId"));
  if (get == nullptr || number == nullptr) return cudaErrorNotSupported;
  CUcontext current = nullptr;
  if (get(&current) != CUDA_SUCCESS || current == nullptr) {
    const cudaError_t e = cudaSetDevice(dev);
    if (e != cudaSuccess) return e;
    if (get(&current) != CUDA_SUCCESS) return cudaErrorDeviceUninitialized;
  }
  if (number(current, id) != CUDA_SUCCESS) return cudaErrorDeviceUninitialized;
  ++*id;  // (above 0)
  return cudaSuccess;
}

static rkl_status device_setup(int* sms) {
  int dev = 0;
  unsigned long long context = 0;
  RKL_CUDA(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return fail(RKL_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
  RKL_CUDA(need_context(dev, &context));
  std::lock_guard<std::mutex> lk(g_dev_mu);
  DevState& d = g_devs[dev];
  if (std::find(d.ready, d.ready + 8, context) == d.ready + 8) {
    int major = 0, minor = 0;
    RKL_CUDA(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev));
    RKL_CUDA(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev));
    if (major != 10 || minor != 0)
      return fail(RKL_ERR_UNSUPPORTED, "device %d is sm_%d%d; this library is built for sm_100a (B200)", dev, major,
                  minor);
    int count = 0;
    RKL_CUDA(cudaDeviceGetAttribute(&count, cudaDevAttrMultiProcessorCount, dev));
    RKL_CUDA(tc_setup(dev));
    RKL_CUDA(ffn_tc_setup());
    d.sms = count;
    d.ready[d.next] = context;
    d.next = (d.next + 1) % 8;
  }
  *sms = d.sms;
  return RKL_OK;
}

// ------------------------------------------------------------------ TMA maps
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = reinterpret_cast<EncodeTiledFn>(driver_entry("cuTensorMapEncodeTiled"));
  return fn;
}

// 2-D row-major map: `inner` contiguous elements per row, `outer` rows,
// `pitch` bytes between rows; out-of-bounds reads give 0.
static rkl_status make_map(CUtensorMap* m, const void* ptr, bool f32, uint64_t inner, uint64_t outer,
                           uint64_t pitch, uint32_t box_inner, uint32_t box_outer,
                           CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(RKL_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {pitch};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                  const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(RKL_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d) for %llux%llu pitch %llu box %ux%u", (int)r,
                (unsigned long long)inner, (unsigned long long)outer, (unsigned long long)pitch, box_inner,
                box_outer);
  return RKL_OK;
}

// ------------------------------------------------------------------ plan
constexpr int kVcBf16 = 65536;  // widest vocab chunk of the backward (multiple of kFBN)
constexpr int kVcF32 = 1024;
constexpr int kSimtSplits = 37;

struct Plan {
  int n_pad = 0, es = 2, S = 1, VT = 1, Vc = 0, nchunks = 1;
  size_t off_hcs = 0, off_hct = 0, off_part = 0, off_rowc = 0, off_lse = 0, off_dz = 0, off_dh = 0, off_cnt = 0,
         off_slot = 0, off_kslot = 0, off_rowk = 0, off_z = 0, total = 0;
  int zrows = 0;      // top-k, hidden payload: rows of a logit block
  long long zpitch = 0;  // its row pitch (floats)
};

constexpr int kTopkBlockRows = 2048;  // top-k, hidden payload: rows whose logits are written at a time

static size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Workspace layout.  S = number of partial-statistics groups of the forward:
// groups of kGroupTiles vocab tiles on the tensor-core path, kSimtSplits
// vocab splits on the fp32 path -- both depend on V only.  With a teacher per
// row (n_teachers > 1) the rows are regrouped by teacher into whole 256-row
// tiles: sum_g ceil(n_g / 256) <= ceil(N / 256) + n_teachers - 1 tiles, plus
// the slot maps.
static Plan make_plan(rkl_payload payload, rkl_dtype dtype, int64_t n_max, int64_t H, int64_t V,
                      int n_teachers = 1) {
  Plan p;
  const bool bf16 = dtype == RKL_BF16;
  const int tile_v = bf16 ? kFBN : kSimtBN;
  p.es = bf16 ? 2 : 4;
  const int64_t n = n_max < 1 ? 1 : n_max;
  p.n_pad = static_cast<int>(((n + 2 * kBM - 1) / (2 * kBM)) * (2 * kBM));  // whole 256-row pair tiles
  if (n_teachers > 1) p.n_pad += 2 * kBM * (n_teachers - 1);
  p.VT = static_cast<int>((V + tile_v - 1) / tile_v);
  // tensor-core path: fwd_slots statistics slots (column parts) per group of
  // the forward kernel of this payload (two GEMMs on the hidden payloads)
  const int ng = (payload == RKL_PAYLOAD_HIDDEN || payload == RKL_PAYLOAD_TOPK_HIDDEN) ? 2 : 1;
  p.S = bf16 ? fwd_slots(ng) * ((p.VT + kGroupTiles - 1) / kGroupTiles) : (p.VT < kSimtSplits ? p.VT : kSimtSplits);
  // Backward vocab chunks: as few as the widest chunk allows, of equal width
  // (a multiple of the 256-column tile), so that every gradient launch has the
  // same work and the tails of the persistent kernels are paid few times.
  const int vc = bf16 ? kVcBf16 : kVcF32;
  const int64_t vround = ((V + kFBN - 1) / kFBN) * kFBN;
  if (bf16) {
    const int64_t nch = (vround + vc - 1) / vc;
    const int64_t w = (vround + nch - 1) / nch;
    p.Vc = static_cast<int>(((w + kFBN - 1) / kFBN) * kFBN);
  } else {
    p.Vc = static_cast<int>(vround < vc ? vround : vc);
  }
  p.nchunks = static_cast<int>((V + p.Vc - 1) / p.Vc);
  size_t off = 256;  // header
  p.off_hcs = off;
  off = align256(off + size_t(p.n_pad) * H * p.es);
  p.off_hct = off;
  if (payload == RKL_PAYLOAD_HIDDEN || payload == RKL_PAYLOAD_TOPK_HIDDEN)
    off = align256(off + size_t(p.n_pad) * H * p.es);
  p.off_part = off;
  off = align256(off + size_t(p.S) * kStatVals * p.n_pad * sizeof(float));
  p.off_rowc = off;
  off = align256(off + size_t(3) * p.n_pad * sizeof(float));
  p.off_lse = off;
  off = align256(off + size_t(p.n_pad) * sizeof(float));
  p.off_dz = off;
  off = align256(off + size_t(p.n_pad) * p.Vc * p.es);
  p.off_dh = off;
  off = align256(off + size_t(p.n_pad) * H * sizeof(float));
  p.off_cnt = off;
  off = align256(off + size_t(p.nchunks) * sizeof(int));
  if (n_teachers > 1) {
    p.off_slot = off;
    off = align256(off + size_t(p.n_pad) * sizeof(int32_t));
    p.off_kslot = off;
    off = align256(off + size_t(n) * sizeof(int32_t));
  }
  if (payload == RKL_PAYLOAD_TOPK_HIDDEN || payload == RKL_PAYLOAD_TOPK_LOGITS) {
    // per-row constants of the top-k dz pass, and the fp32 z_s (hidden
    // payload: and z_t) of one block of rows: never more than
    // kTopkBlockRows rows of logits at a time.  The teacher-logits payload
    // selects against the shipped bf16 teacher rows directly.
    p.off_rowk = off;
    off = align256(off + size_t(6) * p.n_pad * sizeof(float));
    p.zrows = p.n_pad < kTopkBlockRows ? p.n_pad : kTopkBlockRows;
    p.zpitch = ((V + 3) / 4) * 4;
    p.off_z = off;
    const size_t zblocks = payload == RKL_PAYLOAD_TOPK_HIDDEN ? 2 : 1;
    off = align256(off + zblocks * p.zrows * p.zpitch * sizeof(float));
  }
  p.total = off;
  return p;
}

// Teacher-grouped row layout of the per-row-teacher mode (host side).
struct MultiTeacher {
  int n = 0;                         // teachers (> 1)
  const int32_t* teacher_idx = nullptr;  // [B, Sm1] device
  const void* W_t = nullptr;         // stacked heads [n, V, H]
  TeacherSlots ts{};
  int n_rows = 0;                    // slots in use (sum of 256-rounded counts)
  int group_row_end[kMaxTeachers] = {};
};

static rkl_status make_multi(int n_teachers, const int32_t* teacher_idx, const int32_t* counts, int32_t N,
                             MultiTeacher* mt) {
  if (n_teachers < 1 || n_teachers > kMaxTeachers)
    return fail(RKL_ERR_SHAPE, "n_teachers = %d outside [1, %d]", n_teachers, kMaxTeachers);
  if (teacher_idx == nullptr || counts == nullptr) return fail(RKL_ERR_NULL, "teacher_idx and counts must be non-NULL");
  if ((reinterpret_cast<uintptr_t>(teacher_idx) & 15) != 0)
    return fail(RKL_ERR_ALIGN, "teacher_idx is not 16-byte aligned");
  mt->n = n_teachers;
  mt->teacher_idx = teacher_idx;
  mt->ts.n = n_teachers;
  long long sum = 0;
  int base = 0;
  for (int g = 0; g < n_teachers; ++g) {
    if (counts[g] < 0) return fail(RKL_ERR_SHAPE, "counts[%d] = %d is negative", g, counts[g]);
    sum += counts[g];
    mt->ts.count[g] = counts[g];
    mt->ts.base[g] = base;
    if (sum > N) break;
    base += ((counts[g] + 2 * kBM - 1) / (2 * kBM)) * (2 * kBM);
    mt->group_row_end[g] = base;
  }
  if (sum != N)
    return fail(RKL_ERR_SHAPE,
                "per-teacher counts add up to %lld but N = %d (a trainable row has a teacher index outside "
                "[0, n_teachers), or the counts belong to another mask)",
                sum, N);
  mt->n_rows = base;
  return RKL_OK;
}

// ------------------------------------------------------------------ checks
static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

static rkl_status check_common(rkl_payload payload, rkl_dtype dtype, int64_t B, int64_t Sm1, int64_t H, int64_t V,
                               int32_t N, int reduction) {
  if (dtype != RKL_BF16 && dtype != RKL_FP32) return fail(RKL_ERR_DTYPE, "unknown dtype %d", (int)dtype);
  if (payload != RKL_PAYLOAD_HIDDEN && payload != RKL_PAYLOAD_LOGITS && payload != RKL_PAYLOAD_LOGITS_PAIR &&
      payload != RKL_PAYLOAD_TOPK_HIDDEN && payload != RKL_PAYLOAD_TOPK_LOGITS)
    return fail(RKL_ERR_DTYPE, "unknown payload %d", (int)payload);
  if (payload == RKL_PAYLOAD_LOGITS_PAIR) H = 64;  // no hidden dimension in this mode
  if (reduction < 0 || reduction > 2) return fail(RKL_ERR_DTYPE, "unknown reduction %d", reduction);
  if (B < 1 || Sm1 < 1 || H < 1 || V < 1) return fail(RKL_ERR_SHAPE, "B, Sm1, H, V must be >= 1");
  if (B * Sm1 >= (int64_t(1) << 31)) return fail(RKL_ERR_SHAPE, "B*Sm1 = %lld exceeds 2^31-1", (long long)(B * Sm1));
  if (H > 65536) return fail(RKL_ERR_SHAPE, "H = %lld exceeds 65536", (long long)H);
  if (V >= (int64_t(1) << 30)) return fail(RKL_ERR_SHAPE, "V = %lld too large", (long long)V);
  if (N < 0 || N > B * Sm1) return fail(RKL_ERR_SHAPE, "N = %d outside [0, B*Sm1]", N);
  if (dtype == RKL_BF16) {
    if (H % 64 != 0) return fail(RKL_ERR_SHAPE, "bf16 requires H %% 64 == 0 (H = %lld)", (long long)H);
    if ((payload == RKL_PAYLOAD_LOGITS || payload == RKL_PAYLOAD_TOPK_LOGITS) && V % 8 != 0)
      return fail(RKL_ERR_SHAPE, "bf16 logits payload requires V %% 8 == 0 (V = %lld)", (long long)V);
  }
  return RKL_OK;
}

static rkl_status check_ptr(const void* p, const char* name, bool required = true) {
  if (p == nullptr) return required ? fail(RKL_ERR_NULL, "%s is NULL", name) : RKL_OK;
  if (!aligned16(p)) return fail(RKL_ERR_ALIGN, "%s is not 16-byte aligned", name);
  return RKL_OK;
}

// Element counts of the tensors of an optimizer step or a gradient norm.
static rkl_status check_tensor_counts(int32_t n, const int64_t* numel) {
  if (n < 0) return fail(RKL_ERR_SHAPE, "n = %d is negative", n);
  if (n > 0 && numel == nullptr) return fail(RKL_ERR_NULL, "numel is NULL");
  for (int32_t i = 0; i < n; ++i)
    if (numel[i] < 0 || numel[i] >= (int64_t(1) << 37))
      return fail(RKL_ERR_SHAPE, "tensor %d has %lld elements", i, (long long)numel[i]);
  return RKL_OK;
}

// Whether 8 consecutive elements can move as one access a lane.
static bool wide_access(const void* p, int32_t dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (dtype == RKL_BF16 ? 15 : 31)) == 0;
}

// The optional device row count: one int32, 4-byte aligned.
static rkl_status check_n_dev(const int32_t* n_dev) {
  if (n_dev != nullptr && (reinterpret_cast<uintptr_t>(n_dev) & 3) != 0)
    return fail(RKL_ERR_ALIGN, "n_dev is not 4-byte aligned");
  return RKL_OK;
}

#define RKL_TRY(x)                   \
  do {                               \
    rkl_status s__ = (x);            \
    if (s__ != RKL_OK) return s__;   \
  } while (0)

static uint8_t* ws_at(void* ws, size_t off) { return static_cast<uint8_t*>(ws) + off; }

// ------------------------------------------------------------------ forward
static rkl_status forward_impl(rkl_payload payload, const void* h_s, const void* teacher, const void* W_s,
                               const void* W_t, rkl_dtype dtype, int64_t B, int64_t Sm1, int64_t H, int64_t V,
                               const int32_t* row_idx, int32_t N, const int32_t* n_dev, rkl_reduction reduction,
                               float* loss_tok, float* loss, float* saved, void* workspace, size_t workspace_bytes,
                               void* stream_, bool forward_only_workspace = false, const int32_t* targets = nullptr,
                               float* entropy = nullptr, float* target_logprob = nullptr,
                               const MultiTeacher* mt = nullptr) {
  RKL_TRY(check_common(payload, dtype, B, Sm1, H, V, N, reduction));
  RKL_TRY(check_n_dev(n_dev));
  if (mt && n_dev)
    return fail(RKL_ERR_UNSUPPORTED, "a teacher per row needs the per-teacher counts on the host (n_dev must be NULL)");
  RKL_TRY(check_ptr(h_s, "h_s"));
  RKL_TRY(check_ptr(teacher, payload == RKL_PAYLOAD_HIDDEN ? "h_t" : "teacher_logits"));
  RKL_TRY(check_ptr(W_s, "W_s"));
  if (payload == RKL_PAYLOAD_HIDDEN) RKL_TRY(check_ptr(W_t, "W_t"));
  RKL_TRY(check_ptr(row_idx, "row_idx"));
  RKL_TRY(check_ptr(loss_tok, "loss_tok", false));
  RKL_TRY(check_ptr(loss, "loss", false));
  RKL_TRY(check_ptr(saved, "saved", N > 0));
  RKL_TRY(check_ptr(workspace, "workspace"));
  RKL_TRY(check_ptr(targets, "targets", false));
  RKL_TRY(check_ptr(entropy, "entropy", false));
  RKL_TRY(check_ptr(target_logprob, "target_logprob", false));
  if (target_logprob && !targets) return fail(RKL_ERR_NULL, "target_logprob needs targets");
  const Plan pl = make_plan(payload, dtype, N, H, V, mt ? mt->n : 1);
  // The forward touches only the regions in front of the dz chunk.
  const size_t needed = forward_only_workspace ? pl.off_dz : pl.total;
  if (workspace_bytes < needed)
    return fail(RKL_ERR_WORKSPACE, "workspace is %zu bytes, %zu needed", workspace_bytes, needed);
  int sms = 0;
  RKL_TRY(device_setup(&sms));
  cudaStream_t s = static_cast<cudaStream_t>(stream_);
  const long long T = B * Sm1;
  const bool bf16 = dtype == RKL_BF16;
  const bool hidden = payload == RKL_PAYLOAD_HIDDEN;

  // Per-row entropy / target log-prob reuse regions of the backward's row
  // constants (3 x n_pad floats), which the forward does not otherwise use.
  float* rowc = reinterpret_cast<float*>(ws_at(workspace, pl.off_rowc));
  float* tlogit = targets ? rowc : nullptr;
  float* ent_rows = entropy ? rowc + pl.n_pad : nullptr;
  float* lp_rows = target_logprob ? rowc + 2 * pl.n_pad : nullptr;
  // A target id outside [0, V) is never found by the kernels: its log-prob
  // reads back the NaN written here.
  if (tlogit && N > 0) RKL_CUDA(cudaMemsetAsync(tlogit, 0xFF, size_t(pl.n_pad) * sizeof(float), s));
  if (N > 0) {
    float* part = reinterpret_cast<float*>(ws_at(workspace, pl.off_part));
    float* lse_ext = reinterpret_cast<float*>(ws_at(workspace, pl.off_lse));
    // Teacher per row: rows regrouped by teacher into whole pair tiles.
    int32_t* slot_k = nullptr;
    int n_rows = N;
    if (mt) {
      slot_k = reinterpret_cast<int32_t*>(ws_at(workspace, pl.off_slot));
      n_rows = mt->n_rows;
      RKL_CUDA(cudaMemsetAsync(slot_k, 0xFF, size_t(n_rows) * sizeof(int32_t), s));
      RKL_CUDA(launch_build_slots(row_idx, mt->teacher_idx, N, mt->ts, slot_k,
                                  reinterpret_cast<int32_t*>(ws_at(workspace, pl.off_kslot)), s));
    }
    // S2: compact the rows (skipped when every row is known to be trainable).
    const bool identity = N == T && !mt && !n_dev;
    const void* as = h_s;
    const void* at = teacher;
    if (!identity) {
      as = ws_at(workspace, pl.off_hcs);
      at = hidden ? ws_at(workspace, pl.off_hct) : nullptr;
      RKL_CUDA(launch_gather(h_s, hidden ? teacher : nullptr, const_cast<void*>(as), const_cast<void*>(at), row_idx,
                             slot_k, n_rows, n_dev, static_cast<int>(H * pl.es), T, s));
    }
    // S8: teacher log-sum-exp from the shipped logits.
    if (!hidden)
      RKL_CUDA(launch_teacher_lse(teacher, bf16, row_idx, N, n_dev, static_cast<int>(V), V, lse_ext, T, s));
    const int ng = hidden ? 2 : 1;
    if (bf16) {
      FusedArgs a;
      memset(&a, 0, sizeof(a));
      RKL_TRY(make_map(&a.tm_as, as, false, H, n_rows, H * 2, kBK, kBM));
      RKL_TRY(make_map(&a.tm_bs, W_s, false, H, V, H * 2, kBK, kFBN / 2));
      if (hidden) {
        RKL_TRY(make_map(&a.tm_at, at, false, H, n_rows, H * 2, kBK, kBM));
        RKL_TRY(make_map(&a.tm_bt, W_t, false, H, V * (mt ? mt->n : 1), H * 2, kBK, kFBN / 2));
        if (mt) {
          a.tgroups = mt->n;
          for (int g = 0; g < mt->n; ++g) a.group_row_end[g] = mt->group_row_end[g];
        }
      } else {
        a.teacher = static_cast<const uint16_t*>(teacher);
        a.teacher_rows = identity ? nullptr : row_idx;
        a.teacher_pitch = V;
      }
      a.part = part;
      a.row_idx = row_idx;
      a.targets = targets;
      a.tlogit = tlogit;
      a.N = n_rows;
      a.n_dev = n_dev;
      a.n_pad = pl.n_pad;
      a.H = static_cast<int>(H);
      a.V = static_cast<int>(V);
      a.KB = static_cast<int>(H / kBK);
      a.IT = pl.VT;
      a.vt_base = 0;
      a.GT = kGroupTiles;
      a.G = pl.S / fwd_slots(ng);
      const int units = ((n_rows + 2 * kBM - 1) / (2 * kBM)) * a.G;  // at most; the kernel takes the live count
      RKL_CUDA(launch_fused(ng, false, a, 2 * units < sms ? 2 * units : sms, s));
    } else {
      SimtArgs a;
      memset(&a, 0, sizeof(a));
      a.as = static_cast<const float*>(as);
      a.bs = static_cast<const float*>(W_s);
      if (hidden) {
        a.at = static_cast<const float*>(at);
        a.bt = static_cast<const float*>(W_t);
        if (mt) {
          a.tgroups = mt->n;
          for (int g = 0; g < mt->n; ++g) a.group_row_end[g] = mt->group_row_end[g];
        }
      } else {
        a.teacher = static_cast<const float*>(teacher);
        a.teacher_rows = identity ? nullptr : row_idx;
        a.teacher_pitch = V;
      }
      a.part = part;
      a.row_idx = row_idx;
      a.targets = targets;
      a.tlogit = tlogit;
      a.N = n_rows;
      a.n_dev = n_dev;
      a.n_pad = pl.n_pad;
      a.H = static_cast<int>(H);
      a.V = static_cast<int>(V);
      a.IT = pl.VT;
      a.S = pl.S;
      a.ng = ng;
      const int MT = (n_rows + kSimtBN - 1) / kSimtBN;
      RKL_CUDA(launch_simt_fused(false, a, dim3(MT, pl.S), s));
    }
    // S4
    RKL_CUDA(launch_combine(part, pl.S, pl.n_pad, n_rows, n_dev, hidden, lse_ext, tlogit, saved, ent_rows, lp_rows,
                            slot_k, s));
  }
  if (loss_tok) RKL_CUDA(launch_scatter_loss(saved, row_idx, N, n_dev, T, loss_tok, s));
  if (entropy) RKL_CUDA(launch_scatter_rows(ent_rows, row_idx, N, n_dev, T, entropy, s));
  if (target_logprob) RKL_CUDA(launch_scatter_rows(lp_rows, row_idx, N, n_dev, T, target_logprob, s));
  if (loss && reduction != RKL_REDUCE_NONE)
    RKL_CUDA(launch_reduce(saved, row_idx, N, n_dev, static_cast<int>(B), static_cast<int>(Sm1), reduction, loss, s));
  return RKL_OK;
}

// ------------------------------------------------------------------ backward
static rkl_status backward_impl(rkl_payload payload, const void* h_s, const void* teacher, const void* W_s,
                                const void* W_t, rkl_dtype dtype, int64_t B, int64_t Sm1, int64_t H, int64_t V,
                                const int32_t* row_idx, int32_t N, const int32_t* n_dev, rkl_reduction reduction,
                                const float* saved, const float* grad_loss, const float* grad_tok, float* dH_s,
                                float* dW_s, void* workspace, size_t workspace_bytes, void* stream_,
                                const MultiTeacher* mt = nullptr, const int32_t* topk_targets = nullptr) {
  RKL_TRY(check_common(payload, dtype, B, Sm1, H, V, N, reduction));
  RKL_TRY(check_n_dev(n_dev));
  if (mt && n_dev)
    return fail(RKL_ERR_UNSUPPORTED, "a teacher per row needs the per-teacher counts on the host (n_dev must be NULL)");
  const bool topk = payload == RKL_PAYLOAD_TOPK_HIDDEN || payload == RKL_PAYLOAD_TOPK_LOGITS;
  const bool hidden = payload == RKL_PAYLOAD_HIDDEN || payload == RKL_PAYLOAD_TOPK_HIDDEN;
  RKL_TRY(check_ptr(h_s, "h_s"));
  RKL_TRY(check_ptr(teacher, hidden ? "h_t" : "teacher_logits"));
  RKL_TRY(check_ptr(W_s, "W_s"));
  if (hidden) RKL_TRY(check_ptr(W_t, "W_t"));
  if (topk && dtype != RKL_BF16)
    return fail(RKL_ERR_UNSUPPORTED, "the top-k estimator on the tensor-core payloads needs bf16 inputs");
  if (topk) RKL_TRY(check_ptr(topk_targets, "targets"));
  RKL_TRY(check_ptr(row_idx, "row_idx"));
  RKL_TRY(check_ptr(saved, "saved", N > 0));
  RKL_TRY(check_ptr(grad_loss, "grad_loss", false));
  RKL_TRY(check_ptr(grad_tok, "grad_tok", false));
  RKL_TRY(check_ptr(dH_s, "dH_s"));
  RKL_TRY(check_ptr(dW_s, "dW_s"));
  RKL_TRY(check_ptr(workspace, "workspace"));
  const Plan pl = make_plan(payload, dtype, N, H, V, mt ? mt->n : 1);
  if (workspace_bytes < pl.total)
    return fail(RKL_ERR_WORKSPACE, "workspace is %zu bytes, %zu needed", workspace_bytes, pl.total);
  int sms = 0;
  RKL_TRY(device_setup(&sms));
  cudaStream_t s = static_cast<cudaStream_t>(stream_);
  const long long T = B * Sm1;
  const bool bf16 = dtype == RKL_BF16;
  float* dHc = reinterpret_cast<float*>(ws_at(workspace, pl.off_dh));

  if (N == 0) {
    RKL_CUDA(cudaMemsetAsync(dW_s, 0, size_t(V) * H * sizeof(float), s));
    RKL_CUDA(launch_scatter_dh(dHc, row_idx, nullptr, 0, nullptr, T, static_cast<int>(H), dH_s, s));
    return RKL_OK;
  }
  // Teacher per row: rows regrouped by teacher into whole pair tiles.
  int32_t* slot_k = nullptr;
  int32_t* k_slot = nullptr;
  int n_rows = N;
  if (mt) {
    slot_k = reinterpret_cast<int32_t*>(ws_at(workspace, pl.off_slot));
    k_slot = reinterpret_cast<int32_t*>(ws_at(workspace, pl.off_kslot));
    n_rows = mt->n_rows;
    RKL_CUDA(cudaMemsetAsync(slot_k, 0xFF, size_t(n_rows) * sizeof(int32_t), s));
    RKL_CUDA(launch_build_slots(row_idx, mt->teacher_idx, N, mt->ts, slot_k, k_slot, s));
  }
  const bool identity = N == T && !mt && !n_dev;
  const void* as = h_s;
  const void* at = teacher;
  if (!identity) {
    as = ws_at(workspace, pl.off_hcs);
    at = hidden ? ws_at(workspace, pl.off_hct) : nullptr;
    RKL_CUDA(launch_gather(h_s, hidden ? teacher : nullptr, const_cast<void*>(as), const_cast<void*>(at), row_idx,
                           slot_k, n_rows, n_dev, static_cast<int>(H * pl.es), T, s));
  }
  float* rowc = reinterpret_cast<float*>(ws_at(workspace, pl.off_rowc));
  RKL_CUDA(launch_row_weights(saved, row_idx, N, n_dev, pl.n_pad, static_cast<int>(B), static_cast<int>(Sm1),
                              reduction, grad_loss, grad_tok, rowc, slot_k, s));
  float* rowk = nullptr;
  if (topk) {
    rowk = reinterpret_cast<float*>(ws_at(workspace, pl.off_rowk));
    RKL_CUDA(launch_topk_rowk(saved, saved + 3 * size_t(N), row_idx, topk_targets, N, n_dev, pl.n_pad, rowk, s));
  }
  void* dz = ws_at(workspace, pl.off_dz);
  const int ng = hidden ? 2 : 1;
  const int nchunks = static_cast<int>((V + pl.Vc - 1) / pl.Vc);

  if (bf16) {
    FusedArgs a;
    memset(&a, 0, sizeof(a));
    RKL_TRY(make_map(&a.tm_as, as, false, H, n_rows, H * 2, kBK, kBM));
    RKL_TRY(make_map(&a.tm_bs, W_s, false, H, V, H * 2, kBK, kFBN / 2));
    if (hidden) {
      RKL_TRY(make_map(&a.tm_at, at, false, H, n_rows, H * 2, kBK, kBM));
      RKL_TRY(make_map(&a.tm_bt, W_t, false, H, V * (mt ? mt->n : 1), H * 2, kBK, kFBN / 2));
      if (mt) {
        a.tgroups = mt->n;
        for (int g = 0; g < mt->n; ++g) a.group_row_end[g] = mt->group_row_end[g];
      }
    } else {
      a.teacher = static_cast<const uint16_t*>(teacher);
      a.teacher_rows = identity ? nullptr : row_idx;
      a.teacher_pitch = V;
    }
    a.rowc = rowc;
    a.rowk = rowk;
    a.N = n_rows;
    a.n_dev = n_dev;
    a.n_pad = pl.n_pad;
    a.H = static_cast<int>(H);
    a.V = static_cast<int>(V);
    a.KB = static_cast<int>(H / kBK);
    const int MT = (n_rows + 2 * kBM - 1) / (2 * kBM);  // at most; the kernels take the live count

    int* counters = reinterpret_cast<int*>(ws_at(workspace, pl.off_cnt));
    RKL_CUDA(cudaMemsetAsync(counters, 0, size_t(nchunks) * sizeof(int), s));
    GradArgs g;
    memset(&g, 0, sizeof(g));
    RKL_TRY(make_map(&g.tm_hs_mn, as, false, H, n_rows, H * 2, 64, 64));
    RKL_TRY(make_map(&g.tm_ws_mn, W_s, false, H, V, H * 2, 64, 64));
    RKL_TRY(make_map(&g.tm_dw, dW_s, true, H, V, H * 4, 32, 32));
    RKL_TRY(make_map(&g.tm_dh, dHc, true, H, n_rows, H * 4, 32, 32));
    g.N = n_rows;
    g.n_dev = n_dev;
    g.dw = dW_s;
    g.dh = dHc;
    g.dw_rows = static_cast<int>(V);
    g.dh_rows = n_rows;
    g.H = static_cast<int>(H);
    g.NT = static_cast<int>(H / kGradBN) + (H % kGradBN ? 1 : 0);

    for (int c = 0; c < nchunks; ++c) {
      const int cv0 = c * pl.Vc;
      const int cw = static_cast<int>((V - cv0) < pl.Vc ? (V - cv0) : pl.Vc);
      // S6: recompute the logits of this chunk and write dz (bf16) [N, cw].
      RKL_TRY(make_map(&a.tm_dz, dz, false, cw, n_rows, size_t(pl.Vc) * 2, 64, 32));
      a.IT = (cw + kFBN - 1) / kFBN;
      a.vt_base = cv0 / kFBN;
      a.chunk_v0 = cv0;
      a.GT = 1;
      a.G = a.IT;
      const int units = MT * a.IT;
      const int fgrid = 2 * units < sms ? 2 * units : sms;
      if (topk)
        RKL_CUDA(launch_fused_topk(2, ng, a, fgrid, s));
      else
        RKL_CUDA(launch_fused(ng, true, a, fgrid, s));
      // S7: dW_s[chunk] = dz^T hc_s and dHc (+)= dz W_s[chunk].
      RKL_TRY(make_map(&g.tm_dz_k, dz, false, cw, n_rows, size_t(pl.Vc) * 2, 64, 128));
      RKL_TRY(make_map(&g.tm_dz_mn, dz, false, cw, n_rows, size_t(pl.Vc) * 2, 64, 64));
      g.cw = cw;
      g.cv0 = cv0;
      g.MTW = (cw + 2 * kBM - 1) / (2 * kBM);
      g.nW = g.MTW * g.NT;
      g.KBH = (cw + kBK - 1) / kBK;
      g.dh_accumulate = c > 0;
      g.tile_counter = counters + c;
      const int pairs = g.nW + MT * g.NT;  // at most
      RKL_CUDA(launch_grad(g, 2 * pairs < sms ? 2 * pairs : sms, s));
    }
  } else {
    SimtArgs a;
    memset(&a, 0, sizeof(a));
    a.as = static_cast<const float*>(as);
    a.bs = static_cast<const float*>(W_s);
    if (hidden) {
      a.at = static_cast<const float*>(at);
      a.bt = static_cast<const float*>(W_t);
      if (mt) {
        a.tgroups = mt->n;
        for (int g = 0; g < mt->n; ++g) a.group_row_end[g] = mt->group_row_end[g];
      }
    } else {
      a.teacher = static_cast<const float*>(teacher);
      a.teacher_rows = identity ? nullptr : row_idx;
      a.teacher_pitch = V;
    }
    a.rowc = rowc;
    a.dz = static_cast<float*>(dz);
    a.N = n_rows;
    a.n_dev = n_dev;
    a.n_pad = pl.n_pad;
    a.H = static_cast<int>(H);
    a.V = static_cast<int>(V);
    a.ng = ng;
    const int MT = (n_rows + kSimtBN - 1) / kSimtBN;
    for (int c = 0; c < nchunks; ++c) {
      const int cv0 = c * pl.Vc;
      const int cw = static_cast<int>((V - cv0) < pl.Vc ? (V - cv0) : pl.Vc);
      a.cw = cw;
      a.IT = (cw + kSimtBN - 1) / kSimtBN;
      a.vt_base = cv0 / kSimtBN;
      a.chunk_v0 = cv0;
      const int items = MT * a.IT;
      RKL_CUDA(launch_simt_fused(true, a, dim3(items < 4 * sms ? items : 4 * sms), s));
      const float* dzf = static_cast<const float*>(dz);
      // dW_s[cv0 + m, n] = sum_k dz[k, m] hc_s[k, n]
      RKL_CUDA(launch_simt_gemm(dzf, 1, cw, a.as, H, 1, dW_s + size_t(cv0) * H, H, cw, static_cast<int>(H), n_rows,
                                0, n_dev, 2, s));
      // dHc[m, n] (+)= sum_k dz[m, k] W_s[cv0 + k, n]
      RKL_CUDA(launch_simt_gemm(dzf, cw, 1, a.bs + size_t(cv0) * H, H, 1, dHc, H, n_rows, static_cast<int>(H), cw,
                                c > 0, n_dev, 1, s));
    }
  }
  RKL_CUDA(launch_scatter_dh(dHc, row_idx, k_slot, N, n_dev, T, static_cast<int>(H), dH_s, s));
  return RKL_OK;
}

}  // namespace rkl

// ====================================================================== C ABI
using namespace rkl;

extern "C" {

#ifdef RKL_DEBUG
const char* rkl_version(void) { return "rkl 0.2 (sm_100a, debug bounds checks)"; }
#else
const char* rkl_version(void) { return "rkl 0.2 (sm_100a)"; }
#endif

const char* rkl_last_error(void) { return g_last_error.c_str(); }

// Workspace of the logits-pair mode: only the per-row constants of the backward.
static size_t pair_workspace_bytes(int64_t n_max) {
  const int64_t n = n_max < 1 ? 1 : n_max;
  const size_t n_pad = size_t(((n + 255) / 256) * 256);
  return 256 + align256(3 * n_pad * sizeof(float));
}

rkl_status rkl_workspace_size(rkl_payload payload, rkl_dtype dtype, int64_t n_max, int64_t B, int64_t Sm1, int64_t H,
                              int64_t V, size_t* bytes) {
  if (bytes == nullptr) return fail(RKL_ERR_NULL, "bytes is NULL");
  RKL_TRY(check_common(payload, dtype, B, Sm1, H, V, 0, 0));
  if (n_max < 0 || n_max > B * Sm1) return fail(RKL_ERR_SHAPE, "n_max outside [0, B*Sm1]");
  *bytes = payload == RKL_PAYLOAD_LOGITS_PAIR ? pair_workspace_bytes(n_max) : make_plan(payload, dtype, n_max, H, V).total;
  return RKL_OK;
}

rkl_status rkl_forward_logits_pair(const void* student_logits, const void* teacher_logits, rkl_dtype dtype, int64_t B,
                                   int64_t Sm1, int64_t V, const int32_t* row_idx, int32_t N, const int32_t* n_dev,
                                   rkl_reduction reduction, float* loss_tok, float* loss, float* saved,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  RKL_NVTX_RANGE();
  RKL_TRY(check_common(RKL_PAYLOAD_LOGITS_PAIR, dtype, B, Sm1, 64, V, N, reduction));
  RKL_TRY(check_n_dev(n_dev));
  RKL_TRY(check_ptr(student_logits, "student_logits"));
  RKL_TRY(check_ptr(teacher_logits, "teacher_logits"));
  RKL_TRY(check_ptr(row_idx, "row_idx"));
  RKL_TRY(check_ptr(loss_tok, "loss_tok", false));
  RKL_TRY(check_ptr(loss, "loss", false));
  RKL_TRY(check_ptr(saved, "saved", N > 0));
  RKL_TRY(check_ptr(workspace, "workspace"));
  if (workspace_bytes < pair_workspace_bytes(N))
    return fail(RKL_ERR_WORKSPACE, "workspace is %zu bytes, %zu needed", workspace_bytes, pair_workspace_bytes(N));
  int sms = 0;
  RKL_TRY(device_setup(&sms));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const long long T = B * Sm1;
  RKL_CUDA(launch_pair_fwd(student_logits, teacher_logits, dtype == RKL_BF16, row_idx, N, n_dev, static_cast<int>(V),
                           saved, s));
  if (loss_tok) RKL_CUDA(launch_scatter_loss(saved, row_idx, N, n_dev, T, loss_tok, s));
  if (loss && reduction != RKL_REDUCE_NONE)
    RKL_CUDA(launch_reduce(saved, row_idx, N, n_dev, static_cast<int>(B), static_cast<int>(Sm1), reduction, loss, s));
  return RKL_OK;
}

rkl_status rkl_backward_logits_pair(const void* student_logits, const void* teacher_logits, rkl_dtype dtype,
                                    int64_t B, int64_t Sm1, int64_t V, const int32_t* row_idx, int32_t N,
                                    const int32_t* n_dev, rkl_reduction reduction, const float* saved,
                                    const float* grad_loss, const float* grad_tok, void* dz, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  RKL_NVTX_RANGE();
  RKL_TRY(check_common(RKL_PAYLOAD_LOGITS_PAIR, dtype, B, Sm1, 64, V, N, reduction));
  RKL_TRY(check_n_dev(n_dev));
  RKL_TRY(check_ptr(student_logits, "student_logits"));
  RKL_TRY(check_ptr(teacher_logits, "teacher_logits"));
  RKL_TRY(check_ptr(row_idx, "row_idx"));
  RKL_TRY(check_ptr(saved, "saved", N > 0));
  RKL_TRY(check_ptr(grad_loss, "grad_loss", false));
  RKL_TRY(check_ptr(grad_tok, "grad_tok", false));
  RKL_TRY(check_ptr(dz, "dz"));
  RKL_TRY(check_ptr(workspace, "workspace"));
  if (workspace_bytes < pair_workspace_bytes(N))
    return fail(RKL_ERR_WORKSPACE, "workspace is %zu bytes, %zu needed", workspace_bytes, pair_workspace_bytes(N));
  int sms = 0;
  RKL_TRY(device_setup(&sms));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const long long T = B * Sm1;
  const int64_t n = N < 1 ? 1 : N;
  const int n_pad = static_cast<int>(((n + 255) / 256) * 256);
  float* rowc = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + 256);
  if (N > 0)
    RKL_CUDA(launch_row_weights(saved, row_idx, N, n_dev, n_pad, static_cast<int>(B), static_cast<int>(Sm1),
                                reduction, grad_loss, grad_tok, rowc, nullptr, s));
  RKL_CUDA(launch_pair_bwd(student_logits, teacher_logits, dtype == RKL_BF16, row_idx, N, n_dev, n_pad, T,
                           static_cast<int>(V), rowc, dz, s));
  return RKL_OK;
}

// ---------------------------------------------------------------- top-k estimator
static rkl_status check_topk(const void* zs, const void* zt, rkl_dtype dtype, int64_t B, int64_t Sm1, int64_t V,
                             const int32_t* row_idx, int32_t N, const int32_t* n_dev, int64_t k,
                             const int32_t* targets, int reduction, void* workspace, size_t workspace_bytes) {
  RKL_TRY(check_common(RKL_PAYLOAD_LOGITS_PAIR, dtype, B, Sm1, 64, V, N, reduction));
  RKL_TRY(check_n_dev(n_dev));
  RKL_TRY(check_ptr(zs, "student_logits"));
  RKL_TRY(check_ptr(zt, "teacher_logits"));
  RKL_TRY(check_ptr(row_idx, "row_idx"));
  RKL_TRY(check_ptr(targets, "targets"));
  RKL_TRY(check_ptr(workspace, "workspace"));
  if (k < 0) return fail(RKL_ERR_SHAPE, "k = %lld is negative", (long long)k);
  if (workspace_bytes < pair_workspace_bytes(N))
    return fail(RKL_ERR_WORKSPACE, "workspace is %zu bytes, %zu needed", workspace_bytes, pair_workspace_bytes(N));
  return RKL_OK;
}

rkl_status rkl_forward_topk_pair(const void* student_logits, const void* teacher_logits, rkl_dtype dtype, int64_t B,
                                 int64_t Sm1, int64_t V, const int32_t* row_idx, int32_t N, const int32_t* n_dev,
                                 int64_t k, const int32_t* targets, rkl_reduction reduction, float* loss_tok,
                                 float* loss, float* saved, void* workspace, size_t workspace_bytes, void* stream) {
  RKL_NVTX_RANGE();
  RKL_TRY(check_topk(student_logits, teacher_logits, dtype, B, Sm1, V, row_idx, N, n_dev, k, targets, reduction,
                     workspace, workspace_bytes));
  RKL_TRY(check_ptr(loss_tok, "loss_tok", false));
  RKL_TRY(check_ptr(loss, "loss", false));
  RKL_TRY(check_ptr(saved, "saved", N > 0));
  int sms = 0;
  RKL_TRY(device_setup(&sms));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const long long T = B * Sm1;
  RKL_CUDA(launch_topk_fwd(student_logits, teacher_logits, dtype == RKL_BF16, row_idx, targets, N, n_dev, 0,
                           static_cast<int>(V), k, saved, saved + 3 * size_t(N), V, false, s));
  if (loss_tok) RKL_CUDA(launch_scatter_loss(saved, row_idx, N, n_dev, T, loss_tok, s));
  if (loss && reduction != RKL_REDUCE_NONE)
    RKL_CUDA(launch_reduce(saved, row_idx, N, n_dev, static_cast<int>(B), static_cast<int>(Sm1), reduction, loss, s));
  return RKL_OK;
}

rkl_status rkl_backward_topk_pair(const void* student_logits, const void* teacher_logits, rkl_dtype dtype,
                                  int64_t B, int64_t Sm1, int64_t V, const int32_t* row_idx, int32_t N,
                                  const int32_t* n_dev, const int32_t* targets, rkl_reduction reduction,
                                  const float* saved, const float* grad_loss, const float* grad_tok, void* dz,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  RKL_NVTX_RANGE();
  RKL_TRY(check_topk(student_logits, teacher_logits, dtype, B, Sm1, V, row_idx, N, n_dev, 0, targets, reduction,
                     workspace, workspace_bytes));
  RKL_TRY(check_ptr(saved, "saved", N > 0));
  RKL_TRY(check_ptr(grad_loss, "grad_loss", false));
  RKL_TRY(check_ptr(grad_tok, "grad_tok", false));
  RKL_TRY(check_ptr(dz, "dz"));
  int sms = 0;
  RKL_TRY(device_setup(&sms));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const long long T = B * Sm1;
  const int64_t n = N < 1 ? 1 : N;
  const int n_pad = static_cast<int>(((n + 255) / 256) * 256);
  float* rowc = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + 256);
  if (N > 0)
    RKL_CUDA(launch_row_weights(saved, row_idx, N, n_dev, n_pad, static_cast<int>(B), static_cast<int>(Sm1),
                                reduction, grad_loss, grad_tok, rowc, nullptr, s));
  RKL_CUDA(launch_topk_bwd(student_logits, teacher_logits, dtype == RKL_BF16, row_idx, targets, N, n_dev, n_pad, T,
                           static_cast<int>(V), saved, N > 0 ? saved + 3 * size_t(N) : nullptr, rowc, dz, s));
  return RKL_OK;
}

// Top-k estimator on the hidden payload.  Forward: per block of up to
// kTopkBlockRows compacted rows, the tcgen05 kernel writes z_s and z_t (fp32)
// of the block, and the selection / estimate kernel of the logits-pair form
// runs on those rows.  Backward: the recompute + dz kernel with the top-k
// formula (membership from the same fp32 logits, bit for bit), then the
// gradient GEMMs of the exact path.
// Top-k forward of both tensor-core payloads.  Per block of up to
// kTopkBlockRows compacted rows, a tcgen05 kernel writes z_s and z_t (fp32)
// of the block -- on the hidden payload both by the tensor core, on the
// logits payload z_s by the tensor core and z_t copied (exactly) from the
// shipped bf16 teacher rows -- and the selection / estimate kernel of the
// logits-pair form runs on those rows.
static rkl_status forward_topk_impl(rkl_payload payload, const void* h_s, const void* teacher, const void* W_s,
                                    const void* W_t, rkl_dtype dtype, int64_t B, int64_t Sm1, int64_t H, int64_t V,
                                    const int32_t* row_idx, int32_t N, const int32_t* n_dev, int64_t k,
                                    const int32_t* targets, rkl_reduction reduction, float* loss_tok, float* loss,
                                    float* saved, void* workspace, size_t workspace_bytes, void* stream) {
  const bool hidden = payload == RKL_PAYLOAD_TOPK_HIDDEN;
  RKL_TRY(check_common(payload, dtype, B, Sm1, H, V, N, reduction));
  RKL_TRY(check_n_dev(n_dev));
  if (dtype != RKL_BF16)
    return fail(RKL_ERR_UNSUPPORTED, "the top-k estimator on the tensor-core payloads needs bf16 inputs");
  if (k < 0) return fail(RKL_ERR_SHAPE, "k = %lld is negative", (long long)k);
  RKL_TRY(check_ptr(h_s, "h_s"));
  RKL_TRY(check_ptr(teacher, hidden ? "h_t" : "teacher_logits"));
  RKL_TRY(check_ptr(W_s, "W_s"));
  if (hidden) RKL_TRY(check_ptr(W_t, "W_t"));
  RKL_TRY(check_ptr(row_idx, "row_idx"));
  RKL_TRY(check_ptr(targets, "targets"));
  RKL_TRY(check_ptr(loss_tok, "loss_tok", false));
  RKL_TRY(check_ptr(loss, "loss", false));
  RKL_TRY(check_ptr(saved, "saved", N > 0));
  RKL_TRY(check_ptr(workspace, "workspace"));
  const Plan pl = make_plan(payload, dtype, N, H, V);
  if (workspace_bytes < pl.total)
    return fail(RKL_ERR_WORKSPACE, "workspace is %zu bytes, %zu needed", workspace_bytes, pl.total);
  int sms = 0;
  RKL_TRY(device_setup(&sms));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const long long T = B * Sm1;
  if (N > 0) {
    const uint8_t* as = static_cast<const uint8_t*>(h_s);
    const uint8_t* at = hidden ? static_cast<const uint8_t*>(teacher) : nullptr;
    if (N < T || n_dev) {
      as = ws_at(workspace, pl.off_hcs);
      at = hidden ? ws_at(workspace, pl.off_hct) : nullptr;
      RKL_CUDA(launch_gather(h_s, hidden ? teacher : nullptr, const_cast<uint8_t*>(as), const_cast<uint8_t*>(at),
                             row_idx, nullptr, N, n_dev, static_cast<int>(H * 2), T, s));
    }
    float* zs = reinterpret_cast<float*>(ws_at(workspace, pl.off_z));
    float* zt = hidden ? zs + size_t(pl.zrows) * pl.zpitch : nullptr;
    for (int r0 = 0; r0 < N; r0 += pl.zrows) {
      const int nb = (N - r0) < pl.zrows ? (N - r0) : pl.zrows;
      FusedArgs a;
      memset(&a, 0, sizeof(a));
      RKL_TRY(make_map(&a.tm_as, as + size_t(r0) * H * 2, false, H, nb, H * 2, kBK, kBM));
      RKL_TRY(make_map(&a.tm_bs, W_s, false, H, V, H * 2, kBK, kFBN / 2));
      if (hidden) {
        RKL_TRY(make_map(&a.tm_at, at + size_t(r0) * H * 2, false, H, nb, H * 2, kBK, kBM));
        RKL_TRY(make_map(&a.tm_bt, W_t, false, H, V, H * 2, kBK, kFBN / 2));
      } else {
        // row p of the block is compacted row r0 + p: token row row_idx[r0 + p]
        a.teacher = static_cast<const uint16_t*>(teacher);
        a.teacher_rows = row_idx + r0;
        a.teacher_pitch = V;
      }
      RKL_TRY(make_map(&a.tm_zs, zs, true, V, nb, size_t(pl.zpitch) * 4, 32, 32));
      if (hidden) RKL_TRY(make_map(&a.tm_zt, zt, true, V, nb, size_t(pl.zpitch) * 4, 32, 32));
      a.N = nb;
      a.n_dev = n_dev;
      a.n_base = r0;
      a.n_pad = pl.n_pad;
      a.H = static_cast<int>(H);
      a.V = static_cast<int>(V);
      a.KB = static_cast<int>(H / kBK);
      a.IT = pl.VT;
      a.vt_base = 0;
      a.GT = 1;
      a.G = pl.VT;
      const int units = ((nb + 2 * kBM - 1) / (2 * kBM)) * a.G;  // at most
      RKL_CUDA(launch_fused_topk(1, hidden ? 2 : 1, a, 2 * units < sms ? 2 * units : sms, s));
      if (hidden)
        RKL_CUDA(launch_topk_fwd(zs, zt, false, row_idx + r0, targets, nb, n_dev, r0, static_cast<int>(V), k,
                                 saved + 3 * size_t(r0), saved + 3 * size_t(N) + 4 * size_t(r0), pl.zpitch, true, s));
      else
        RKL_CUDA(launch_topk_fwd_tlogits(zs, static_cast<const uint16_t*>(teacher), V, row_idx + r0, targets, nb,
                                         n_dev, r0, static_cast<int>(V), k, saved + 3 * size_t(r0),
                                         saved + 3 * size_t(N) + 4 * size_t(r0), pl.zpitch, s));
    }
  }
  if (loss_tok) RKL_CUDA(launch_scatter_loss(saved, row_idx, N, n_dev, T, loss_tok, s));
  if (loss && reduction != RKL_REDUCE_NONE)
    RKL_CUDA(launch_reduce(saved, row_idx, N, n_dev, static_cast<int>(B), static_cast<int>(Sm1), reduction, loss, s));
  return RKL_OK;
}

rkl_status rkl_forward_topk_hidden(const void* h_s, const void* h_t, const void* W_s, const void* W_t,
                                   rkl_dtype dtype, int64_t B, int64_t Sm1, int64_t H, int64_t V,
                                   const int32_t* row_idx, int32_t N, const int32_t* n_dev, int64_t k,
                                   const int32_t* targets, rkl_reduction reduction, float* loss_tok, float* loss,
                                   float* saved, void* workspace, size_t workspace_bytes, void* stream) {
  RKL_NVTX_RANGE();
  return forward_topk_impl(RKL_PAYLOAD_TOPK_HIDDEN, h_s, h_t, W_s, W_t, dtype, B, Sm1, H, V, row_idx, N, n_dev, k,
                           targets, reduction, loss_tok, loss, saved, workspace, workspace_bytes, stream);
}

rkl_status rkl_forward_topk_logits(const void* h_s, const void* W_s, const void* teacher_logits, rkl_dtype dtype,
                                   int64_t B, int64_t Sm1, int64_t H, int64_t V, const int32_t* row_idx, int32_t N,
                                   const int32_t* n_dev, int64_t k, const int32_t* targets, rkl_reduction reduction,
                                   float* loss_tok, float* loss, float* saved, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  RKL_NVTX_RANGE();
  return forward_topk_impl(RKL_PAYLOAD_TOPK_LOGITS, h_s, teacher_logits, W_s, nullptr, dtype, B, Sm1, H, V, row_idx,
                           N, n_dev, k, targets, reduction, loss_tok, loss, saved, workspace, workspace_bytes, stream);
}

rkl_status rkl_backward_topk_logits(const void* h_s, const void* W_s, const void* teacher_logits, rkl_dtype dtype,
                                    int64_t B, int64_t Sm1, int64_t H, int64_t V, const int32_t* row_idx, int32_t N,
                                    const int32_t* n_dev, const int32_t* targets, rkl_reduction reduction,
                                    const float* saved, const float* grad_loss, const float* grad_tok, float* dH_s,
                                    float* dW_s, void* workspace, size_t workspace_bytes, void* stream) {
  RKL_NVTX_RANGE();
  return backward_impl(RKL_PAYLOAD_TOPK_LOGITS, h_s, teacher_logits, W_s, nullptr, dtype, B, Sm1, H, V, row_idx, N,
                       n_dev, reduction, saved, grad_loss, grad_tok, dH_s, dW_s, workspace, workspace_bytes, stream,
                       nullptr, targets);
}

rkl_status rkl_backward_topk_hidden(const void* h_s, const void* h_t, const void* W_s, const void* W_t,
                                    rkl_dtype dtype, int64_t B, int64_t Sm1, int64_t H, int64_t V,
                                    const int32_t* row_idx, int32_t N, const int32_t* n_dev, const int32_t* targets,
                                    rkl_reduction reduction, const float* saved, const float* grad_loss,
                                    const float* grad_tok, float* dH_s, float* dW_s, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  RKL_NVTX_RANGE();
  return backward_impl(RKL_PAYLOAD_TOPK_HIDDEN, h_s, h_t, W_s, W_t, dtype, B, Sm1, H, V, row_idx, N, n_dev,
                       reduction, saved, grad_loss, grad_tok, dH_s, dW_s, workspace, workspace_bytes, stream, nullptr,
                       targets);
}

rkl_status rkl_compact_rows(const uint8_t* mask, int64_t B, int64_t Sm1, int32_t* row_idx, int32_t* n_dev,
                            void* stream) {
  RKL_NVTX_RANGE();
  if (mask == nullptr || row_idx == nullptr || n_dev == nullptr)
    return fail(RKL_ERR_NULL, "mask, row_idx and n_dev must be non-NULL");
  if (!aligned16(row_idx)) return fail(RKL_ERR_ALIGN, "row_idx is not 16-byte aligned");
  if (B < 1 || Sm1 < 1) return fail(RKL_ERR_SHAPE, "B and Sm1 must be >= 1");
  if (B * Sm1 >= (int64_t(1) << 31)) return fail(RKL_ERR_SHAPE, "B*Sm1 exceeds 2^31-1");
  int sms = 0;
  RKL_TRY(device_setup(&sms));
  RKL_CUDA(launch_compact(mask, B * Sm1, row_idx, n_dev, static_cast<cudaStream_t>(stream)));
  return RKL_OK;
}

rkl_status rkl_forward_hidden(const void* h_s, const void* h_t, const void* W_s, const void* W_t, rkl_dtype dtype,
                              int64_t B, int64_t Sm1, int64_t H, int64_t V, const int32_t* row_idx, int32_t N,
                              const int32_t* n_dev, rkl_reduction reduction, float* loss_tok, float* loss,
                              float* saved, void* workspace, size_t workspace_bytes, void* stream) {
  RKL_NVTX_RANGE();
  return forward_impl(RKL_PAYLOAD_HIDDEN, h_s, h_t, W_s, W_t, dtype, B, Sm1, H, V, row_idx, N, n_dev, reduction,
                      loss_tok, loss, saved, workspace, workspace_bytes, stream);
}

rkl_status rkl_forward_logits(const void* h_s, const void* W_s, const void* teacher_logits, rkl_dtype dtype,
                              int64_t B, int64_t Sm1, int64_t H, int64_t V, const int32_t* row_idx, int32_t N,
                              const int32_t* n_dev, rkl_reduction reduction, float* loss_tok, float* loss,
                              float* saved, void* workspace, size_t workspace_bytes, void* stream) {
  RKL_NVTX_RANGE();
  return forward_impl(RKL_PAYLOAD_LOGITS, h_s, teacher_logits, W_s, nullptr, dtype, B, Sm1, H, V, row_idx, N, n_dev,
                      reduction, loss_tok, loss, saved, workspace, workspace_bytes, stream);
}

rkl_status rkl_forward_hidden_ex(const void* h_s, const void* h_t, const void* W_s, const void* W_t, rkl_dtype dtype,
                                 int64_t B, int64_t Sm1, int64_t H, int64_t V, const int32_t* row_idx, int32_t N,
                                 const int32_t* n_dev, rkl_reduction reduction, float* loss_tok, float* loss,
                                 float* saved, const int32_t* targets, float* entropy, float* target_logprob,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  RKL_NVTX_RANGE();
  return forward_impl(RKL_PAYLOAD_HIDDEN, h_s, h_t, W_s, W_t, dtype, B, Sm1, H, V, row_idx, N, n_dev, reduction,
                      loss_tok, loss, saved, workspace, workspace_bytes, stream, false, targets, entropy,
                      target_logprob);
}

rkl_status rkl_forward_logits_ex(const void* h_s, const void* W_s, const void* teacher_logits, rkl_dtype dtype,
                                 int64_t B, int64_t Sm1, int64_t H, int64_t V, const int32_t* row_idx, int32_t N,
                                 const int32_t* n_dev, rkl_reduction reduction, float* loss_tok, float* loss,
                                 float* saved, const int32_t* targets, float* entropy, float* target_logprob,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  RKL_NVTX_RANGE();
  return forward_impl(RKL_PAYLOAD_LOGITS, h_s, teacher_logits, W_s, nullptr, dtype, B, Sm1, H, V, row_idx, N, n_dev,
                      reduction, loss_tok, loss, saved, workspace, workspace_bytes, stream, false, targets, entropy,
                      target_logprob);
}

rkl_status rkl_backward(rkl_payload payload, const void* h_s, const void* teacher, const void* W_s, const void* W_t,
                        rkl_dtype dtype, int64_t B, int64_t Sm1, int64_t H, int64_t V, const int32_t* row_idx,
                        int32_t N, const int32_t* n_dev, rkl_reduction reduction, const float* saved,
                        const float* grad_loss, const float* grad_tok, float* dH_s, float* dW_s, void* workspace,
                        size_t workspace_bytes, void* stream) {
  RKL_NVTX_RANGE();
  return backward_impl(payload, h_s, teacher, W_s, W_t, dtype, B, Sm1, H, V, row_idx, N, n_dev, reduction, saved,
                       grad_loss, grad_tok, dH_s, dW_s, workspace, workspace_bytes, stream);
}

// ---------------------------------------------------------------- teacher per row
rkl_status rkl_compact_rows_multi(const uint8_t* mask, const int32_t* teacher_idx, int64_t B, int64_t Sm1,
                                  int32_t n_teachers, int32_t* row_idx, int32_t* n_dev, int32_t* counts,
                                  void* stream) {
  RKL_NVTX_RANGE();
  if (mask == nullptr || teacher_idx == nullptr || row_idx == nullptr || n_dev == nullptr || counts == nullptr)
    return fail(RKL_ERR_NULL, "mask, teacher_idx, row_idx, n_dev and counts must be non-NULL");
  if (!aligned16(row_idx) || !aligned16(teacher_idx))
    return fail(RKL_ERR_ALIGN, "row_idx and teacher_idx must be 16-byte aligned");
  if (B < 1 || Sm1 < 1) return fail(RKL_ERR_SHAPE, "B and Sm1 must be >= 1");
  if (B * Sm1 >= (int64_t(1) << 31)) return fail(RKL_ERR_SHAPE, "B*Sm1 exceeds 2^31-1");
  if (n_teachers < 1 || n_teachers > kMaxTeachers)
    return fail(RKL_ERR_SHAPE, "n_teachers = %d outside [1, %d]", n_teachers, kMaxTeachers);
  int sms = 0;
  RKL_TRY(device_setup(&sms));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  RKL_CUDA(cudaMemsetAsync(counts, 0, size_t(n_teachers + 1) * sizeof(int32_t), s));
  RKL_CUDA(launch_compact(mask, B * Sm1, row_idx, n_dev, s));
  RKL_CUDA(launch_count_teachers(mask, teacher_idx, B * Sm1, n_teachers, counts, s));
  return RKL_OK;
}

rkl_status rkl_workspace_size_multi(rkl_dtype dtype, int64_t n_max, int32_t n_teachers, int64_t B, int64_t Sm1,
                                    int64_t H, int64_t V, size_t* bytes) {
  if (bytes == nullptr) return fail(RKL_ERR_NULL, "bytes is NULL");
  RKL_TRY(check_common(RKL_PAYLOAD_HIDDEN, dtype, B, Sm1, H, V, 0, 0));
  if (n_max < 0 || n_max > B * Sm1) return fail(RKL_ERR_SHAPE, "n_max outside [0, B*Sm1]");
  if (n_teachers < 1 || n_teachers > kMaxTeachers)
    return fail(RKL_ERR_SHAPE, "n_teachers = %d outside [1, %d]", n_teachers, kMaxTeachers);
  *bytes = make_plan(RKL_PAYLOAD_HIDDEN, dtype, n_max, H, V, n_teachers).total;
  return RKL_OK;
}

rkl_status rkl_forward_hidden_multi(const void* h_s, const void* h_t, const void* W_s, const void* W_t,
                                   int32_t n_teachers, const int32_t* teacher_idx, const int32_t* counts,
                                   rkl_dtype dtype, int64_t B, int64_t Sm1, int64_t H, int64_t V,
                                   const int32_t* row_idx, int32_t N, rkl_reduction reduction, float* loss_tok,
                                   float* loss, float* saved, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  RKL_NVTX_RANGE();
  MultiTeacher mt;
  RKL_TRY(make_multi(n_teachers, teacher_idx, counts, N, &mt));
  return forward_impl(RKL_PAYLOAD_HIDDEN, h_s, h_t, W_s, W_t, dtype, B, Sm1, H, V, row_idx, N, nullptr, reduction,
                      loss_tok, loss, saved, workspace, workspace_bytes, stream, false, nullptr, nullptr, nullptr,
                      n_teachers > 1 ? &mt : nullptr);
}

rkl_status rkl_backward_hidden_multi(const void* h_s, const void* h_t, const void* W_s, const void* W_t,
                                    int32_t n_teachers, const int32_t* teacher_idx, const int32_t* counts,
                                    rkl_dtype dtype, int64_t B, int64_t Sm1, int64_t H, int64_t V,
                                    const int32_t* row_idx, int32_t N, rkl_reduction reduction, const float* saved,
                                    const float* grad_loss, const float* grad_tok, float* dH_s, float* dW_s,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  RKL_NVTX_RANGE();
  MultiTeacher mt;
  RKL_TRY(make_multi(n_teachers, teacher_idx, counts, N, &mt));
  return backward_impl(RKL_PAYLOAD_HIDDEN, h_s, h_t, W_s, W_t, dtype, B, Sm1, H, V, row_idx, N, nullptr, reduction,
                       saved, grad_loss, grad_tok, dH_s, dW_s, workspace, workspace_bytes, stream,
                       n_teachers > 1 ? &mt : nullptr);
}

rkl_status rkl_device_error(int32_t* code) {
  if (code == nullptr) return fail(RKL_ERR_NULL, "code is NULL");
  RKL_CUDA(cudaDeviceSynchronize());
  int v = 0, waits = 0, line_tc = 0, line_small = 0, line_optim = 0, line_ffn = 0;
  RKL_CUDA(read_and_clear_device_error(&v));
  RKL_CUDA(read_and_clear_bounds_tc(&line_tc));
  RKL_CUDA(read_and_clear_bounds_small(&line_small));
  RKL_CUDA(read_and_clear_bounds_optim(&line_optim));
  RKL_CUDA(read_and_clear_bounds_ffn(&line_ffn));
  RKL_CUDA(read_and_clear_ffn_error(&waits));
  v |= waits;
  if (line_tc || line_small || line_optim || line_ffn) v |= ERR_BOUNDS;
  *code = v;
  if (line_tc || line_small || line_optim || line_ffn)
    return fail(RKL_ERR_DEVICE,
                "a bounds check failed (tc_kernels.cu line %d, small_kernels.cu line %d, optim_kernels.cu line %d, "
                "ffn_tc_kernels.cu line %d; 0 = none); the access was skipped and the outputs are invalid (bits 0x%x)",
                line_tc, line_small, line_optim, line_ffn, v);
  if (v != 0) return fail(RKL_ERR_DEVICE, "a kernel wait ran out (bits 0x%x); its outputs are invalid", v);
  return RKL_OK;
}

// ====================================================================== optimizer step
rkl_status rkl_adamw_state_size(int32_t n, const int64_t* numel, int64_t* at, int64_t* total) {
  if (total == nullptr) return fail(RKL_ERR_NULL, "total is NULL");
  RKL_TRY(check_tensor_counts(n, numel));
  int64_t sum = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (at != nullptr) at[i] = sum;
    sum += (numel[i] + kOptBlock - 1) / kOptBlock * kOptBlock;
  }
  *total = sum;
  return RKL_OK;
}

rkl_status rkl_adamw_step(int32_t n, void* const* params, const void* const* grads, const int64_t* numel,
                          const int32_t* param_dtype, const int32_t* grad_dtype, const float* weight_decay,
                          int32_t state_bits, void* exp_avg, void* exp_avg_sq, float* exp_avg_scale,
                          float* exp_avg_sq_scale, float* master, int32_t* control, double lr, const float* lr_dev,
                          double beta1, double beta2, double eps, uint32_t seed, const float* norm, double max_norm,
                          void* stream) {
  RKL_NVTX_RANGE();
  RKL_TRY(check_tensor_counts(n, numel));
  if (n > 0 && (params == nullptr || grads == nullptr || param_dtype == nullptr || grad_dtype == nullptr ||
                weight_decay == nullptr))
    return fail(RKL_ERR_NULL, "params, grads, param_dtype, grad_dtype and weight_decay must be non-NULL");
  if (state_bits != 32 && state_bits != 8) return fail(RKL_ERR_DTYPE, "state_bits = %d is neither 32 nor 8", state_bits);
  if (control == nullptr) return fail(RKL_ERR_NULL, "control is NULL");
  if (reinterpret_cast<uintptr_t>(control) & 7) return fail(RKL_ERR_ALIGN, "control is not 8-byte aligned");
  if (!(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1))
    return fail(RKL_ERR_SHAPE, "betas (%g, %g) outside [0, 1)", beta1, beta2);
  if (!(eps >= 0)) return fail(RKL_ERR_SHAPE, "eps = %g is negative", eps);
  if (lr_dev == nullptr && !(lr >= 0)) return fail(RKL_ERR_SHAPE, "lr = %g is negative", lr);
  if (norm != nullptr && !(max_norm > 0)) return fail(RKL_ERR_SHAPE, "max_norm = %g is not positive", max_norm);
  for (const float* p : {lr_dev, norm})
    if (reinterpret_cast<uintptr_t>(p) & 3) return fail(RKL_ERR_ALIGN, "lr_dev or norm is not 4-byte aligned");
  int64_t total = 0;
  RKL_TRY(rkl_adamw_state_size(n, numel, nullptr, &total));
  if (total > 0) {
    // the state is read and written 8 elements a lane
    const struct { const void* p; const char* name; bool need; } state[] = {
        {exp_avg, "exp_avg", true},
        {exp_avg_sq, "exp_avg_sq", true},
        {exp_avg_scale, "exp_avg_scale", state_bits == 8},
        {exp_avg_sq_scale, "exp_avg_sq_scale", state_bits == 8},
        {master, "master", false}};
    for (const auto& x : state) {
      if (x.need && x.p == nullptr) return fail(RKL_ERR_NULL, "%s is NULL", x.name);
      if (reinterpret_cast<uintptr_t>(x.p) & 31) return fail(RKL_ERR_ALIGN, "%s is not 32-byte aligned", x.name);
    }
  }
  for (int32_t i = 0; i < n; ++i) {
    if (param_dtype[i] != RKL_BF16 && param_dtype[i] != RKL_FP32)
      return fail(RKL_ERR_DTYPE, "unknown dtype %d of parameter %d", param_dtype[i], i);
    if (grad_dtype[i] != RKL_BF16 && grad_dtype[i] != RKL_FP32)
      return fail(RKL_ERR_DTYPE, "unknown dtype %d of gradient %d", grad_dtype[i], i);
    if (numel[i] == 0 || grads[i] == nullptr) continue;
    if (params[i] == nullptr) return fail(RKL_ERR_NULL, "parameter %d is NULL", i);
    if (reinterpret_cast<uintptr_t>(params[i]) & (param_dtype[i] == RKL_BF16 ? 1 : 3))
      return fail(RKL_ERR_ALIGN, "parameter %d is not aligned to its elements", i);
    if (reinterpret_cast<uintptr_t>(grads[i]) & (grad_dtype[i] == RKL_BF16 ? 1 : 3))
      return fail(RKL_ERR_ALIGN, "gradient %d is not aligned to its elements", i);
  }
  int sms = 0;
  RKL_TRY(device_setup(&sms));
  AdamwArgs a;
  a.total = total;
  a.m = exp_avg;
  a.v = exp_avg_sq;
  a.m_scale = exp_avg_scale;
  a.v_scale = exp_avg_sq_scale;
  a.master = master;
  a.control = control;
  a.norm = norm;
  a.lr_dev = lr_dev;
  a.lr = static_cast<float>(lr);
  a.beta1 = static_cast<float>(beta1);
  a.beta2 = static_cast<float>(beta2);
  a.omb1 = static_cast<float>(1 - beta1);
  a.omb2 = static_cast<float>(1 - beta2);
  a.log_beta1 = static_cast<float>(log(beta1));  // -inf for 0: 1 - b^t = 1
  a.log_beta2 = static_cast<float>(log(beta2));
  // With v = 0 too, 0 / eps has to stay 0 (the elements between two tensors): no
  // less than the smallest number whose reciprocal the kernels' approximation has.
  // 8-bit states: no less than what v below fp32's normal numbers, which that kernel
  // takes as 0, comes from (gradients of 3.4e-18 with beta2 = 0.999; blocks of v up
  // to 2^-100, gradients of 3e-14, have no digits there at all).
  const float least_eps = state_bits == 8 ? 3.469446951953614e-18f : FLT_MIN;
  a.eps = eps < least_eps ? least_eps : static_cast<float>(eps);
  a.beta1_64 = beta1;
  a.beta2_64 = beta2;
  a.max_norm = max_norm;
  a.seed = seed;
  a.n = 0;
  a.blocks = 0;
  int64_t at = 0;
  for (int32_t i = 0; i <= n; ++i) {
    const int64_t blocks = i < n ? (numel[i] + kOptBlock - 1) / kOptBlock : 0;
    const bool taken = i < n && numel[i] > 0 && grads[i] != nullptr;
    if (i == n || (taken && (a.n == kOptTensors || a.blocks + blocks > INT32_MAX / 2))) {
      // (a step with nothing to update still counts)
      a.advance = i == n;
      const int64_t need = (a.blocks + kOptWarps - 1) / kOptWarps;
      const int64_t most = int64_t(sms) * (state_bits == 8 ? kOpt8PerSm : kOptPerSm);
      RKL_CUDA(launch_adamw(state_bits, a, static_cast<int>(need < 1 ? 1 : (need < most ? need : most)),
                            static_cast<cudaStream_t>(stream)));
      a.n = 0;
      a.blocks = 0;
    }
    if (taken) {
      AdamwTensor& x = a.t[a.n];
      x.param = params[i];
      x.grad = grads[i];
      x.n = numel[i];
      x.at = at;
      x.decay = weight_decay[i];
      x.flags = (param_dtype[i] == RKL_BF16 ? OPT_PARAM_BF16 : 0u) | (grad_dtype[i] == RKL_BF16 ? OPT_GRAD_BF16 : 0u) |
                (wide_access(params[i], param_dtype[i]) ? OPT_WIDE_PARAM : 0u) |
                (wide_access(grads[i], grad_dtype[i]) ? OPT_WIDE_GRAD : 0u);
      a.first[a.n++] = a.blocks;
      a.blocks += static_cast<int>(blocks);
    }
    at += blocks * kOptBlock;
  }
  return RKL_OK;
}

rkl_status rkl_grad_norm_workspace_size(int32_t n, size_t* bytes) {
  if (bytes == nullptr) return fail(RKL_ERR_NULL, "bytes is NULL");
  if (n < 0) return fail(RKL_ERR_SHAPE, "n = %d is negative", n);
  const size_t launches = n <= kOptTensors ? 1 : (n + kOptTensors - 1) / kOptTensors;
  *bytes = launches * kNormMaxGrid * sizeof(double);
  return RKL_OK;
}

rkl_status rkl_grad_norm(int32_t n, const void* const* grads, const int64_t* numel, const int32_t* grad_dtype,
                         float* norm, void* workspace, size_t workspace_bytes, void* stream) {
  RKL_NVTX_RANGE();
  RKL_TRY(check_tensor_counts(n, numel));
  if (n > 0 && (grads == nullptr || grad_dtype == nullptr))
    return fail(RKL_ERR_NULL, "grads and grad_dtype must be non-NULL");
  if (norm == nullptr) return fail(RKL_ERR_NULL, "norm is NULL");
  if (reinterpret_cast<uintptr_t>(norm) & 3) return fail(RKL_ERR_ALIGN, "norm is not 4-byte aligned");
  for (int32_t i = 0; i < n; ++i) {
    if (grad_dtype[i] != RKL_BF16 && grad_dtype[i] != RKL_FP32)
      return fail(RKL_ERR_DTYPE, "unknown dtype %d of gradient %d", grad_dtype[i], i);
    if (reinterpret_cast<uintptr_t>(grads[i]) & (grad_dtype[i] == RKL_BF16 ? 1 : 3))
      return fail(RKL_ERR_ALIGN, "gradient %d is not aligned to its elements", i);
    if ((numel[i] + kNormChunk - 1) / kNormChunk > INT32_MAX / 2)
      return fail(RKL_ERR_SHAPE, "gradient %d has too many elements", i);
  }
  size_t need_ws = 0;
  RKL_TRY(rkl_grad_norm_workspace_size(n, &need_ws));
  if (workspace == nullptr || workspace_bytes < need_ws)
    return fail(RKL_ERR_WORKSPACE, "workspace is NULL or smaller than %zu bytes", need_ws);
  RKL_TRY(check_ptr(workspace, "workspace"));
  int sms = 0;
  RKL_TRY(device_setup(&sms));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  NormArgs a;
  a.n = 0;
  int64_t chunks = 0;
  int partials = 0;
  for (int32_t i = 0; i <= n; ++i) {
    const int64_t more = i < n ? (numel[i] + kNormChunk - 1) / kNormChunk : 0;
    const bool taken = i < n && numel[i] > 0 && grads[i] != nullptr;
    // a full table, or (a launch's chunks are counted in 32 bits) too many elements, begins another launch
    if (a.n > 0 && (i == n || (taken && (a.n == kOptTensors || chunks + more > INT32_MAX / 2)))) {
      a.chunks = static_cast<int>(chunks);
      const int64_t need = (chunks + kOptWarps - 1) / kOptWarps;
      const int most = sms * kNormPerSm < kNormMaxGrid ? sms * kNormPerSm : kNormMaxGrid;
      const int grid = static_cast<int>(need < most ? need : most);
      if ((partials + grid) * sizeof(double) > workspace_bytes)
        return fail(RKL_ERR_SHAPE, "the gradients have too many elements for %d tensors", n);
      a.partial = static_cast<double*>(workspace) + partials;
      RKL_CUDA(launch_norm_partial(a, grid, s));
      partials += grid;
      a.n = 0;
      chunks = 0;
    }
    if (taken) {
      a.t[a.n].grad = grads[i];
      a.t[a.n].n = numel[i];
      a.t[a.n].flags = (grad_dtype[i] == RKL_BF16 ? OPT_GRAD_BF16 : 0u) |
                       (wide_access(grads[i], grad_dtype[i]) ? OPT_WIDE_GRAD : 0u);
      a.first[a.n++] = static_cast<int>(chunks);
      chunks += more;
    }
  }
  RKL_CUDA(launch_norm_final(static_cast<const double*>(workspace), partials, norm, s));
  return RKL_OK;
}

// ====================================================================== gated feed-forward block
static rkl_status check_ffn(rkl_dtype dtype, int activation, int64_t T, int64_t H, int64_t F, int64_t O) {
  if (dtype != RKL_BF16 && dtype != RKL_FP32) return fail(RKL_ERR_DTYPE, "unknown dtype %d", (int)dtype);
  if (activation < ACT_SILU || activation > ACT_RELU) return fail(RKL_ERR_DTYPE, "unknown activation %d", activation);
  if (T < 0 || H < 1 || F < 1 || O < 1) return fail(RKL_ERR_SHAPE, "T must be >= 0 and H, F, O >= 1");
  if (T >= (int64_t(1) << 30) || H > (1 << 20) || F > (1 << 20) || O > (1 << 20))
    return fail(RKL_ERR_SHAPE, "T = %lld, H = %lld, F = %lld, O = %lld: too large", (long long)T, (long long)H,
                (long long)F, (long long)O);
  return RKL_OK;
}

// fp32 tensors are aligned to their elements; so are bf16 ones of odd widths,
// which are copied; TMA reads the others where they lie.
static unsigned ffn_alignment(rkl_dtype dtype, int64_t H, int64_t F, int64_t O) {
  return dtype == RKL_FP32 ? 4 : (H % 8 || F % 8 || O % 8) ? 2 : 16;
}

static rkl_status check_ffn_ptr(const void* p, const char* name, unsigned alignment, bool required = true) {
  if (p == nullptr) return required ? fail(RKL_ERR_NULL, "%s is NULL", name) : RKL_OK;
  if (reinterpret_cast<uintptr_t>(p) & (alignment - 1))
    return fail(RKL_ERR_ALIGN, "%s is not %u-byte aligned", name, alignment);
  return RKL_OK;
}

// ---- plan of the gated block, by its sizes and type alone
constexpr int kPlanSms = 148;

// ffn_skinny_kernel's share: `per` steps a CTA (4 at least: a part is written
// and read again), and the most parts a tile has.
struct SkinnyPlan {
  int tiles = 0, tiles_first = 0, steps = 0, grid = 0, parts = 0, pitch = 0;
  long long per = 0;
};

static SkinnyPlan skinny_plan(int64_t rows_first, int64_t rows_second, int64_t K) {
  SkinnyPlan p;
  p.tiles_first = static_cast<int>((rows_first + 127) / 128);
  p.tiles = p.tiles_first + static_cast<int>((rows_second + 127) / 128);
  p.steps = static_cast<int>((K + kBK - 1) / kBK);
  const long long all = static_cast<long long>(p.tiles) * p.steps;
  p.per = (all + kPlanSms - 1) / kPlanSms;
  if (p.per < 4) p.per = 4;
  p.grid = static_cast<int>((all + p.per - 1) / p.per);
  // a tile of `steps` that begins anywhere in a CTA's share touches this many CTAs at most
  p.parts = static_cast<int>((p.steps - 2 + p.per) / p.per) + 1;
  p.pitch = p.tiles * 128;
  return p;
}

// Parts of K for a product of `tiles` pair tiles of `steps` 128-deep steps
// (0.58 us each) beside `others` steps of the same launch: what the longest
// pair of CTAs takes, plus the parts' way through memory (8 bytes a result and
// part at 5 TB/s, and 3 us for the join).
static int pair_parts(int64_t tiles, int64_t steps, int64_t others, int64_t M, int64_t N) {
  const int64_t pairs = kPlanSms / 2;
  double best = 0;
  int parts = 1;
  for (int n = 1; n <= 16 && n <= steps; ++n) {
    const int64_t chain = (steps + n - 1) / n;
    int64_t longest = (tiles * n + pairs - 1) / pairs * chain;
    if (others > 0) {
      const int64_t fair = (tiles * steps + others + pairs - 1) / pairs;
      longest = chain > fair ? chain : fair;
    }
    const double us = 0.58 * static_cast<double>(longest) +
                      (n > 1 ? 3.0 + 8.0 * n * static_cast<double>(M) * static_cast<double>(N) / 5e6 : 0.0);
    if (n == 1 || us < best) {
      best = us;
      parts = n;
    }
  }
  return parts;
}

static int64_t tiles_of(int64_t n, int64_t t) { return (n + t - 1) / t; }

struct FfnPlan {
  bool tc = false, skinny = false;     // on the tensor cores (bf16); few rows
  int terms = 1;                       // bf16 terms of a, dg and du
  SkinnyPlan up, down;
  int parts = 1, part_rows = 0;        // of y (forward) or dx (backward)
  size_t plane = 0;                    // bytes of a [T, F] operand
  size_t off_counter = 0, off_part = 0, total = 0;
  bool padded = false;                 // bf16 of odd widths: copies at off_pad (backward, two terms: x and dy)
  size_t off_pad = 0;
  int64_t inner = 0;                   // F without its padding
};

static FfnPlan ffn_plan(rkl_dtype dtype, int64_t T, int64_t H, int64_t F, int64_t O, bool backward) {
  FfnPlan p;
  p.tc = dtype == RKL_BF16 && T > 0;
  if (p.tc && (H % 8 || F % 8 || O % 8)) {
    // rows of whole 16 bytes: the padded problem's plan, and copies behind its workspace
    const int64_t Hp = (H + 7) / 8 * 8, Fp = (F + 7) / 8 * 8, Op = (O + 7) / 8 * 8;
    p = ffn_plan(dtype, T, Hp, Fp, Op, backward);
    p.padded = true;
    p.inner = F;
    p.off_pad = align256(p.total);
    const size_t x = align256(T * Hp * 2), wide = align256(Fp * Hp * 2), down = align256(Op * Fp * 2),
                 y = align256(T * Op * 2);
    p.total = p.off_pad + (backward ? p.terms * (x + y) + x + 2 * (2 * wide + down) : x + 2 * wide + down + y);
    return p;
  }
  if (p.tc && T <= kFfnTermRows && (T * F <= kFfnTermElements || T * (backward ? H : O) <= kFfnTermResults)) p.terms = 2;
  p.inner = F;
  p.plane = size_t(T) * F * (dtype == RKL_BF16 ? 2 * p.terms : 4);
  p.off_counter = align256((backward ? 3 : 1) * p.plane);
  p.off_part = p.off_counter + 256;
  p.total = p.off_part;
  if (!p.tc) return p;
  p.part_rows = static_cast<int>((p.terms * T + 31) / 32 * 32);
  if (backward) {
    const int64_t mt = tiles_of(T, 256), steps_t = tiles_of(T, 128);
    const int64_t others =
        (2 * tiles_of(F, 256) * tiles_of(H, 256) + tiles_of(O, 256) * tiles_of(F, 256)) * steps_t;
    p.parts = pair_parts(mt * tiles_of(H, 256), 2 * tiles_of(F, 128), others, p.terms * T, H);
    if (p.parts > 1 || p.terms > 1) p.total += size_t(p.parts) * p.part_rows * H * 4;
    if (p.terms > 1) {
      p.off_pad = align256(p.total);
      p.total = p.off_pad + align256(2 * T * H * 2) + align256(2 * T * O * 2);
    }
    return p;
  }
  p.skinny = T <= kFfnSkinnyRows;
  if (p.skinny) {
    p.up = skinny_plan(F, F, H);
    p.down = skinny_plan(O, 0, F);
    const size_t up = size_t(p.up.parts) * T * p.up.pitch * 4, down = size_t(p.down.parts) * p.terms * T * p.down.pitch * 4;
    p.total += up > down ? up : down;
    return p;
  }
  p.parts = pair_parts(tiles_of(T, 256) * tiles_of(O, 256), tiles_of(F, 128), 0, T, O);
  if (p.parts > 1) p.total += size_t(p.parts) * p.part_rows * O * 4;
  return p;
}

// Map of a bf16 operand: `rows` x `cols` row-major, read K-major (K = columns)
// or MN-major (K = rows).  live > 0: columns from there on read as zeros.
static rkl_status operand_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, bool mn, int64_t live = 0) {
  return make_map(m, p, false, live > 0 ? live : cols, rows, cols * 2, kBK, mn ? kBK : 128);
}

// Map of a bf16 result, stored in 32 x 32 boxes.
static rkl_status result_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols) {
  return make_map(m, p, false, cols, rows, cols * 2, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
}

// One product of a launch's list: A and B row-major as they lie, `*_mn` where K
// is their row index.  a_live > 0: columns of A (K-major) from there on are
// padding, which may hold anything: act(g) u of an infinite row of x is infinity
// x 0 there.
static rkl_status pair_product(FfnPairArgs& a, const void* A, const void* A2, bool a_mn, const void* B, const void* B2,
                               bool b_mn, void* C, int64_t M, int64_t N, int64_t K, bool up, int64_t a_live = 0,
                               int parts = 1, int part_rows = 0) {
  FfnPairProduct& p = a.p[a.n++];
  RKL_TRY(operand_map(&p.a[0], A, a_mn ? K : M, a_mn ? M : K, a_mn, a_live));
  p.a[1] = p.a[0];
  if (A2) RKL_TRY(operand_map(&p.a[1], A2, a_mn ? K : M, a_mn ? M : K, a_mn, a_live));
  RKL_TRY(operand_map(&p.b[0], B, b_mn ? K : N, b_mn ? N : K, b_mn));
  p.b[1] = p.b[0];
  if (B2) RKL_TRY(operand_map(&p.b[1], B2, b_mn ? K : N, b_mn ? N : K, b_mn));
  if (part_rows > 0)
    RKL_TRY(make_map(&p.c, C, true, N, int64_t(parts) * part_rows, N * 4, 32, 32));
  else
    RKL_TRY(result_map(&p.c, C, M, N));
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.mt = static_cast<int>(tiles_of(M, 256));
  p.nt = static_cast<int>(tiles_of(N, up ? 128 : 256));
  p.steps = static_cast<int>(tiles_of(K, 128));
  p.segments = A2 ? 2 : 1;
  p.a_mn = a_mn;
  p.b_mn = b_mn;
  p.parts = parts;
  p.part_rows = part_rows;
  p.first = a.items;
  a.items += p.mt * p.nt * parts;
  return RKL_OK;
}

// (x_live: as a_live above)
static rkl_status skinny_product(const SkinnyPlan& p, const void* x, const void* W1, int64_t R1, const void* W2, int64_t T,
                                 int64_t K, int64_t x_live, float* part, bool follows, cudaStream_t s) {
  FfnSkinnyArgs a = {};
  a.cols = static_cast<int>((T + 15) / 16 * 16);
  RKL_TRY(operand_map(&a.w1, W1, R1, K, false));
  a.w2 = a.w1;
  if (W2) RKL_TRY(operand_map(&a.w2, W2, R1, K, false));
  RKL_TRY(make_map(&a.x, x, false, x_live, T, K * 2, kBK, a.cols));
  a.part = part;
  a.per = p.per;
  a.tiles = p.tiles;
  a.tiles_first = p.tiles_first;
  a.steps = p.steps;
  a.T = static_cast<int>(T);
  a.pitch = p.pitch;
  a.parts = p.parts;
  a.follows = follows;
  RKL_CUDA(launch_ffn_skinny(a, p.grid, s));
  return RKL_OK;
}

static FfnJoinArgs join_args(const float* part, void* out, int64_t T, int64_t N) {
  FfnJoinArgs j = {};
  j.part = part;
  j.out = static_cast<uint16_t*>(out);
  j.T = static_cast<int>(T);
  j.N = static_cast<int>(N);
  return j;
}

static rkl_status join_skinny(const SkinnyPlan& p, int act, const float* part, void* out, void* rest, float* saved,
                              int64_t T, int64_t N, int terms, cudaStream_t s) {
  FfnJoinArgs j = join_args(part, out, T, N);
  j.rest = static_cast<uint16_t*>(rest);
  j.saved = saved;
  j.terms = terms;
  j.pitch = p.pitch;
  j.slab = (act < 0 ? terms : 1) * T * p.pitch;  // (two terms: as many rows more)
  j.per = p.per;
  j.second = p.tiles_first * 128;
  j.steps = p.steps;
  RKL_CUDA(launch_ffn_join(act, j, s));
  return RKL_OK;
}

static rkl_status join_pair(const FfnPlan& p, const float* part, void* out, int64_t T, int64_t N, cudaStream_t s) {
  FfnJoinArgs j = join_args(part, out, T, N);
  j.pitch = N;
  j.slab = int64_t(p.part_rows) * N;
  j.parts = p.parts;
  j.terms = p.terms;
  RKL_CUDA(launch_ffn_join(-1, j, s));
  return RKL_OK;
}

static rkl_status ffn_forward_tc(const FfnPlan& p, const void* x, const void* W_gate, const void* W_up,
                                 const void* W_down, int act, int64_t T, int64_t H, int64_t F, int64_t O, void* y,
                                 float* saved, uint8_t* ws, int sms, cudaStream_t s) {
  float* part = reinterpret_cast<float*>(ws + p.off_part);
  if (p.skinny) {
    RKL_TRY(skinny_product(p.up, x, W_gate, F, W_up, T, H, H, part, false, s));
    RKL_TRY(join_skinny(p.up, act, part, ws, p.terms > 1 ? ws + p.plane / 2 : nullptr, saved, T, F, p.terms, s));
    RKL_TRY(skinny_product(p.down, ws, W_down, O, nullptr, p.terms * T, F, p.inner, part, true, s));
    return join_skinny(p.down, -1, part, y, nullptr, nullptr, T, O, p.terms, s);
  }
  FfnPairArgs a = {};
  RKL_TRY(pair_product(a, x, nullptr, false, W_gate, W_up, false, ws, T, F, H, true));
  a.saved = saved;
  RKL_CUDA(launch_ffn_pair(FFN_UP, act, a, sms, s));
  FfnPairArgs d = {};
  d.follows = true;
  RKL_TRY(pair_product(d, ws, nullptr, false, W_down, nullptr, false, p.parts > 1 ? static_cast<void*>(part) : y, T, O, F,
                       false, p.inner, p.parts, p.parts > 1 ? p.part_rows : 0));
  RKL_CUDA(launch_ffn_pair(FFN_GEMM, act, d, sms, s));
  return p.parts > 1 ? join_pair(p, part, y, T, O, s) : RKL_OK;
}

// p.terms = 2: x and dy hold their T rows twice, for the weights' gradients of
// the 2 T rows that a, dg and du then are.
static rkl_status ffn_backward_tc(const FfnPlan& p, const void* x, const void* W_gate, const void* W_up,
                                  const void* W_down, int act, int64_t T, int64_t H, int64_t F, int64_t O,
                                  const void* dy, const float* saved, void* dx, void* dW_gate, void* dW_up,
                                  void* dW_down, uint8_t* ws, int sms, cudaStream_t s) {
  void *a_plane = ws, *dg = ws + p.plane, *du = ws + 2 * p.plane;
  int* counter = reinterpret_cast<int*>(ws + p.off_counter);
  float* part = reinterpret_cast<float*>(ws + p.off_part);
  FfnPairArgs a = {};
  RKL_TRY(pair_product(a, dy, nullptr, false, W_down, nullptr, true, a_plane, T, F, O, false));
  RKL_TRY(result_map(&a.c2, dg, T, F));
  RKL_TRY(result_map(&a.c3, du, T, F));
  if (p.terms > 1)
    for (int i = 0; i < 3; ++i) RKL_TRY(result_map(&a.rest[i], ws + i * p.plane + p.plane / 2, T, F));
  a.saved = const_cast<float*>(saved);
  a.zero_counter = counter;
  RKL_CUDA(launch_ffn_pair(p.terms > 1 ? FFN_DGATE_TERMS : FFN_DGATE, act, a, sms, s));
  // longest items (K = 2 F) first
  FfnPairArgs d = {};
  d.follows = true;
  d.counter = counter;
  const int64_t rows = p.terms * T;
  const bool joined = p.parts > 1 || p.terms > 1;
  if (dx)
    RKL_TRY(pair_product(d, dg, du, false, W_gate, W_up, true, joined ? static_cast<void*>(part) : dx, rows, H, F, false,
                         p.inner, p.parts, joined ? p.part_rows : 0));
  if (dW_gate) RKL_TRY(pair_product(d, dg, nullptr, true, x, nullptr, true, dW_gate, F, H, rows, false));
  if (dW_up) RKL_TRY(pair_product(d, du, nullptr, true, x, nullptr, true, dW_up, F, H, rows, false));
  if (dW_down) RKL_TRY(pair_product(d, dy, nullptr, true, a_plane, nullptr, true, dW_down, O, F, rows, false));
  RKL_CUDA(launch_ffn_pair(FFN_GEMM, act, d, sms, s));
  return dx && joined ? join_pair(p, part, dx, T, H, s) : RKL_OK;
}

// Matrices laid out anew: the odd-width problem's in rows of whole 16 bytes, and
// x and dy twice where a backward pass has two terms.
struct Padding {
  FfnPadArgs in = {}, out = {};
  uint8_t* at;

  explicit Padding(uint8_t* ws) : at(ws) {}
  static int up8(int64_t n) { return static_cast<int>((n + 7) / 8 * 8); }
  uint16_t* take(int64_t rows, int64_t cols) {
    uint16_t* p = reinterpret_cast<uint16_t*>(at);
    at += align256(size_t(rows) * cols * 2);
    return p;
  }
  static void add(FfnPadArgs& a, const void* src, void* dst, int64_t rows, int64_t cols, int64_t src_pitch,
                  int64_t dst_rows, int64_t dst_cols) {
    a.item[a.n++] = {static_cast<const uint16_t*>(src), static_cast<uint16_t*>(dst), static_cast<int>(rows),
                     static_cast<int>(cols),            static_cast<int>(src_pitch), static_cast<int>(dst_rows),
                     static_cast<int>(dst_cols),        a.total};
    a.total += dst_rows * dst_cols;
  }
  // A copy of an input, its rows padded too where they are an odd width elsewhere.
  const void* input(const void* src, int64_t rows, int64_t cols, bool pad_rows, int times = 1) {
    const int64_t r = pad_rows ? up8(rows) : rows, c = up8(cols);
    uint16_t* p = take(times * r, c);
    for (int i = 0; i < times; ++i) add(in, src, p + i * r * c, rows, cols, cols, r, c);
    return p;
  }
  // Where an output is computed; `finish` copies it to dst (nullptr: left out).
  void* output(void* dst, int64_t rows, int64_t cols, bool pad_rows) {
    if (dst == nullptr) return nullptr;
    const int64_t r = pad_rows ? up8(rows) : rows, c = up8(cols);
    uint16_t* p = take(r, c);
    add(out, p, dst, rows, cols, c, rows, cols);
    return p;
  }
};

rkl_status rkl_ffn_workspace_size(rkl_dtype dtype, int64_t T, int64_t H, int64_t F, int64_t O, int32_t backward,
                                  size_t* bytes) {
  if (bytes == nullptr) return fail(RKL_ERR_NULL, "bytes is NULL");
  RKL_TRY(check_ffn(dtype, ACT_SILU, T, H, F, O));
  *bytes = ffn_plan(dtype, T, H, F, O, backward != 0).total;
  return RKL_OK;
}

rkl_status rkl_ffn_saved_size(int64_t T, int64_t F, int64_t* elements) {
  if (elements == nullptr) return fail(RKL_ERR_NULL, "elements is NULL");
  RKL_TRY(check_ffn(RKL_FP32, ACT_SILU, T, 1, F, 1));
  *elements = 2 * ffn_saved_plane(T, F);
  return RKL_OK;
}

rkl_status rkl_ffn_forward(const void* x, const void* W_gate, const void* W_up, const void* W_down, rkl_dtype dtype,
                           int32_t activation, int64_t T, int64_t H, int64_t F, int64_t O, void* y, float* saved,
                           void* workspace, size_t workspace_bytes, void* stream) {
  RKL_NVTX_RANGE();
  RKL_TRY(check_ffn(dtype, activation, T, H, F, O));
  const unsigned align = ffn_alignment(dtype, H, F, O);
  RKL_TRY(check_ffn_ptr(W_gate, "W_gate", align));
  RKL_TRY(check_ffn_ptr(W_up, "W_up", align));
  RKL_TRY(check_ffn_ptr(W_down, "W_down", align));
  if (T == 0) return RKL_OK;
  RKL_TRY(check_ffn_ptr(x, "x", align));
  RKL_TRY(check_ffn_ptr(y, "y", align));
  RKL_TRY(check_ptr(saved, "saved", false));
  const FfnPlan plan = ffn_plan(dtype, T, H, F, O, false);
  if (workspace == nullptr || workspace_bytes < plan.total)
    return fail(RKL_ERR_WORKSPACE, "workspace is NULL or smaller than %zu bytes", plan.total);
  RKL_TRY(check_ptr(workspace, "workspace"));
  int sms = 0;
  RKL_TRY(device_setup(&sms));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (plan.padded) {
    Padding pad(ws + plan.off_pad);
    const void* px = pad.input(x, T, H, false);
    const void* pg = pad.input(W_gate, F, H, true);
    const void* pu = pad.input(W_up, F, H, true);
    const void* pd = pad.input(W_down, O, F, true);
    void* py = pad.output(y, T, O, false);
    RKL_CUDA(launch_ffn_pad(pad.in, s));
    RKL_TRY(ffn_forward_tc(plan, px, pg, pu, pd, activation, T, Padding::up8(H), Padding::up8(F), Padding::up8(O), py,
                           saved, ws, sms, s));
    RKL_CUDA(launch_ffn_pad(pad.out, s));
    return RKL_OK;
  }
  if (plan.tc) return ffn_forward_tc(plan, x, W_gate, W_up, W_down, activation, T, H, F, O, y, saved, ws, sms, s);
  const auto f32 = [](const void* p) { return static_cast<const float*>(p); };
  float* act = reinterpret_cast<float*>(ws);
  FfnSimtArgs a = {};
  a.n = 1;
  a.act = activation;
  a.saved = saved;
  // a = act(x Wg^T) (x Wu^T)
  a.p[0] = {{f32(x), nullptr}, {f32(W_gate), f32(W_up)}, act, T, F, H, H, 1, 1, H, 1, 0};
  RKL_CUDA(launch_ffn_simt(FFN_UP, a, sms, s));
  // y = a Wd^T
  a.p[0] = {{act, nullptr}, {f32(W_down), nullptr}, static_cast<float*>(y), T, O, F, F, 1, 1, F, 1, 0};
  RKL_CUDA(launch_ffn_simt(FFN_GEMM, a, sms, s));
  return RKL_OK;
}

rkl_status rkl_ffn_backward(const void* x, const void* W_gate, const void* W_up, const void* W_down, rkl_dtype dtype,
                            int32_t activation, int64_t T, int64_t H, int64_t F, int64_t O, const void* dy,
                            const float* saved, void* dx, void* dW_gate, void* dW_up, void* dW_down, void* workspace,
                            size_t workspace_bytes, void* stream) {
  RKL_NVTX_RANGE();
  RKL_TRY(check_ffn(dtype, activation, T, H, F, O));
  const unsigned align = ffn_alignment(dtype, H, F, O);
  RKL_TRY(check_ffn_ptr(W_gate, "W_gate", align));
  RKL_TRY(check_ffn_ptr(W_up, "W_up", align));
  RKL_TRY(check_ffn_ptr(W_down, "W_down", align));
  RKL_TRY(check_ffn_ptr(dx, "dx", align, false));
  RKL_TRY(check_ffn_ptr(dW_gate, "dW_gate", align, false));
  RKL_TRY(check_ffn_ptr(dW_up, "dW_up", align, false));
  RKL_TRY(check_ffn_ptr(dW_down, "dW_down", align, false));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t es = dtype == RKL_BF16 ? 2 : 4;
  if (T == 0) {  // no rows: the weights' gradients are zero
    if (dW_gate) RKL_CUDA(cudaMemsetAsync(dW_gate, 0, size_t(F) * H * es, s));
    if (dW_up) RKL_CUDA(cudaMemsetAsync(dW_up, 0, size_t(F) * H * es, s));
    if (dW_down) RKL_CUDA(cudaMemsetAsync(dW_down, 0, size_t(O) * F * es, s));
    return RKL_OK;
  }
  RKL_TRY(check_ffn_ptr(x, "x", align));
  RKL_TRY(check_ffn_ptr(dy, "dy", align));
  RKL_TRY(check_ptr(saved, "saved"));
  const FfnPlan plan = ffn_plan(dtype, T, H, F, O, true);
  if (workspace == nullptr || workspace_bytes < plan.total)
    return fail(RKL_ERR_WORKSPACE, "workspace is NULL or smaller than %zu bytes", plan.total);
  RKL_TRY(check_ptr(workspace, "workspace"));
  if (!dx && !dW_gate && !dW_up && !dW_down) return RKL_OK;
  int sms = 0;
  RKL_TRY(device_setup(&sms));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (plan.padded) {
    Padding pad(ws + plan.off_pad);
    const void* px = pad.input(x, T, H, false, plan.terms);
    const void* pg = pad.input(W_gate, F, H, true);
    const void* pu = pad.input(W_up, F, H, true);
    const void* pd = pad.input(W_down, O, F, true);
    const void* pdy = pad.input(dy, T, O, false, plan.terms);
    void* pdx = pad.output(dx, T, H, false);
    void* pdg = pad.output(dW_gate, F, H, true);
    void* pdu = pad.output(dW_up, F, H, true);
    void* pdd = pad.output(dW_down, O, F, true);
    RKL_CUDA(launch_ffn_pad(pad.in, s));
    RKL_TRY(ffn_backward_tc(plan, px, pg, pu, pd, activation, T, Padding::up8(H), Padding::up8(F), Padding::up8(O), pdy,
                            saved, pdx, pdg, pdu, pdd, ws, sms, s));
    RKL_CUDA(launch_ffn_pad(pad.out, s));
    return RKL_OK;
  }
  if (plan.tc && plan.terms > 1) {
    Padding twice(ws + plan.off_pad);
    x = twice.input(x, T, H, false, 2);
    dy = twice.input(dy, T, O, false, 2);
    RKL_CUDA(launch_ffn_pad(twice.in, s));
  }
  if (plan.tc)
    return ffn_backward_tc(plan, x, W_gate, W_up, W_down, activation, T, H, F, O, dy, saved, dx, dW_gate, dW_up, dW_down,
                           ws, sms, s);
  const auto f32 = [](const void* p) { return static_cast<const float*>(p); };
  const auto out = [](void* p) { return static_cast<float*>(p); };
  FfnSimtArgs a = {};
  a.act = activation;
  a.saved = const_cast<float*>(saved);
  float* act = reinterpret_cast<float*>(ws);  // a, dg and du, [T, F] each
  const float *dg = act + T * F, *du = dg + T * F;
  // da = dy Wd -> a, dg, du
  a.n = 1;
  a.p[0] = {{f32(dy), nullptr}, {f32(W_down), nullptr}, act, T, F, O, O, 1, F, 1, 1, 0};
  RKL_CUDA(launch_ffn_simt(FFN_DGATE, a, sms, s));
  a.n = 0;
  if (dx) a.p[a.n++] = {{dg, du}, {f32(W_gate), f32(W_up)}, out(dx), T, H, F, F, 1, H, 1, 2, 0};
  if (dW_gate) a.p[a.n++] = {{dg, nullptr}, {f32(x), nullptr}, out(dW_gate), F, H, T, 1, F, H, 1, 1, 0};
  if (dW_up) a.p[a.n++] = {{du, nullptr}, {f32(x), nullptr}, out(dW_up), F, H, T, 1, F, H, 1, 1, 0};
  if (dW_down) a.p[a.n++] = {{f32(dy), nullptr}, {act, nullptr}, out(dW_down), O, F, T, 1, O, F, 1, 1, 0};
  RKL_CUDA(launch_ffn_simt(FFN_GEMM, a, sms, s));
  return RKL_OK;
}

int32_t rkl_kernel_count(void) { return K_COUNT; }

const char* rkl_kernel_name(int32_t kernel_id) { return kernel_name(kernel_id); }

rkl_status rkl_profile_enable(int32_t enable) {
  g_profile.store(enable != 0);
  return RKL_OK;
}

static rkl_status drain_profile() {
  std::vector<ProfRec> pend;
  {
    std::lock_guard<std::mutex> lk(g_prof_mu);
    pend.swap(g_prof_pending);
  }
  for (const ProfRec& r : pend) {
    float ms = 0.f;
    cudaError_t e = cudaEventSynchronize(r.b);
    if (e == cudaSuccess) e = cudaEventElapsedTime(&ms, r.a, r.b);
    cudaEventDestroy(r.a);
    cudaEventDestroy(r.b);
    if (e != cudaSuccess) return fail(RKL_ERR_CUDA, "profile event: %s", cudaGetErrorString(e));
    std::lock_guard<std::mutex> lk(g_prof_mu);
    g_prof_ms[r.id] += ms;
    g_prof_n[r.id] += 1;
  }
  return RKL_OK;
}

rkl_status rkl_profile_reset(void) {
  RKL_TRY(drain_profile());
  std::lock_guard<std::mutex> lk(g_prof_mu);
  for (int i = 0; i < K_COUNT; ++i) {
    g_prof_ms[i] = 0.0;
    g_prof_n[i] = 0;
  }
  return RKL_OK;
}

rkl_status rkl_profile_read(int32_t kernel_id, double* total_ms, int64_t* launches) {
  if (kernel_id < 0 || kernel_id >= K_COUNT) return fail(RKL_ERR_SHAPE, "kernel id %d out of range", kernel_id);
  if (total_ms == nullptr || launches == nullptr) return fail(RKL_ERR_NULL, "outputs are NULL");
  RKL_TRY(drain_profile());
  std::lock_guard<std::mutex> lk(g_prof_mu);
  *total_ms = g_prof_ms[kernel_id];
  *launches = g_prof_n[kernel_id];
  return RKL_OK;
}

int64_t rkl_launch_count(void) { return g_launches.load(); }

}  // extern "C"

// ====================================================================== no-allocation forward
// Scratch of rkl_forward_hidden_noalloc: one array in the library's device
// image.  Every GPU on which the library's kernels are loaded holds these
// bytes until the process exits, whether or not it ever calls that entry
// point.  Host code only sees a stand-in symbol for it; the device address is
// looked up per device below.
namespace rkl {
constexpr size_t kStaticScratchBytes = size_t(32) << 20;  // 32 MiB
static __device__ __align__(256) uint8_t g_static_scratch[kStaticScratchBytes];

static std::mutex g_static_mu;
static void* g_static_ptr[64];  // device address of g_static_scratch, per device

// Looks up (once per device, with that device current) the device address of
// the static scratch array.
static rkl_status static_scratch_ptr(void** out) {
  int dev = 0;
  RKL_CUDA(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return fail(RKL_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
  std::lock_guard<std::mutex> lk(g_static_mu);
  if (g_static_ptr[dev] == nullptr) {
    void* ptr = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&ptr, g_static_scratch);
    if (e != cudaSuccess || ptr == nullptr)
      return fail(RKL_ERR_CUDA, "cudaGetSymbolAddress(static scratch) failed on device %d: %s", dev,
                  cudaGetErrorString(e));
    g_static_ptr[dev] = ptr;
  }
  *out = g_static_ptr[dev];
  return RKL_OK;
}
}  // namespace rkl

extern "C" rkl_status rkl_forward_hidden_noalloc(const void* h_s, const void* h_t, const void* W_s, const void* W_t,
                                                 rkl_dtype dtype, int64_t B, int64_t Sm1, int64_t H, int64_t V,
                                                 const int32_t* row_idx, int32_t N, rkl_reduction reduction,
                                                 float* loss_tok, float* loss, float* saved, void* stream) {
  RKL_NVTX_RANGE();
  // Size check first, from the same layout the workspace path uses; nothing
  // on the device is touched when the problem does not fit.
  RKL_TRY(check_common(RKL_PAYLOAD_HIDDEN, dtype, B, Sm1, H, V, N, reduction));
  const Plan pl = make_plan(RKL_PAYLOAD_HIDDEN, dtype, N, H, V);
  if (pl.off_dz > kStaticScratchBytes)
    return fail(RKL_ERR_WORKSPACE,
                "rkl_forward_hidden_noalloc: this problem needs %zu bytes of scratch, the static limit is %zu "
                "bytes (%zu MiB); use rkl_forward_hidden with a caller workspace",
                pl.off_dz, kStaticScratchBytes, kStaticScratchBytes >> 20);
  void* scratch = nullptr;
  RKL_TRY(static_scratch_ptr(&scratch));
  // Every region of the scratch that the forward reads is written earlier in
  // the same call, so nothing needs clearing between calls.
  return forward_impl(RKL_PAYLOAD_HIDDEN, h_s, h_t, W_s, W_t, dtype, B, Sm1, H, V, row_idx, N, nullptr, reduction,
                      loss_tok, loss, saved, scratch, kStaticScratchBytes, stream, /*forward_only_workspace=*/true);
}
