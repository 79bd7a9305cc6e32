// C-ABI entry points of the exact-attention library (declared in include/fa_attention.h).
//
// This layer validates arguments on the host (nothing is launched for a bad
// call), encodes the TMA descriptors of the [B*H, N, d] tensors, lays out the
// backward workspace, and owns the device error word that the kernels' bounded
// waits write.  It allocates no device memory.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <utility>
#include <vector>

#include "../../include/fa_attention.h"
#include "fa_internal.h"
#include "fa_kv4.h"
#include "fa_kv4_plan.h"
#include "fa_marks.h"
#include "fa_nvtx.h"
#include "fa_rotary.h"
#include "ptx.cuh"

namespace fa {

// Device error record the kernels write when a bounded wait gives up (one per
// device that loads the library): bits, first failure code, its CTA, its barrier.
__device__ uint32_t g_error_word[4];

namespace {

constexpr int kMaxDevices = 64;
uint32_t g_last_detail[4] = {0, 0, 0, 0};

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// The current CUDA context (driver API, looked up through the runtime's entry-point
// query so the library needs no link against libcuda), or nullptr.
using CtxGetCurrentFn = CUresult (*)(CUcontext*);
CUcontext current_context() {
  static CtxGetCurrentFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<CtxGetCurrentFn>(p);
  });
  CUcontext c = nullptr;
  if (fn && fn(&c) != CUDA_SUCCESS) c = nullptr;
  return c;
}

// Device address of a __device__ symbol on the current device, cached per device
// and keyed on the device's current context: after cudaDeviceReset (a new primary
// context) the address is looked up again instead of reusing a stale one.
struct SymbolCache {
  std::mutex mu;
  CUcontext ctx[kMaxDevices] = {};
  void* ptr[kMaxDevices] = {};
  void* get(const void* symbol) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    // (before the first runtime call on a thread no context may be current yet: the
    // lookup below makes it current, and the next call re-keys the cache once)
    const CUcontext c = current_context();
    std::lock_guard<std::mutex> lock(mu);
    if (!ptr[dev] || c != ctx[dev]) {
      void* p = nullptr;
      if (cudaGetSymbolAddress(&p, symbol) != cudaSuccess) return nullptr;
      ptr[dev] = p;
      ctx[dev] = c;
    }
    return ptr[dev];
  }
};

int sm_count() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 1;
  return sms > 0 ? sms : 1;
}

// Address of the error word on the current device.
uint32_t* error_word_ptr() {
  static SymbolCache cache;
  return static_cast<uint32_t*>(cache.get(g_error_word));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Checks shared by both passes.  Returns FA_OK or the first problem found.
fa_status check_common(int B, int H, int H_kv, int Nq, int Nk, int d, float scale, int dtype) {
  if (B < 0 || H < 0 || H_kv < 0 || Nq < 0 || Nk < 0) return FA_ERR_INVALID_ARG;
  if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128 && d != 256) return FA_ERR_UNSUPPORTED;
  if (H > 0 && (H_kv < 1 || H % H_kv != 0)) return FA_ERR_INVALID_ARG;
  const long long BH = (long long)B * H;
  // grid size and 32-bit index limits of the kernels
  if (BH > (1LL << 24) || Nq > (1 << 28) || Nk > (1 << 28)) return FA_ERR_UNSUPPORTED;
  if (BH * ((Nq + 127) / 128) * 2 > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  if ((long long)B * H_kv * ((Nk + 127) / 128) * 2 > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  // the d = 256 backward launches both kinds of CTA in one grid
  if (BH * ((Nq + 127) / 128) + (long long)B * H_kv * ((Nk + 127) / 128) * 2 > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  // Queries with an empty key set are not a supported problem.
  if (BH * Nq > 0 && Nk == 0) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

fa_status check_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
  // The first call of a thread may find no context current, and the queries below need none; the encoding
  // of a TMA descriptor does.
  if (!current_context() && cudaSetDevice(dev) != cudaSuccess) return FA_ERR_CUDA;
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess) return FA_ERR_CUDA;
  if (cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) return FA_ERR_CUDA;
  if (major != 10 || minor != 3) return FA_ERR_UNSUPPORTED;  // the kernels are built for sm_103a only
  return FA_OK;
}

// TMA descriptor of a [BH, N, d] 16-bit tensor read or written in boxes of
// 64 columns (128 B, 128-byte swizzle) x `box_rows` rows of one head.
bool make_map(CUtensorMap* m, const void* ptr, long long BH, int N, int d, bool bf16, int box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)N, (cuuint64_t)BH};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)N * d * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                   const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

constexpr float kLog2e = 1.4426950408889634f;

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Library-owned events for the measurement hook.
struct Profile {
  std::vector<std::pair<cudaEvent_t, cudaEvent_t>> ev;
  std::vector<int> kind;
  int used = 0;
  bool on = false;
  bool open = false;  // a begin mark is waiting for its end mark
  void release() {
    for (auto& e : ev) {
      if (e.first) cudaEventDestroy(e.first);
      if (e.second) cudaEventDestroy(e.second);
    }
    ev.clear();
    kind.clear();
    used = 0;
    on = false;
    open = false;
  }
};
Profile& profile() {
  static Profile p;
  return p;
}

}  // namespace

void profile_mark_begin(cudaStream_t stream) {
  Profile& p = profile();
  if (!p.on || p.used >= (int)p.ev.size()) return;
  if (cudaEventRecord(p.ev[p.used].first, stream) == cudaSuccess) p.open = true;
}

namespace {
// The host-buffer pipeline's dK/dV mark (one per thread: calls on other threads
// are not affected).
thread_local cudaEvent_t t_dkdv_mark = nullptr;
thread_local bool t_dkdv_recorded = false;
}  // namespace

void arm_dkdv_mark(cudaEvent_t ev) {
  t_dkdv_mark = ev;
  t_dkdv_recorded = false;
}

bool take_dkdv_mark() {
  const bool r = t_dkdv_recorded;
  t_dkdv_mark = nullptr;
  t_dkdv_recorded = false;
  return r;
}

void profile_mark_end(cudaStream_t stream, int kind) {
  if (t_dkdv_mark && (kind == kProfileBwdKV || kind == kProfileBwdFused)) {
    t_dkdv_recorded = cudaEventRecord(t_dkdv_mark, stream) == cudaSuccess;
    t_dkdv_mark = nullptr;
  }
  Profile& p = profile();
  if (!p.on || !p.open) return;
  p.open = false;
  if (cudaEventRecord(p.ev[p.used].second, stream) == cudaSuccess) p.kind[p.used++] = kind;
}

size_t bwd_delta_offset(long long BH, int N) { return round_up((size_t)BH * bwd_npad(N) * sizeof(float), 256); }
size_t bwd_workspace_bytes(long long BH, int N) {
  return bwd_delta_offset(BH, N) + round_up((size_t)BH * bwd_npad(N) * sizeof(float), 256);
}

}  // namespace fa

using namespace fa;

namespace fa {

// cta_head_group for a given number of SMs (also the host query fa_cta_head_group).
static int cta_head_group_for(long long nheads, int nblocks, size_t bytes_per_head, bool causal, int num_sms) {
  if (nheads <= 1 || nblocks <= 0) return 1;
  const long long sms = std::max(num_sms, 1);
  const long long nb = nblocks;
  const long long work = causal ? nb * (nb + 1) / 2 : nb * nb;  // steps per head; the longest CTA takes nb
  const long long g_tail = (sms * nb + work - 1) / work;
  const long long g_l2 = std::max<long long>(1, (48ll << 20) / (long long)std::max<size_t>(bytes_per_head, 1));
  const long long g = std::min(std::max(g_tail, g_l2), nheads);
  // Equal groups: a short last group would hold heavy CTAs with too little work
  // around them.  Take the smallest divisor of nheads in [g, 2g] if there is one.
  for (long long c = g; c <= std::min(2 * g, nheads); ++c)
    if (nheads % c == 0) return (int)c;
  return (int)g;
}

int cta_head_group(long long nheads, int nblocks, size_t bytes_per_head, bool causal) {
  return cta_head_group_for(nheads, nblocks, bytes_per_head, causal, sm_count());
}

}  // namespace fa

extern "C" {

fa_status fa_fwd_ex(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int H_kv,
                    int N_q, int N_k, int d, float scale, int causal, fa_dtype dtype, fa_stream_t stream) {
  const fa::NvtxRange range("fa_fwd_ex");
  fa_status st = check_common(B, H, H_kv, N_q, N_k, d, scale, (int)dtype);
  if (st != FA_OK) return st;
  if ((long long)B * H * N_q == 0) return FA_OK;  // empty problem
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse)) return FA_ERR_MISALIGNED;
  if ((st = check_device()) != FA_OK) return st;
  const bool bf16 = dtype == FA_BF16;
  const long long BH = (long long)B * H, BHkv = (long long)B * H_kv;
  CUtensorMap mq, mk, mv, mo;
  if (!make_map(&mq, q, BH, N_q, d, bf16, 128) || !make_map(&mk, k, BHkv, N_k, d, bf16, 128) ||
      !make_map(&mv, v, BHkv, N_k, d, bf16, 128) || !make_map(&mo, o, BH, N_q, d, bf16, 128))
    return FA_ERR_CUDA;
  FwdArgs a{};
  a.lse = lse;
  a.N = N_q;
  a.Nk = N_k;
  a.BH = (int)BH;
  a.H = H;
  a.group = H / H_kv;
  const int rows = fwd_rows_per_cta(d, BH, N_q, sm_count());
  a.num_qblocks = (N_q + rows - 1) / rows;
  a.scale = scale;
  a.scale_log2 = scale * kLog2e;
  a.causal = causal ? 1 : 0;
  a.head_group = cta_head_group(BH, a.num_qblocks, (size_t)4 * (N_q + N_k) * d, causal != 0);
  a.err = error_word_ptr();
  if (!a.err) return FA_ERR_CUDA;
  cudaError_t e = launch_fwd(d, bf16, rows, mq, mk, mv, mo, a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N, int d,
                 float scale, int causal, fa_dtype dtype, fa_stream_t stream) {
  return fa_fwd_ex(q, k, v, o, lse, B, H, H, N, N, d, scale, causal, dtype, stream);
}

size_t fa_bwd_workspace_size(int B, int H, int N, int d) {
  if (check_common(B, H, H > 0 ? 1 : 0, N, N, d, 1.f, FA_FP16) != FA_OK) return 0;
  if ((size_t)B * H * N == 0) return 0;
  return bwd_workspace_bytes((long long)B * H, N);
}

fa_status fa_bwd_ex(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
                    void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes, int B, int H, int H_kv,
                    int N_q, int N_k, int d, float scale, int causal, fa_dtype dtype, fa_stream_t stream) {
  const fa::NvtxRange range("fa_bwd_ex");
  fa_status st = check_common(B, H, H_kv, N_q, N_k, d, scale, (int)dtype);
  if (st != FA_OK) return st;
  if ((long long)B * H * N_q == 0) {
    // No query rows: nothing flows back, so dK = dV = 0.
    const size_t kv_bytes = (size_t)B * H_kv * N_k * d * 2;
    if (kv_bytes == 0) return FA_OK;
    if (!dk || !dv) return FA_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (cudaMemsetAsync(dk, 0, kv_bytes, s) != cudaSuccess || cudaMemsetAsync(dv, 0, kv_bytes, s) != cudaSuccess)
      return FA_ERR_CUDA;
    return FA_OK;
  }
  if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dout) || !aligned16(lse) ||
      !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
    return FA_ERR_MISALIGNED;
  const size_t need = fa_bwd_workspace_size(B, H, N_q, d);
  if (!workspace || workspace_bytes < need) return FA_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return FA_ERR_MISALIGNED;
  if ((st = check_device()) != FA_OK) return st;
  const bool bf16 = dtype == FA_BF16;
  const long long BH = (long long)B * H, BHkv = (long long)B * H_kv;
  const int rows = bwd_box_rows(d);
  CUtensorMap mq, mk, mv, mdo;
  if (!make_map(&mq, q, BH, N_q, d, bf16, rows) || !make_map(&mk, k, BHkv, N_k, d, bf16, rows) ||
      !make_map(&mv, v, BHkv, N_k, d, bf16, rows) || !make_map(&mdo, dout, BH, N_q, d, bf16, rows))
    return FA_ERR_CUDA;
  BwdArgs a{};
  a.q = q;
  a.k = k;
  a.o = o;
  a.dout = dout;
  a.lse = lse;
  a.lse_log2 = static_cast<float*>(workspace);
  a.delta = reinterpret_cast<float*>(static_cast<char*>(workspace) + bwd_delta_offset(BH, N_q));
  a.Npad = bwd_npad(N_q);
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.N = N_q;
  a.Nk = N_k;
  a.d = d;
  a.BH = (int)BH;
  a.BHkv = (int)BHkv;
  a.H = H;
  a.group = H / H_kv;
  a.scale = scale;
  a.scale_log2 = scale * kLog2e;
  a.causal = causal ? 1 : 0;
  a.head_group_kv = cta_head_group(BHkv, (N_k + 127) / 128, (size_t)4 * ((size_t)a.group * N_q + N_k) * d, causal != 0);
  a.head_group_q = cta_head_group(BH, (N_q + 127) / 128, (size_t)4 * (N_q + N_k) * d, causal != 0);
  a.err = error_word_ptr();
  if (!a.err) return FA_ERR_CUDA;
  cudaError_t e = launch_bwd(d, bf16, mq, mk, mv, mdo, a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
                 void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes, int B, int H, int N, int d,
                 float scale, int causal, fa_dtype dtype, fa_stream_t stream) {
  return fa_bwd_ex(q, k, v, o, dout, lse, dq, dk, dv, workspace, workspace_bytes, B, H, H, N, N, d, scale, causal,
                   dtype, stream);
}

}  // extern "C"

namespace fa {
namespace {

// Checks of a score rule (host values and pointers; device contents are not read).  The ids of
// a side without rows may be null: an array without elements need not have an address.
fa_status check_rule(const fa_score_rule* r, float scale, bool no_queries, bool no_keys) {
  if (!r) return FA_ERR_INVALID_ARG;
  if (!(std::isfinite(r->cap) && r->cap >= 0.f)) return FA_ERR_INVALID_ARG;
  if (r->cap > 0.f && !std::isfinite(scale / r->cap * 4.f)) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(r->cap * kLog2e)) return FA_ERR_INVALID_ARG;
  if ((r->q_doc && !r->k_doc && !no_keys) || (r->k_doc && !r->q_doc && !no_queries)) return FA_ERR_INVALID_ARG;
  for (const void* p : {(const void*)r->slopes, (const void*)r->q_doc, (const void*)r->k_doc, (const void*)r->prefix})
    if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0) return FA_ERR_MISALIGNED;
  return FA_OK;
}

RuleArgs rule_args(const fa_score_rule& r, float scale) {
  RuleArgs a{};
  a.slopes = r.slopes;
  a.prefix = r.prefix;
  if (r.cap > 0.f) {
    const double k = (double)scale / r.cap;
    a.cap_x = (float)k;
    a.cap2 = r.cap * kLog2e;
    // The polynomial of fa_rule.cuh in the raw score.  A k above 1e4, whose powers leave
    // fp32's range, takes the other form for every score but 0.  Of a small k the high powers
    // lose their bits: those terms are left out, and the range ends where they would show.
    const int terms = k >= 0x1p-19 ? 3 : k >= 1e-7 ? 2 : k >= 1e-12 ? 1 : 0;
    constexpr double kTop[4] = {2e-4, 0.02, 0.09, 0.35};
    a.tanh_top = k <= 1e4 ? (float)(kTop[terms] / k) : -1.f;
    a.tanh_a1 = terms < 1 ? 0.f : (float)(-0.33332669734954834 * k * k * k);
    a.tanh_a2 = terms < 2 ? 0.f : (float)(0.13300010561943054 * k * k * k * k * k);
    a.tanh_a3 = terms < 3 ? 0.f : (float)(-0.049159303307533264 * k * k * k * k * k * k * k);
  }
  return a;
}

// Bytes of the row vectors at the start of a backward workspace.
size_t bwd_rows_bytes(int B, int H, int N) { return round_up(bwd_workspace_bytes((long long)B * H, N), 256); }

}  // namespace
}  // namespace fa

extern "C" {

size_t fa_fwd_rule_workspace_size(int B, int H, int N_q, int N_k, int d, int docs) {
  if (check_common(B, H, H > 0 ? 1 : 0, N_q, N_k, d, 1.f, FA_FP16) != FA_OK) return 0;
  if (!docs || (size_t)B * H * N_q == 0) return 0;
  return rule_plan(B, N_q, N_k, 128, false).bytes;
}

size_t fa_bwd_rule_workspace_size(int B, int H, int N_q, int N_k, int d, int docs) {
  if (check_common(B, H, H > 0 ? 1 : 0, N_q, N_k, d, 1.f, FA_FP16) != FA_OK) return 0;
  if ((size_t)B * H * N_q == 0) return 0;
  return bwd_rows_bytes(B, H, N_q) + (docs ? rule_plan(B, N_q, N_k, 128, true).bytes : 0);
}

fa_status fa_fwd_rule(const void* q, const void* k, const void* v, void* o, float* lse, const fa_score_rule* rule,
                      void* workspace, size_t workspace_bytes, int B, int H, int H_kv, int N_q, int N_k, int d,
                      float scale, fa_dtype dtype, fa_stream_t stream) {
  const fa::NvtxRange range("fa_fwd_rule");
  fa_status st = check_common(B, H, H_kv, N_q, N_k, d, scale, (int)dtype);
  if (st != FA_OK) return st;
  if ((st = check_rule(rule, scale, (long long)B * N_q == 0, (long long)B * N_k == 0)) != FA_OK) return st;
  if ((long long)B * H * N_q == 0) return FA_OK;  // empty problem
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse)) return FA_ERR_MISALIGNED;
  const bool docs = rule->q_doc != nullptr;
  if (docs) {
    if (!workspace || workspace_bytes < fa_fwd_rule_workspace_size(B, H, N_q, N_k, d, 1)) return FA_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return FA_ERR_MISALIGNED;
  }
  if ((st = check_device()) != FA_OK) return st;
  const bool bf16 = dtype == FA_BF16;
  const long long BH = (long long)B * H, BHkv = (long long)B * H_kv;
  CUtensorMap mq, mk, mv, mo;
  if (!make_map(&mq, q, BH, N_q, d, bf16, 128) || !make_map(&mk, k, BHkv, N_k, d, bf16, 128) ||
      !make_map(&mv, v, BHkv, N_k, d, bf16, 128) || !make_map(&mo, o, BH, N_q, d, bf16, 128))
    return FA_ERR_CUDA;
  FwdRuleArgs a{};
  a.lse = lse;
  a.N = N_q;
  a.Nk = N_k;
  a.BH = (int)BH;
  a.H = H;
  a.group = H / H_kv;
  const int rows = fwd_rows_per_cta(d, BH, N_q, sm_count());
  a.num_qblocks = (N_q + rows - 1) / rows;
  a.scale = scale;
  a.scale_log2 = scale * kLog2e;
  a.causal = rule->causal ? 1 : 0;
  a.head_group = cta_head_group(BH, a.num_qblocks, (size_t)4 * (N_q + N_k) * d, a.causal != 0);
  a.err = error_word_ptr();
  if (!a.err) return FA_ERR_CUDA;
  a.rule = rule_args(*rule, scale);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (docs) {
    const RulePlan p = rule_plan(B, N_q, N_k, rows, false);
    char* ws = static_cast<char*>(workspace);
    if (launch_rule_plan(p, ws, rule->q_doc, rule->k_doc, rule->prefix, B, N_q, N_k, rows, a.causal, s) != cudaSuccess)
      return FA_ERR_CUDA;
    rule_plan_args(a.rule, p, ws);
  }
  const int kind = rule_kind(a.rule);
  return launch_fwd_rule(kind, d, bf16, rows, mq, mk, mv, mo, a, s) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_bwd_rule(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
                      void* dq, void* dk, void* dv, const fa_score_rule* rule, void* workspace,
                      size_t workspace_bytes, int B, int H, int H_kv, int N_q, int N_k, int d, float scale,
                      fa_dtype dtype, fa_stream_t stream) {
  const fa::NvtxRange range("fa_bwd_rule");
  fa_status st = check_common(B, H, H_kv, N_q, N_k, d, scale, (int)dtype);
  if (st != FA_OK) return st;
  if ((st = check_rule(rule, scale, (long long)B * N_q == 0, (long long)B * N_k == 0)) != FA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if ((long long)B * H * N_q == 0) {
    // No query rows: nothing flows back, so dK = dV = 0.
    const size_t kv_bytes = (size_t)B * H_kv * N_k * d * 2;
    if (kv_bytes == 0) return FA_OK;
    if (!dk || !dv) return FA_ERR_INVALID_ARG;
    if (cudaMemsetAsync(dk, 0, kv_bytes, s) != cudaSuccess || cudaMemsetAsync(dv, 0, kv_bytes, s) != cudaSuccess)
      return FA_ERR_CUDA;
    return FA_OK;
  }
  if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dout) || !aligned16(lse) ||
      !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
    return FA_ERR_MISALIGNED;
  const bool docs = rule->q_doc != nullptr;
  const size_t need = fa_bwd_rule_workspace_size(B, H, N_q, N_k, d, docs);
  if (!workspace || workspace_bytes < need) return FA_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return FA_ERR_MISALIGNED;
  if ((st = check_device()) != FA_OK) return st;
  const bool bf16 = dtype == FA_BF16;
  const long long BH = (long long)B * H, BHkv = (long long)B * H_kv;
  const int rows = bwd_box_rows(d);
  CUtensorMap mq, mk, mv, mdo;
  if (!make_map(&mq, q, BH, N_q, d, bf16, rows) || !make_map(&mk, k, BHkv, N_k, d, bf16, rows) ||
      !make_map(&mv, v, BHkv, N_k, d, bf16, rows) || !make_map(&mdo, dout, BH, N_q, d, bf16, rows))
    return FA_ERR_CUDA;
  char* ws = static_cast<char*>(workspace);
  BwdRuleArgs a{};
  a.q = q;
  a.k = k;
  a.o = o;
  a.dout = dout;
  a.lse = lse;
  a.lse_log2 = reinterpret_cast<float*>(ws);
  a.delta = reinterpret_cast<float*>(ws + bwd_delta_offset(BH, N_q));
  a.Npad = bwd_npad(N_q);
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.N = N_q;
  a.Nk = N_k;
  a.d = d;
  a.BH = (int)BH;
  a.BHkv = (int)BHkv;
  a.H = H;
  a.group = H / H_kv;
  a.scale = scale;
  a.scale_log2 = scale * kLog2e;
  a.causal = rule->causal ? 1 : 0;
  a.head_group_kv = cta_head_group(BHkv, (N_k + 127) / 128, (size_t)4 * ((size_t)a.group * N_q + N_k) * d, a.causal != 0);
  a.head_group_q = cta_head_group(BH, (N_q + 127) / 128, (size_t)4 * (N_q + N_k) * d, a.causal != 0);
  a.err = error_word_ptr();
  if (!a.err) return FA_ERR_CUDA;
  a.rule = rule_args(*rule, scale);
  if (docs) {
    char* pws = ws + bwd_rows_bytes(B, H, N_q);
    const RulePlan p = rule_plan(B, N_q, N_k, 128, true);
    if (launch_rule_plan(p, pws, rule->q_doc, rule->k_doc, rule->prefix, B, N_q, N_k, 128, a.causal, s) != cudaSuccess)
      return FA_ERR_CUDA;
    rule_plan_args(a.rule, p, pws);
    a.kv_list = reinterpret_cast<int*>(pws + p.k_list);
    a.kv_count = reinterpret_cast<int*>(pws + p.k_count);
    a.kv_list_stride = p.k_list_stride;
  }
  const int kind = rule_kind(a.rule);
  return launch_bwd_rule(kind, d, bf16, mq, mk, mv, mdo, a, rule->q_doc, s) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"

namespace fa {
namespace {

// Checks of a cache and its page table (host values and pointers only).
fa_status check_cache(const fa_kv4_cache* c, const int32_t* table, int max_pages, int B, int N) {
  if (!c || B < 0 || N < 0 || c->num_pages < 0 || c->H_kv < 1 || max_pages < 0) return FA_ERR_INVALID_ARG;
  if (c->dtype != FA_FP16 && c->dtype != FA_BF16) return FA_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128 && c->d != 256) return FA_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0) return FA_ERR_UNSUPPORTED;
  if ((long long)max_pages * c->page_size > (1LL << 30)) return FA_ERR_UNSUPPORTED;
  // the row kernels number B x H_kv x N rows of keys and of values in 32 bits
  if (c->H_kv > (1 << 20) || (long long)B * c->H_kv > (1LL << 24) || N > (1 << 28)) return FA_ERR_UNSUPPORTED;
  if ((long long)B * c->H_kv * N >= (1LL << 30)) return FA_ERR_UNSUPPORTED;
  if ((long long)B * N == 0) return FA_OK;
  if (c->num_pages > 0 && (!c->k_codes || !c->k_params || !c->v_codes || !c->v_params)) return FA_ERR_INVALID_ARG;
  if (!table && max_pages > 0) return FA_ERR_INVALID_ARG;
  if (!aligned16(c->k_codes) || !aligned16(c->k_params) || !aligned16(c->v_codes) || !aligned16(c->v_params))
    return FA_ERR_MISALIGNED;
  return FA_OK;
}
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

Kv4Pool pool_of(const fa_kv4_cache& c, const int32_t* table, int max_pages) {
  Kv4Pool p{};
  p.codes[0] = static_cast<uint8_t*>(c.k_codes);
  p.codes[1] = static_cast<uint8_t*>(c.v_codes);
  p.params[0] = static_cast<uint32_t*>(c.k_params);
  p.params[1] = static_cast<uint32_t*>(c.v_params);
  p.table = table;
  p.num_pages = c.num_pages;
  while ((1 << p.page_shift) < c.page_size) ++p.page_shift;
  p.max_pages = max_pages;
  p.H_kv = c.H_kv;
  p.err = error_word_ptr();
  return p;
}

struct Kv4Parts {
  int unit_cols, col_tiles;
  size_t slots, ml_offset, bytes;
};
Kv4Parts kv4_parts(int H, int H_kv, int N_q, int d) {
  Kv4Parts p{};
  const int cols = H / H_kv * N_q;
  p.unit_cols = kv4_unit_cols(d, cols);
  p.col_tiles = (cols + p.unit_cols - 1) / p.unit_cols;
  p.slots = 2 * kKv4MaxCtas;  // the units that a CTA's stretch cuts: its first and its last
  p.ml_offset = round_up(p.slots * p.unit_cols * d * 4, 256);
  p.bytes = p.ml_offset + round_up(p.slots * p.unit_cols * 8, 256);
  return p;
}
bool kv4_sizes_ok(int B, int H, int H_kv, int N_q, int d) {
  if (B < 0 || H < 0 || N_q < 0 || H_kv < 1 || H % H_kv != 0) return false;
  if (d != 64 && d != 128 && d != 256) return false;
  return B <= kKv4MaxBatch && (long long)B * H <= (1LL << 24) && N_q <= (1 << 20) && (long long)H * N_q <= (1LL << 28) &&
         (long long)B * H * N_q <= (1LL << 32);
}

// Parts of the kernel for trees with many rows: none where it is not used.
struct WideParts {
  size_t ml_offset, bytes;
};
WideParts wide_parts(int H, int H_kv, int N_q, int d) {
  WideParts p{};
  if (!kv4_tree_wide(d, H / H_kv * N_q)) return p;
  p.ml_offset = (size_t)2 * kWideMaxCtas * kWideRows * d * 4;
  p.bytes = p.ml_offset + (size_t)2 * kWideMaxCtas * kWideRows * 8 + (size_t)kWideMaxCtas * 32;  // and the cuts
  return p;
}

// Checks of an attention call over the cache, and its arguments; tokens: of all units, at most, -1
// for an empty problem.
fa_status attend_args(Kv4AttendArgs& a, long long& tokens, const void* q, const fa_kv4_cache* cache,
                      const int32_t* page_table, int max_pages, const int32_t* lengths, void* o, float* lse, int causal,
                      float cap, const float* slopes, void* workspace, size_t workspace_bytes, int B, int H, int N_q,
                      float scale) {
  fa_status st = check_cache(cache, page_table, max_pages, B, N_q);
  if (st != FA_OK) return st;
  if (H < 0 || H % cache->H_kv != 0) return FA_ERR_INVALID_ARG;
  if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
  fa_score_rule rule{};
  rule.causal = causal;
  rule.cap = cap;
  rule.slopes = slopes;
  if ((st = check_rule(&rule, scale, true, true)) != FA_OK) return st;
  if (!kv4_sizes_ok(B, H, cache->H_kv, N_q, cache->d)) return FA_ERR_UNSUPPORTED;
  tokens = -1;
  if ((long long)B * H * N_q == 0) return FA_OK;
  if (!q || !lengths || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o) || !aligned16(lse) || !aligned4(page_table) || !aligned4(lengths))
    return FA_ERR_MISALIGNED;
  const Kv4Parts parts = kv4_parts(H, cache->H_kv, N_q, cache->d);
  if (!workspace || workspace_bytes < parts.bytes) return FA_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return FA_ERR_MISALIGNED;
  // pieces of 128 tokens over all units: the kernels count them in 32 bits
  const long long per_unit = ((long long)max_pages * cache->page_size + 127) / 128;
  const long long units = (long long)B * cache->H_kv * parts.col_tiles;
  if (per_unit * units > (1LL << 30) || units * parts.unit_cols * cache->d > (1LL << 37)) return FA_ERR_UNSUPPORTED;
  if ((st = check_device()) != FA_OK) return st;
  const RuleArgs r = rule_args(rule, scale);
  a.pool = pool_of(*cache, page_table, max_pages);
  if (!a.pool.err) return FA_ERR_CUDA;
  a.q = q;
  a.lengths = lengths;
  a.o = o;
  a.lse = lse;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + parts.ml_offset);
  a.B = B;
  a.H = H;
  a.N_q = N_q;
  a.group = H / cache->H_kv;
  a.cols = a.group * N_q;
  a.col_tiles = parts.col_tiles;
  a.causal = causal ? 1 : 0;
  a.cap = cap > 0.f ? 1 : 0;
  a.scale_log2 = scale * kLog2e;
  a.rule = r;
  tokens = per_unit * 128 * units;
  return FA_OK;
}

// Rows of a rotary call: 16-byte accesses, output rows that do not overlap.
fa_status check_rotary_rows(const fa_rotary_rows& r, int B, int H, int N, int d) {
  if (!r.in || !r.out) return FA_ERR_INVALID_ARG;
  if (!aligned16(r.in) || !aligned16(r.out)) return FA_ERR_MISALIGNED;
  const int sizes[3] = {B, H, N};
  for (int i = 0; i < 3; ++i) {
    if (sizes[i] < 2) continue;
    if (r.in_stride[i] < 0 || r.out_stride[i] < d) return FA_ERR_INVALID_ARG;
    if (r.in_stride[i] % 8 != 0 || r.out_stride[i] % 8 != 0) return FA_ERR_MISALIGNED;
  }
  return FA_OK;
}

}  // namespace
}  // namespace fa

extern "C" {

fa_status fa_kv4_append(const fa_kv4_cache* cache, const void* k, const void* v, const int32_t* page_table,
                        int max_pages, const int32_t* start, const int32_t* count, int B, int N, fa_stream_t stream) {
  const fa::NvtxRange range("fa_kv4_append");
  fa_status st = check_cache(cache, page_table, max_pages, B, N);
  if (st != FA_OK || (long long)B * N == 0) return st;
  if (!k || !v || !start) return FA_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned4(page_table) || !aligned4(start) || !aligned4(count))
    return FA_ERR_MISALIGNED;
  if ((st = check_device()) != FA_OK) return st;
  const Kv4Pool p = pool_of(*cache, page_table, max_pages);
  if (!p.err) return FA_ERR_CUDA;
  return launch_kv4_append(p, cache->d, cache->dtype == FA_BF16, k, v, start, count, B, N, sm_count(),
                           reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

fa_status fa_kv4_read(const fa_kv4_cache* cache, const int32_t* page_table, int max_pages, const int32_t* start,
                      const int32_t* lengths, void* k, void* v, int B, int N, fa_stream_t stream) {
  const fa::NvtxRange range("fa_kv4_read");
  fa_status st = check_cache(cache, page_table, max_pages, B, N);
  if (st != FA_OK || (long long)B * N == 0) return st;
  if (!k || !v || !start || !lengths) return FA_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned4(page_table) || !aligned4(start) || !aligned4(lengths))
    return FA_ERR_MISALIGNED;
  if ((st = check_device()) != FA_OK) return st;
  const Kv4Pool p = pool_of(*cache, page_table, max_pages);
  if (!p.err) return FA_ERR_CUDA;
  return launch_kv4_read(p, cache->d, cache->dtype == FA_BF16, start, lengths, k, v, B, N, sm_count(),
                         reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

size_t fa_kv4_attend_workspace_size(int B, int H, int H_kv, int N_q, int d) {
  if (!kv4_sizes_ok(B, H, H_kv, N_q, d) || (long long)B * H * N_q == 0) return 0;
  return kv4_parts(H, H_kv, N_q, d).bytes;
}

fa_status fa_kv4_attend(const void* q, const fa_kv4_cache* cache, const int32_t* page_table, int max_pages,
                        const int32_t* lengths, void* o, float* lse, int causal, float cap, const float* slopes,
                        void* workspace, size_t workspace_bytes, int B, int H, int N_q, float scale,
                        fa_stream_t stream) {
  const fa::NvtxRange range("fa_kv4_attend");
  Kv4AttendArgs a{};
  long long tokens = 0;
  const fa_status st = attend_args(a, tokens, q, cache, page_table, max_pages, lengths, o, lse, causal, cap, slopes,
                                   workspace, workspace_bytes, B, H, N_q, scale);
  if (st != FA_OK || tokens < 0) return st;
  return launch_kv4_attend(a, cache->d, cache->dtype == FA_BF16, tokens, sm_count(), reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

size_t fa_kv4_attend_tree_workspace_size(int B, int H, int H_kv, int N_q, int d) {
  if (N_q > kKv4MaxDraft) return 0;
  const size_t bytes = fa_kv4_attend_workspace_size(B, H, H_kv, N_q, d);
  return bytes ? std::max(bytes, wide_parts(H, H_kv, N_q, d).bytes) : 0;
}

int fa_kv4_tree_many_rows(int B, int H, int H_kv, int N_q, int d, long long room, int num_sms) {
  if (!kv4_sizes_ok(B, H, H_kv, N_q, d) || N_q > kKv4MaxDraft || room < 0 || room > (1LL << 30)) return -1;
  if ((long long)B * H * N_q == 0) return 0;
  return kv4_tree_many_rows(B, H_kv, H / H_kv * N_q, d, room, num_sms > 0 ? num_sms : sm_count()) ? 1 : 0;
}

fa_status fa_kv4_attend_tree(const void* q, const fa_kv4_cache* cache, const int32_t* page_table, int max_pages,
                             const int32_t* lengths, const int32_t* parents, const int32_t* count, void* o,
                             float* lse, float cap, const float* slopes, void* workspace, size_t workspace_bytes,
                             int B, int H, int N_q, float scale, fa_stream_t stream) {
  const fa::NvtxRange range("fa_kv4_attend_tree");
  Kv4TreeArgs a{};
  long long tokens = 0;
  if (N_q > kKv4MaxDraft) return FA_ERR_UNSUPPORTED;
  const bool some = (long long)B * H * N_q > 0;
  if (some && !parents) return FA_ERR_INVALID_ARG;
  if (some && (!aligned4(parents) || !aligned4(count))) return FA_ERR_MISALIGNED;
  const fa_status st = attend_args(a, tokens, q, cache, page_table, max_pages, lengths, o, lse, 1, cap, slopes, workspace,
                                   workspace_bytes, B, H, N_q, scale);
  if (st != FA_OK || tokens < 0) return st;
  const WideParts parts = wide_parts(H, cache->H_kv, N_q, cache->d);
  if (parts.bytes) {
    if (workspace_bytes < parts.bytes) return FA_ERR_WORKSPACE;
    a.part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + parts.ml_offset);
  }
  a.tree.parents = parents;
  a.tree.count = count;
  return launch_kv4_tree(a, cache->d, cache->dtype == FA_BF16, tokens, sm_count(), reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

fa_status fa_kv4_keep(const fa_kv4_cache* cache, const int32_t* page_table, int max_pages, const int32_t* start,
                      const int32_t* path, const int32_t* kept, int B, int N, fa_stream_t stream) {
  const fa::NvtxRange range("fa_kv4_keep");
  fa_status st = check_cache(cache, page_table, max_pages, B, N);
  if (st != FA_OK) return st;
  if (N > kKv4MaxDraft) return FA_ERR_UNSUPPORTED;
  if ((long long)B * N == 0) return FA_OK;
  if (!start || !path || !kept) return FA_ERR_INVALID_ARG;
  if (!aligned4(page_table) || !aligned4(start) || !aligned4(path) || !aligned4(kept)) return FA_ERR_MISALIGNED;
  if ((st = check_device()) != FA_OK) return st;
  const Kv4Pool p = pool_of(*cache, page_table, max_pages);
  if (!p.err) return FA_ERR_CUDA;
  return launch_kv4_keep(p, cache->d, start, path, kept, B, N, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

fa_status fa_kv4_plan(int32_t* page_table, int32_t* held, int max_pages, int32_t* free_pages, int num_free,
                      int32_t* free_count, int page_size, const int32_t* start, const int32_t* count,
                      const int32_t* parents, int32_t* out_count, int32_t* lengths, int64_t* slots,
                      int32_t* positions, int B, int N, fa_stream_t stream) {
  const fa::NvtxRange range("fa_kv4_plan");
  if (B < 0 || N < 0 || max_pages < 0 || num_free < 0) return FA_ERR_INVALID_ARG;
  if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)) != 0) return FA_ERR_UNSUPPORTED;
  if ((long long)max_pages * page_size > (1LL << 30) || B > kKv4MaxBatch) return FA_ERR_UNSUPPORTED;
  if ((long long)B * N > INT_MAX || (parents && N > kKv4MaxDraft)) return FA_ERR_UNSUPPORTED;
  if (B == 0) return FA_OK;
  if (!held || !free_count || !start || !count || !out_count || !lengths) return FA_ERR_INVALID_ARG;
  if ((!page_table && max_pages > 0) || (!free_pages && num_free > 0) || (N > 0 && (!slots || !positions)))
    return FA_ERR_INVALID_ARG;
  if (!aligned4(page_table) || !aligned4(held) || !aligned4(free_pages) || !aligned4(free_count) || !aligned4(start) ||
      !aligned4(count) || !aligned4(parents) || !aligned4(out_count) || !aligned4(lengths) || !aligned4(positions) ||
      (reinterpret_cast<uintptr_t>(slots) & 7u) != 0)
    return FA_ERR_MISALIGNED;
  const fa_status st = check_device();
  if (st != FA_OK) return st;
  Kv4PlanArgs a{page_table, held, free_pages, free_count, start, count, N > 0 ? parents : nullptr, out_count, lengths,
                slots, positions, B, N, max_pages, num_free, 0};
  while ((1 << a.page_shift) < page_size) ++a.page_shift;
  return launch_kv4_plan(a, sm_count(), reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_rotary(const fa_rotary_rows* q, const fa_rotary_rows* k, const int32_t* positions, const double* freqs,
                    int dims, int interleaved, int backward, float amplitude, int B, int H, int H_kv, int N, int d,
                    fa_dtype dtype, fa_stream_t stream) {
  const fa::NvtxRange range("fa_rotary");
  if (B < 0 || H < 0 || H_kv < 0 || N < 0 || !std::isfinite(amplitude)) return FA_ERR_INVALID_ARG;
  if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128 && d != 256) return FA_ERR_UNSUPPORTED;
  if (dims < 16 || dims > d || dims % 16 != 0) return FA_ERR_UNSUPPORTED;
  // rows and heads as the kernel's grid counts them
  if ((long long)B * N > INT_MAX || (long long)H + H_kv > 65535) return FA_ERR_UNSUPPORTED;
  if ((long long)B * N == 0 || H + H_kv == 0) return FA_OK;
  if (!freqs || (H > 0 && !q) || (H_kv > 0 && !k)) return FA_ERR_INVALID_ARG;
  if (!aligned4(positions) || (reinterpret_cast<uintptr_t>(freqs) & 7u) != 0) return FA_ERR_MISALIGNED;
  RotaryArgs a{};
  const fa_rotary_rows* rows[2] = {H > 0 ? q : nullptr, H_kv > 0 ? k : nullptr};
  for (int i = 0; i < 2; ++i) {
    if (!rows[i]) continue;
    const fa_rotary_rows& r = *rows[i];
    const fa_status st = check_rotary_rows(r, B, i ? H_kv : H, N, d);
    if (st != FA_OK) return st;
    a.part[i] = RotaryRows{r.in, r.out, r.in_stride[0], r.in_stride[1], r.in_stride[2],
                           r.out_stride[0], r.out_stride[1], r.out_stride[2]};
    if (dims < d && r.in != r.out) a.tail = 1;
  }
  const fa_status st = check_device();
  if (st != FA_OK) return st;
  a.positions = positions;
  a.freqs = freqs;
  a.B = B;
  a.H = H;
  a.H_kv = H_kv;
  a.N = N;
  a.dims = dims;
  a.backward = backward ? 1 : 0;
  a.amplitude = amplitude;
  return launch_rotary(a, d, dtype == FA_BF16, interleaved != 0, sm_count(), reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

uint64_t fa_rotary_turns(double freq) { return turns_of(freq); }

long long fa_kv4_row(const int32_t* pages, int max_pages, int page_size, int num_pages, long long pos) {
  if (!pages || max_pages < 0 || page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)) != 0) return -1;
  int shift = 0;
  while ((1 << shift) < page_size) ++shift;
  return kv4_row(pages, max_pages, shift, num_pages, pos);
}

}  // extern "C"

namespace fa {
namespace {
// Fixed scratch of fa_bwd_noalloc (the backward workspace: fp32 L log2 e and D
// rows).  Its name in host code is only a host-side stand-in; the device address
// comes from cudaGetSymbolAddress on each device.
constexpr size_t kNoAllocScratchBytes = size_t(32) << 20;
__device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];

// Device address of the scratch on the current device.
void* noalloc_scratch_ptr() {
  static SymbolCache cache;
  return cache.get(g_noalloc_scratch);
}
}  // namespace
}  // namespace fa

extern "C" {

fa_status fa_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const void* dout,
                         const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d, float scale,
                         int causal, fa_dtype dtype, fa_stream_t stream) {
  const fa::NvtxRange range("fa_bwd_noalloc");
  fa_status st = check_common(B, H, H, N, N, d, scale, (int)dtype);
  if (st != FA_OK) return st;
  if ((long long)B * H * N == 0) return FA_OK;
  if (fa_bwd_workspace_size(B, H, N, d) > kNoAllocScratchBytes) return FA_ERR_WORKSPACE;
  if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv) return FA_ERR_INVALID_ARG;
  if ((st = check_device()) != FA_OK) return st;
  void* scratch = noalloc_scratch_ptr();
  if (!scratch) return FA_ERR_CUDA;
  return fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, scratch, kNoAllocScratchBytes, B, H, N, d, scale, causal, dtype,
                stream);
}

int fa_cta_head_group(long long nheads, int nblocks, size_t bytes_per_head, int causal, int num_sms) {
  if (nheads < 1 || nblocks < 0) return -1;
  return cta_head_group_for(nheads, nblocks, bytes_per_head, causal != 0, num_sms > 0 ? num_sms : sm_count());
}

fa_status fa_check_device_status(fa_stream_t stream) {
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return FA_ERR_CUDA;
  uint32_t rec[4] = {0, 0, 0, 0};
  if (cudaMemcpyFromSymbol(rec, g_error_word, sizeof(rec)) != cudaSuccess) return FA_ERR_CUDA;
  for (int i = 0; i < 4; ++i) g_last_detail[i] = rec[i];
  if (rec[0] != 0) {
    const uint32_t zero[4] = {0, 0, 0, 0};
    if (cudaMemcpyToSymbol(g_error_word, zero, sizeof(zero)) != cudaSuccess) return FA_ERR_CUDA;
    // the first failure decides: a debug-build check (code kDbgBase | kind) or a wait
    return (rec[1] & kDbgBase) ? FA_ERR_DEVICE_CHECK : FA_ERR_DEVICE_TIMEOUT;
  }
  return FA_OK;
}

fa_status fa_selftest_device_check(int kind, fa_stream_t stream) {
#ifdef FA_DEBUG
  if (kind < (int)kDbgTmaCol || kind > (int)kDbgPhase) return FA_ERR_INVALID_ARG;
  fa_status st = check_device();
  if (st != FA_OK) return st;
  uint32_t* err = error_word_ptr();
  if (!err) return FA_ERR_CUDA;
  return launch_selftest_check(err, kind, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK
                                                                                                  : FA_ERR_CUDA;
#else
  (void)kind;
  (void)stream;
  return FA_ERR_UNSUPPORTED;  // the checks are compiled out of this build
#endif
}

fa_status fa_selftest_wait_timeout(uint32_t limit_us, fa_stream_t stream) {
  if (limit_us == 0 || limit_us > 1000000u) return FA_ERR_INVALID_ARG;
  fa_status st = check_device();
  if (st != FA_OK) return st;
  uint32_t* err = error_word_ptr();
  if (!err) return FA_ERR_CUDA;
  return launch_selftest_wait(err, 1000ull * limit_us, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

uint32_t fa_last_device_error_bits(void) { return g_last_detail[0]; }

void fa_last_device_error_detail(uint32_t* out4) {
  if (!out4) return;
  for (int i = 0; i < 4; ++i) out4[i] = g_last_detail[i];
}

const char* fa_status_string(fa_status s) {
  switch (s) {
    case FA_OK: return "FA_OK";
    case FA_ERR_INVALID_ARG: return "FA_ERR_INVALID_ARG";
    case FA_ERR_UNSUPPORTED: return "FA_ERR_UNSUPPORTED";
    case FA_ERR_MISALIGNED: return "FA_ERR_MISALIGNED";
    case FA_ERR_WORKSPACE: return "FA_ERR_WORKSPACE";
    case FA_ERR_CUDA: return "FA_ERR_CUDA";
    case FA_ERR_DEVICE_TIMEOUT: return "FA_ERR_DEVICE_TIMEOUT";
    case FA_ERR_DEVICE_CHECK: return "FA_ERR_DEVICE_CHECK";
  }
  return "FA_ERR_UNKNOWN";
}

fa_status fa_profile_begin(int n) {
  if (n < 0 || n > 65536) return FA_ERR_INVALID_ARG;
  Profile& p = profile();
  p.release();
  p.ev.resize((size_t)n);
  p.kind.assign((size_t)n, 0);
  for (auto& e : p.ev) {
    if (cudaEventCreate(&e.first) != cudaSuccess || cudaEventCreate(&e.second) != cudaSuccess) {
      p.release();
      return FA_ERR_CUDA;
    }
  }
  p.used = 0;
  p.open = false;
  p.on = n > 0;
  return FA_OK;
}

int fa_profile_end(float* out_ms, int* out_kind, int max_out) {
  Profile& p = profile();
  int written = 0;
  bool failed = false;
  for (int i = 0; i < p.used && i < max_out; ++i) {
    float ms = 0.f;
    if (cudaEventSynchronize(p.ev[i].second) != cudaSuccess ||
        cudaEventElapsedTime(&ms, p.ev[i].first, p.ev[i].second) != cudaSuccess) {
      failed = true;
      break;
    }
    if (out_ms) out_ms[i] = ms;
    if (out_kind) out_kind[i] = p.kind[i];
    ++written;
  }
  p.release();
  return failed ? -1 : written;
}

uint32_t fa_version(void) { return (1u << 16) | 0u; }

}  // extern "C"
