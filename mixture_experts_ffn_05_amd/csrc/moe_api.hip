// libmoe C ABI: argument validation (on the host, before any HIP call) and
// dispatch to the kernel launchers.  Declarations and the contract of every
// call are in include/libmoe.h.
#include "libmoe.h"
#include "moe_common.h"

#include <rocprofiler-sdk-roctx/roctx.h>

#include <algorithm>
#include <math.h>
#include <mutex>
#include <new>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>
#include <string>
#include <vector>

namespace {

constexpr int kVersion = 100;  // 0.1.0
constexpr int64_t kMaxRows = (int64_t)1 << 28;

thread_local std::string g_last_error;

moe_status fail(moe_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return st;
}

moe_status hip_result(hipError_t err, const char* call) {
  if (err == hipSuccess) return MOE_OK;
  return fail(MOE_ERR_HIP, "%s: HIP error %d (%s)", call, (int)err, hipGetErrorString(err));
}

int cu_count() {
  static std::mutex mu;
  static int cache[64] = {0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  std::lock_guard<std::mutex> lock(mu);
  if (cache[dev] == 0) {
    int v = 0;
    if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v <= 0) v = 256;
    cache[dev] = v;
  }
  return cache[dev];
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

int elem_size(moe_dtype dt) { return dt == MOE_BF16 ? 2 : 4; }

// Validation helpers: each returns MOE_OK or records a message naming the argument.
#define MOE_CHECK(expr)                 \
  do {                                  \
    moe_status _st = (expr);            \
    if (_st != MOE_OK) return _st;      \
  } while (0)

moe_status need_ptr(const void* p, const char* fn, const char* name) {
  return p ? MOE_OK : fail(MOE_ERR_INVALID_ARGUMENT, "%s: %s must not be NULL", fn, name);
}

moe_status need_pos(int64_t v, const char* fn, const char* name) {
  return v >= 1 ? MOE_OK : fail(MOE_ERR_INVALID_ARGUMENT, "%s: %s must be >= 1 (got %lld)", fn, name, (long long)v);
}

moe_status need_dtype(moe_dtype dt, const char* fn) {
  return (dt == MOE_F32 || dt == MOE_BF16) ? MOE_OK
                                          : fail(MOE_ERR_INVALID_ARGUMENT, "%s: dt must be MOE_F32 or MOE_BF16 (got %d)",
                                                 fn, (int)dt);
}

moe_status need_layout(moe_weight_layout wl, const char* fn) {
  return (wl == MOE_W_KN || wl == MOE_W_NK)
             ? MOE_OK
             : fail(MOE_ERR_INVALID_ARGUMENT, "%s: weight layout must be MOE_W_KN or MOE_W_NK (got %d)", fn, (int)wl);
}

moe_status need_mult8(int64_t v, const char* fn, const char* name) {
  return v % 8 == 0 ? MOE_OK
                    : fail(MOE_ERR_UNSUPPORTED, "%s: %s must be a multiple of 8 (got %lld)", fn, name, (long long)v);
}

moe_status need_experts(int64_t E, const char* fn) {
  MOE_CHECK(need_pos(E, fn, "E"));
  return E <= moe::kMaxExperts ? MOE_OK
                               : fail(MOE_ERR_UNSUPPORTED, "%s: E must be <= %d (got %lld)", fn, moe::kMaxExperts,
                                      (long long)E);
}

moe_status need_topk(int64_t k, const char* fn) {
  if (k < 1) return fail(MOE_ERR_INVALID_ARGUMENT, "%s: top_k must be positive (got %lld)", fn, (long long)k);
  return k <= moe::kMaxTopK ? MOE_OK
                            : fail(MOE_ERR_UNSUPPORTED, "%s: top_k must be <= %d (got %lld)", fn, moe::kMaxTopK,
                                   (long long)k);
}

moe_status need_rows(int64_t rows, const char* fn, const char* what) {
  return rows < kMaxRows ? MOE_OK
                         : fail(MOE_ERR_UNSUPPORTED, "%s: %s must be < 2^28 (got %lld)", fn, what, (long long)rows);
}

// A call's argument as memory; outputs (and the workspace, which a call writes) have out set.
struct Span {
  const void* p;
  size_t bytes;
  const char* name;
  bool out;
};

// No output may overlap another argument.  Arguments that are NULL overlap nothing.
template <size_t N>
moe_status need_apart(const Span (&a)[N], const char* fn) {
  for (size_t i = 0; i < N; ++i)
    for (size_t j = 0; j < i; ++j) {
      if (!a[i].p || !a[j].p || !(a[i].out || a[j].out)) continue;
      const uintptr_t x = (uintptr_t)a[i].p, y = (uintptr_t)a[j].p;
      if (x < y + a[j].bytes && y < x + a[i].bytes)
        return fail(MOE_ERR_INVALID_ARGUMENT, "%s: %s overlaps %s", fn, a[i].name, a[j].name);
    }
  return MOE_OK;
}

moe_status need_flag(int32_t v, const char* fn, const char* name) {
  return (v == 0 || v == 1) ? MOE_OK
                            : fail(MOE_ERR_INVALID_ARGUMENT, "%s: %s must be 0 or 1 (got %d)", fn, name, (int)v);
}


// Stage of every call, in the stage vocabulary of the PLENA pages
// (PLENA_Compiler PR #69, sections "Group B" and "Group E"; PLENA_Simulator
// PR #97, section "Stage attribution"); '+' joins the stages of a call that
// serves several.  The routed SwiGLU runs in the fc1 epilogue, so it bills to
// expert_projection; the combine overwrites its output, so no separate
// accumulator_init launch exists.  Backward calls carry a "backward:" prefix.
struct CallStage {
  const char* call;
  const char* stage;
};
constexpr CallStage kCallStages[] = {
    {"moe_route", "router_topk"},
    {"moe_route_and_scatter", "router_topk+gather"},
    {"moe_route_and_scatter_noalloc", "router_topk+gather"},
    {"moe_build_scatter", "gather"},
    {"moe_grouped_swiglu_fc1", "expert_projection"},
    {"moe_grouped_fc2", "expert_projection"},
    {"moe_gather_combine", "scatter_combine"},
    {"moe_shared_expert", "shared_expert_projection"},
    {"moe_shared_expert:gated", "shared_expert_gate+shared_expert_projection"},
    {"moe_grouped_swiglu_fc1_mx8", "expert_projection"},
    {"moe_grouped_fc2_mx8", "expert_projection"},
    {"moe_shared_expert_mx8", "shared_expert_projection"},
    {"moe_shared_expert_mx8:gated", "shared_expert_gate+shared_expert_projection"},
    {"moe_grouped_swiglu_fc1_and_shared_mx8", "expert_projection+shared_expert_projection"},
    {"moe_grouped_fc2_and_shared_mx8", "expert_projection+shared_expert_projection"},
    {"moe_grouped_fc2_and_shared_mx8:gated", "expert_projection+shared_expert_gate+shared_expert_projection"},
    {"moe_grouped_swiglu_fc1_and_shared", "expert_projection+shared_expert_projection"},
    {"moe_grouped_swiglu_fc1_gather", "expert_projection"},
    {"moe_grouped_swiglu_fc1_and_shared_gather", "expert_projection+shared_expert_projection"},
    {"moe_grouped_fc2_and_shared", "expert_projection+shared_expert_projection"},
    {"moe_grouped_fc2_and_shared:gated", "expert_projection+shared_expert_gate+shared_expert_projection"},
    {"moe_grouped_swiglu_fc1_save", "expert_projection"},
    {"moe_scatter_grad", "backward:scatter_combine"},
    {"moe_grouped_fc2_backward", "backward:expert_projection"},
    {"moe_grouped_fc1_backward", "backward:expert_projection+backward:gather"},
    {"moe_shared_fc1_save", "shared_expert_projection"},
    {"moe_shared_fc2_save", "shared_expert_projection"},
    {"moe_shared_fc2_save:gated", "shared_expert_gate+shared_expert_projection"},
    {"moe_shared_fc2_backward", "backward:shared_expert_projection"},
    {"moe_shared_fc2_backward:gated", "backward:shared_expert_gate+backward:shared_expert_projection"},
    {"moe_shared_fc1_backward", "backward:shared_expert_projection"},
    {"moe_shared_fc1_backward:gated", "backward:shared_expert_gate+backward:shared_expert_projection"},
    {"moe_route_backward", "backward:router_topk"},
    {"moe_balance_loss", "router_topk"},
    {"moe_route_balance_backward", "backward:router_topk"},
    {"moe_norm_residual", "residual_setup"},
    {"moe_norm_residual_backward", "backward:residual_setup"},
    {"moe_orthogonal_update", "backward:other"},
    {"moe_grad_norm", "backward:other"},
    {"moe_grad_clip", "backward:other"},
};

const char* stage_of(const char* call) {
  for (const CallStage& c : kCallStages)
    if (strcmp(c.call, call) == 0) return c.stage;
  return "other";
}

// roctx range around one call, named with its stage: a rocprofv3 marker
// trace then attributes every launch to a stage.
struct StageRange {
  explicit StageRange(const char* stage) { roctxRangePushA(stage); }
  ~StageRange() { roctxRangePop(); }
  StageRange(const StageRange&) = delete;
  StageRange& operator=(const StageRange&) = delete;
};

}  // namespace

extern "C" {

const char* moe_status_name(int status) {
  switch (status) {
    case MOE_OK: return "MOE_OK";
    case MOE_ERR_INVALID_ARGUMENT: return "MOE_ERR_INVALID_ARGUMENT";
    case MOE_ERR_UNSUPPORTED: return "MOE_ERR_UNSUPPORTED";
    case MOE_ERR_WORKSPACE: return "MOE_ERR_WORKSPACE";
    case MOE_ERR_HIP: return "MOE_ERR_HIP";
    default: return "MOE_STATUS_UNKNOWN";
  }
}

const char* moe_last_error(void) { return g_last_error.c_str(); }

int moe_version(void) { return kVersion; }

const char* moe_call_stage(const char* call, int32_t gated) {
  if (!call) return "other";
  if (gated) {
    const std::string g = std::string(call) + ":gated";
    for (const CallStage& c : kCallStages)
      if (g == c.call) return c.stage;
  }
  return stage_of(call);
}

size_t moe_route_workspace_bytes(moe_dtype dt, int32_t T, int32_t H, int32_t E) {
  if (T < 1 || H < 1 || E < 1 || (dt != MOE_F32 && dt != MOE_BF16)) return 0;
  return moe_launch::route_workspace_bytes((int)dt, T, H, E);
}

moe_status moe_route(moe_dtype dt, const void* x, const void* w_router, const float* logit_bias, int32_t T, int32_t H,
                     int32_t E, int32_t top_k, int32_t* topk_ids, float* topk_weights, float* logits, void* workspace,
                     size_t workspace_bytes, void* stream) {
  const char* fn = "moe_route";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_dtype(dt, fn));
  MOE_CHECK(need_ptr(x, fn, "x"));
  MOE_CHECK(need_ptr(w_router, fn, "w_router"));
  MOE_CHECK(need_ptr(topk_ids, fn, "topk_ids"));
  MOE_CHECK(need_ptr(topk_weights, fn, "topk_weights"));
  MOE_CHECK(need_ptr(logits, fn, "logits"));
  MOE_CHECK(need_pos(T, fn, "T"));
  MOE_CHECK(need_pos(H, fn, "H"));
  MOE_CHECK(need_experts(E, fn));
  MOE_CHECK(need_topk(top_k, fn));
  if (top_k > E) return fail(MOE_ERR_INVALID_ARGUMENT, "moe_route: top_k (%d) exceeds E (%d)", top_k, E);
  MOE_CHECK(need_mult8(H, fn, "H"));
  MOE_CHECK(need_rows((int64_t)T * top_k, fn, "T*top_k"));
  MOE_CHECK(need_rows((int64_t)T * E / 8, fn, "T*E/8"));
  const size_t need = moe_launch::route_workspace_bytes((int)dt, T, H, E);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(MOE_ERR_WORKSPACE, "moe_route: workspace needs %zu bytes (got %zu%s)", need, workspace_bytes,
                workspace ? "" : ", NULL pointer");
  return hip_result(moe_launch::route((int)dt, x, w_router, logit_bias, T, H, E, top_k, topk_ids, topk_weights, logits,
                                      workspace, (hipStream_t)stream),
                    fn);
}

size_t moe_route_and_scatter_workspace_bytes(moe_dtype dt, int32_t T, int32_t H, int32_t E, int32_t top_k) {
  if (T < 1 || H < 1 || E < 1 || top_k < 1 || (dt != MOE_F32 && dt != MOE_BF16)) return 0;
  const size_t r = moe_launch::route_workspace_bytes((int)dt, T, H, E);
  const size_t sc = moe_launch::scatter_workspace_bytes(T, top_k, E);
  return r > sc ? r : sc;
}

}  // extern "C"

namespace {

// Argument checks of moe_route_and_scatter and its no-allocation variant
// (everything but the workspace).
moe_status check_route_and_scatter(const char* fn, moe_dtype dt, const void* x, const void* w_router, int32_t T,
                                   int32_t H, int32_t E, int32_t top_k, const int32_t* topk_ids,
                                   const float* topk_weights, const float* logits, const int32_t* scatter_index,
                                   const int32_t* row_token, const int32_t* expert_offsets,
                                   const int32_t* status_words) {
  MOE_CHECK(need_dtype(dt, fn));
  MOE_CHECK(need_ptr(x, fn, "x"));
  MOE_CHECK(need_ptr(w_router, fn, "w_router"));
  MOE_CHECK(need_ptr(topk_ids, fn, "topk_ids"));
  MOE_CHECK(need_ptr(topk_weights, fn, "topk_weights"));
  MOE_CHECK(need_ptr(logits, fn, "logits"));
  MOE_CHECK(need_ptr(scatter_index, fn, "scatter_index"));
  MOE_CHECK(need_ptr(row_token, fn, "row_token"));
  MOE_CHECK(need_ptr(expert_offsets, fn, "expert_offsets"));
  MOE_CHECK(need_ptr(status_words, fn, "status_words"));
  // x_scattered may be NULL: the rows are then not copied (the *_gather fc1 calls read x instead)
  MOE_CHECK(need_pos(T, fn, "T"));
  MOE_CHECK(need_pos(H, fn, "H"));
  MOE_CHECK(need_experts(E, fn));
  MOE_CHECK(need_topk(top_k, fn));
  if (top_k > E) return fail(MOE_ERR_INVALID_ARGUMENT, "%s: top_k (%d) exceeds E (%d)", fn, top_k, E);
  MOE_CHECK(need_mult8(H, fn, "H"));
  MOE_CHECK(need_rows((int64_t)T * top_k, fn, "T*top_k"));
  MOE_CHECK(need_rows((int64_t)T * E / 8, fn, "T*E/8"));
  return MOE_OK;
}

// The kernels of moe_route_and_scatter on a validated call, with `workspace`
// holding at least moe_route_and_scatter_workspace_bytes bytes.
moe_status run_route_and_scatter(const char* fn, moe_dtype dt, const void* x, const void* w_router,
                                 const float* logit_bias, int32_t T, int32_t H, int32_t E, int32_t top_k,
                                 int32_t* topk_ids, float* topk_weights, float* logits, int32_t* scatter_index,
                                 int32_t* row_token, int32_t* expert_offsets, int32_t* status_words,
                                 void* x_scattered, void* workspace, void* stream) {
  const hipStream_t s = (hipStream_t)stream;
  if (moe_launch::router_small((int)dt, T, E) && moe_launch::route_scatter_fusable(T, top_k, E)) {
    int nsplit = 0;
    hipError_t err = moe_launch::route_partials_small(x, w_router, T, H, E, workspace, &nsplit, s);
    if (err == hipSuccess)
      err = moe_launch::route_scatter_fused((int)dt, (const float*)workspace, nsplit, logit_bias, logits, T, H, E,
                                            top_k, topk_ids, topk_weights, x, scatter_index, row_token,
                                            expert_offsets, status_words, x_scattered, s);
    return hip_result(err, fn);
  }
  hipError_t err = moe_launch::route((int)dt, x, w_router, logit_bias, T, H, E, top_k, topk_ids, topk_weights,
                                     logits, workspace, s);
  if (err == hipSuccess)
    err = moe_launch::build_scatter((int)dt, x, topk_ids, T, H, E, top_k, scatter_index, row_token, expert_offsets,
                                    status_words, x_scattered, workspace, s);
  return hip_result(err, fn);
}

// Scratch of the no-allocation entry point: one array per GPU, allocated
// when the code object loads and held until the process ends.  Host code
// must not pass `scratch` itself to a kernel (on the host it names a
// stand-in, not device memory); it uses the device address that
// hipGetSymbolAddress returns, looked up once per device with that device
// current and kept in scratch_addr.
constexpr size_t kScratchBytes = (size_t)64 << 20;

}  // namespace

static __device__ __align__(256) unsigned char scratch[kScratchBytes];

namespace {

std::mutex g_scratch_mu;
void* g_scratch_addr[64] = {};

moe_status scratch_address(const char* fn, void** out) {
  int dev = 0;
  hipError_t err = hipGetDevice(&dev);
  if (err != hipSuccess) return hip_result(err, fn);
  if (dev < 0 || dev >= 64) return fail(MOE_ERR_UNSUPPORTED, "%s: device ordinal %d is beyond 63", fn, dev);
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_addr[dev]) {
    void* p = nullptr;
    err = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (err != hipSuccess) return hip_result(err, fn);
    if (!p) return fail(MOE_ERR_HIP, "%s: hipGetSymbolAddress returned no address for the scratch array", fn);
    g_scratch_addr[dev] = p;
  }
  *out = g_scratch_addr[dev];
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_route_and_scatter(moe_dtype dt, const void* x, const void* w_router, const float* logit_bias,
                                 int32_t T, int32_t H, int32_t E, int32_t top_k, int32_t* topk_ids,
                                 float* topk_weights, float* logits, int32_t* scatter_index, int32_t* row_token,
                                 int32_t* expert_offsets, int32_t* status_words, void* x_scattered, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  const char* fn = "moe_route_and_scatter";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(check_route_and_scatter(fn, dt, x, w_router, T, H, E, top_k, topk_ids, topk_weights, logits,
                                    scatter_index, row_token, expert_offsets, status_words));
  const size_t need = moe_route_and_scatter_workspace_bytes(dt, T, H, E, top_k);
  if (!workspace || workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace needs %zu bytes (got %zu%s)", fn, need, workspace_bytes,
                workspace ? "" : ", NULL pointer");
  return run_route_and_scatter(fn, dt, x, w_router, logit_bias, T, H, E, top_k, topk_ids, topk_weights, logits,
                               scatter_index, row_token, expert_offsets, status_words, x_scattered, workspace,
                               stream);
}

size_t moe_route_and_scatter_noalloc_max_bytes(void) { return kScratchBytes; }

moe_status moe_route_and_scatter_noalloc(moe_dtype dt, const void* x, const void* w_router, const float* logit_bias,
                                         int32_t T, int32_t H, int32_t E, int32_t top_k, int32_t* topk_ids,
                                         float* topk_weights, float* logits, int32_t* scatter_index,
                                         int32_t* row_token, int32_t* expert_offsets, int32_t* status_words,
                                         void* x_scattered, void* stream) {
  const char* fn = "moe_route_and_scatter_noalloc";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(check_route_and_scatter(fn, dt, x, w_router, T, H, E, top_k, topk_ids, topk_weights, logits,
                                    scatter_index, row_token, expert_offsets, status_words));
  const size_t need = moe_route_and_scatter_workspace_bytes(dt, T, H, E, top_k);
  if (need > kScratchBytes)
    return fail(MOE_ERR_UNSUPPORTED, "%s: these sizes need %zu bytes of scratch, more than the %zu bytes the "
                "library holds per device (use moe_route_and_scatter with a workspace)", fn, need, kScratchBytes);
  void* ws = nullptr;
  MOE_CHECK(scratch_address(fn, &ws));
  return run_route_and_scatter(fn, dt, x, w_router, logit_bias, T, H, E, top_k, topk_ids, topk_weights, logits,
                               scatter_index, row_token, expert_offsets, status_words, x_scattered, ws, stream);
}

size_t moe_build_scatter_workspace_bytes(int32_t T, int32_t top_k, int32_t E) {
  if (T < 1 || top_k < 1 || E < 1) return 0;
  return moe_launch::scatter_workspace_bytes(T, top_k, E);
}

moe_status moe_build_scatter(moe_dtype dt, const void* x, const int32_t* topk_ids, int32_t T, int32_t H, int32_t E,
                             int32_t top_k, int32_t* scatter_index, int32_t* row_token, int32_t* expert_offsets,
                             int32_t* status_words, void* x_scattered, void* workspace, size_t workspace_bytes,
                             void* stream) {
  const char* fn = "moe_build_scatter";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_dtype(dt, fn));
  MOE_CHECK(need_ptr(x, fn, "x"));
  MOE_CHECK(need_ptr(topk_ids, fn, "topk_ids"));
  MOE_CHECK(need_ptr(scatter_index, fn, "scatter_index"));
  MOE_CHECK(need_ptr(row_token, fn, "row_token"));
  MOE_CHECK(need_ptr(expert_offsets, fn, "expert_offsets"));
  MOE_CHECK(need_ptr(status_words, fn, "status_words"));
  // x_scattered may be NULL: the rows are then not copied (the *_gather fc1 calls read x instead)
  MOE_CHECK(need_pos(T, fn, "T"));
  MOE_CHECK(need_pos(H, fn, "H"));
  MOE_CHECK(need_experts(E, fn));
  MOE_CHECK(need_topk(top_k, fn));
  MOE_CHECK(need_mult8(H, fn, "H"));
  MOE_CHECK(need_rows((int64_t)T * top_k, fn, "T*top_k"));
  const size_t need = moe_launch::scatter_workspace_bytes(T, top_k, E);
  if (!workspace || workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "moe_build_scatter: workspace needs %zu bytes (got %zu%s)", need, workspace_bytes,
                workspace ? "" : ", NULL pointer");
  return hip_result(moe_launch::build_scatter((int)dt, x, topk_ids, T, H, E, top_k, scatter_index, row_token,
                                              expert_offsets, status_words, x_scattered, workspace,
                                              (hipStream_t)stream),
                    fn);
}

moe_status moe_grouped_swiglu_fc1(moe_dtype dt, moe_weight_layout wl, const void* x_scattered,
                                  const int32_t* expert_offsets, const void* w1, int32_t R, int32_t H, int32_t E,
                                  int32_t I, void* act, void* stream) {
  const char* fn = "moe_grouped_swiglu_fc1";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_dtype(dt, fn));
  MOE_CHECK(need_layout(wl, fn));
  MOE_CHECK(need_ptr(x_scattered, fn, "x_scattered"));
  MOE_CHECK(need_ptr(expert_offsets, fn, "expert_offsets"));
  MOE_CHECK(need_ptr(w1, fn, "w1"));
  MOE_CHECK(need_ptr(act, fn, "act"));
  MOE_CHECK(need_pos(R, fn, "R"));
  MOE_CHECK(need_pos(H, fn, "H"));
  MOE_CHECK(need_experts(E, fn));
  MOE_CHECK(need_pos(I, fn, "I"));
  MOE_CHECK(need_mult8(H, fn, "H"));
  MOE_CHECK(need_mult8(I, fn, "I"));
  MOE_CHECK(need_rows(R, fn, "R"));
  return hip_result(moe_launch::grouped_swiglu_fc1((int)dt, (int)wl, x_scattered, expert_offsets, E, R, w1,
                                                   (int64_t)H * 2 * I, H, I, act, 0, cu_count(), (hipStream_t)stream),
                    fn);
}

moe_status moe_grouped_fc2(moe_dtype dt, moe_weight_layout wl, const void* act, const int32_t* expert_offsets,
                           const void* w2, int32_t R, int32_t I, int32_t E, int32_t H, float* y_rows, void* stream) {
  const char* fn = "moe_grouped_fc2";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_dtype(dt, fn));
  MOE_CHECK(need_layout(wl, fn));
  MOE_CHECK(need_ptr(act, fn, "act"));
  MOE_CHECK(need_ptr(expert_offsets, fn, "expert_offsets"));
  MOE_CHECK(need_ptr(w2, fn, "w2"));
  MOE_CHECK(need_ptr(y_rows, fn, "y_rows"));
  MOE_CHECK(need_pos(R, fn, "R"));
  MOE_CHECK(need_pos(I, fn, "I"));
  MOE_CHECK(need_experts(E, fn));
  MOE_CHECK(need_pos(H, fn, "H"));
  MOE_CHECK(need_mult8(H, fn, "H"));
  MOE_CHECK(need_mult8(I, fn, "I"));
  MOE_CHECK(need_rows(R, fn, "R"));
  return hip_result(moe_launch::grouped_fc2((int)dt, (int)wl, act, expert_offsets, E, R, w2, (int64_t)I * H, I, H,
                                            y_rows, nullptr, 0, 1, 0, cu_count(), (hipStream_t)stream),
                    fn);
}

moe_status moe_gather_combine(const float* y_rows, const int32_t* scatter_index, const float* topk_weights, int32_t T,
                              int32_t H, int32_t top_k, int32_t accumulate, float* y, void* stream) {
  const char* fn = "moe_gather_combine";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_ptr(y_rows, fn, "y_rows"));
  MOE_CHECK(need_ptr(scatter_index, fn, "scatter_index"));
  MOE_CHECK(need_ptr(topk_weights, fn, "topk_weights"));
  MOE_CHECK(need_ptr(y, fn, "y"));
  MOE_CHECK(need_pos(T, fn, "T"));
  MOE_CHECK(need_pos(H, fn, "H"));
  MOE_CHECK(need_topk(top_k, fn));
  MOE_CHECK(need_mult8(H, fn, "H"));
  MOE_CHECK(need_flag(accumulate, fn, "accumulate"));
  MOE_CHECK(need_rows((int64_t)T * top_k, fn, "T*top_k"));
  return hip_result(moe_launch::gather_combine(y_rows, scatter_index, topk_weights, T, H, top_k, accumulate, y,
                                               (hipStream_t)stream),
                    fn);
}

size_t moe_shared_expert_workspace_bytes(moe_dtype dt, int32_t T, int32_t I_s) {
  if (T < 1 || I_s < 1 || (dt != MOE_F32 && dt != MOE_BF16)) return 0;
  return align256((size_t)T * I_s * elem_size(dt)) + align256((size_t)T * sizeof(float));
}

moe_status moe_shared_expert(moe_dtype dt, moe_weight_layout wl, const void* x, const void* ws1, const void* ws2,
                             const void* w_gate, int32_t T, int32_t H, int32_t I_s, int32_t accumulate, float* y,
                             void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "moe_shared_expert";
  StageRange stage_range(stage_of(w_gate ? "moe_shared_expert:gated" : fn));
  MOE_CHECK(need_dtype(dt, fn));
  MOE_CHECK(need_layout(wl, fn));
  MOE_CHECK(need_ptr(x, fn, "x"));
  MOE_CHECK(need_ptr(ws1, fn, "ws1"));
  MOE_CHECK(need_ptr(ws2, fn, "ws2"));
  MOE_CHECK(need_ptr(y, fn, "y"));
  MOE_CHECK(need_pos(T, fn, "T"));
  MOE_CHECK(need_pos(H, fn, "H"));
  MOE_CHECK(need_pos(I_s, fn, "I_s"));
  MOE_CHECK(need_mult8(H, fn, "H"));
  MOE_CHECK(need_mult8(I_s, fn, "I_s"));
  MOE_CHECK(need_flag(accumulate, fn, "accumulate"));
  MOE_CHECK(need_rows(T, fn, "T"));
  const size_t need = moe_shared_expert_workspace_bytes(dt, T, I_s);
  if (!workspace || workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "moe_shared_expert: workspace needs %zu bytes (got %zu%s)", need, workspace_bytes,
                workspace ? "" : ", NULL pointer");
  hipStream_t s = (hipStream_t)stream;
  char* ws = (char*)workspace;
  void* act = ws;
  float* gate = w_gate ? (float*)(ws + align256((size_t)T * I_s * elem_size(dt))) : nullptr;
  const int cus = cu_count();
  if (gate) MOE_CHECK(hip_result(moe_launch::shared_gate((int)dt, x, w_gate, T, H, gate, s), fn));
  MOE_CHECK(hip_result(
      moe_launch::grouped_swiglu_fc1((int)dt, (int)wl, x, nullptr, 1, T, ws1, 0, H, I_s, act, 1, cus, s), fn));
  return hip_result(
      moe_launch::grouped_fc2((int)dt, (int)wl, act, nullptr, 1, T, ws2, 0, I_s, H, y, gate, accumulate, 0, 1, cus, s),
      fn);
}

moe_status need_mult128(int64_t v, const char* fn, const char* name) {
  return v % 128 == 0 ? MOE_OK
                      : fail(MOE_ERR_UNSUPPORTED, "%s: %s must be a multiple of 128 for MXFP8 weights (got %lld)", fn,
                             name, (long long)v);
}

moe_status moe_grouped_swiglu_fc1_mx8(const void* x_scattered, const int32_t* expert_offsets, const uint8_t* w1q,
                                      const uint8_t* w1s, int32_t R, int32_t H, int32_t E, int32_t I, void* act,
                                      void* stream) {
  const char* fn = "moe_grouped_swiglu_fc1_mx8";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_ptr(x_scattered, fn, "x_scattered"));
  MOE_CHECK(need_ptr(expert_offsets, fn, "expert_offsets"));
  MOE_CHECK(need_ptr(w1q, fn, "w1q"));
  MOE_CHECK(need_ptr(w1s, fn, "w1s"));
  MOE_CHECK(need_ptr(act, fn, "act"));
  MOE_CHECK(need_pos(R, fn, "R"));
  MOE_CHECK(need_pos(H, fn, "H"));
  MOE_CHECK(need_experts(E, fn));
  MOE_CHECK(need_pos(I, fn, "I"));
  MOE_CHECK(need_mult8(I, fn, "I"));
  MOE_CHECK(need_mult128(H, fn, "H"));
  MOE_CHECK(need_rows(R, fn, "R"));
  return hip_result(moe_launch::grouped_swiglu_fc1_mx8(x_scattered, expert_offsets, E, R, w1q, w1s, H, I, act, 0,
                                                       cu_count(), (hipStream_t)stream),
                    fn);
}

moe_status moe_grouped_fc2_mx8(const void* act, const int32_t* expert_offsets, const uint8_t* w2q,
                               const uint8_t* w2s, int32_t R, int32_t I, int32_t E, int32_t H, float* y_rows,
                               void* stream) {
  const char* fn = "moe_grouped_fc2_mx8";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_ptr(act, fn, "act"));
  MOE_CHECK(need_ptr(expert_offsets, fn, "expert_offsets"));
  MOE_CHECK(need_ptr(w2q, fn, "w2q"));
  MOE_CHECK(need_ptr(w2s, fn, "w2s"));
  MOE_CHECK(need_ptr(y_rows, fn, "y_rows"));
  MOE_CHECK(need_pos(R, fn, "R"));
  MOE_CHECK(need_pos(I, fn, "I"));
  MOE_CHECK(need_experts(E, fn));
  MOE_CHECK(need_pos(H, fn, "H"));
  MOE_CHECK(need_mult8(H, fn, "H"));
  MOE_CHECK(need_mult128(I, fn, "I"));
  MOE_CHECK(need_rows(R, fn, "R"));
  return hip_result(moe_launch::grouped_fc2_mx8(act, expert_offsets, E, R, w2q, w2s, I, H, y_rows, nullptr, 0, 1, 0,
                                                cu_count(), (hipStream_t)stream),
                    fn);
}

moe_status moe_shared_expert_mx8(const void* x, const uint8_t* ws1q, const uint8_t* ws1s, const uint8_t* ws2q,
                                 const uint8_t* ws2s, const void* w_gate, int32_t T, int32_t H, int32_t I_s,
                                 int32_t accumulate, float* y, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  const char* fn = "moe_shared_expert_mx8";
  StageRange stage_range(stage_of(w_gate ? "moe_shared_expert_mx8:gated" : fn));
  MOE_CHECK(need_ptr(x, fn, "x"));
  MOE_CHECK(need_ptr(ws1q, fn, "ws1q"));
  MOE_CHECK(need_ptr(ws1s, fn, "ws1s"));
  MOE_CHECK(need_ptr(ws2q, fn, "ws2q"));
  MOE_CHECK(need_ptr(ws2s, fn, "ws2s"));
  MOE_CHECK(need_ptr(y, fn, "y"));
  MOE_CHECK(need_pos(T, fn, "T"));
  MOE_CHECK(need_pos(H, fn, "H"));
  MOE_CHECK(need_pos(I_s, fn, "I_s"));
  MOE_CHECK(need_mult128(H, fn, "H"));
  MOE_CHECK(need_mult128(I_s, fn, "I_s"));
  MOE_CHECK(need_flag(accumulate, fn, "accumulate"));
  MOE_CHECK(need_rows(T, fn, "T"));
  const size_t need = moe_shared_expert_workspace_bytes(MOE_BF16, T, I_s);
  if (!workspace || workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace needs %zu bytes (got %zu%s)", fn, need, workspace_bytes,
                workspace ? "" : ", NULL pointer");
  hipStream_t s = (hipStream_t)stream;
  char* ws = (char*)workspace;
  void* act = ws;
  float* gate = w_gate ? (float*)(ws + align256((size_t)T * I_s * elem_size(MOE_BF16))) : nullptr;
  const int cus = cu_count();
  if (gate) MOE_CHECK(hip_result(moe_launch::shared_gate(1, x, w_gate, T, H, gate, s), fn));
  MOE_CHECK(hip_result(moe_launch::grouped_swiglu_fc1_mx8(x, nullptr, 1, T, ws1q, ws1s, H, I_s, act, 1, cus, s), fn));
  return hip_result(moe_launch::grouped_fc2_mx8(act, nullptr, 1, T, ws2q, ws2s, I_s, H, y, gate, accumulate, 0, 1, cus,
                                                s),
                    fn);
}

moe_status moe_grouped_swiglu_fc1_and_shared_mx8(const void* x_scattered, const int32_t* expert_offsets,
                                                 const uint8_t* w1q, const uint8_t* w1s, int32_t R, int32_t H,
                                                 int32_t E, int32_t I, void* act, const void* x, const uint8_t* ws1q,
                                                 const uint8_t* ws1s, int32_t T, int32_t I_s, void* act_shared,
                                                 void* stream) {
  const char* fn = "moe_grouped_swiglu_fc1_and_shared_mx8";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_ptr(x_scattered, fn, "x_scattered"));
  MOE_CHECK(need_ptr(expert_offsets, fn, "expert_offsets"));
  MOE_CHECK(need_ptr(w1q, fn, "w1q"));
  MOE_CHECK(need_ptr(w1s, fn, "w1s"));
  MOE_CHECK(need_ptr(act, fn, "act"));
  MOE_CHECK(need_ptr(x, fn, "x"));
  MOE_CHECK(need_ptr(ws1q, fn, "ws1q"));
  MOE_CHECK(need_ptr(ws1s, fn, "ws1s"));
  MOE_CHECK(need_ptr(act_shared, fn, "act_shared"));
  MOE_CHECK(need_pos(R, fn, "R"));
  MOE_CHECK(need_pos(H, fn, "H"));
  MOE_CHECK(need_experts(E, fn));
  MOE_CHECK(need_pos(I, fn, "I"));
  MOE_CHECK(need_pos(T, fn, "T"));
  MOE_CHECK(need_pos(I_s, fn, "I_s"));
  MOE_CHECK(need_mult128(H, fn, "H"));
  MOE_CHECK(need_mult128(I, fn, "I"));
  MOE_CHECK(need_mult128(I_s, fn, "I_s"));
  MOE_CHECK(need_rows(R, fn, "R"));
  MOE_CHECK(need_rows(T, fn, "T"));
  return hip_result(moe_launch::fused_fc1_mx8(x_scattered, expert_offsets, E, R, w1q, w1s, H, I, act, x, T, ws1q,
                                              ws1s, I_s, act_shared, cu_count(), (hipStream_t)stream),
                    fn);
}

moe_status moe_grouped_fc2_and_shared_mx8(const void* act, const int32_t* expert_offsets, const uint8_t* w2q,
                                          const uint8_t* w2s, int32_t R, int32_t I, int32_t E, int32_t H,
                                          float* y_rows, const void* act_shared, const uint8_t* ws2q,
                                          const uint8_t* ws2s, const void* x, const void* w_gate, int32_t T,
                                          int32_t I_s, int32_t accumulate, float* y, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  const char* fn = "moe_grouped_fc2_and_shared_mx8";
  StageRange stage_range(stage_of(w_gate ? "moe_grouped_fc2_and_shared_mx8:gated" : fn));
  MOE_CHECK(need_ptr(act, fn, "act"));
  MOE_CHECK(need_ptr(expert_offsets, fn, "expert_offsets"));
  MOE_CHECK(need_ptr(w2q, fn, "w2q"));
  MOE_CHECK(need_ptr(w2s, fn, "w2s"));
  MOE_CHECK(need_ptr(y_rows, fn, "y_rows"));
  MOE_CHECK(need_ptr(act_shared, fn, "act_shared"));
  MOE_CHECK(need_ptr(ws2q, fn, "ws2q"));
  MOE_CHECK(need_ptr(ws2s, fn, "ws2s"));
  MOE_CHECK(need_ptr(y, fn, "y"));
  if (w_gate) MOE_CHECK(need_ptr(x, fn, "x (needed for the gate)"));
  MOE_CHECK(need_pos(R, fn, "R"));
  MOE_CHECK(need_pos(I, fn, "I"));
  MOE_CHECK(need_experts(E, fn));
  MOE_CHECK(need_pos(H, fn, "H"));
  MOE_CHECK(need_pos(T, fn, "T"));
  MOE_CHECK(need_pos(I_s, fn, "I_s"));
  MOE_CHECK(need_mult8(H, fn, "H"));
  MOE_CHECK(need_mult128(I, fn, "I"));
  MOE_CHECK(need_mult128(I_s, fn, "I_s"));
  MOE_CHECK(need_flag(accumulate, fn, "accumulate"));
  MOE_CHECK(need_rows(R, fn, "R"));
  MOE_CHECK(need_rows(T, fn, "T"));
  const size_t need = moe_shared_expert_workspace_bytes(MOE_BF16, T, I_s);
  if (!workspace || workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace needs %zu bytes (got %zu%s)", fn, need, workspace_bytes,
                workspace ? "" : ", NULL pointer");
  hipStream_t s = (hipStream_t)stream;
  float* gate = w_gate ? (float*)((char*)workspace + align256((size_t)T * I_s * elem_size(MOE_BF16))) : nullptr;
  if (gate) MOE_CHECK(hip_result(moe_launch::shared_gate(1, x, w_gate, T, H, gate, s), fn));
  return hip_result(moe_launch::fused_fc2_mx8(act, expert_offsets, E, R, w2q, w2s, I, H, y_rows, act_shared, T, ws2q,
                                              ws2s, I_s, gate, accumulate, y, cu_count(), s),
                    fn);
}

int32_t moe_grouped_gemm_tile(moe_dtype dt, int32_t call, int32_t R, int32_t H, int32_t E, int32_t I, int32_t T,
                              int32_t I_s) {
  if ((dt != MOE_F32 && dt != MOE_BF16) || (call != 0 && call != 1) || R < 1 || H < 1 || E < 1 || I < 1 ||
      E > moe::kMaxExperts || I_s < 0 || (I_s > 0 && T < 1))
    return -1;
  return moe_launch::tile_config((int)dt, call, R, H, E, I, T, I_s, cu_count());
}

int32_t moe_and_shared_launches(moe_dtype dt, int32_t R, int32_t H, int32_t E, int32_t I, int32_t T, int32_t I_s) {
  if (R < 1 || H < 1 || E < 1 || I < 1 || T < 1 || I_s < 1 || (dt != MOE_F32 && dt != MOE_BF16)) return 0;
  return moe_launch::fused_supported((int)dt, H, I, I_s, E, R, T) ? 1 : 2;
}

moe_status moe_grouped_swiglu_fc1_and_shared(moe_dtype dt, moe_weight_layout wl, const void* x_scattered,
                                             const int32_t* expert_offsets, const void* w1, int32_t R, int32_t H,
                                             int32_t E, int32_t I, void* act, const void* x, const void* ws1,
                                             int32_t T, int32_t I_s, void* act_shared, void* stream) {
  const char* fn = "moe_grouped_swiglu_fc1_and_shared";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_dtype(dt, fn));
  MOE_CHECK(need_layout(wl, fn));
  MOE_CHECK(need_ptr(x_scattered, fn, "x_scattered"));
  MOE_CHECK(need_ptr(expert_offsets, fn, "expert_offsets"));
  MOE_CHECK(need_ptr(w1, fn, "w1"));
  MOE_CHECK(need_ptr(act, fn, "act"));
  MOE_CHECK(need_ptr(x, fn, "x"));
  MOE_CHECK(need_ptr(ws1, fn, "ws1"));
  MOE_CHECK(need_ptr(act_shared, fn, "act_shared"));
  MOE_CHECK(need_pos(R, fn, "R"));
  MOE_CHECK(need_pos(H, fn, "H"));
  MOE_CHECK(need_experts(E, fn));
  MOE_CHECK(need_pos(I, fn, "I"));
  MOE_CHECK(need_pos(T, fn, "T"));
  MOE_CHECK(need_pos(I_s, fn, "I_s"));
  MOE_CHECK(need_mult8(H, fn, "H"));
  MOE_CHECK(need_mult8(I, fn, "I"));
  MOE_CHECK(need_mult8(I_s, fn, "I_s"));
  MOE_CHECK(need_rows(R, fn, "R"));
  MOE_CHECK(need_rows(T, fn, "T"));
  hipStream_t s = (hipStream_t)stream;
  const int cus = cu_count();
  if (moe_launch::fused_supported((int)dt, H, I, I_s, E, R, T))
    return hip_result(moe_launch::fused_fc1((int)wl, x_scattered, expert_offsets, E, R, w1, H, I, act, x, T, ws1,
                                            I_s, act_shared, cus, s),
                      fn);
  MOE_CHECK(hip_result(moe_launch::grouped_swiglu_fc1((int)dt, (int)wl, x_scattered, expert_offsets, E, R, w1,
                                                      (int64_t)H * 2 * I, H, I, act, 0, cus, s),
                       fn));
  return hip_result(
      moe_launch::grouped_swiglu_fc1((int)dt, (int)wl, x, nullptr, 1, T, ws1, 0, H, I_s, act_shared, 1, cus, s), fn);
}

moe_status moe_grouped_swiglu_fc1_gather(moe_dtype dt, moe_weight_layout wl, const void* x, const int32_t* row_token,
                                         const int32_t* expert_offsets, const void* w1, int32_t T, int32_t R,
                                         int32_t H, int32_t E, int32_t I, void* act, void* stream) {
  const char* fn = "moe_grouped_swiglu_fc1_gather";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_dtype(dt, fn));
  MOE_CHECK(need_layout(wl, fn));
  MOE_CHECK(need_ptr(x, fn, "x"));
  MOE_CHECK(need_ptr(row_token, fn, "row_token"));
  MOE_CHECK(need_ptr(expert_offsets, fn, "expert_offsets"));
  MOE_CHECK(need_ptr(w1, fn, "w1"));
  MOE_CHECK(need_ptr(act, fn, "act"));
  MOE_CHECK(need_pos(T, fn, "T"));
  MOE_CHECK(need_pos(R, fn, "R"));
  MOE_CHECK(need_pos(H, fn, "H"));
  MOE_CHECK(need_experts(E, fn));
  MOE_CHECK(need_pos(I, fn, "I"));
  MOE_CHECK(need_mult8(H, fn, "H"));
  MOE_CHECK(need_mult8(I, fn, "I"));
  MOE_CHECK(need_rows(R, fn, "R"));
  MOE_CHECK(need_rows(T, fn, "T"));
  return hip_result(moe_launch::grouped_swiglu_fc1((int)dt, (int)wl, x, expert_offsets, E, R, w1, (int64_t)H * 2 * I,
                                                   H, I, act, 0, cu_count(), (hipStream_t)stream, row_token, T),
                    fn);
}

moe_status moe_grouped_swiglu_fc1_and_shared_gather(moe_dtype dt, moe_weight_layout wl, const void* x,
                                                    const int32_t* row_token, const int32_t* expert_offsets,
                                                    const void* w1, int32_t R, int32_t H, int32_t E, int32_t I,
                                                    void* act, const void* ws1, int32_t T, int32_t I_s,
                                                    void* act_shared, void* stream) {
  const char* fn = "moe_grouped_swiglu_fc1_and_shared_gather";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_dtype(dt, fn));
  MOE_CHECK(need_layout(wl, fn));
  MOE_CHECK(need_ptr(x, fn, "x"));
  MOE_CHECK(need_ptr(row_token, fn, "row_token"));
  MOE_CHECK(need_ptr(expert_offsets, fn, "expert_offsets"));
  MOE_CHECK(need_ptr(w1, fn, "w1"));
  MOE_CHECK(need_ptr(act, fn, "act"));
  MOE_CHECK(need_ptr(ws1, fn, "ws1"));
  MOE_CHECK(need_ptr(act_shared, fn, "act_shared"));
  MOE_CHECK(need_pos(R, fn, "R"));
  MOE_CHECK(need_pos(H, fn, "H"));
  MOE_CHECK(need_experts(E, fn));
  MOE_CHECK(need_pos(I, fn, "I"));
  MOE_CHECK(need_pos(T, fn, "T"));
  MOE_CHECK(need_pos(I_s, fn, "I_s"));
  MOE_CHECK(need_mult8(H, fn, "H"));
  MOE_CHECK(need_mult8(I, fn, "I"));
  MOE_CHECK(need_mult8(I_s, fn, "I_s"));
  MOE_CHECK(need_rows(R, fn, "R"));
  MOE_CHECK(need_rows(T, fn, "T"));
  hipStream_t s = (hipStream_t)stream;
  const int cus = cu_count();
  if (moe_launch::fused_supported((int)dt, H, I, I_s, E, R, T))
    return hip_result(moe_launch::fused_fc1((int)wl, x, expert_offsets, E, R, w1, H, I, act, x, T, ws1, I_s,
                                            act_shared, cus, s, row_token),
                      fn);
  MOE_CHECK(hip_result(moe_launch::grouped_swiglu_fc1((int)dt, (int)wl, x, expert_offsets, E, R, w1,
                                                      (int64_t)H * 2 * I, H, I, act, 0, cus, s, row_token, T),
                       fn));
  return hip_result(
      moe_launch::grouped_swiglu_fc1((int)dt, (int)wl, x, nullptr, 1, T, ws1, 0, H, I_s, act_shared, 1, cus, s), fn);
}

moe_status moe_grouped_fc2_and_shared(moe_dtype dt, moe_weight_layout wl, const void* act,
                                      const int32_t* expert_offsets, const void* w2, int32_t R, int32_t I, int32_t E,
                                      int32_t H, float* y_rows, const void* act_shared, const void* ws2,
                                      const void* x, const void* w_gate, int32_t T, int32_t I_s, int32_t accumulate,
                                      float* y, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "moe_grouped_fc2_and_shared";
  StageRange stage_range(stage_of(w_gate ? "moe_grouped_fc2_and_shared:gated" : fn));
  MOE_CHECK(need_dtype(dt, fn));
  MOE_CHECK(need_layout(wl, fn));
  MOE_CHECK(need_ptr(act, fn, "act"));
  MOE_CHECK(need_ptr(expert_offsets, fn, "expert_offsets"));
  MOE_CHECK(need_ptr(w2, fn, "w2"));
  MOE_CHECK(need_ptr(y_rows, fn, "y_rows"));
  MOE_CHECK(need_ptr(act_shared, fn, "act_shared"));
  MOE_CHECK(need_ptr(ws2, fn, "ws2"));
  MOE_CHECK(need_ptr(y, fn, "y"));
  if (w_gate) MOE_CHECK(need_ptr(x, fn, "x (needed for the gate)"));
  MOE_CHECK(need_pos(R, fn, "R"));
  MOE_CHECK(need_pos(I, fn, "I"));
  MOE_CHECK(need_experts(E, fn));
  MOE_CHECK(need_pos(H, fn, "H"));
  MOE_CHECK(need_pos(T, fn, "T"));
  MOE_CHECK(need_pos(I_s, fn, "I_s"));
  MOE_CHECK(need_mult8(H, fn, "H"));
  MOE_CHECK(need_mult8(I, fn, "I"));
  MOE_CHECK(need_mult8(I_s, fn, "I_s"));
  MOE_CHECK(need_flag(accumulate, fn, "accumulate"));
  MOE_CHECK(need_rows(R, fn, "R"));
  MOE_CHECK(need_rows(T, fn, "T"));
  const size_t need = moe_shared_expert_workspace_bytes(dt, T, I_s);
  if (!workspace || workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "moe_grouped_fc2_and_shared: workspace needs %zu bytes (got %zu%s)", need,
                workspace_bytes, workspace ? "" : ", NULL pointer");
  hipStream_t s = (hipStream_t)stream;
  float* gate = w_gate ? (float*)((char*)workspace + align256((size_t)T * I_s * elem_size(dt))) : nullptr;
  const int cus = cu_count();
  if (gate) MOE_CHECK(hip_result(moe_launch::shared_gate((int)dt, x, w_gate, T, H, gate, s), fn));
  if (moe_launch::fused_supported((int)dt, H, I, I_s, E, R, T))
    return hip_result(moe_launch::fused_fc2((int)wl, act, expert_offsets, E, R, w2, I, H, y_rows, act_shared, T,
                                            ws2, I_s, gate, accumulate, y, cus, s),
                      fn);
  MOE_CHECK(hip_result(moe_launch::grouped_fc2((int)dt, (int)wl, act, expert_offsets, E, R, w2, (int64_t)I * H, I, H,
                                               y_rows, nullptr, 0, 1, 0, cus, s),
                       fn));
  return hip_result(moe_launch::grouped_fc2((int)dt, (int)wl, act_shared, nullptr, 1, T, ws2, 0, I_s, H, y, gate,
                                            accumulate, 0, 1, cus, s),
                    fn);
}

// ------------------------------------------------------------------------------------------
// Backward of the routed experts
// ------------------------------------------------------------------------------------------
moe_status moe_grouped_swiglu_fc1_save(moe_dtype dt, moe_weight_layout wl, const void* x_scattered,
                                       const int32_t* expert_offsets, const void* w1, int32_t R, int32_t H,
                                       int32_t E, int32_t I, void* act, void* h_pre, void* stream) {
  const char* fn = "moe_grouped_swiglu_fc1_save";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_dtype(dt, fn));
  MOE_CHECK(need_layout(wl, fn));
  MOE_CHECK(need_ptr(x_scattered, fn, "x_scattered"));
  MOE_CHECK(need_ptr(expert_offsets, fn, "expert_offsets"));
  MOE_CHECK(need_ptr(w1, fn, "w1"));
  MOE_CHECK(need_ptr(act, fn, "act"));
  MOE_CHECK(need_ptr(h_pre, fn, "h_pre"));
  MOE_CHECK(need_pos(R, fn, "R"));
  MOE_CHECK(need_pos(H, fn, "H"));
  MOE_CHECK(need_experts(E, fn));
  MOE_CHECK(need_pos(I, fn, "I"));
  MOE_CHECK(need_mult8(H, fn, "H"));
  MOE_CHECK(need_mult8(I, fn, "I"));
  MOE_CHECK(need_rows(R, fn, "R"));
  return hip_result(moe_launch::grouped_swiglu_fc1_save((int)dt, (int)wl, x_scattered, expert_offsets, E, R, w1,
                                                        (int64_t)H * 2 * I, H, I, act, h_pre, cu_count(),
                                                        (hipStream_t)stream),
                    fn);
}

moe_status moe_scatter_grad(moe_dtype dt, const float* dy, const float* y_rows, const float* topk_weights,
                            const int32_t* scatter_index, int32_t T, int32_t H, int32_t top_k, int32_t R,
                            void* d_rows, float* d_topk_weights, void* stream) {
  const char* fn = "moe_scatter_grad";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_dtype(dt, fn));
  MOE_CHECK(need_ptr(dy, fn, "dy"));
  MOE_CHECK(need_ptr(y_rows, fn, "y_rows"));
  MOE_CHECK(need_ptr(topk_weights, fn, "topk_weights"));
  MOE_CHECK(need_ptr(scatter_index, fn, "scatter_index"));
  MOE_CHECK(need_ptr(d_rows, fn, "d_rows"));
  MOE_CHECK(need_ptr(d_topk_weights, fn, "d_topk_weights"));
  MOE_CHECK(need_pos(T, fn, "T"));
  MOE_CHECK(need_pos(H, fn, "H"));
  MOE_CHECK(need_topk(top_k, fn));
  MOE_CHECK(need_pos(R, fn, "R"));
  MOE_CHECK(need_mult8(H, fn, "H"));
  MOE_CHECK(need_rows((int64_t)T * top_k, fn, "T*top_k"));
  MOE_CHECK(need_rows(R, fn, "R"));
  return hip_result(moe_launch::scatter_grad((int)dt, dy, y_rows, topk_weights, scatter_index, T, H, top_k, R, d_rows,
                                             d_topk_weights, (hipStream_t)stream),
                    fn);
}

moe_status moe_grouped_fc2_backward(moe_dtype dt, moe_weight_layout wl, const void* d_rows, const void* act,
                                    const void* h_pre, const int32_t* expert_offsets, const void* w2, int32_t R,
                                    int32_t I, int32_t E, int32_t H, void* d_h, void* d_w2, void* stream) {
  const char* fn = "moe_grouped_fc2_backward";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_dtype(dt, fn));
  MOE_CHECK(need_layout(wl, fn));
  MOE_CHECK(need_ptr(d_rows, fn, "d_rows"));
  MOE_CHECK(need_ptr(act, fn, "act"));
  MOE_CHECK(need_ptr(h_pre, fn, "h_pre"));
  MOE_CHECK(need_ptr(expert_offsets, fn, "expert_offsets"));
  MOE_CHECK(need_ptr(w2, fn, "w2"));
  MOE_CHECK(need_ptr(d_h, fn, "d_h"));
  MOE_CHECK(need_ptr(d_w2, fn, "d_w2"));
  MOE_CHECK(need_pos(R, fn, "R"));
  MOE_CHECK(need_pos(I, fn, "I"));
  MOE_CHECK(need_experts(E, fn));
  MOE_CHECK(need_pos(H, fn, "H"));
  MOE_CHECK(need_mult8(H, fn, "H"));
  MOE_CHECK(need_mult8(I, fn, "I"));
  MOE_CHECK(need_rows(R, fn, "R"));
  const hipStream_t s = (hipStream_t)stream;
  const int cus = cu_count();
  hipError_t err = moe_launch::grouped_fc2_dgrad_swiglu((int)dt, (int)wl, d_rows, expert_offsets, E, R, w2, I, H,
                                                        h_pre, d_h, cus, s);
  // d_w2 in the layout of w2: [I, H] = act^T d_rows, or [H, I] = d_rows^T act.
  if (err == hipSuccess)
    err = wl == MOE_W_KN ? moe_launch::grouped_wgrad((int)dt, act, d_rows, expert_offsets, E, R, I, H, d_w2, 2, cus, s)
                         : moe_launch::grouped_wgrad((int)dt, d_rows, act, expert_offsets, E, R, H, I, d_w2, 2, cus, s);
  return hip_result(err, fn);
}

size_t moe_grouped_fc1_backward_workspace_bytes(int32_t R, int32_t H) {
  if (R < 1 || H < 1) return 0;
  return align256((size_t)R * H * sizeof(float));
}

moe_status moe_grouped_fc1_backward(moe_dtype dt, moe_weight_layout wl, const void* d_h, const void* x_scattered,
                                    const int32_t* expert_offsets, const void* w1, int32_t R, int32_t H, int32_t E,
                                    int32_t I, const int32_t* scatter_index, int32_t T, int32_t top_k,
                                    int32_t accumulate, float* d_x, void* d_w1, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  const char* fn = "moe_grouped_fc1_backward";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_dtype(dt, fn));
  MOE_CHECK(need_layout(wl, fn));
  MOE_CHECK(need_ptr(d_h, fn, "d_h"));
  MOE_CHECK(need_ptr(x_scattered, fn, "x_scattered"));
  MOE_CHECK(need_ptr(expert_offsets, fn, "expert_offsets"));
  MOE_CHECK(need_ptr(w1, fn, "w1"));
  MOE_CHECK(need_ptr(scatter_index, fn, "scatter_index"));
  MOE_CHECK(need_ptr(d_x, fn, "d_x"));
  MOE_CHECK(need_ptr(d_w1, fn, "d_w1"));
  MOE_CHECK(need_pos(R, fn, "R"));
  MOE_CHECK(need_pos(H, fn, "H"));
  MOE_CHECK(need_experts(E, fn));
  MOE_CHECK(need_pos(I, fn, "I"));
  MOE_CHECK(need_pos(T, fn, "T"));
  MOE_CHECK(need_topk(top_k, fn));
  MOE_CHECK(need_flag(accumulate, fn, "accumulate"));
  MOE_CHECK(need_mult8(H, fn, "H"));
  MOE_CHECK(need_mult8(I, fn, "I"));
  MOE_CHECK(need_rows(R, fn, "R"));
  MOE_CHECK(need_rows((int64_t)T * top_k, fn, "T*top_k"));
  const size_t need = moe_grouped_fc1_backward_workspace_bytes(R, H);
  if (!workspace || workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace needs %zu bytes (got %zu%s)", fn, need, workspace_bytes,
                workspace ? "" : ", NULL pointer");
  const hipStream_t s = (hipStream_t)stream;
  const int cus = cu_count();
  float* d_xs = (float*)workspace;
  hipError_t err = moe_launch::grouped_fc1_dgrad((int)dt, (int)wl, d_h, expert_offsets, E, R, w1, H, I, d_xs, cus, s);
  if (err == hipSuccess)
    err = moe_launch::gather_combine(d_xs, scatter_index, nullptr, T, H, top_k, accumulate, d_x, s);
  // d_w1 in the layout of w1: [H, 2I] = x_scattered^T d_h, or [2I, H] = d_h^T x_scattered.
  if (err == hipSuccess)
    err = wl == MOE_W_KN
              ? moe_launch::grouped_wgrad((int)dt, x_scattered, d_h, expert_offsets, E, R, H, 2 * I, d_w1, 1, cus, s)
              : moe_launch::grouped_wgrad((int)dt, d_h, x_scattered, expert_offsets, E, R, 2 * I, H, d_w1, 1, cus, s);
  return hip_result(err, fn);
}

// ------------------------------------------------------------------------------------------
// Training of the shared expert, backward of the router, gradient norm and clipping
// ------------------------------------------------------------------------------------------
namespace {

constexpr int32_t kMaxWidth = 1 << 18;

moe_status need_align(const void* p, size_t a, const char* fn, const char* name) {
  return ((uintptr_t)p & (a - 1)) == 0
             ? MOE_OK
             : fail(MOE_ERR_INVALID_ARGUMENT, "%s: %s must be %zu-byte aligned", fn, name, a);
}

// A required device tensor read or written 16 bytes at a time.
moe_status need_tensor(const void* p, const char* fn, const char* name) {
  MOE_CHECK(need_ptr(p, fn, name));
  return need_align(p, 16, fn, name);
}

// A tensor that must be given exactly when `wanted`.
moe_status need_iff(const void* p, bool wanted, const char* fn, const char* name, const char* when) {
  if (wanted) return need_tensor(p, fn, name);
  return p ? fail(MOE_ERR_INVALID_ARGUMENT, "%s: %s must be NULL without %s", fn, name, when) : MOE_OK;
}

moe_status need_width(int32_t v, const char* fn, const char* name) {
  MOE_CHECK(need_pos(v, fn, name));
  MOE_CHECK(need_mult8(v, fn, name));
  return v <= kMaxWidth ? MOE_OK
                        : fail(MOE_ERR_UNSUPPORTED, "%s: %s must be <= 2^18 (got %d)", fn, name, (int)v);
}

moe_status need_workspace(const void* ws, size_t have, size_t need, const char* fn) {
  if (!ws || have < need)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace needs %zu bytes (got %zu%s)", fn, need, have,
                ws ? "" : ", NULL pointer");
  return need_align(ws, 16, fn, "workspace");
}

// A launch of `blocks` workgroups of 256 threads: at most 2^32 - 1 threads.
moe_status need_launch(int64_t blocks, const char* fn) {
  return blocks < (int64_t)1 << 24
             ? MOE_OK
             : fail(MOE_ERR_UNSUPPORTED, "%s: too large for one launch (%lld workgroups, 2^24 - 1 allowed)", fn,
                    (long long)blocks);
}

// call: as in moe_shared_train_tiles
moe_status need_shared_sizes(moe_dtype dt, int32_t call, moe_weight_layout wl, int32_t T, int32_t H, int32_t I_s,
                             const char* fn) {
  MOE_CHECK(need_dtype(dt, fn));
  MOE_CHECK(need_layout(wl, fn));
  MOE_CHECK(need_pos(T, fn, "T"));
  MOE_CHECK(need_width(H, fn, "H"));
  MOE_CHECK(need_width(I_s, fn, "I_s"));
  if ((int64_t)H * I_s >= (int64_t)1 << 28)
    return fail(MOE_ERR_UNSUPPORTED, "%s: H * I_s must be < 2^28 (got %d * %d)", fn, (int)H, (int)I_s);
  MOE_CHECK(need_rows(T, fn, "T"));
  return dt == MOE_F32 ? need_launch(moe_launch::shared_f32_blocks(call, T, H, I_s), fn) : MOE_OK;
}

}  // namespace

size_t moe_shared_train_workspace_bytes(moe_dtype dt, int32_t T, int32_t H, int32_t I_s) {
  if (T < 1 || H < 1 || I_s < 1 || H > kMaxWidth || I_s > kMaxWidth || (dt != MOE_F32 && dt != MOE_BF16)) return 0;
  return moe_launch::shared_train_workspace_bytes((int)dt, T, H, I_s);
}

int32_t moe_shared_train_tiles(moe_dtype dt, int32_t call, moe_weight_layout wl, int32_t T, int32_t H, int32_t I_s,
                               int32_t* splits) {
  if (!splits || call < 0 || call > 3 || need_shared_sizes(dt, call, wl, T, H, I_s, "moe_shared_train_tiles") != MOE_OK)
    return -1;
  return moe_launch::shared_train_tiles((int)dt, call, (int)wl, T, H, I_s, cu_count(), splits);
}

moe_status moe_shared_fc1_save(moe_dtype dt, moe_weight_layout wl, const void* x, const void* ws1, int32_t T,
                               int32_t H, int32_t I_s, void* act, void* h_pre, void* workspace,
                               size_t workspace_bytes, void* stream) {
  const char* fn = "moe_shared_fc1_save";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_shared_sizes(dt, 0, wl, T, H, I_s, fn));
  MOE_CHECK(need_tensor(x, fn, "x"));
  MOE_CHECK(need_tensor(ws1, fn, "ws1"));
  MOE_CHECK(need_tensor(act, fn, "act"));
  MOE_CHECK(need_tensor(h_pre, fn, "h_pre"));
  MOE_CHECK(need_workspace(workspace, workspace_bytes, moe_shared_train_workspace_bytes(dt, T, H, I_s), fn));
  const size_t e = dt == MOE_BF16 ? 2 : 4, t = (size_t)T, h = (size_t)H, i = (size_t)I_s;
  const Span spans[] = {
      {x, e * t * h, "x", false},
      {ws1, e * h * 2 * i, "ws1", false},
      {act, e * t * i, "act", true},
      {h_pre, e * t * 2 * i, "h_pre", true},
      {workspace, moe_shared_train_workspace_bytes(dt, T, H, I_s), "workspace", true}};
  MOE_CHECK(need_apart(spans, fn));
  return hip_result(moe_launch::shared_fc1_save((int)dt, (int)wl, x, ws1, T, H, I_s, act, h_pre, workspace,
                                                cu_count(), (hipStream_t)stream),
                    fn);
}

moe_status moe_shared_fc2_save(moe_dtype dt, moe_weight_layout wl, const void* act, const void* ws2, const void* x,
                               const void* w_gate, int32_t T, int32_t H, int32_t I_s, int32_t accumulate, float* y,
                               float* y_shared, float* gate, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "moe_shared_fc2_save";
  const bool gated = w_gate != nullptr;
  StageRange stage_range(stage_of(gated ? "moe_shared_fc2_save:gated" : fn));
  MOE_CHECK(need_shared_sizes(dt, 1, wl, T, H, I_s, fn));
  MOE_CHECK(need_flag(accumulate, fn, "accumulate"));
  MOE_CHECK(need_tensor(act, fn, "act"));
  MOE_CHECK(need_tensor(ws2, fn, "ws2"));
  if (gated) {
    MOE_CHECK(need_tensor(w_gate, fn, "w_gate"));
    MOE_CHECK(need_tensor(x, fn, "x (needed for the gate)"));
  }
  MOE_CHECK(need_tensor(y, fn, "y"));
  MOE_CHECK(need_iff(y_shared, gated, fn, "y_shared", "w_gate"));
  MOE_CHECK(need_iff(gate, gated, fn, "gate", "w_gate"));
  MOE_CHECK(need_workspace(workspace, workspace_bytes, moe_shared_train_workspace_bytes(dt, T, H, I_s), fn));
  const size_t e = dt == MOE_BF16 ? 2 : 4, t = (size_t)T, h = (size_t)H, i = (size_t)I_s;
  const Span spans[] = {
      {act, e * t * i, "act", false},
      {ws2, e * i * h, "ws2", false},
      {gated ? x : nullptr, e * t * h, "x", false},
      {w_gate, e * h, "w_gate", false},
      {y, 4 * t * h, "y", true},
      {y_shared, 4 * t * h, "y_shared", true},
      {gate, 4 * t, "gate", true},
      {workspace, moe_shared_train_workspace_bytes(dt, T, H, I_s), "workspace", true}};
  MOE_CHECK(need_apart(spans, fn));
  return hip_result(moe_launch::shared_fc2_save((int)dt, (int)wl, act, ws2, x, w_gate, T, H, I_s, accumulate, y,
                                                y_shared, gate, workspace, cu_count(), (hipStream_t)stream),
                    fn);
}

moe_status moe_shared_fc2_backward(moe_dtype dt, moe_weight_layout wl, const float* dy, const void* act,
                                   const void* h_pre, const void* ws2, const float* y_shared, const float* gate,
                                   int32_t T, int32_t H, int32_t I_s, void* d_h, void* d_ws2, float* d_gate_logit,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "moe_shared_fc2_backward";
  const bool gated = gate != nullptr;
  StageRange stage_range(stage_of(gated ? "moe_shared_fc2_backward:gated" : fn));
  MOE_CHECK(need_shared_sizes(dt, 2, wl, T, H, I_s, fn));
  MOE_CHECK(need_tensor(dy, fn, "dy"));
  MOE_CHECK(need_tensor(act, fn, "act"));
  MOE_CHECK(need_tensor(h_pre, fn, "h_pre"));
  MOE_CHECK(need_tensor(ws2, fn, "ws2"));
  MOE_CHECK(need_iff(y_shared, gated, fn, "y_shared", "gate"));
  if (gated) MOE_CHECK(need_tensor(gate, fn, "gate"));
  MOE_CHECK(need_tensor(d_h, fn, "d_h"));
  MOE_CHECK(need_tensor(d_ws2, fn, "d_ws2"));
  MOE_CHECK(need_iff(d_gate_logit, gated, fn, "d_gate_logit", "gate"));
  MOE_CHECK(need_workspace(workspace, workspace_bytes, moe_shared_train_workspace_bytes(dt, T, H, I_s), fn));
  const size_t e = dt == MOE_BF16 ? 2 : 4, t = (size_t)T, h = (size_t)H, i = (size_t)I_s;
  const Span spans[] = {
      {dy, 4 * t * h, "dy", false},
      {act, e * t * i, "act", false},
      {h_pre, e * t * 2 * i, "h_pre", false},
      {ws2, e * i * h, "ws2", false},
      {y_shared, 4 * t * h, "y_shared", false},
      {gate, 4 * t, "gate", false},
      {d_h, e * t * 2 * i, "d_h", true},
      {d_ws2, e * i * h, "d_ws2", true},
      {d_gate_logit, 4 * t, "d_gate_logit", true},
      {workspace, moe_shared_train_workspace_bytes(dt, T, H, I_s), "workspace", true}};
  MOE_CHECK(need_apart(spans, fn));
  return hip_result(moe_launch::shared_fc2_backward((int)dt, (int)wl, dy, act, h_pre, ws2, y_shared, gate, T, H, I_s,
                                                    d_h, d_ws2, d_gate_logit, workspace, cu_count(),
                                                    (hipStream_t)stream),
                    fn);
}

moe_status moe_shared_fc1_backward(moe_dtype dt, moe_weight_layout wl, const void* d_h, const void* x,
                                   const void* ws1, const float* d_gate_logit, const void* w_gate, int32_t T,
                                   int32_t H, int32_t I_s, int32_t accumulate, float* d_x, void* d_ws1,
                                   void* d_w_gate, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "moe_shared_fc1_backward";
  const bool gated = w_gate != nullptr;
  StageRange stage_range(stage_of(gated ? "moe_shared_fc1_backward:gated" : fn));
  MOE_CHECK(need_shared_sizes(dt, 3, wl, T, H, I_s, fn));
  MOE_CHECK(need_flag(accumulate, fn, "accumulate"));
  MOE_CHECK(need_tensor(d_h, fn, "d_h"));
  MOE_CHECK(need_tensor(x, fn, "x"));
  MOE_CHECK(need_tensor(ws1, fn, "ws1"));
  MOE_CHECK(need_iff(d_gate_logit, gated, fn, "d_gate_logit", "w_gate"));
  if (gated) MOE_CHECK(need_tensor(w_gate, fn, "w_gate"));
  MOE_CHECK(need_tensor(d_x, fn, "d_x"));
  MOE_CHECK(need_tensor(d_ws1, fn, "d_ws1"));
  MOE_CHECK(need_iff(d_w_gate, gated, fn, "d_w_gate", "w_gate"));
  MOE_CHECK(need_workspace(workspace, workspace_bytes, moe_shared_train_workspace_bytes(dt, T, H, I_s), fn));
  const size_t e = dt == MOE_BF16 ? 2 : 4, t = (size_t)T, h = (size_t)H, i = (size_t)I_s;
  const Span spans[] = {
      {d_h, e * t * 2 * i, "d_h", false},
      {x, e * t * h, "x", false},
      {ws1, e * h * 2 * i, "ws1", false},
      {d_gate_logit, 4 * t, "d_gate_logit", false},
      {w_gate, e * h, "w_gate", false},
      {d_x, 4 * t * h, "d_x", true},
      {d_ws1, e * h * 2 * i, "d_ws1", true},
      {d_w_gate, e * h, "d_w_gate", true},
      {workspace, moe_shared_train_workspace_bytes(dt, T, H, I_s), "workspace", true}};
  MOE_CHECK(need_apart(spans, fn));
  return hip_result(moe_launch::shared_fc1_backward((int)dt, (int)wl, d_h, x, ws1, d_gate_logit, w_gate, T, H, I_s,
                                                    accumulate, d_x, d_ws1, d_w_gate, workspace, cu_count(),
                                                    (hipStream_t)stream),
                    fn);
}

size_t moe_route_backward_workspace_bytes(moe_dtype dt, int32_t T, int32_t H, int32_t E, int32_t top_k) {
  if (T < 1 || H < 1 || H > kMaxWidth || E < 1 || E > moe::kMaxExperts || top_k < 1 || top_k > moe::kMaxTopK ||
      (dt != MOE_F32 && dt != MOE_BF16))
    return 0;
  return moe_launch::route_backward_workspace_bytes((int)dt, T, H, E, top_k, cu_count());
}

moe_status moe_route_backward(moe_dtype dt, const void* x, const void* w_router, const int32_t* topk_ids,
                              const float* topk_weights, const float* d_topk_weights, int32_t T, int32_t H, int32_t E,
                              int32_t top_k, int32_t accumulate, float* d_x, void* d_w_router, float* d_logit_bias,
                              void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "moe_route_backward";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_dtype(dt, fn));
  MOE_CHECK(need_pos(T, fn, "T"));
  MOE_CHECK(need_width(H, fn, "H"));
  MOE_CHECK(need_experts(E, fn));
  MOE_CHECK(need_topk(top_k, fn));
  MOE_CHECK(need_flag(accumulate, fn, "accumulate"));
  MOE_CHECK(need_rows((int64_t)T * top_k, fn, "T*top_k"));
  MOE_CHECK(need_launch(moe_launch::route_backward_blocks(T, H, E), fn));
  MOE_CHECK(need_tensor(x, fn, "x"));
  MOE_CHECK(need_tensor(w_router, fn, "w_router"));
  MOE_CHECK(need_ptr(topk_ids, fn, "topk_ids"));
  MOE_CHECK(need_align(topk_ids, 4, fn, "topk_ids"));
  MOE_CHECK(need_ptr(topk_weights, fn, "topk_weights"));
  MOE_CHECK(need_align(topk_weights, 4, fn, "topk_weights"));
  MOE_CHECK(need_ptr(d_topk_weights, fn, "d_topk_weights"));
  MOE_CHECK(need_align(d_topk_weights, 4, fn, "d_topk_weights"));
  MOE_CHECK(need_tensor(d_x, fn, "d_x"));
  MOE_CHECK(need_tensor(d_w_router, fn, "d_w_router"));
  MOE_CHECK(need_align(d_logit_bias, 4, fn, "d_logit_bias"));
  const size_t need = moe_route_backward_workspace_bytes(dt, T, H, E, top_k);
  MOE_CHECK(need_workspace(workspace, workspace_bytes, need, fn));
  const size_t e = dt == MOE_BF16 ? 2 : 4, t = (size_t)T, h = (size_t)H, pairs = t * (size_t)top_k;
  const Span spans[] = {{x, e * t * h, "x", false},
                        {w_router, e * h * E, "w_router", false},
                        {topk_ids, 4 * pairs, "topk_ids", false},
                        {topk_weights, 4 * pairs, "topk_weights", false},
                        {d_topk_weights, 4 * pairs, "d_topk_weights", false},
                        {d_x, 4 * t * h, "d_x", true},
                        {d_w_router, e * h * E, "d_w_router", true},
                        {d_logit_bias, 4 * (size_t)E, "d_logit_bias", true},
                        {workspace, need, "workspace", true}};
  MOE_CHECK(need_apart(spans, fn));
  return hip_result(moe_launch::route_backward((int)dt, x, w_router, topk_ids, topk_weights, d_topk_weights, T, H, E,
                                               top_k, accumulate, d_x, d_w_router, d_logit_bias, workspace, cu_count(),
                                               (hipStream_t)stream),
                    fn);
}

namespace {

moe_status need_grad_list(int32_t n, const void* const* grads, const int64_t* numel, const int32_t* dts,
                          const char* fn) {
  MOE_CHECK(need_pos(n, fn, "n"));
  MOE_CHECK(need_ptr(grads, fn, "grads"));
  MOE_CHECK(need_ptr(numel, fn, "numel"));
  MOE_CHECK(need_ptr(dts, fn, "dts"));
  int64_t left = (int64_t)1 << 43;
  for (int32_t i = 0; i < n; ++i) {
    if (dts[i] != MOE_F32 && dts[i] != MOE_BF16)
      return fail(MOE_ERR_INVALID_ARGUMENT, "%s: dts[%d] must be MOE_F32 or MOE_BF16 (got %d)", fn, (int)i,
                  (int)dts[i]);
    if (numel[i] < 0)
      return fail(MOE_ERR_INVALID_ARGUMENT, "%s: numel[%d] must be >= 0 (got %lld)", fn, (int)i, (long long)numel[i]);
    if (numel[i] >= left) return fail(MOE_ERR_UNSUPPORTED, "%s: the tensors must hold fewer than 2^43 elements", fn);
    left -= numel[i];
    if (numel[i] == 0) continue;
    if (!grads[i]) return fail(MOE_ERR_INVALID_ARGUMENT, "%s: grads[%d] must not be NULL", fn, (int)i);
    if ((uintptr_t)grads[i] % (dts[i] == MOE_BF16 ? 2 : 4))
      return fail(MOE_ERR_INVALID_ARGUMENT, "%s: grads[%d] must be aligned to its element type", fn, (int)i);
  }
  return MOE_OK;
}

// No output, coef among them, may overlap norm or another tensor of either list (a tensor's own
// input in place excepted): every workgroup reads norm, while others write.
moe_status need_disjoint_outs(int32_t n, const void* const* grads, void* const* outs, const int64_t* numel,
                              const int32_t* dts, const float* norm, const float* coef, const char* fn) {
  struct Range {
    uintptr_t lo, hi;
    int32_t i;   // n: norm, n + 1: coef
    bool out;
  };
  try {
    std::vector<Range> r;
    r.reserve(2 * (size_t)n + 2);
    r.push_back(Range{(uintptr_t)norm, (uintptr_t)norm + 4, n, false});
    if (coef) r.push_back(Range{(uintptr_t)coef, (uintptr_t)coef + 4, n + 1, true});
    for (int32_t i = 0; i < n; ++i) {
      if (numel[i] == 0) continue;
      const uintptr_t bytes = (uintptr_t)numel[i] * (dts[i] == MOE_BF16 ? 2 : 4);
      r.push_back(Range{(uintptr_t)outs[i], (uintptr_t)outs[i] + bytes, i, true});
      if (outs[i] != grads[i]) r.push_back(Range{(uintptr_t)grads[i], (uintptr_t)grads[i] + bytes, i, false});
    }
    std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
    uintptr_t out_end = 0, in_end = 0;  // furthest ends so far
    for (const Range& a : r) {
      if ((a.lo < out_end || (a.out && a.lo < in_end)) && a.i >= n)
        return fail(MOE_ERR_INVALID_ARGUMENT, "%s: %s overlaps another argument", fn, a.i == n ? "norm" : "coef");
      if (a.lo < out_end || (a.out && a.lo < in_end))
        return fail(MOE_ERR_INVALID_ARGUMENT, "%s: %s[%d] overlaps another argument (allowed: a tensor in place)", fn,
                    a.out ? "outs" : "grads", (int)a.i);
      uintptr_t& end = a.out ? out_end : in_end;
      end = std::max(end, a.hi);
    }
  } catch (const std::bad_alloc&) {
    return fail(MOE_ERR_UNSUPPORTED, "%s: no host memory to check %d tensors", fn, (int)n);
  }
  return MOE_OK;
}

}  // namespace

size_t moe_grad_norm_workspace_bytes(int32_t n) { return n < 1 ? 0 : moe_launch::grad_norm_workspace_bytes(n); }

moe_status moe_grad_norm(int32_t n, const void* const* grads, const int64_t* numel, const int32_t* dts, float* norm,
                         double* sum_sq, void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "moe_grad_norm";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_grad_list(n, grads, numel, dts, fn));
  MOE_CHECK(need_ptr(norm, fn, "norm"));
  MOE_CHECK(need_align(norm, 4, fn, "norm"));
  MOE_CHECK(need_align(sum_sq, 8, fn, "sum_sq"));
  const size_t need = moe_grad_norm_workspace_bytes(n);
  if (!workspace || workspace_bytes < need)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace needs %zu bytes (got %zu%s)", fn, need, workspace_bytes,
                workspace ? "" : ", NULL pointer");
  MOE_CHECK(need_align(workspace, 8, fn, "workspace"));
  const Span outs[] = {{norm, 4, "norm", true}, {sum_sq, 8, "sum_sq", true}, {workspace, need, "workspace", true}};
  MOE_CHECK(need_apart(outs, fn));
  for (int32_t i = 0; i < n; ++i) {
    if (numel[i] == 0) continue;
    const uintptr_t lo = (uintptr_t)grads[i], hi = lo + (uintptr_t)numel[i] * (dts[i] == MOE_BF16 ? 2 : 4);
    for (const Span& o : outs)
      if (o.p && (uintptr_t)o.p < hi && lo < (uintptr_t)o.p + o.bytes)
        return fail(MOE_ERR_INVALID_ARGUMENT, "%s: %s overlaps grads[%d]", fn, o.name, (int)i);
  }
  return hip_result(moe_launch::grad_norm(n, grads, numel, dts, norm, sum_sq, workspace, (hipStream_t)stream), fn);
}

moe_status moe_grad_clip(int32_t n, const void* const* grads, void* const* outs, const int64_t* numel,
                         const int32_t* dts, const float* norm, float max_norm, float* coef, void* stream) {
  const char* fn = "moe_grad_clip";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_grad_list(n, grads, numel, dts, fn));
  MOE_CHECK(need_ptr(outs, fn, "outs"));
  for (int32_t i = 0; i < n; ++i) {
    if (numel[i] == 0) continue;
    if (!outs[i]) return fail(MOE_ERR_INVALID_ARGUMENT, "%s: outs[%d] must not be NULL", fn, (int)i);
    if ((uintptr_t)outs[i] % (dts[i] == MOE_BF16 ? 2 : 4))
      return fail(MOE_ERR_INVALID_ARGUMENT, "%s: outs[%d] must be aligned to its element type", fn, (int)i);
  }
  MOE_CHECK(need_ptr(norm, fn, "norm"));
  MOE_CHECK(need_align(norm, 4, fn, "norm"));
  MOE_CHECK(need_align(coef, 4, fn, "coef"));
  MOE_CHECK(need_disjoint_outs(n, grads, outs, numel, dts, norm, coef, fn));
  if (!isfinite(max_norm) || max_norm < 0.f)
    return fail(MOE_ERR_INVALID_ARGUMENT, "%s: max_norm must be finite and >= 0 (got %g)", fn, (double)max_norm);
  return hip_result(moe_launch::grad_clip(n, grads, outs, numel, dts, norm, max_norm, coef, (hipStream_t)stream), fn);
}

// ------------------------------------------------------------------------------------------
// Around the layer: auxiliary losses of the router, norms and residual, orthogonalised update
// ------------------------------------------------------------------------------------------
namespace {

moe_status need_finite(float v, const char* fn, const char* name) {
  return isfinite(v) ? MOE_OK
                     : fail(MOE_ERR_INVALID_ARGUMENT, "%s: %s must be finite (got %g)", fn, name, (double)v);
}

// A required device array aligned to its 4-byte elements.
moe_status need_words(const void* p, const char* fn, const char* name) {
  MOE_CHECK(need_ptr(p, fn, name));
  return need_align(p, 4, fn, name);
}

// An array that must be NULL unless `allowed`.
moe_status need_absent(const void* p, bool allowed, const char* fn, const char* name, const char* when) {
  return p && !allowed ? fail(MOE_ERR_INVALID_ARGUMENT, "%s: %s must be NULL without %s", fn, name, when) : MOE_OK;
}

}  // namespace

size_t moe_balance_loss_workspace_bytes(int32_t T, int32_t E) {
  if (T < 1 || E < 1 || E > moe::kMaxExperts) return 0;
  return moe_launch::balance_loss_workspace_bytes(T, E);
}

moe_status moe_balance_loss(const float* logits, const int32_t* topk_ids, const uint8_t* token_mask, int32_t T,
                            int32_t E, int32_t top_k, float balance_coef, float z_coef, float* losses,
                            int32_t* counts, int32_t* tokens, float* prob_sums, float* lse, void* workspace,
                            size_t workspace_bytes, void* stream) {
  const char* fn = "moe_balance_loss";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_pos(T, fn, "T"));
  MOE_CHECK(need_experts(E, fn));
  MOE_CHECK(need_topk(top_k, fn));
  MOE_CHECK(need_rows((int64_t)T * top_k, fn, "T*top_k"));
  MOE_CHECK(need_finite(balance_coef, fn, "balance_coef"));
  MOE_CHECK(need_finite(z_coef, fn, "z_coef"));
  MOE_CHECK(need_words(logits, fn, "logits"));
  MOE_CHECK(need_words(topk_ids, fn, "topk_ids"));
  MOE_CHECK(need_words(losses, fn, "losses"));
  MOE_CHECK(need_words(counts, fn, "counts"));
  MOE_CHECK(need_words(tokens, fn, "tokens"));
  MOE_CHECK(need_words(prob_sums, fn, "prob_sums"));
  MOE_CHECK(need_words(lse, fn, "lse"));
  const size_t need = moe_balance_loss_workspace_bytes(T, E), t = (size_t)T, e = (size_t)E;
  MOE_CHECK(need_workspace(workspace, workspace_bytes, need, fn));
  const Span spans[] = {{logits, 4 * t * e, "logits", false},
                        {topk_ids, 4 * t * top_k, "topk_ids", false},
                        {token_mask, t, "token_mask", false},
                        {losses, 8, "losses", true},
                        {counts, 4 * e, "counts", true},
                        {tokens, 4, "tokens", true},
                        {prob_sums, 4 * e, "prob_sums", true},
                        {lse, 4 * t, "lse", true},
                        {workspace, need, "workspace", true}};
  MOE_CHECK(need_apart(spans, fn));
  return hip_result(moe_launch::balance_loss(logits, topk_ids, token_mask, T, E, top_k, balance_coef, z_coef, losses,
                                             counts, tokens, prob_sums, lse, workspace, (hipStream_t)stream),
                    fn);
}

size_t moe_route_balance_backward_workspace_bytes(moe_dtype dt, int32_t T, int32_t H, int32_t E) {
  if (T < 1 || H < 1 || H > kMaxWidth || E < 1 || E > moe::kMaxExperts || (dt != MOE_F32 && dt != MOE_BF16)) return 0;
  return moe_launch::route_balance_backward_workspace_bytes((int)dt, T, H, E, cu_count());
}

moe_status moe_route_balance_backward(moe_dtype dt, const void* x, const void* w_router, const float* logits,
                                      const float* lse, const int32_t* topk_ids, const float* topk_weights,
                                      const float* d_topk_weights, const uint8_t* token_mask, const int32_t* counts,
                                      const int32_t* tokens, int32_t T, int32_t H, int32_t E, int32_t top_k,
                                      float balance_coef, float z_coef, int32_t accumulate, float* d_x,
                                      void* d_w_router, float* d_logit_bias, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  const char* fn = "moe_route_balance_backward";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_dtype(dt, fn));
  MOE_CHECK(need_pos(T, fn, "T"));
  MOE_CHECK(need_width(H, fn, "H"));
  MOE_CHECK(need_experts(E, fn));
  MOE_CHECK(need_topk(top_k, fn));
  MOE_CHECK(need_flag(accumulate, fn, "accumulate"));
  MOE_CHECK(need_finite(balance_coef, fn, "balance_coef"));
  MOE_CHECK(need_finite(z_coef, fn, "z_coef"));
  MOE_CHECK(need_rows((int64_t)T * top_k, fn, "T*top_k"));
  MOE_CHECK(need_launch(moe_launch::route_balance_backward_blocks((int)dt, T, H, E), fn));
  MOE_CHECK(need_tensor(x, fn, "x"));
  MOE_CHECK(need_tensor(w_router, fn, "w_router"));
  MOE_CHECK(need_words(logits, fn, "logits"));
  MOE_CHECK(need_words(lse, fn, "lse"));
  if (!topk_weights != !d_topk_weights)
    return fail(MOE_ERR_INVALID_ARGUMENT, "%s: topk_weights and d_topk_weights must both be given or both be NULL", fn);
  if (d_topk_weights) {
    MOE_CHECK(need_words(topk_ids, fn, "topk_ids"));
    MOE_CHECK(need_align(topk_weights, 4, fn, "topk_weights"));
    MOE_CHECK(need_align(d_topk_weights, 4, fn, "d_topk_weights"));
  }
  MOE_CHECK(need_words(counts, fn, "counts"));
  MOE_CHECK(need_words(tokens, fn, "tokens"));
  MOE_CHECK(need_tensor(d_x, fn, "d_x"));
  MOE_CHECK(need_tensor(d_w_router, fn, "d_w_router"));
  MOE_CHECK(need_align(d_logit_bias, 4, fn, "d_logit_bias"));
  const size_t need = moe_route_balance_backward_workspace_bytes(dt, T, H, E);
  MOE_CHECK(need_workspace(workspace, workspace_bytes, need, fn));
  const size_t b = dt == MOE_BF16 ? 2 : 4, t = (size_t)T, h = (size_t)H, e = (size_t)E, pairs = t * (size_t)top_k;
  const Span spans[] = {{x, b * t * h, "x", false},
                        {w_router, b * h * e, "w_router", false},
                        {logits, 4 * t * e, "logits", false},
                        {lse, 4 * t, "lse", false},
                        {d_topk_weights ? topk_ids : nullptr, 4 * pairs, "topk_ids", false},
                        {topk_weights, 4 * pairs, "topk_weights", false},
                        {d_topk_weights, 4 * pairs, "d_topk_weights", false},
                        {token_mask, t, "token_mask", false},
                        {counts, 4 * e, "counts", false},
                        {tokens, 4, "tokens", false},
                        {d_x, 4 * t * h, "d_x", true},
                        {d_w_router, b * h * e, "d_w_router", true},
                        {d_logit_bias, 4 * e, "d_logit_bias", true},
                        {workspace, need, "workspace", true}};
  MOE_CHECK(need_apart(spans, fn));
  return hip_result(moe_launch::route_balance_backward((int)dt, x, w_router, logits, lse, topk_ids, topk_weights,
                                                       d_topk_weights, token_mask, counts, tokens, T, H, E, top_k,
                                                       balance_coef, z_coef, accumulate, d_x, d_w_router, d_logit_bias,
                                                       workspace, cu_count(), (hipStream_t)stream),
                    fn);
}

namespace {

moe_status need_norm_sizes(moe_dtype dt, moe_dtype stream_dt, int32_t T, int32_t H, const char* fn) {
  MOE_CHECK(need_dtype(dt, fn));
  if (stream_dt != MOE_F32 && stream_dt != MOE_BF16)
    return fail(MOE_ERR_INVALID_ARGUMENT, "%s: stream_dt must be MOE_F32 or MOE_BF16 (got %d)", fn, (int)stream_dt);
  MOE_CHECK(need_pos(T, fn, "T"));
  MOE_CHECK(need_rows(T, fn, "T"));
  MOE_CHECK(need_pos(H, fn, "H"));
  MOE_CHECK(need_mult8(H, fn, "H"));
  const int most = moe_launch::norm_max_width();
  return H <= most ? MOE_OK : fail(MOE_ERR_UNSUPPORTED, "%s: H must be <= %d (got %d)", fn, most, (int)H);
}

}  // namespace

moe_status moe_norm_residual(moe_dtype dt, moe_dtype stream_dt, const void* h, const float* y, const void* w_post,
                             const void* gate, const void* w_pre, int32_t T, int32_t H, float eps,
                             float weight_offset, float residual_scale, float branch_scale, void* h_out, void* x,
                             float* rstd_post, float* rstd_pre, void* stream) {
  const char* fn = "moe_norm_residual";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_norm_sizes(dt, stream_dt, T, H, fn));
  MOE_CHECK(need_finite(eps, fn, "eps"));
  if (eps < 0.f) return fail(MOE_ERR_INVALID_ARGUMENT, "%s: eps must be >= 0 (got %g)", fn, (double)eps);
  MOE_CHECK(need_finite(weight_offset, fn, "weight_offset"));
  MOE_CHECK(need_finite(residual_scale, fn, "residual_scale"));
  MOE_CHECK(need_finite(branch_scale, fn, "branch_scale"));
  if (!y && !w_pre) return fail(MOE_ERR_INVALID_ARGUMENT, "%s: y and w_pre must not both be NULL", fn);
  MOE_CHECK(need_tensor(h, fn, "h"));
  MOE_CHECK(need_align(y, 16, fn, "y"));
  MOE_CHECK(need_absent(w_post, y, fn, "w_post", "y"));
  MOE_CHECK(need_align(w_post, 16, fn, "w_post"));
  MOE_CHECK(need_absent(gate, y, fn, "gate", "y"));
  MOE_CHECK(need_align(gate, 16, fn, "gate"));
  MOE_CHECK(need_align(w_pre, 16, fn, "w_pre"));
  MOE_CHECK(need_iff(h_out, y != nullptr, fn, "h_out", "y"));
  MOE_CHECK(need_iff(x, w_pre != nullptr, fn, "x", "w_pre"));
  MOE_CHECK(need_absent(rstd_post, w_post, fn, "rstd_post", "w_post"));
  MOE_CHECK(need_align(rstd_post, 4, fn, "rstd_post"));
  MOE_CHECK(need_absent(rstd_pre, w_pre, fn, "rstd_pre", "w_pre"));
  MOE_CHECK(need_align(rstd_pre, 4, fn, "rstd_pre"));
  const size_t e = dt == MOE_BF16 ? 2 : 4, r = stream_dt == MOE_BF16 ? 2 : 4, t = (size_t)T, w = (size_t)H;
  const Span spans[] = {{h_out == h ? nullptr : h, r * t * w, "h", false},
                        {y, 4 * t * w, "y", false},
                        {w_post, e * w, "w_post", false},
                        {gate, e * w, "gate", false},
                        {w_pre, e * w, "w_pre", false},
                        {h_out, r * t * w, "h_out", true},
                        {x, e * t * w, "x", true},
                        {rstd_post, 4 * t, "rstd_post", true},
                        {rstd_pre, 4 * t, "rstd_pre", true}};
  MOE_CHECK(need_apart(spans, fn));
  return hip_result(moe_launch::norm_residual((int)dt, (int)stream_dt, h, y, w_post, gate, w_pre, T, H, eps,
                                              weight_offset, residual_scale, branch_scale, h_out, x, rstd_post,
                                              rstd_pre, (hipStream_t)stream),
                    fn);
}

size_t moe_norm_residual_backward_workspace_bytes(int32_t T, int32_t H) {
  if (T < 1 || H < 1 || H > moe_launch::norm_max_width()) return 0;
  return moe_launch::norm_residual_backward_workspace_bytes(T, H);
}

moe_status moe_norm_residual_backward(moe_dtype dt, moe_dtype stream_dt, const void* d_h_out, const float* d_x,
                                      const void* h_out, const float* rstd_pre, const void* w_pre, const float* y,
                                      const float* rstd_post, const void* w_post, const void* gate, int32_t T,
                                      int32_t H, float weight_offset, float residual_scale, float branch_scale,
                                      void* d_h, float* d_y, void* d_w_pre, void* d_w_post, void* d_gate,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "moe_norm_residual_backward";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_norm_sizes(dt, stream_dt, T, H, fn));
  MOE_CHECK(need_finite(weight_offset, fn, "weight_offset"));
  MOE_CHECK(need_finite(residual_scale, fn, "residual_scale"));
  MOE_CHECK(need_finite(branch_scale, fn, "branch_scale"));
  const bool pre = d_x != nullptr, branch = d_y != nullptr;
  if (!d_h_out && !pre) return fail(MOE_ERR_INVALID_ARGUMENT, "%s: d_h_out and d_x must not both be NULL", fn);
  MOE_CHECK(need_align(d_h_out, 16, fn, "d_h_out"));
  MOE_CHECK(need_align(d_x, 16, fn, "d_x"));
  if (pre) MOE_CHECK(need_tensor(h_out, fn, "h_out"));
  if (!pre) h_out = nullptr;   // not read
  if (pre) MOE_CHECK(need_words(rstd_pre, fn, "rstd_pre"));
  MOE_CHECK(need_absent(rstd_pre, pre, fn, "rstd_pre", "d_x"));
  MOE_CHECK(need_iff(w_pre, pre, fn, "w_pre", "d_x"));
  MOE_CHECK(need_absent(w_post, branch, fn, "w_post", "d_y"));
  MOE_CHECK(need_align(w_post, 16, fn, "w_post"));
  if (w_post) MOE_CHECK(need_words(rstd_post, fn, "rstd_post"));
  MOE_CHECK(need_absent(rstd_post, w_post, fn, "rstd_post", "w_post"));
  MOE_CHECK(need_absent(gate, branch, fn, "gate", "d_y"));
  MOE_CHECK(need_align(gate, 16, fn, "gate"));
  if (w_post || gate) MOE_CHECK(need_ptr(y, fn, "y (needed for w_post or gate)"));
  MOE_CHECK(need_absent(y, branch, fn, "y", "d_y"));
  MOE_CHECK(need_align(y, 16, fn, "y"));
  MOE_CHECK(need_tensor(d_h, fn, "d_h"));
  MOE_CHECK(need_align(d_y, 16, fn, "d_y"));
  MOE_CHECK(need_iff(d_w_pre, pre, fn, "d_w_pre", "w_pre"));
  MOE_CHECK(need_iff(d_w_post, w_post != nullptr, fn, "d_w_post", "w_post"));
  MOE_CHECK(need_iff(d_gate, gate != nullptr, fn, "d_gate", "gate"));
  const size_t need = moe_norm_residual_backward_workspace_bytes(T, H);
  MOE_CHECK(need_workspace(workspace, workspace_bytes, need, fn));
  if (!w_post && !gate) y = nullptr;   // not read
  const size_t e = dt == MOE_BF16 ? 2 : 4, r = stream_dt == MOE_BF16 ? 2 : 4, t = (size_t)T, w = (size_t)H;
  const Span spans[] = {{d_h == d_h_out ? nullptr : d_h_out, r * t * w, "d_h_out", false},
                        {d_x, 4 * t * w, "d_x", false},
                        {h_out, r * t * w, "h_out", false},
                        {rstd_pre, 4 * t, "rstd_pre", false},
                        {w_pre, e * w, "w_pre", false},
                        {y, 4 * t * w, "y", false},
                        {rstd_post, 4 * t, "rstd_post", false},
                        {w_post, e * w, "w_post", false},
                        {gate, e * w, "gate", false},
                        {d_h, r * t * w, "d_h", true},
                        {d_y, 4 * t * w, "d_y", true},
                        {d_w_pre, e * w, "d_w_pre", true},
                        {d_w_post, e * w, "d_w_post", true},
                        {d_gate, e * w, "d_gate", true},
                        {workspace, need, "workspace", true}};
  MOE_CHECK(need_apart(spans, fn));
  if (!branch) residual_scale = 1.0f;
  return hip_result(moe_launch::norm_residual_backward((int)dt, (int)stream_dt, d_h_out, d_x, h_out, rstd_pre, w_pre,
                                                       y, rstd_post, w_post, gate, T, H, weight_offset,
                                                       residual_scale, branch_scale, d_h, d_y, d_w_pre, d_w_post,
                                                       d_gate, workspace, (hipStream_t)stream),
                    fn);
}

namespace {

constexpr int32_t kMaxOrthoSide = 32768, kMaxOrthoMatrices = 65535;

moe_status need_ortho_sizes(moe_dtype dt, moe_dtype out_dt, int32_t batch, int32_t M, int32_t N, int32_t parts,
                            const char* fn) {
  MOE_CHECK(need_dtype(dt, fn));
  if (out_dt != MOE_F32 && out_dt != MOE_BF16)
    return fail(MOE_ERR_INVALID_ARGUMENT, "%s: out_dt must be MOE_F32 or MOE_BF16 (got %d)", fn, (int)out_dt);
  MOE_CHECK(need_pos(batch, fn, "batch"));
  MOE_CHECK(need_pos(M, fn, "M"));
  MOE_CHECK(need_pos(N, fn, "N"));
  MOE_CHECK(need_pos(parts, fn, "parts"));
  if (M > kMaxOrthoSide || N > kMaxOrthoSide)
    return fail(MOE_ERR_UNSUPPORTED, "%s: M and N must be <= %d (got %d and %d)", fn, (int)kMaxOrthoSide, (int)M,
                (int)N);
  if ((int64_t)batch * parts > kMaxOrthoMatrices)
    return fail(MOE_ERR_UNSUPPORTED, "%s: batch * parts must be <= %d (got %lld)", fn, (int)kMaxOrthoMatrices,
                (long long)batch * parts);
  return MOE_OK;
}

}  // namespace

size_t moe_orthogonal_update_workspace_bytes(moe_dtype dt, moe_dtype out_dt, int32_t batch, int32_t M, int32_t N,
                                             int32_t parts, int32_t has_momentum) {
  if (need_ortho_sizes(dt, out_dt, batch, M, N, parts, "moe_orthogonal_update_workspace_bytes") != MOE_OK) return 0;
  return moe_launch::orthogonal_update_workspace_bytes((int)dt, (int)out_dt, batch, M, N, parts, has_momentum != 0,
                                                       cu_count());
}

moe_status moe_orthogonal_update(moe_dtype dt, moe_dtype out_dt, const void* grad, float* momentum, float mu,
                                 int32_t nesterov, int32_t batch, int32_t M, int32_t N, int32_t parts, int32_t steps,
                                 const float* coefs, float eps, float scale, float keep, void* out, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  const char* fn = "moe_orthogonal_update";
  StageRange stage_range(stage_of(fn));
  MOE_CHECK(need_ortho_sizes(dt, out_dt, batch, M, N, parts, fn));
  MOE_CHECK(need_flag(nesterov, fn, "nesterov"));
  MOE_CHECK(need_pos(steps, fn, "steps"));
  if (steps > moe::kOrthoMaxSteps)
    return fail(MOE_ERR_UNSUPPORTED, "%s: steps must be <= %d (got %d)", fn, moe::kOrthoMaxSteps, (int)steps);
  MOE_CHECK(need_ptr(coefs, fn, "coefs"));
  for (int32_t i = 0; i < 3 * steps; ++i) MOE_CHECK(need_finite(coefs[i], fn, "coefs"));
  MOE_CHECK(need_finite(mu, fn, "mu"));
  MOE_CHECK(need_finite(scale, fn, "scale"));
  MOE_CHECK(need_finite(keep, fn, "keep"));
  if (!(eps >= 1e-12f) || !isfinite(eps))
    return fail(MOE_ERR_INVALID_ARGUMENT, "%s: eps must be finite and at least 1e-12 (got %g)", fn, (double)eps);
  double sigma[moe::kOrthoMaxSteps + 1], beta[moe::kOrthoMaxSteps];
  if (!moe_launch::orthogonal_bounds(steps, coefs, sigma, beta))
    return fail(MOE_ERR_UNSUPPORTED, "%s: with these coefs singular values grow beyond 64", fn);
  const size_t e = dt == MOE_BF16 ? 2 : 4, o = out_dt == MOE_BF16 ? 2 : 4;
  const size_t n = (size_t)batch * M * N * parts;
  MOE_CHECK(need_ptr(grad, fn, "grad"));
  MOE_CHECK(need_align(grad, e, fn, "grad"));
  MOE_CHECK(need_align(momentum, 4, fn, "momentum"));
  MOE_CHECK(need_ptr(out, fn, "out"));
  MOE_CHECK(need_align(out, o, fn, "out"));
  const size_t need = moe_orthogonal_update_workspace_bytes(dt, out_dt, batch, M, N, parts, momentum != nullptr);
  MOE_CHECK(need_workspace(workspace, workspace_bytes, need, fn));
  const Span spans[] = {{grad, e * n, "grad", false},
                        {momentum, 4 * n, "momentum", true},
                        {out, o * n, "out", true},
                        {workspace, need, "workspace", true}};
  MOE_CHECK(need_apart(spans, fn));
  return hip_result(moe_launch::orthogonal_update((int)dt, (int)out_dt, grad, momentum, mu, nesterov, batch, M, N,
                                                  parts, steps, coefs, eps, scale, keep, out, workspace, cu_count(),
                                                  (hipStream_t)stream),
                    fn);
}

}  // extern "C"
