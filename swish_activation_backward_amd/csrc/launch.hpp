// Internal launchers (C++ linkage) called by the C ABI layer after validation.
#pragma once

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "plan.hpp"

namespace swg {

// Kernel-duration timing of one entry-point call (swg_time_next_call): caller-created HIP
// events, per host thread, cleared when the timed call returns.
struct CallTiming {
  hipEvent_t start = nullptr;
  hipEvent_t stop = nullptr;
};
CallTiming& call_timing();

// Every kernel of the library is dispatched through this.  While a call is timed, the
// dispatch carries the call's events (hipExtLaunchKernelGGL): the first dispatch records
// `start` when it begins and every dispatch records `stop` when it ends, so the pair spans
// the call's kernels from the first one's start to the last one's end.
#define SWG_LAUNCH(KERNEL, GRID, BLOCK, SHMEM, STREAM, ...)                                 \
  do {                                                                                    \
    ::swg::CallTiming& t_ = ::swg::call_timing();                                         \
    if (t_.stop == nullptr) {                                                             \
      hipLaunchKernelGGL(KERNEL, GRID, BLOCK, SHMEM, STREAM, __VA_ARGS__);                 \
    } else {                                                                              \
      hipExtLaunchKernelGGL(KERNEL, GRID, BLOCK, SHMEM, STREAM, t_.start, t_.stop, 0,       \
                            __VA_ARGS__);                                                 \
      t_.start = nullptr;                                                                 \
    }                                                                                     \
  } while (0)

constexpr int64_t kMaxStreamBlocks = 8192;

hipError_t launch_swish_grad(int dtype, const void* grad, const void* x, void* out, int64_t n,
                             float beta, bool vector_path, hipStream_t stream);

// Strided views for swish_grad: a logical shape in row-major order (after merging the
// dimensions that are contiguous in all three tensors) and each tensor's element strides.
constexpr int kMaxStridedDims = 8;
struct StridedView {
  int nd;
  int64_t size[kMaxStridedDims];
  int64_t stride[3][kMaxStridedDims];   // grad, x, grad_x
};

// grad_x[i] for every logical index i of the view (n = product of the sizes > 0)
hipError_t launch_swish_grad_strided(int dtype, const void* grad, const void* x, void* out,
                                     const StridedView& v, int64_t n, float beta,
                                     hipStream_t stream);

// The device address of the b stage's static scratch array on the current device
// (kBScratchBytes; resolved on the first call per device, no allocation).
hipError_t b_scratch(float** out);

hipError_t launch_b_stage(int dtype, const BPlan& p, const void* dy, const void* g,
                          const void* fc, void* dg, void* dfc, void* db_g, void* db_fc,
                          int64_t M, int64_t N, float* part, hipStream_t stream);

// `cus`: compute units of the device: the GEMM stages launch one persistent workgroup
// per CU (fewer when there is less work).
hipError_t launch_w_stage(int dtype, const WPlan& p, const void* x, const void* dg,
                          const void* dfc, void* dw_g, void* dw_fc, int64_t M, int64_t K,
                          int64_t N, float* ws, int cus, hipStream_t stream);

// fused w + x pass (bf16 / fp16): dx and [dw_g | dw_fc] += x^T [dg | dfc] in one launch
hipError_t launch_wx(int dtype, const WXPlan& p, const void* x, const void* dg, const void* dfc,
                     const void* w_g, const void* w_fc, void* dw_g, void* dw_fc, void* dx,
                     int64_t M, int64_t K, int64_t N, float* ws, hipStream_t stream);

// force_f: tile configuration override (4 or 2; 0 = the planner's choice)
hipError_t launch_x_stage(int dtype, const void* dg, const void* dfc, const void* w_g,
                          const void* w_fc, void* dx, int64_t M, int64_t K, int64_t N,
                          int force_f, int cus, hipStream_t stream);

// fp32 tensors (dtype 2) of the GEMMs; called by launch_x_stage / launch_w_stage / launch_fwd
hipError_t launch_x_stage32(const void* dg, const void* dfc, const void* w_g, const void* w_fc,
                            void* dx, int64_t M, int64_t K, int64_t N, hipStream_t stream);
hipError_t launch_w_stage32(const WPlan& p, const void* x, const void* dg, const void* dfc,
                            void* dw_g, void* dw_fc, int64_t M, int64_t K, int64_t N, float* ws,
                            hipStream_t stream);
hipError_t launch_fwd32(const void* x, const void* w_g, const void* w_fc, const void* b_g,
                        const void* b_fc, void* g, void* fc, void* y, int64_t M, int64_t K,
                        int64_t N, hipStream_t stream);

// SwiGLU forward: g, fc, y [M, N] from x [M, K], W_g, W_fc [K, N], b_g, b_fc [N] (may be
// null); one persistent workgroup per CU.
hipError_t launch_fwd(int dtype, const void* x, const void* w_g, const void* w_fc,
                      const void* b_g, const void* b_fc, void* g, void* fc, void* y, int64_t M,
                      int64_t K, int64_t N, int cus, hipStream_t stream);

hipError_t launch_zero(void* p, size_t bytes, hipStream_t stream);

// Layer norm.  Row strides in elements; w, b, y, mean, rstd (forward) and dx, dw, db
// (backward) may be null.
struct NormArgs {
  const void* x;
  int64_t ldx;
  const void* w;
  const void* b;
  void* y;
  int64_t ldy;
  float* mean;
  float* rstd;
  const void* dy;
  int64_t lddy;
  void* dx;
  int64_t lddx;
  void* dw;
  void* db;
  int accumulate;
  int64_t M, N;
  float eps;
};
hipError_t launch_norm_fwd(int dtype, int wdtype, const NormArgs& a, hipStream_t stream);
hipError_t launch_norm_bwd(int dtype, int wdtype, const NormArgs& a, const NormPlan& p,
                           float* part, hipStream_t stream);

// Rows of logits [R, V] (row stride ld) with what the forward and backward of the token log
// probabilities and of the distillation loss read and write; pointers that a call does not
// use are null.
struct VocabArgs {
  const void* z;
  int64_t ld;
  void* dz;
  int64_t lddz;
  int64_t R, V;
  float inv_t;              // 1 / temperature
  float t;
  // token log probabilities
  const int64_t* target;
  int64_t ignore;
  float* logprob;
  float* entropy;
  float* lse;
  float* top_logprob;
  int64_t* top_id;
  int64_t top;
  const float* lse_in;
  const float* entropy_in;
  const float* dlogprob;
  const float* dentropy;
  // distillation: the teacher's entries [R, k]
  const void* teacher;
  int teacher_dtype;
  const int64_t* ids;
  int64_t k;
  float* loss;
  const float* dloss;
  float* stat;              // [R, 2]: m and ln sum exp(a - m), between the two kernels of a call
};
hipError_t launch_logprobs(int dtype, const VocabArgs& a, const VocabPlan& p, void* ws,
                           hipStream_t stream);
hipError_t launch_logprobs_bwd(int dtype, const VocabArgs& a, hipStream_t stream);
hipError_t launch_distill_fwd(int dtype, const VocabArgs& a, const VocabPlan& p, void* ws,
                              hipStream_t stream);
hipError_t launch_distill_bwd(int dtype, const VocabArgs& a, hipStream_t stream);
hipError_t launch_distill_fwd_bwd(int dtype, const VocabArgs& a, const VocabPlan& p, void* ws,
                                  hipStream_t stream);

}  // namespace swg
