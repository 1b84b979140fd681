// C ABI of the block norm: argument validation, thread mapping, launches.  The
// contract is in include/dcn_core.h.
#define DCN_ERROR_WORD_BY_POINTER
#include "dcn_core.h"

#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdlib>

#include "dcn_block_norm.cuh"
#include "dcn_host.h"

namespace dcn {
namespace {

dcn_status launched() { return cudaGetLastError() == cudaSuccess ? DCN_OK : DCN_ERR_CUDA; }

bool valid_norm(dcn_norm n) {
  return n == DCN_NORM_NONE || n == DCN_NORM_LAYER || n == DCN_NORM_RMS;
}
bool valid_eps(dcn_norm n, float eps) {
  return n == DCN_NORM_NONE || (std::isfinite(eps) && eps >= 0.f);
}
bool valid_dtype(dcn_dtype d) { return d == DCN_F32 || d == DCN_BF16 || d == DCN_F16; }

dcn_status check_norm(const dcn_block_norm* p) {
  if (!p || p->M < 1 || p->C < 1 || p->rows_per_gate < 0) return DCN_ERR_INVALID_ARG;
  if (!valid_dtype(p->stream_dtype) || !valid_dtype(p->branch_dtype)) return DCN_ERR_INVALID_ARG;
  if (!valid_norm(p->post_norm) || !valid_norm(p->pre_norm)) return DCN_ERR_INVALID_ARG;
  if (!valid_eps(p->post_norm, p->post_eps) || !valid_eps(p->pre_norm, p->pre_eps))
    return DCN_ERR_INVALID_ARG;
  if (!std::isfinite(p->residual_scale)) return DCN_ERR_INVALID_ARG;
  if (p->C > kNormMaxC) return DCN_ERR_UNSUPPORTED;
  if (p->stream_dtype != p->branch_dtype && p->stream_dtype != DCN_F32) return DCN_ERR_UNSUPPORTED;
  return DCN_OK;
}

// Calls f(stream value, branch value) with the storage types of the norm.
template <typename F>
auto with_types(const dcn_block_norm* p, F&& f) {
  if (p->stream_dtype == p->branch_dtype)
    return with_storage(p->stream_dtype, [&](auto tag) { return f(tag, tag); });
  if (p->branch_dtype == DCN_BF16) return f(float(), __nv_bfloat16());
  return f(float(), __half());
}

// Calls f(threads a row, vector loads) as constants: the fewest threads that hold
// `groups` groups of four channels, five each.  Rows that do not start on a vector
// boundary take single loads and, to save code, one of three mappings.
template <int N>
struct Int {
  static constexpr int value = N;
};
template <typename F>
auto with_mapping(int64_t groups, bool vec, F&& f) {
  const int64_t tpr = (groups + kNormGroups - 1) / kNormGroups;
  if (!vec) {
    if (tpr <= 32) return f(Int<32>(), Int<0>());
    return tpr <= 64 ? f(Int<64>(), Int<0>()) : f(Int<256>(), Int<0>());
  }
  if (tpr <= 8) return f(Int<8>(), Int<1>());
  if (tpr <= 16) return f(Int<16>(), Int<1>());
  if (tpr <= 32) return f(Int<32>(), Int<1>());
  if (tpr <= 64) return f(Int<64>(), Int<1>());
  if (tpr <= 128) return f(Int<128>(), Int<1>());
  return f(Int<256>(), Int<1>());
}

template <typename Kernel>
dcn_status launch_backward(Kernel k, size_t smem, const NormBwdArgs& a, int ctas,
                           cudaStream_t stream) {
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) !=
      cudaSuccess)
    return DCN_ERR_CUDA;
  k<<<unsigned(ctas), kNormThreads, smem, stream>>>(a);
  return launched();
}

int64_t gates_of(const dcn_block_norm* p, bool gate) {
  return gate && p->rows_per_gate > 0
             ? (int64_t(p->M) + p->rows_per_gate - 1) / p->rows_per_gate
             : 1;
}

// Vector accesses in the backward: rows of both types start on 16-byte boundaries.
bool vector_rows(const dcn_block_norm* p) {
  return (int64_t(p->C) * esize(p->stream_dtype)) % 16 == 0 &&
         (int64_t(p->C) * esize(p->branch_dtype)) % 16 == 0;
}

// The backward's split of the rows and its partial sums.
struct NormSplit {
  int rows_per_cta, ctas;
  size_t s_floats, t_floats;
};

NormSplit norm_split(const dcn_block_norm* p, int64_t gates, int sms) {
  NormSplit s;
  const int64_t most = int64_t(sms);
  // whole steps of the row slots that a CTA has in hand
  const int64_t slots = with_mapping((int64_t(p->C) + 3) / 4, vector_rows(p), [](auto tpr, auto) {
    return kNormThreads / decltype(tpr)::value;
  });
  int64_t rows = (p->M + most - 1) / most;
  rows = std::min<int64_t>((rows + slots - 1) / slots * slots, INT_MAX);
  s.rows_per_cta = int(rows);
  s.ctas = int((p->M + rows - 1) / rows);
  s.s_floats = size_t(s.ctas + gates - 1) * 2 * size_t(p->C);
  s.t_floats = size_t(s.ctas) * 2 * size_t(p->C);
  return s;
}

size_t split_bytes(const NormSplit& s) {
  return (s.s_floats + s.t_floats) * sizeof(float);
}

}  // namespace
}  // namespace dcn

using namespace dcn;

extern "C" {

dcn_status dcn_core_block_norm(const dcn_block_norm* norm, const void* residual,
                               const void* branch, const float* gate, const float* post_gamma,
                               const float* post_beta, const float* pre_gamma,
                               const float* pre_beta, void* residual_out, void* normed,
                               float* normed_scales, float* post_stats, float* pre_stats,
                               cudaStream_t stream) {
  dcn_status st = check_norm(norm);
  if (st != DCN_OK) return st;
  if (!residual || (!residual_out && !normed)) return DCN_ERR_INVALID_ARG;
  const bool post = norm->post_norm != DCN_NORM_NONE, pre = norm->pre_norm != DCN_NORM_NONE;
  if (!branch && (post || gate)) return DCN_ERR_INVALID_ARG;
  if (!post && (post_gamma || post_beta || post_stats)) return DCN_ERR_INVALID_ARG;
  if (!pre && (pre_gamma || pre_beta || pre_stats || normed)) return DCN_ERR_INVALID_ARG;
  if (normed_scales && !normed) return DCN_ERR_INVALID_ARG;
  for (const void* p : {residual, branch, static_cast<const void*>(residual_out),
                        static_cast<const void*>(normed), static_cast<const void*>(gate),
                        static_cast<const void*>(post_gamma), static_cast<const void*>(post_beta),
                        static_cast<const void*>(pre_gamma), static_cast<const void*>(pre_beta)})
    if (!aligned(p, 16)) return DCN_ERR_UNSUPPORTED;
  if (!aligned(normed_scales, 4) || !aligned(post_stats, 4) || !aligned(pre_stats, 4))
    return DCN_ERR_UNSUPPORTED;
  DeviceInfo dev;
  if (device_info(&dev) != DCN_OK) return DCN_ERR_CUDA;
  NormArgs a;
  a.M = norm->M;
  a.C = norm->C;
  a.rows_per_gate = norm->rows_per_gate > 0 ? norm->rows_per_gate : norm->M;
  a.pitch = int(dcn_core_fp8_pitch(norm->C));
  a.post = norm->post_norm;
  a.pre = norm->pre_norm;
  a.post_eps = norm->post_eps;
  a.pre_eps = norm->pre_eps;
  a.residual_scale = norm->residual_scale;
  a.residual = residual;
  a.branch = branch;
  a.gate = gate;
  a.post_gamma = post_gamma;
  a.post_beta = post_beta;
  a.pre_gamma = pre_gamma;
  a.pre_beta = pre_beta;
  a.residual_out = residual_out;
  a.normed = normed;
  a.scales = normed_scales;
  a.post_stats = post_stats;
  a.pre_stats = pre_stats;
  a.error_word = dev.error_word;
  const bool fp8 = normed_scales != nullptr;
  const int64_t groups = ((fp8 ? int64_t(a.pitch) : int64_t(a.C)) + 3) / 4;
  return with_types(norm, [&](auto s, auto b) {
    return with_mapping(groups, a.C % 4 == 0, [&](auto tpr, auto vec) {
      using TS = decltype(s);
      using TB = decltype(b);
      constexpr int kTpr = decltype(tpr)::value;
      constexpr bool kVec = decltype(vec)::value != 0;
      constexpr int kRows = kNormThreads / kTpr;
      // every CTA resident, each with rows to load ahead
      const int64_t grid = std::min<int64_t>((int64_t(a.M) + kRows - 1) / kRows,
                                             int64_t(dev.sms) * kNormCtas);
      auto launch = [&](auto k) {
        k<<<unsigned(grid), kNormThreads, 0, stream>>>(a);
        return launched();
      };
      if constexpr (kVec) {
        // the widths of the stages (160, 320, 640, 1280) leave no thread without channels
        if (a.C == 4 * kNormGroups * kTpr)
          return fp8 ? launch(dcn_block_norm_kernel<TS, TB, kTpr, true, true, true>)
                     : launch(dcn_block_norm_kernel<TS, TB, kTpr, true, true, false>);
      }
      return fp8 ? launch(dcn_block_norm_kernel<TS, TB, kTpr, kVec, false, true>)
                 : launch(dcn_block_norm_kernel<TS, TB, kTpr, kVec, false, false>);
    });
  });
}

size_t dcn_core_block_norm_backward_workspace(const dcn_block_norm* norm) {
  DeviceInfo dev;
  if (check_norm(norm) != DCN_OK || device_info(&dev) != DCN_OK) return 0;
  return split_bytes(norm_split(norm, gates_of(norm, true), dev.sms));
}

dcn_status dcn_core_block_norm_backward(
    const dcn_block_norm* norm, const void* residual_out, const void* branch, const float* gate,
    const float* post_gamma, const float* post_beta, const float* pre_gamma,
    const float* post_stats, const float* pre_stats, const void* grad_residual_out,
    const void* grad_normed, void* grad_residual, void* grad_branch, float* grad_gate,
    float* grad_post_gamma, float* grad_post_beta, float* grad_pre_gamma, float* grad_pre_beta,
    void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  dcn_status st = check_norm(norm);
  if (st != DCN_OK) return st;
  const bool post = norm->post_norm != DCN_NORM_NONE, pre = norm->pre_norm != DCN_NORM_NONE;
  if (pre ? (!residual_out || !pre_stats || !grad_normed)
          : (!grad_residual_out || grad_normed || pre_gamma || pre_stats || grad_pre_gamma ||
             grad_pre_beta))
    return DCN_ERR_INVALID_ARG;
  if (!branch && (post || gate || grad_branch)) return DCN_ERR_INVALID_ARG;
  if (branch && !grad_branch) return DCN_ERR_INVALID_ARG;
  if (post ? !post_stats
           : (post_gamma || post_beta || post_stats || grad_post_gamma || grad_post_beta))
    return DCN_ERR_INVALID_ARG;
  if (grad_gate && !gate) return DCN_ERR_INVALID_ARG;
  if (!grad_residual && !grad_branch && !grad_pre_gamma && !grad_pre_beta)
    return DCN_ERR_INVALID_ARG;
  for (const void* p :
       {residual_out, branch, grad_residual_out, grad_normed,
        static_cast<const void*>(grad_residual), static_cast<const void*>(grad_branch),
        static_cast<const void*>(workspace), static_cast<const void*>(gate),
        static_cast<const void*>(post_gamma), static_cast<const void*>(post_beta),
        static_cast<const void*>(pre_gamma), static_cast<const void*>(grad_gate),
        static_cast<const void*>(grad_post_gamma), static_cast<const void*>(grad_post_beta),
        static_cast<const void*>(grad_pre_gamma), static_cast<const void*>(grad_pre_beta)})
    if (!aligned(p, 16)) return DCN_ERR_UNSUPPORTED;
  if (!aligned(post_stats, 4) || !aligned(pre_stats, 4)) return DCN_ERR_UNSUPPORTED;
  DeviceInfo dev;
  if (device_info(&dev) != DCN_OK) return DCN_ERR_CUDA;
  if (!workspace ||
      workspace_bytes < split_bytes(norm_split(norm, gates_of(norm, true), dev.sms)))
    return DCN_ERR_INVALID_ARG;
  const int64_t gates = gates_of(norm, gate != nullptr);
  const NormSplit split = norm_split(norm, gates, dev.sms);
  const bool s_sums = grad_gate || grad_post_gamma || grad_post_beta;
  const bool t_sums = grad_pre_gamma || grad_pre_beta;
  float* ws = static_cast<float*>(workspace);
  NormBwdArgs a;
  a.M = norm->M;
  a.C = norm->C;
  a.rows_per_gate = gates > 1 ? norm->rows_per_gate : norm->M;
  a.gates = int(gates);
  a.rows_per_cta = split.rows_per_cta;
  a.post = norm->post_norm;
  a.pre = norm->pre_norm;
  a.residual_scale = norm->residual_scale;
  a.r = residual_out;
  a.branch = branch;
  a.gate = gate;
  a.post_gamma = post_gamma;
  a.pre_gamma = pre_gamma;
  a.post_stats = post_stats;
  a.pre_stats = pre_stats;
  a.grad_r = grad_residual_out;
  a.grad_h = grad_normed;
  a.grad_x = grad_residual;
  a.grad_y = grad_branch;
  a.s_part = s_sums ? ws : nullptr;
  a.t_part = t_sums ? ws + split.s_floats : nullptr;
  const char* stall = std::getenv("DCN_CORE_TEST_STALL");
  a.inject_stall = stall != nullptr && std::atoi(stall) == 1;
  a.error_word = dev.error_word;
  st = with_types(norm, [&](auto s, auto b) {
    return with_mapping((int64_t(a.C) + 3) / 4, vector_rows(norm), [&](auto tpr, auto v) {
      using TS = decltype(s);
      using TB = decltype(b);
      constexpr int kTpr = decltype(tpr)::value;
      constexpr bool kVec = decltype(v)::value != 0;
      if constexpr (kVec) {
        // the widths of the stages (160, 320, 640, 1280) leave no thread without channels
        if (a.C == 4 * kNormGroups * kTpr)
          return launch_backward(dcn_block_norm_backward_kernel<TS, TB, kTpr, true, true>,
                                 NormBwdShape<TS, TB>::kSmemBytes, a, split.ctas, stream);
      }
      return launch_backward(dcn_block_norm_backward_kernel<TS, TB, kTpr, kVec, false>,
                             NormBwdShape<TS, TB>::kSmemBytes, a, split.ctas, stream);
    });
  });
  if (st != DCN_OK || (!s_sums && !t_sums)) return st;
  NormSumArgs f;
  f.M = a.M;
  f.C = a.C;
  f.rows_per_gate = a.rows_per_gate;
  f.gates = a.gates;
  f.rows_per_cta = a.rows_per_cta;
  f.ctas = split.ctas;
  f.s_part = a.s_part;
  f.t_part = a.t_part;
  f.gate = gate;
  f.post_gamma = post_gamma;
  f.post_beta = post_beta;
  f.grad_gate = grad_gate;
  f.grad_post_gamma = grad_post_gamma;
  f.grad_post_beta = grad_post_beta;
  f.grad_pre_gamma = grad_pre_gamma;
  f.grad_pre_beta = grad_pre_beta;
  return launch_kernel(dcn_block_norm_sums_kernel, true, dim3(unsigned((a.C + 31) / 32), 2),
                       32 * kSumGroups, 0, stream, f);
}

}  // extern "C"
