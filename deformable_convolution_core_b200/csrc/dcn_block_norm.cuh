// Norms behind one branch of the block and before the next, with the branch's
// gate and the residual scale: forward and backward.
//
//   p = post_norm(y) * gp + bp,  r = a * x + g * p,  h = pre_norm(r) * gq + bq
//
// A row's channels are spread over TPR threads (8 .. 256), each owning up to five
// groups of four consecutive channels, group t + j * TPR for j = 0 .. 4: every
// load of a row's threads is one contiguous run, and a row's values stay in
// registers between its sums (mean, then centred squares) and its outputs, so
// each tensor crosses HBM once.  Rows of fewer than 32 threads share a warp and
// reduce by shuffles; longer ones add one exchange through shared memory.
#pragma once

#include "dcn_fp8.cuh"

namespace dcn {

constexpr int kNormThreads = 256;
constexpr int kNormGroups = 5;                     // groups of four channels a thread
constexpr int kNormMaxC = 4 * kNormGroups * kNormThreads;  // 5120

enum NormKind { kNormNone = 0, kNormLayer = 1, kNormRms = 2 };

struct NormArgs {
  int M, C;
  int rows_per_gate;  // rows of one gate vector (M with one for all)
  int pitch;          // bytes of a row of e4m3 codes
  int post, pre;      // NormKind
  float post_eps, pre_eps, residual_scale;
  const void* residual;
  const void* branch;
  const float* gate;
  const float* post_gamma;
  const float* post_beta;
  const float* pre_gamma;
  const float* pre_beta;
  void* residual_out;
  void* normed;
  float* scales;
  float* post_stats;
  float* pre_stats;
  unsigned int* error_word;
};

// Four consecutive channels c .. c + 3 of a row as fp32, 0 behind the last.
// VEC: rows start on a boundary of four values and C is a multiple of 4.
// Plain loads: residual_out may be the residual's own buffer.
template <typename T, bool VEC>
__device__ __forceinline__ void load4(const T* row, int c, int C, float (&v)[4]) {
  if constexpr (VEC) {
    if (c < C) {
      if constexpr (sizeof(T) == 4) {
        const float4 w = *reinterpret_cast<const float4*>(row + c);
        v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(row + c);
        const uint32_t a[2] = {w.x, w.y};
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = Storage<T>::chan(a, k);
      }
      return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = 0.f;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = c + k < C ? Storage<T>::to_float(row[c + k]) : 0.f;
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store4(T* row, int c, int C, const float (&v)[4]) {
  if constexpr (VEC) {
    if (c < C) {
      if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(row + c) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
        uint32_t a[2];
        Storage<T>::pack(a, v);
        *reinterpret_cast<uint2*>(row + c) = make_uint2(a[0], a[1]);
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c + k < C) Storage<T>::store_float(row + c + k, v[k]);
  }
}

// Four values of an fp32 parameter vector, `dflt` where there is none.
template <bool VEC>
__device__ __forceinline__ void param4(const float* p, int c, int C, float dflt, float (&v)[4]) {
  if (p == nullptr) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = dflt;
  } else if constexpr (VEC) {
    const float4 w = c < C ? __ldg(reinterpret_cast<const float4*>(p + c))
                           : make_float4(0.f, 0.f, 0.f, 0.f);
    v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = c + k < C ? __ldg(p + c + k) : 0.f;
  }
}

// Sums of two values over the TPR threads of a row; every one of them gets both.
// `slots`: the row's shared memory, two sets of (TPR / 32) pairs used in turn, so
// that one barrier a sum is enough; `turn` counts the sums.  The row's threads
// form whole warps for TPR > 32 and meet at named barrier 1 + row slot.
template <int TPR>
__device__ __forceinline__ float2 row_sum2(float2 v, float2* slots, int& turn) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
    v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, o);
  }
  if constexpr (TPR > 32) {
    constexpr int kWarps = TPR / 32;
    const int w = int(threadIdx.x % TPR) >> 5;
    float2* s = slots + (turn & 1) * kWarps;
    ++turn;
    if ((threadIdx.x & 31) == 0) s[w] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + int(threadIdx.x / TPR)), "n"(TPR) : "memory");
    v = s[0];
#pragma unroll
    for (int k = 1; k < kWarps; ++k) {
      v.x += s[k].x;
      v.y += s[k].y;
    }
  }
  return v;
}

template <int TPR>
__device__ __forceinline__ float row_sum(float v, float2* slots, int& turn) {
  return row_sum2<TPR>(make_float2(v, 0.f), slots, turn).x;
}

// Mean (0 for RMS) and 1 / sqrt(variance or mean square + eps) of a row's values,
// which are 0 behind the last channel.  The squares are of centred values: no
// cancellation, however far the mean is from zero.
template <int TPR>
__device__ __forceinline__ float2 row_stats(const float (&v)[kNormGroups][4], int t, int C,
                                            int kind, float eps, float2* slots, int& turn) {
  float mean = 0.f;
  if (kind == kNormLayer) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < kNormGroups; ++j) s += (v[j][0] + v[j][1]) + (v[j][2] + v[j][3]);
    mean = row_sum<TPR>(s, slots, turn) / float(C);
  }
  float q = 0.f;
#pragma unroll
  for (int j = 0; j < kNormGroups; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float d = 4 * (t + j * TPR) + k < C ? v[j][k] - mean : 0.f;
      q = fmaf(d, d, q);
    }
  return make_float2(mean, 1.f / sqrtf(row_sum<TPR>(q, slots, turn) / float(C) + eps));
}

// TS, TB: storage of the residual stream and of the branch; FP8: normed as e4m3.
template <typename TS, typename TB, int TPR, bool VEC, bool FP8>
__global__ void __launch_bounds__(kNormThreads)
    dcn_block_norm_kernel(const NormArgs a) {
  __shared__ float2 s_slots[2 * (kNormThreads / 32)];
  constexpr int kRows = kNormThreads / TPR;  // rows a CTA has in hand
  const int slot = int(threadIdx.x) / TPR, t = int(threadIdx.x) % TPR;
  float2* slots = s_slots + slot * 2 * (TPR / 32);
  int turn = 0;
  const size_t total = size_t(a.M) * a.C;
  for (int64_t base = int64_t(blockIdx.x) * kRows; base < a.M;
       base += int64_t(gridDim.x) * kRows) {
    // the threads of a warp stay together: a row slot behind the last row works on
    // the last row and stores nothing
    const bool live = base + slot < a.M;
    const int64_t row = live ? base + slot : int64_t(a.M) - 1;
    const size_t off = size_t(row) * a.C;
    const TS* x = static_cast<const TS*>(a.residual) + off;
    const TB* y = static_cast<const TB*>(a.branch) + off;
    const float* gate =
        a.gate ? a.gate + size_t(row / a.rows_per_gate) * a.C : nullptr;

    float r[kNormGroups][4], p[kNormGroups][4];
#pragma unroll
    for (int j = 0; j < kNormGroups; ++j) {
      const int c = 4 * (t + j * TPR);
      const int n = min(4, a.C - c);
      const bool in = n <= 0 || in_range_of(a.error_word, off + c, size_t(n), total);
      load4<TS, VEC>(x, in ? c : a.C, a.C, r[j]);
      if (a.branch) load4<TB, VEC>(y, in ? c : a.C, a.C, p[j]);
    }
    if (a.branch) {
      float2 st = make_float2(0.f, 1.f);
      if (a.post != kNormNone) {
        st = row_stats<TPR>(p, t, a.C, a.post, a.post_eps, slots, turn);
        if (a.post_stats && t == 0 && live) {
          a.post_stats[row] = st.x;
          a.post_stats[size_t(a.M) + row] = st.y;
        }
      }
#pragma unroll
      for (int j = 0; j < kNormGroups; ++j) {
        const int c = 4 * (t + j * TPR);
        float gm[4], bt[4], gt[4];
        param4<VEC>(a.post_gamma, c, a.C, 1.f, gm);
        param4<VEC>(a.post_beta, c, a.C, 0.f, bt);
        param4<VEC>(gate, c, a.C, 1.f, gt);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float n = fmaf((p[j][k] - st.x) * st.y, gm[k], bt[k]);
          r[j][k] = c + k < a.C ? fmaf(gt[k], n, a.residual_scale * r[j][k]) : 0.f;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < kNormGroups; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) r[j][k] *= a.residual_scale;
    }
    if (a.residual_out && live) {
      TS* o = static_cast<TS*>(a.residual_out) + off;
#pragma unroll
      for (int j = 0; j < kNormGroups; ++j) {
        const int c = 4 * (t + j * TPR);
        if (c < a.C &&
            in_range_of(a.error_word, off + c, size_t(min(4, a.C - c)), total))
          store4<TS, VEC>(o, c, a.C, r[j]);
      }
    }
    if (a.pre == kNormNone) continue;
    const float2 st = row_stats<TPR>(r, t, a.C, a.pre, a.pre_eps, slots, turn);
    if (a.pre_stats && t == 0 && live) {
      a.pre_stats[row] = st.x;
      a.pre_stats[size_t(a.M) + row] = st.y;
    }
    if (a.normed == nullptr) continue;
#pragma unroll
    for (int j = 0; j < kNormGroups; ++j) {
      const int c = 4 * (t + j * TPR);
      float gm[4], bt[4];
      param4<VEC>(a.pre_gamma, c, a.C, 1.f, gm);
      param4<VEC>(a.pre_beta, c, a.C, 0.f, bt);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        r[j][k] = c + k < a.C ? fmaf((r[j][k] - st.x) * st.y, gm[k], bt[k]) : 0.f;
    }
    if constexpr (!FP8) {
      if (live) {
        TB* o = static_cast<TB*>(a.normed) + off;
#pragma unroll
        for (int j = 0; j < kNormGroups; ++j) {
          const int c = 4 * (t + j * TPR);
          if (c < a.C &&
              in_range_of(a.error_word, off + c, size_t(min(4, a.C - c)), total))
            store4<TB, VEC>(o, c, a.C, r[j]);
        }
      }
    } else {
      // A block of 128 channels is 32 consecutive groups of four: one j of a whole
      // warp, or 2 or 4 consecutive j of the row's 16 or 8 threads.
      constexpr int kSpan = TPR < 32 ? 32 / TPR : 1;
      uint8_t* codes = static_cast<uint8_t*>(a.normed) + size_t(row) * a.pitch;
#pragma unroll
      for (int j0 = 0; j0 < kNormGroups; j0 += kSpan) {
        float m = 0.f;
#pragma unroll
        for (int j = j0; j < j0 + kSpan && j < kNormGroups; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) m = max_nan(m, fabsf(r[j][k]));
#pragma unroll
        for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1)
          m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const BlockScale b = block_scale(m);
        const int c0 = 4 * (t + j0 * TPR);
        if (live && c0 < a.C && (t % (TPR < 32 ? TPR : 32)) == 0)
          a.scales[size_t(c0 / kFp8Block) * a.M + row] = b.scale;
#pragma unroll
        for (int j = j0; j < j0 + kSpan && j < kNormGroups; ++j) {
          const int c = 4 * (t + j * TPR);
          float q[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) q[k] = c + k < a.C ? __fmul_rn(r[j][k], b.inv) : 0.f;
          if (live && c < a.pitch &&
              in_range_of(a.error_word, size_t(row) * a.pitch + c, 4, size_t(a.M) * a.pitch))
            *reinterpret_cast<uint32_t*>(codes + c) = e4m3x4(q[0], q[1], q[2], q[3]);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Backward.  With n and m the normalised branch and stream, and back(.) the
// gradient of a normalisation, dv = rstd * (d - <d> - n <d n>) (no <d> for RMS):
//   dr = dr_out + back(dh * gq),   dx = a * dr,   dy = back(g * dr * gp),
// and over the rows, with S1_b = sum dr * n and S0_b = sum dr of gate vector b:
//   dgq = sum dh * m, dbq = sum dh, dg_b = gp * S1_b + bp * S0_b,
//   dgp = sum_b g_b * S1_b, dbp = sum_b g_b * S0_b:
// four running sums a channel give the gradients of five parameter vectors.
// CTA c takes the rows [c R, (c + 1) R); it writes its S sums whenever the gate
// vector changes and its dh sums at its end.  The (CTA, gate) pairs that meet form
// a staircase, so c + b numbers them without a gap or a clash.
// ---------------------------------------------------------------------------
struct NormBwdArgs {
  int M, C;
  int rows_per_gate, gates;
  int rows_per_cta;
  int post, pre;
  float residual_scale;
  const void* r;
  const void* branch;
  const float* gate;
  const float* post_gamma;
  const float* pre_gamma;
  const float* post_stats;
  const float* pre_stats;
  const void* grad_r;
  const void* grad_h;
  void* grad_x;
  void* grad_y;
  float* s_part;  // (ctas + gates - 1, 2, C): S1, S0 of each meeting pair, or null
  float* t_part;  // (ctas, 2, C): sums of dh * m and dh, or null
  unsigned int* error_word;
};

// Sum the CTA's row slots' running sums of one array and write them out, fixed order.
template <int TPR>
__device__ __forceinline__ void flush_sums(float (&acc)[kNormGroups][4], float* buf, float* out,
                                           int C) {
  constexpr int kRows = kNormThreads / TPR;
  constexpr int kCols = 4 * kNormGroups * TPR;  // kRows * kCols = 5120 floats
  const int slot = int(threadIdx.x) / TPR, t = int(threadIdx.x) % TPR;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kNormGroups; ++j) {
    *reinterpret_cast<float4*>(buf + slot * kCols + 4 * (t + j * TPR)) =
        make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[j][k] = 0.f;
  }
  __syncthreads();
  for (int c = int(threadIdx.x); c < C && c < kCols; c += kNormThreads) {
    float s = 0.f;
#pragma unroll 8
    for (int k = 0; k < kRows; ++k) s += buf[k * kCols + c];
    out[c] = s;
  }
}

template <typename TS, typename TB, int TPR, bool VEC>
__global__ void __launch_bounds__(kNormThreads, 1)
    dcn_block_norm_backward_kernel(const NormBwdArgs a) {
  __shared__ float2 s_slots[2 * (kNormThreads / 32)];
  __shared__ __align__(16) float s_buf[kNormMaxC];
  constexpr int kRows = kNormThreads / TPR;
  const int slot = int(threadIdx.x) / TPR, t = int(threadIdx.x) % TPR;
  float2* slots = s_slots + slot * 2 * (TPR / 32);
  int turn = 0;
  const size_t total = size_t(a.M) * a.C;
  const int64_t begin = int64_t(blockIdx.x) * a.rows_per_cta;
  const int64_t end = min(begin + a.rows_per_cta, int64_t(a.M));
  const float inv_c = 1.f / float(a.C);

  float s1[kNormGroups][4], s0[kNormGroups][4], t1[kNormGroups][4], t0[kNormGroups][4];
#pragma unroll
  for (int j = 0; j < kNormGroups; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) s1[j][k] = s0[j][k] = t1[j][k] = t0[j][k] = 0.f;

  for (int64_t seg = begin; seg < end;) {
    const int64_t b = seg / a.rows_per_gate;
    const int64_t seg_end = min(end, (b + 1) * int64_t(a.rows_per_gate));
    const float* gate = a.gate ? a.gate + size_t(b) * a.C : nullptr;
    for (int64_t base = seg; base < seg_end; base += kRows) {
      const bool live = base + slot < seg_end;
      const int64_t row = live ? base + slot : seg_end - 1;
      const size_t off = size_t(row) * a.C;
      float dr[kNormGroups][4], n[kNormGroups][4];
#pragma unroll
      for (int j = 0; j < kNormGroups; ++j) {
        const int c = 4 * (t + j * TPR);
        const int w = min(4, a.C - c);
        const bool in = w <= 0 || in_range_of(a.error_word, off + c, size_t(w), total);
        if (a.grad_r) {
          load4<TS, VEC>(static_cast<const TS*>(a.grad_r) + off, in ? c : a.C, a.C, dr[j]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) dr[j][k] = 0.f;
        }
      }
      if (a.pre != kNormNone) {
        const float mean = a.pre_stats[row], rstd = a.pre_stats[size_t(a.M) + row];
        float dh[kNormGroups][4];
        float2 dots = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < kNormGroups; ++j) {
          const int c = 4 * (t + j * TPR);
          const int w = min(4, a.C - c);
          const bool in = w <= 0 || in_range_of(a.error_word, off + c, size_t(w), total);
          load4<TB, VEC>(static_cast<const TB*>(a.grad_h) + off, in ? c : a.C, a.C, dh[j]);
          load4<TS, VEC>(static_cast<const TS*>(a.r) + off, in ? c : a.C, a.C, n[j]);
          float gm[4];
          param4<VEC>(a.pre_gamma, c, a.C, 1.f, gm);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            n[j][k] = c + k < a.C ? (n[j][k] - mean) * rstd : 0.f;
            if (live) {
              t1[j][k] = fmaf(dh[j][k], n[j][k], t1[j][k]);
              t0[j][k] += dh[j][k];
            }
            dh[j][k] *= gm[k];
            dots.x += dh[j][k];
            dots.y = fmaf(dh[j][k], n[j][k], dots.y);
          }
        }
        dots = row_sum2<TPR>(dots, slots, turn);
        const float d0 = a.pre == kNormLayer ? dots.x * inv_c : 0.f, d1 = dots.y * inv_c;
#pragma unroll
        for (int j = 0; j < kNormGroups; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            dr[j][k] = fmaf(rstd, dh[j][k] - fmaf(n[j][k], d1, d0), dr[j][k]);
      }
      if (a.grad_x && live) {
        TS* o = static_cast<TS*>(a.grad_x) + off;
#pragma unroll
        for (int j = 0; j < kNormGroups; ++j) {
          const int c = 4 * (t + j * TPR);
          float v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = a.residual_scale * dr[j][k];
          if (c < a.C && in_range_of(a.error_word, off + c, size_t(min(4, a.C - c)), total))
            store4<TS, VEC>(o, c, a.C, v);
        }
      }
      if (a.branch == nullptr) continue;
      const bool norm = a.post != kNormNone;
      const float mean = norm ? a.post_stats[row] : 0.f;
      const float rstd = norm ? a.post_stats[size_t(a.M) + row] : 1.f;
      float2 dots = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < kNormGroups; ++j) {
        const int c = 4 * (t + j * TPR);
        const int w = min(4, a.C - c);
        const bool in = w <= 0 || in_range_of(a.error_word, off + c, size_t(w), total);
        load4<TB, VEC>(static_cast<const TB*>(a.branch) + off, in ? c : a.C, a.C, n[j]);
        float gm[4], gt[4];
        param4<VEC>(a.post_gamma, c, a.C, 1.f, gm);
        param4<VEC>(gate, c, a.C, 1.f, gt);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          n[j][k] = c + k < a.C ? (n[j][k] - mean) * rstd : 0.f;
          if (c + k >= a.C) dr[j][k] = 0.f;
          if (live) {
            s1[j][k] = fmaf(dr[j][k], n[j][k], s1[j][k]);
            s0[j][k] += dr[j][k];
          }
          dr[j][k] *= gt[k] * gm[k];
          dots.x += dr[j][k];
          dots.y = fmaf(dr[j][k], n[j][k], dots.y);
        }
      }
      if (norm) {
        dots = row_sum2<TPR>(dots, slots, turn);
        const float d0 = a.post == kNormLayer ? dots.x * inv_c : 0.f, d1 = dots.y * inv_c;
#pragma unroll
        for (int j = 0; j < kNormGroups; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) dr[j][k] = rstd * (dr[j][k] - fmaf(n[j][k], d1, d0));
      }
      if (live) {
        TB* o = static_cast<TB*>(a.grad_y) + off;
#pragma unroll
        for (int j = 0; j < kNormGroups; ++j) {
          const int c = 4 * (t + j * TPR);
          if (c < a.C && in_range_of(a.error_word, off + c, size_t(min(4, a.C - c)), total))
            store4<TB, VEC>(o, c, a.C, dr[j]);
        }
      }
    }
    if (a.s_part) {
      float* o = a.s_part + (size_t(blockIdx.x) + size_t(b)) * 2 * a.C;
      flush_sums<TPR>(s1, s_buf, o, a.C);
      flush_sums<TPR>(s0, s_buf, o + a.C, a.C);
    }
    seg = seg_end;
  }
  if (a.t_part) {
    float* o = a.t_part + size_t(blockIdx.x) * 2 * a.C;
    flush_sums<TPR>(t1, s_buf, o, a.C);
    flush_sums<TPR>(t0, s_buf, o + a.C, a.C);
  }
}

struct NormSumArgs {
  int M, C;
  int rows_per_gate, gates, rows_per_cta, ctas;
  const float* s_part;
  const float* t_part;
  const float* gate;
  const float* post_gamma;
  const float* post_beta;
  float* grad_gate;
  float* grad_post_gamma;
  float* grad_post_beta;
  float* grad_pre_gamma;
  float* grad_pre_beta;
  float* gated;  // (gates, 2, C): g_b * S1_b, g_b * S0_b with several gate vectors, else null
};

// Sums of the pairs (v[i][0][c], v[i][1][c]), i in [first, last), by 8 threads a
// column in a fixed order; valid in the threads with g = 0.
__device__ __forceinline__ float2 pair_sum(const float* v, size_t first, size_t last, int C, int c,
                                           int g, float2 (*s)[33]) {
  float2 a = make_float2(0.f, 0.f);
  if (c < C) {
#pragma unroll 4
    for (size_t i = first + g; i < last; i += 8) {
      a.x += v[(2 * i) * C + c];
      a.y += v[(2 * i + 1) * C + c];
    }
  }
  s[g][threadIdx.x & 31] = a;
  __syncthreads();
  if (g == 0)
#pragma unroll
    for (int k = 1; k < 8; ++k) {
      a.x += s[k][threadIdx.x & 31].x;
      a.y += s[k][threadIdx.x & 31].y;
    }
  return a;
}

// blockIdx.y < gates: the S sums of one gate vector; blockIdx.y = gates: the dh sums.
__global__ void __launch_bounds__(256) dcn_block_norm_sums_kernel(const NormSumArgs a) {
  __shared__ float2 s[8][33];
  const int c = int(blockIdx.x) * 32 + int(threadIdx.x & 31), g = int(threadIdx.x >> 5);
  const bool writes = g == 0 && c < a.C;
  for (int64_t b = blockIdx.y; b <= a.gates; b += gridDim.y) {
    __syncthreads();
    if (b == a.gates) {
      if (a.t_part == nullptr) continue;
      const float2 v = pair_sum(a.t_part, 0, size_t(a.ctas), a.C, c, g, s);
      if (writes && a.grad_pre_gamma) a.grad_pre_gamma[c] = v.x;
      if (writes && a.grad_pre_beta) a.grad_pre_beta[c] = v.y;
      continue;
    }
    if (a.s_part == nullptr) continue;
    const int64_t r0 = b * a.rows_per_gate;
    const int64_t r1 = min(r0 + a.rows_per_gate, int64_t(a.M));
    const size_t first = size_t(r0 / a.rows_per_cta) + size_t(b);
    const size_t last = size_t((r1 - 1) / a.rows_per_cta) + size_t(b) + 1;
    const float2 v = pair_sum(a.s_part, first, last, a.C, c, g, s);
    if (!writes) continue;
    const float gp = a.post_gamma ? a.post_gamma[c] : 1.f;
    const float bp = a.post_beta ? a.post_beta[c] : 0.f;
    const float gt = a.gate ? a.gate[size_t(b) * a.C + c] : 1.f;
    if (a.grad_gate) a.grad_gate[size_t(b) * a.C + c] = fmaf(gp, v.x, bp * v.y);
    if (a.gated) {
      a.gated[size_t(2 * b) * a.C + c] = gt * v.x;
      a.gated[size_t(2 * b + 1) * a.C + c] = gt * v.y;
    } else {
      if (a.grad_post_gamma) a.grad_post_gamma[c] = gt * v.x;
      if (a.grad_post_beta) a.grad_post_beta[c] = gt * v.y;
    }
  }
}

// The post norm's parameters over several gate vectors.
__global__ void __launch_bounds__(256) dcn_block_norm_gated_sum_kernel(const NormSumArgs a) {
  __shared__ float2 s[8][33];
  const int c = int(blockIdx.x) * 32 + int(threadIdx.x & 31), g = int(threadIdx.x >> 5);
  const float2 v = pair_sum(a.gated, 0, size_t(a.gates), a.C, c, g, s);
  if (g == 0 && c < a.C) {
    if (a.grad_post_gamma) a.grad_post_gamma[c] = v.x;
    if (a.grad_post_beta) a.grad_post_beta[c] = v.y;
  }
}

}  // namespace dcn
