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

#include <type_traits>

#include "dcn_chain.cuh"
#include "dcn_fp8.cuh"
#include "dcn_ptx.cuh"

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

__device__ __forceinline__ float2 splat(float v) { return make_float2(v, v); }

// Channel of value i = 4 j + k of a row's thread t: with VEC groups of four
// consecutive channels (vector accesses), else every TPR-th channel, so that single
// accesses of neighbouring threads are neighbours too.
template <int TPR, bool VEC>
__device__ __forceinline__ int norm_channel(int t, int j, int k) {
  return VEC ? 4 * (t + j * TPR) + k : t + (4 * j + k) * TPR;
}

// Four values of a staged row as two pairs, 0 behind the last channel (FULL: there is
// none behind it).
template <typename T, int TPR, bool VEC, bool FULL>
__device__ __forceinline__ void staged4(const T* row, int t, int j, int C, float2 (&v)[2]) {
  if constexpr (VEC) {
    if (FULL || 4 * (t + j * TPR) < C) {
      if constexpr (sizeof(T) == 4) {
        const float4 w = *reinterpret_cast<const float4*>(row + 4 * (t + j * TPR));
        v[0] = make_float2(w.x, w.y);
        v[1] = make_float2(w.z, w.w);
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(row + 4 * (t + j * TPR));
        const uint32_t a[2] = {w.x, w.y};
        v[0] = make_float2(Storage<T>::chan(a, 0), Storage<T>::chan(a, 1));
        v[1] = make_float2(Storage<T>::chan(a, 2), Storage<T>::chan(a, 3));
      }
    } else {
      v[0] = v[1] = make_float2(0.f, 0.f);
    }
  } else {
    float x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = t + (4 * j + k) * TPR;
      x[k] = c < C ? Storage<T>::to_float(row[c]) : 0.f;
    }
    v[0] = make_float2(x[0], x[1]);
    v[1] = make_float2(x[2], x[3]);
  }
}

// The same of an fp32 parameter vector in global memory, `dflt` where there is none.
template <int TPR, bool VEC, bool FULL>
__device__ __forceinline__ void param_pairs(const float* p, int t, int j, int C, float dflt,
                                            float2 (&v)[2]) {
  if (p == nullptr) {
    v[0] = v[1] = make_float2(dflt, dflt);
  } else if constexpr (VEC) {
    const int c = 4 * (t + j * TPR);
    const float4 w = FULL || c < C ? __ldg(reinterpret_cast<const float4*>(p + c))
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
    v[0] = make_float2(w.x, w.y);
    v[1] = make_float2(w.z, w.w);
  } else {
    float x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = t + (4 * j + k) * TPR;
      x[k] = c < C ? __ldg(p + c) : 0.f;
    }
    v[0] = make_float2(x[0], x[1]);
    v[1] = make_float2(x[2], x[3]);
  }
}

template <typename T, int TPR, bool VEC, bool FULL>
__device__ __forceinline__ void store_pairs(T* row, int t, int j, int C, const float2 (&v)[2]) {
  const float x[4] = {v[0].x, v[0].y, v[1].x, v[1].y};
  if constexpr (VEC) {
    if (FULL || 4 * (t + j * TPR) < C) store4<T, true>(row, 4 * (t + j * TPR), C, x);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = t + (4 * j + k) * TPR;
      if (c < C) Storage<T>::store_float(row + c, x[k]);
    }
  }
}


// A thread's values of a row as they lie in memory, loaded a row ahead: vectors of four
// (VEC; kept packed until the row's turn) or single values.
template <typename T, int TPR, bool VEC, bool FULL>
struct RowAhead {
  using Unit = typename std::conditional<
      VEC, typename std::conditional<sizeof(T) == 4, float4, uint2>::type, float4>::type;
  Unit u[kNormGroups];
  __device__ __forceinline__ void load(const T* row, int t, int C) {
#pragma unroll
    for (int j = 0; j < kNormGroups; ++j) {
      const int c = 4 * (t + j * TPR);
      if constexpr (VEC) {
        u[j] = FULL || c < C ? *reinterpret_cast<const Unit*>(row + c) : Unit{};
      } else {
        float x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = c + k < C ? Storage<T>::to_float(row[c + k]) : 0.f;
        u[j] = make_float4(x[0], x[1], x[2], x[3]);
      }
    }
  }
  __device__ __forceinline__ void widen(int j, float2 (&v)[2]) const {
    if constexpr (VEC && sizeof(T) == 2) {
      const uint32_t a[2] = {u[j].x, u[j].y};
      v[0] = make_float2(Storage<T>::chan(a, 0), Storage<T>::chan(a, 1));
      v[1] = make_float2(Storage<T>::chan(a, 2), Storage<T>::chan(a, 3));
    } else {
      v[0] = make_float2(u[j].x, u[j].y);
      v[1] = make_float2(u[j].z, u[j].w);
    }
  }
};

// Four values of an fp32 parameter vector of the forward's mapping (groups of four
// consecutive channels), `dflt` where there is none.
template <int TPR, bool VEC, bool FULL>
__device__ __forceinline__ void group_params(const float* p, int t, int j, int C, float dflt,
                                             float2 (&v)[2]) {
  if constexpr (VEC) {
    param_pairs<TPR, true, FULL>(p, t, j, C, dflt, v);
  } else {
    float x[4];
    param4<false>(p, 4 * (t + j * TPR), C, dflt, x);
    v[0] = make_float2(x[0], x[1]);
    v[1] = make_float2(x[2], x[3]);
  }
}

template <typename T, int TPR, bool VEC, bool FULL>
__device__ __forceinline__ void store_group(T* row, int t, int j, int C, const float2 (&v)[2]) {
  const int c = 4 * (t + j * TPR);
  const float x[4] = {v[0].x, v[0].y, v[1].x, v[1].y};
  if (FULL || c < C) store4<T, VEC>(row, c, C, x);
}

// Mean (0 for RMS) and 1 / sqrt(variance or mean square + eps) of a row's values,
// which are 0 behind the last channel.  The squares are of centred values: no
// cancellation, however far the mean is from zero.
template <int TPR, bool FULL>
__device__ __forceinline__ float2 row_stats(const float2 (&v)[kNormGroups][2], int t, int C,
                                            float inv_c, int kind, float eps, float2* slots,
                                            int& turn) {
  float mean = 0.f;
  if (kind == kNormLayer) {
    float2 s = splat(0.f);
#pragma unroll
    for (int j = 0; j < kNormGroups; ++j) s = __fadd2_rn(s, __fadd2_rn(v[j][0], v[j][1]));
    mean = row_sum<TPR>(s.x + s.y, slots, turn) * inv_c;
  }
  const float2 m2 = splat(-mean);
  float2 q = splat(0.f);
#pragma unroll
  for (int j = 0; j < kNormGroups; ++j)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float2 d = __fadd2_rn(v[j][k], m2);
      if (!FULL) {
        const int c = 4 * (t + j * TPR) + 2 * k;
        if (c >= C) d.x = 0.f;
        if (c + 1 >= C) d.y = 0.f;
      }
      q = __ffma2_rn(d, d, q);
    }
  // rsqrtf is within 2 units in the last place, of 2^-24 relative half steps
  return make_float2(mean, rsqrtf(fmaf(row_sum<TPR>(q.x + q.y, slots, turn), inv_c, eps)));
}

// CTAs an SM holds (128 registers a thread).  With the next rows loaded ahead, 16 warps
// keep about 40 KB in flight, and HBM is at 89% of its copy rate at 589,824 x 160 bf16;
// three CTAs of 80 registers spill and take 209 us there instead of 132.  With e4m3 output
// (9216 x 1280, 29.8 us of which the bytes need 20) a block's maximum is reduced too.
constexpr int kNormCtas = 2;

// TS, TB: storage of the residual stream and of the branch; FULL: every thread has all
// of its 20 channels (C = 20 TPR); FP8: normed as e4m3.  Each row's values are loaded
// while the row before is reduced and stored.
template <typename TS, typename TB, int TPR, bool VEC, bool FULL, bool FP8>
__global__ void __launch_bounds__(kNormThreads, kNormCtas)
    dcn_block_norm_kernel(const NormArgs a) {
  __shared__ float2 s_slots[2 * (kNormThreads / 32)];
  constexpr int kRows = kNormThreads / TPR;  // rows a CTA has in hand
  const int slot = int(threadIdx.x) / TPR, t = int(threadIdx.x) % TPR;
  float2* slots = s_slots + slot * 2 * (TPR / 32);
  int turn = 0;
  const float inv_c = 1.f / float(a.C);
  const size_t total = size_t(a.M) * a.C;
  const int64_t step = int64_t(gridDim.x) * kRows;
  RowAhead<TS, TPR, VEC, FULL> xa;
  RowAhead<TB, TPR, VEC, FULL> ya;
  auto load = [&](int64_t row) {
    if (row >= a.M || !in_range_of(a.error_word, size_t(row) * a.C, size_t(a.C), total)) return;
    xa.load(static_cast<const TS*>(a.residual) + size_t(row) * a.C, t, a.C);
    if (a.branch) ya.load(static_cast<const TB*>(a.branch) + size_t(row) * a.C, t, a.C);
  };
#pragma unroll
  for (int j = 0; j < kNormGroups; ++j) {
    xa.u[j] = {};
    ya.u[j] = {};
  }
  const int64_t first = int64_t(blockIdx.x) * kRows;
  load(first + slot);
  // The parameters are read between the row's sums, one trip to L2 or HBM after the
  // other; asked for here, those trips run under the first row's own.
  if (slot == 0) {
#pragma unroll
    for (int j = 0; j < kNormGroups; ++j) {
      const int c = 4 * (t + j * TPR);
      if ((c & 31) == 0 && c < a.C) {  // one thread a 128-byte line
        for (const float* p : {a.post_gamma, a.post_beta, a.pre_gamma, a.pre_beta, a.gate})
          if (p) asm volatile("prefetch.global.L2 [%0];" ::"l"(p + c));
      }
    }
  }
  for (int64_t base = first; base < a.M; base += step) {
    // the threads of a warp stay together: a row slot behind the last row works on
    // what it has and stores nothing
    const bool live = base + slot < a.M;
    const int row = live ? int(base + slot) : a.M - 1;
    const size_t off = size_t(row) * a.C;
    float2 r[kNormGroups][2], p[kNormGroups][2];
#pragma unroll
    for (int j = 0; j < kNormGroups; ++j) {
      xa.widen(j, r[j]);
      if (a.branch) ya.widen(j, p[j]);
    }
    load(base + step + slot);
    const float2 alpha = splat(a.residual_scale);
    if (a.branch) {
      float2 st = make_float2(0.f, 1.f);
      if (a.post != kNormNone) {
        st = row_stats<TPR, FULL>(p, t, a.C, inv_c, a.post, a.post_eps, slots, turn);
        if (a.post_stats && t == 0 && live) {
          a.post_stats[row] = st.x;
          a.post_stats[size_t(a.M) + row] = st.y;
        }
      }
      const float* gate = a.gate;
      if (gate && a.rows_per_gate < a.M) gate += size_t(row / a.rows_per_gate) * a.C;
      const float2 m2 = splat(-st.x), r2 = splat(st.y);
#pragma unroll
      for (int j = 0; j < kNormGroups; ++j) {
        float2 gt[2];
        if (a.post != kNormNone) {
          float2 gm[2], bt[2];
          group_params<TPR, VEC, FULL>(a.post_gamma, t, j, a.C, 1.f, gm);
          group_params<TPR, VEC, FULL>(a.post_beta, t, j, a.C, 0.f, bt);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            p[j][k] = __ffma2_rn(__fmul2_rn(__fadd2_rn(p[j][k], m2), r2), gm[k], bt[k]);
        }
        group_params<TPR, VEC, FULL>(gate, t, j, a.C, 1.f, gt);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          r[j][k] = __ffma2_rn(gt[k], p[j][k], __fmul2_rn(alpha, r[j][k]));
          if (!FULL) {
            const int c = 4 * (t + j * TPR) + 2 * k;
            if (c >= a.C) r[j][k].x = 0.f;
            if (c + 1 >= a.C) r[j][k].y = 0.f;
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < kNormGroups; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) r[j][k] = __fmul2_rn(alpha, r[j][k]);
    }
    if (a.residual_out && live) {
#pragma unroll
      for (int j = 0; j < kNormGroups; ++j)
        store_group<TS, TPR, VEC, FULL>(static_cast<TS*>(a.residual_out) + off, t, j, a.C, r[j]);
    }
    if (a.pre == kNormNone) continue;
    const float2 st = row_stats<TPR, FULL>(r, t, a.C, inv_c, a.pre, a.pre_eps, slots, turn);
    if (a.pre_stats && t == 0 && live) {
      a.pre_stats[row] = st.x;
      a.pre_stats[size_t(a.M) + row] = st.y;
    }
    if (a.normed == nullptr) continue;
    const float2 m2 = splat(-st.x), r2 = splat(st.y);
#pragma unroll
    for (int j = 0; j < kNormGroups; ++j) {
      float2 gm[2], bt[2];
      group_params<TPR, VEC, FULL>(a.pre_gamma, t, j, a.C, 1.f, gm);
      group_params<TPR, VEC, FULL>(a.pre_beta, t, j, a.C, 0.f, bt);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        r[j][k] = __ffma2_rn(__fmul2_rn(__fadd2_rn(r[j][k], m2), r2), gm[k], bt[k]);
        if (!FULL) {
          const int c = 4 * (t + j * TPR) + 2 * k;
          if (c >= a.C) r[j][k].x = 0.f;
          if (c + 1 >= a.C) r[j][k].y = 0.f;
        }
      }
    }
    if constexpr (!FP8) {
      if (live) {
#pragma unroll
        for (int j = 0; j < kNormGroups; ++j)
          store_group<TB, TPR, VEC, FULL>(static_cast<TB*>(a.normed) + off, t, j, a.C, r[j]);
      }
    } else {
      // A block of 128 channels is 32 consecutive groups of four: one j of a whole
      // warp, or 2 or 4 consecutive j of the row's 16 or 8 threads.  Maxima are taken
      // of the magnitudes' bits, which order as the values do, NaN above all; lane b of
      // the block's threads then divides for block b, once, and hands inv around.
      constexpr int kSpan = TPR < 32 ? 32 / TPR : 1;
      constexpr int kBlocks = (kNormGroups + kSpan - 1) / kSpan;
      constexpr int kGroup = TPR < 32 ? TPR : 32;  // threads of a block
      uint32_t top[kBlocks];
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        uint32_t m = 0;
#pragma unroll
        for (int j = b * kSpan; j < (b + 1) * kSpan && j < kNormGroups; ++j)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            m = max(m, max(__float_as_uint(fabsf(r[j][k].x)), __float_as_uint(fabsf(r[j][k].y))));
        if constexpr (kGroup == 32) {
          m = __reduce_max_sync(0xFFFFFFFFu, m);
        } else {
#pragma unroll
          for (int o = kGroup / 2; o > 0; o >>= 1)
            m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        }
        top[b] = m;
      }
      const int tg = t % kGroup;
      uint32_t mine = top[0];
#pragma unroll
      for (int b = 1; b < kBlocks; ++b) mine = tg == b ? top[b] : mine;
      const BlockScale scale = block_scale(__uint_as_float(mine));
      uint8_t* codes = static_cast<uint8_t*>(a.normed) + size_t(row) * a.pitch;
      // block b of this thread's group starts at channel 4 (t - tg + b kSpan TPR)
      if (tg < kBlocks) {
        const int c0 = 4 * (t - tg + tg * kSpan * TPR);
        if (live && c0 < a.C) a.scales[size_t(c0 / kFp8Block) * a.M + row] = scale.scale;
      }
#pragma unroll
      for (int j = 0; j < kNormGroups; ++j) {
        const float inv = __shfl_sync(0xFFFFFFFFu, scale.inv, j / kSpan, kGroup);
        const int c = 4 * (t + j * TPR);
        float q[4] = {__fmul_rn(r[j][0].x, inv), __fmul_rn(r[j][0].y, inv),
                      __fmul_rn(r[j][1].x, inv), __fmul_rn(r[j][1].y, inv)};
        if (!FULL) {  // zeros behind the row, in a block of NaN scale too
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (c + k >= a.C) q[k] = 0.f;
        }
        if (live && (FULL || c < a.pitch) &&
            in_range_of(a.error_word, size_t(row) * a.pitch + c, 4, size_t(a.M) * a.pitch))
          *reinterpret_cast<uint32_t*>(codes + c) = e4m3x4(q[0], q[1], q[2], q[3]);
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
  int inject_stall;  // test knob: 1 = a CTA's first rows never arrive, so the waits expire
  float* s_part;  // (ctas + gates - 1, 2, C): S1, S0 of each meeting pair, or null
  float* t_part;  // (ctas, 2, C): sums of dh * m and dh, or null
  unsigned int* error_word;
};

// The barrier of the CTA's eight warps (0 to 8 are the rows').
__device__ __forceinline__ void norm_sync() {
  asm volatile("bar.sync 9, %0;" ::"n"(kNormThreads) : "memory");
}

// Untiled copy of whole 16-byte units from global to shared memory.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}

// Sum the CTA's row slots' running sums of one array and write them out, fixed order.
template <int TPR, bool VEC>
__device__ __forceinline__ void flush_sums(float2 (&acc)[kNormGroups][2], float* buf, float* out,
                                           int C) {
  constexpr int kRows = kNormThreads / TPR;
  constexpr int kCols = 4 * kNormGroups * TPR;  // kRows * kCols = 5120 floats
  const int slot = int(threadIdx.x) / TPR, t = int(threadIdx.x) % TPR;
  norm_sync();
#pragma unroll
  for (int j = 0; j < kNormGroups; ++j) {
    const float x[4] = {acc[j][0].x, acc[j][0].y, acc[j][1].x, acc[j][1].y};
#pragma unroll
    for (int k = 0; k < 4; ++k) buf[slot * kCols + norm_channel<TPR, VEC>(t, j, k)] = x[k];
    acc[j][0] = acc[j][1] = make_float2(0.f, 0.f);
  }
  norm_sync();
  for (int c = int(threadIdx.x); c < C; c += kNormThreads) {
    float s = 0.f;
#pragma unroll 8
    for (int k = 0; k < kRows; ++k) s += buf[k * kCols + c];
    out[c] = s;
  }
}

// The rows [base, base + rows) of one step of a CTA: rows of one gate vector, at most
// as many as it has row slots.
struct NormSteps {
  int64_t base, seg_end, end, gate;
  int per_gate;
  __device__ __forceinline__ NormSteps(const NormBwdArgs& a) {
    base = int64_t(blockIdx.x) * a.rows_per_cta;
    end = min(base + a.rows_per_cta, int64_t(a.M));
    per_gate = a.rows_per_gate;
    gate = base / per_gate;
    seg_end = min(end, (gate + 1) * per_gate);
  }
  __device__ __forceinline__ bool valid() const { return base < end; }
  // Moves on by `rows` row slots; true at the end of a gate vector's rows.
  __device__ __forceinline__ bool next(int rows) {
    base += rows;
    if (base < seg_end) return false;
    base = seg_end;
    ++gate;
    seg_end = min(end, (gate + 1) * per_gate);
    return true;
  }
};

// What a step brings to shared memory: the rows' bytes of up to four tensors, copied
// as they lie in memory.  A copy starts on a 16-byte boundary at or before the rows;
// `shift` is where they begin in the buffer.
struct NormCopy {
  size_t from;     // first byte copied
  uint32_t bytes;  // whole 16-byte units copied
  uint32_t tail;   // bytes behind them, at the tensor's end
  uint32_t shift;
};

__device__ __forceinline__ NormCopy norm_copy(int64_t base, int rows, int C, int esize,
                                              size_t total) {
  NormCopy c;
  const size_t first = size_t(base) * C * esize, last = first + size_t(rows) * C * esize;
  c.from = first & ~size_t(15);
  const size_t most = total & ~size_t(15);  // nothing behind the tensor is read
  size_t to = (last + 15) & ~size_t(15);
  to = to < most ? to : most;
  c.bytes = uint32_t(to > c.from ? to - c.from : 0);
  c.tail = uint32_t(last > c.from + c.bytes ? last - c.from - c.bytes : 0);
  c.shift = uint32_t(first - c.from);
  return c;
}

template <typename TS, typename TB>
struct NormBwdShape {
  // A step's rows have at most kNormMaxC values; 32 bytes for the shift and the end.
  static constexpr uint32_t kTileS = kNormMaxC * sizeof(TS) + 32;
  static constexpr uint32_t kTileB = kNormMaxC * sizeof(TB) + 32;
  static constexpr uint32_t kStageBytes = 2 * kTileS + 2 * kTileB;
  static constexpr int kStages = int(166 * 1024 / kStageBytes);  // 2 (fp32) to 4 (2-byte types)
  static constexpr uint32_t kParamBytes = 2 * kNormMaxC * 4;     // pre_gamma, gate * post_gamma
  static constexpr size_t kSmemBytes = size_t(kStages) * kStageBytes + kParamBytes + 128;
};

// Eight warps keep the four running sums of their channels (80 registers a thread) and
// a row's normalised values and gradients (40); the warps in turn have the steps' rows
// copied into a ring in shared memory, so that what is in flight does not depend on registers.  (A
// ninth warp for the copies would leave 168 registers to each, by the granularity of
// their allocation, and spill where a width leaves threads without channels: 41 us for
// 4001 x 773 fp32 against 34.  One thread of one warp for all copies: 129 us at 320.)
// pre_gamma and gate * post_gamma of the rows at hand stand in shared
// memory too, ones where there are none.  Each step is a chain of waits (the rows, two
// sums over a row, the stores): 107 us for 147,456 x 320 bf16 with gates and both norms,
// 5.3 TB/s or 81% of the copy rate (124 with the rows' statistics loaded when needed).
template <typename TS, typename TB, int TPR, bool VEC, bool FULL>
__global__ void __launch_bounds__(kNormThreads, 1)
    dcn_block_norm_backward_kernel(const NormBwdArgs a) {
  chain_release();
  using S = NormBwdShape<TS, TB>;
  extern __shared__ __align__(128) unsigned char nb_smem[];
  __shared__ float2 s_slots[2 * (kNormThreads / 32)];
  __shared__ __align__(16) float s_buf[kNormMaxC];
  __shared__ uint64_t full[S::kStages], empty[S::kStages];
  __shared__ int s_abort;
  __shared__ uint32_t s_copied;  // steps whose copies have been issued
  constexpr int kRows = kNormThreads / TPR;
  const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
  volatile int* abort_flag = &s_abort;
  volatile uint32_t* copied = &s_copied;
  if (threadIdx.x == 0) {
    s_copied = 0;
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&full[i], 4);
      mbar_init(&empty[i], kNormThreads / 32);
    }
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  const size_t total = size_t(a.M) * a.C;
  // A wait that gives up sets the error word; the roles then run on to their ends
  // without waiting (the row barriers need every thread).
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (*abort_flag) return false;
    if (mbar_wait_bounded(bar, parity)) return true;
    atomicOr(a.error_word, kErrTimeout);
    *abort_flag = 1;
    return false;
  };
  // ---- copies: the warps take the steps in turn, lanes 0 to 3 of one a tensor each ----
  const bool of_branch = lane >= 2;
  const int size = int(of_branch ? sizeof(TB) : sizeof(TS));
  const char* src = static_cast<const char*>(lane == 0   ? a.grad_r
                                             : lane == 1 ? a.r
                                             : lane == 2 ? a.grad_h
                                             : lane == 3 ? a.branch
                                                         : nullptr);
  if (a.pre == kNormNone && (lane == 1 || lane == 2)) src = nullptr;
  const uint32_t src_at = of_branch ? 2 * S::kTileS + (lane & 1) * S::kTileB : (lane & 1) * S::kTileS;
  auto copy_step = [&](const NormSteps& step, uint32_t n) {
    if (lane >= 4 || (a.inject_stall && n == 0)) return;  // test knob
    const int i = int(n % S::kStages);
    const int rows = int(min(int64_t(kRows), step.seg_end - step.base));
    const NormCopy c = norm_copy(step.base, rows, a.C, size, total * size);
    if (src != nullptr &&
        !in_range_of(a.error_word, c.from, size_t(c.bytes) + c.tail, total * size))
      src = nullptr;  // the bounds-checked build: no copies of it from here on
    const uint32_t bytes = src != nullptr ? c.bytes : 0;
    unsigned char* d = nb_smem + size_t(i) * S::kStageBytes + src_at;
    if (src != nullptr)  // the tensor's last bytes, fewer than a unit
      for (uint32_t e = 0; e < c.tail; ++e)
        d[c.bytes + e] = static_cast<unsigned char>(src[c.from + c.bytes + e]);
    mbar_arrive_expect_tx(&full[i], bytes);
    if (bytes > 0) bulk_load(d, src + c.from, bytes, &full[i]);
    if (lane == 0) *copied = n + 1;
  };
  NormSteps next(a);  // the first step that is not copied yet
  for (int i = 0; i < S::kStages && next.valid(); ++i, next.next(kRows))
    if (warp == 0) copy_step(next, uint32_t(i));
  const int slot = int(threadIdx.x) / TPR, t = int(threadIdx.x) % TPR;
  float2* slots = s_slots + slot * 2 * (TPR / 32);
  int turn = 0;
  const float inv_c = 1.f / float(a.C);
  float* p_gamma = reinterpret_cast<float*>(nb_smem + size_t(S::kStages) * S::kStageBytes);
  float* p_weight = p_gamma + kNormMaxC;
  const bool pre = a.pre != kNormNone, post = a.post != kNormNone;
  for (int c = int(threadIdx.x); c < a.C; c += kNormThreads)
    p_gamma[c] = a.pre_gamma ? __ldg(a.pre_gamma + c) : 1.f;
  auto set_weight = [&](int64_t b) {  // gate b times post_gamma
    norm_sync();
    const float* gate = a.gate ? a.gate + size_t(b) * a.C : nullptr;
    for (int c = int(threadIdx.x); c < a.C; c += kNormThreads)
      p_weight[c] = (gate ? __ldg(gate + c) : 1.f) * (a.post_gamma ? __ldg(a.post_gamma + c) : 1.f);
    norm_sync();
  };
  // a group of channels behind the row for every thread
  auto skip = [&](int j) { return !FULL && 4 * j * TPR >= a.C; };
  float2 s1[kNormGroups][2], s0[kNormGroups][2], t1[kNormGroups][2], t0[kNormGroups][2];
#pragma unroll
  for (int j = 0; j < kNormGroups; ++j)
#pragma unroll
    for (int k = 0; k < 2; ++k) s1[j][k] = s0[j][k] = t1[j][k] = t0[j][k] = splat(0.f);

  uint32_t it = 0;
  NormSteps st(a);
  auto row_at = [&](const NormSteps& s) { return min(s.base + slot, s.seg_end - 1); };
  // a row's statistics, loaded a step ahead: their way from HBM would stand in every step
  struct RowStats {
    float m_mean, m_rstd, n_mean, n_rstd;
  } ahead = {0.f, 0.f, 0.f, 1.f};
  auto load_stats = [&](int64_t row) {
    if (pre) {
      ahead.m_mean = __ldg(a.pre_stats + row);
      ahead.m_rstd = __ldg(a.pre_stats + size_t(a.M) + row);
    }
    if (post) {
      ahead.n_mean = __ldg(a.post_stats + row);
      ahead.n_rstd = __ldg(a.post_stats + size_t(a.M) + row);
    }
  };
  if (st.valid()) {
    load_stats(row_at(st));
    set_weight(st.gate);
  }
  while (st.valid()) {
    const int i = int(it % S::kStages);
    const bool live = st.base + slot < st.seg_end;
    const int64_t row = row_at(st);
    const int at = int(row - st.base) * a.C;
    const size_t off = size_t(row) * a.C;
    const unsigned char* stage = nb_smem + size_t(i) * S::kStageBytes;
    // vector rows start on 16-byte boundaries
    const uint32_t shift_s = VEC ? 0u : uint32_t(size_t(st.base) * a.C * sizeof(TS)) & 15u;
    const uint32_t shift_b = VEC ? 0u : uint32_t(size_t(st.base) * a.C * sizeof(TB)) & 15u;
    const TS* g_r = reinterpret_cast<const TS*>(stage + shift_s) + at;
    const TS* x_r = reinterpret_cast<const TS*>(stage + S::kTileS + shift_s) + at;
    const TB* g_h = reinterpret_cast<const TB*>(stage + 2 * S::kTileS + shift_b) + at;
    const TB* y = reinterpret_cast<const TB*>(stage + 2 * S::kTileS + S::kTileB + shift_b) + at;
    const auto [m_mean, m_rstd, n_mean, n_rstd] = ahead;
    const size_t b = size_t(st.gate);
    const bool gate_ends = st.next(kRows);
    if (st.valid()) load_stats(row_at(st));
    (void)wait(&full[i], (it / S::kStages) & 1);

    float2 dr[kNormGroups][2], n[kNormGroups][2];  // the gradient; the normalised row
    if (pre) {
      const float2 mean2 = splat(-m_mean), rstd2 = splat(m_rstd);
      float2 sum = splat(0.f), dot = splat(0.f);
#pragma unroll
      for (int j = 0; j < kNormGroups; ++j) {
        if (skip(j)) continue;
        float2 d[2], gm[2];
        staged4<TB, TPR, VEC, FULL>(g_h, t, j, a.C, d);
        staged4<TS, TPR, VEC, FULL>(x_r, t, j, a.C, n[j]);
        staged4<float, TPR, VEC, FULL>(p_gamma, t, j, a.C, gm);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          n[j][k] = __fmul2_rn(__fadd2_rn(n[j][k], mean2), rstd2);  // times d = 0 behind the row
          if (live) {
            t1[j][k] = __ffma2_rn(d[k], n[j][k], t1[j][k]);
            t0[j][k] = __fadd2_rn(t0[j][k], d[k]);
          }
          dr[j][k] = __fmul2_rn(d[k], gm[k]);
          sum = __fadd2_rn(sum, dr[j][k]);
          dot = __ffma2_rn(dr[j][k], n[j][k], dot);
        }
      }
      const float2 dots =
          row_sum2<TPR>(make_float2(sum.x + sum.y, dot.x + dot.y), slots, turn);
      // dr = dr_out + rstd * (d - d0 - m d1), with m = (r - mean) * rstd
      const float2 d0 = splat(a.pre == kNormLayer ? -dots.x * inv_c : 0.f);
      const float2 d1 = splat(-dots.y * inv_c);
#pragma unroll
      for (int j = 0; j < kNormGroups; ++j) {
        if (skip(j)) continue;
        float2 g[2] = {splat(0.f), splat(0.f)};
        if (a.grad_r) staged4<TS, TPR, VEC, FULL>(g_r, t, j, a.C, g);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 v = __ffma2_rn(n[j][k], d1, __fadd2_rn(dr[j][k], d0));
          dr[j][k] = __ffma2_rn(rstd2, v, g[k]);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < kNormGroups; ++j)
        if (!skip(j)) staged4<TS, TPR, VEC, FULL>(g_r, t, j, a.C, dr[j]);
    }
    // the stage of the step before, which every warp has read or is about to have, takes
    // the step that is a ring ahead of it
    if (it > 0 && next.valid()) {
      if (warp == int(it % (kNormThreads / 32)) &&
          wait(&empty[(it - 1) % S::kStages], ((it - 1) / S::kStages) & 1))
        copy_step(next, it - 1 + S::kStages);
      next.next(kRows);
      __syncwarp();
    }
    if (a.grad_x && live) {
      TS* o = static_cast<TS*>(a.grad_x) + off;
      const float2 scale = splat(a.residual_scale);
#pragma unroll
      for (int j = 0; j < kNormGroups; ++j) {
        if (skip(j)) continue;
        const float2 v[2] = {__fmul2_rn(dr[j][0], scale), __fmul2_rn(dr[j][1], scale)};
        store_pairs<TS, TPR, VEC, FULL>(o, t, j, a.C, v);
      }
    }
    if (a.branch != nullptr) {
      const float2 mean2 = splat(-n_mean), rstd2 = splat(n_rstd);
      float2 sum = splat(0.f), dot = splat(0.f);
#pragma unroll
      for (int j = 0; j < kNormGroups; ++j) {
        if (skip(j)) continue;
        float2 w[2];
        staged4<TB, TPR, VEC, FULL>(y, t, j, a.C, n[j]);
        staged4<float, TPR, VEC, FULL>(p_weight, t, j, a.C, w);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          n[j][k] = __fmul2_rn(__fadd2_rn(n[j][k], mean2), rstd2);
          if (!FULL) {  // neither is 0 behind the row
            if (norm_channel<TPR, VEC>(t, j, 2 * k) >= a.C) dr[j][k].x = n[j][k].x = 0.f;
            if (norm_channel<TPR, VEC>(t, j, 2 * k + 1) >= a.C) dr[j][k].y = n[j][k].y = 0.f;
          }
          if (live) {
            s1[j][k] = __ffma2_rn(dr[j][k], n[j][k], s1[j][k]);
            s0[j][k] = __fadd2_rn(s0[j][k], dr[j][k]);
          }
          dr[j][k] = __fmul2_rn(dr[j][k], w[k]);
          sum = __fadd2_rn(sum, dr[j][k]);
          dot = __ffma2_rn(dr[j][k], n[j][k], dot);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[i]);  // the step's rows have all been read
      TB* o = static_cast<TB*>(a.grad_y) + off;
      if (post) {
        const float2 dots =
            row_sum2<TPR>(make_float2(sum.x + sum.y, dot.x + dot.y), slots, turn);
        const float2 d0 = splat(a.post == kNormLayer ? -dots.x * inv_c : 0.f);
        const float2 d1 = splat(-dots.y * inv_c);
#pragma unroll
        for (int j = 0; j < kNormGroups; ++j)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (!skip(j))
              dr[j][k] = __fmul2_rn(rstd2, __ffma2_rn(n[j][k], d1, __fadd2_rn(dr[j][k], d0)));
      }
      if (live) {
#pragma unroll
        for (int j = 0; j < kNormGroups; ++j)
          if (!skip(j)) store_pairs<TB, TPR, VEC, FULL>(o, t, j, a.C, dr[j]);
      }
    } else {
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[i]);
    }
    ++it;
    if (gate_ends) {
      if (a.s_part) {
        float* o = a.s_part + (size_t(blockIdx.x) + b) * 2 * a.C;
        flush_sums<TPR, VEC>(s1, s_buf, o, a.C);
        flush_sums<TPR, VEC>(s0, s_buf, o + a.C, a.C);
      }
      if (st.valid() && a.gate) set_weight(st.gate);
    }
  }
  norm_sync();
  if (*abort_flag && threadIdx.x == 0)  // the last copies may still be landing
    for (uint32_t j = *copied > uint32_t(S::kStages) ? *copied - S::kStages : 0; j < *copied; ++j)
      if (!(a.inject_stall && j == 0))
        (void)mbar_wait_bounded(&full[j % S::kStages], (j / S::kStages) & 1);
  __syncwarp();
  if (a.t_part) {
    float* o = a.t_part + size_t(blockIdx.x) * 2 * a.C;
    flush_sums<TPR, VEC>(t1, s_buf, o, a.C);
    flush_sums<TPR, VEC>(t0, s_buf, o + a.C, a.C);
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
};

constexpr int kSumGroups = 32;  // warps of a CTA that share 32 columns

// The sum of the warps' values, by warp 0 in the warps' order (valid there).
__device__ __forceinline__ float2 join_groups(float2 v, int g, float2 (*s)[32]) {
  __syncthreads();
  s[g][threadIdx.x & 31] = v;
  __syncthreads();
  if (g == 0) {
#pragma unroll 8
    for (int k = 1; k < kSumGroups; ++k) {
      v.x += s[k][threadIdx.x & 31].x;
      v.y += s[k][threadIdx.x & 31].y;
    }
  }
  return v;
}

// The CTAs' partial sums to the parameters' gradients: 32 columns a CTA, a lane a
// column.  Many gate vectors are dealt out to the 32 warps; the partial sums of few, and
// those of dh (blockIdx.y = 1), are.
__global__ void __launch_bounds__(32 * kSumGroups)
    dcn_block_norm_sums_kernel(const NormSumArgs a) {
  chain_wait();
  __shared__ float2 s[kSumGroups][32];
  const int c = int(blockIdx.x) * 32 + int(threadIdx.x & 31), g = int(threadIdx.x >> 5);
  const bool in = c < a.C;
  auto add = [&](const float* v, size_t i, float2& to) {
    to.x += v[(2 * i) * a.C + c];
    to.y += v[(2 * i + 1) * a.C + c];
  };
  if (a.s_part && blockIdx.y == 0) {
    const float gp = in && a.post_gamma ? a.post_gamma[c] : 1.f;
    const float bp = in && a.post_beta ? a.post_beta[c] : 0.f;
    float2 gated = make_float2(0.f, 0.f);
    // the gradient of gate b, and its part of the post norm's parameters
    auto finish = [&](int64_t b, float2 v) {
      const float gt = a.gate ? a.gate[size_t(b) * a.C + c] : 1.f;
      if (a.grad_gate) a.grad_gate[size_t(b) * a.C + c] = fmaf(gp, v.x, bp * v.y);
      gated.x = fmaf(gt, v.x, gated.x);
      gated.y = fmaf(gt, v.y, gated.y);
    };
    const bool deal = a.gates >= kSumGroups;
    for (int64_t b = deal ? g : 0; b < a.gates; b += deal ? kSumGroups : 1) {
      // rows fit 31 bits: 32-bit divisions
      const uint32_t r0 = uint32_t(b * a.rows_per_gate);
      const uint32_t r1 = uint32_t(min((b + 1) * a.rows_per_gate, int64_t(a.M)));
      const size_t first = size_t(r0 / uint32_t(a.rows_per_cta)) + size_t(b);
      const size_t last = size_t((r1 - 1) / uint32_t(a.rows_per_cta)) + size_t(b) + 1;
      float2 v = make_float2(0.f, 0.f);
      if (in)
#pragma unroll 4
        for (size_t i = first + (deal ? 0 : g); i < last; i += deal ? 1 : kSumGroups)
          add(a.s_part, i, v);
      if (!deal) v = join_groups(v, g, s);
      if (in && (deal || g == 0)) finish(b, v);
    }
    if (deal) gated = join_groups(gated, g, s);
    if (in && g == 0) {
      if (a.grad_post_gamma) a.grad_post_gamma[c] = gated.x;
      if (a.grad_post_beta) a.grad_post_beta[c] = gated.y;
    }
  }
  if (a.t_part && blockIdx.y == 1) {
    float2 v = make_float2(0.f, 0.f);
    if (in)
#pragma unroll 4
      for (int i = g; i < a.ctas; i += kSumGroups) add(a.t_part, size_t(i), v);
    v = join_groups(v, g, s);
    if (in && g == 0) {
      if (a.grad_pre_gamma) a.grad_pre_gamma[c] = v.x;
      if (a.grad_pre_beta) a.grad_pre_beta[c] = v.y;
    }
  }
}

}  // namespace dcn
