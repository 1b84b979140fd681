// Quantiser to block-scaled e4m3 (dcn_fp8.cuh).
#pragma once

#include "dcn_fp8.cuh"

namespace dcn {

// 8 consecutive values of a row as fp32; values at or behind column `cols` are 0.
// VEC: the row starts on a vector boundary and cols is a multiple of 8.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, int col, int cols, float (&v)[8]) {
  if constexpr (VEC) {
    if (col < cols) {
      constexpr int kPer = 16 / int(sizeof(T));
#pragma unroll
      for (int h = 0; h < 8 / kPer; ++h) {
        Vec<16> w;
        ldg_nc(w, row + col + h * kPer);
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[h * kPer + j] = Storage<T>::chan(w.w, j);
      }
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = col + j < cols ? Storage<T>::to_float(row[col + j]) : 0.f;
  }
}

struct QuantArgs {
  const void* x;
  int rows, cols;
  int pitch, pitch_t;  // bytes of a row of q and of q_t
  int col_tiles;       // ceil(cols / 128)
  int row_tiles;       // ceil(rows / 128)
  uint8_t* q;          // (rows, pitch), or null
  float* scales;       // (col_tiles, rows), or (col_tiles, row_tiles) with whole blocks
  uint8_t* q_t;        // (cols, pitch_t), or null
  float* scales_t;     // (row_tiles, cols), or (row_tiles, col_tiles)
  float* col_sums;     // (row_tiles, cols): sums over the tile's rows, or null
  unsigned int* error_word;
};

constexpr int kQuantThreads = 256;

// One 128 x 128 tile a CTA, held in registers, so that the input is read once
// whatever is written.  Sixteen lanes own a row's 128 columns (8 each: a 16-byte
// load of a 2-byte type), and a lane owns 8 consecutive rows, i.e. an 8 x 8
// patch: a row's maximum is a shuffle over 16 lanes, a column's goes over the
// patch, the other half-warp and the 8 warps (through shared memory).  For the
// transpose a patch column packs into 8 bytes, written to shared memory at unit
// (u ^ (c / 8)) of column c's 128 bytes: the sixteen lanes of a half-warp then
// meet sixteen different bank pairs, and each column leaves as one 128-byte run.
// Memory bound: the input once, one byte a value for each code tensor.
template <typename T, bool VEC, bool WHOLE, bool ROWS, bool TRANS>
__global__ void __launch_bounds__(kQuantThreads)
    dcn_quantize_kernel(const QuantArgs a) {
  __shared__ float s_col[8][kFp8Block];            // per warp and column: maximum
  __shared__ float s_sum[8][kFp8Block];            // per warp and column: sum
  __shared__ __align__(16) uint8_t s_t[TRANS ? kFp8Block * kFp8Block : 16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = lane >> 4, l = lane & 15;
  const int rt = int(blockIdx.x / unsigned(a.col_tiles));
  const int ct = int(blockIdx.x - unsigned(rt) * unsigned(a.col_tiles));
  const int r0 = rt * kFp8Block + warp * 16 + half * 8;  // the patch's first row
  const int c0 = ct * kFp8Block + l * 8;                 // and column
  const T* x = static_cast<const T*>(a.x);
  const size_t total = size_t(a.rows) * a.cols;

  float v[8][8];  // [row][column]
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const size_t row = size_t(r0 + i);
    const int n = min(8, a.cols - c0);
    if (r0 + i < a.rows && n > 0 &&
        in_range_of(a.error_word, row * a.cols + c0, size_t(n), total)) {
      load8<T, VEC>(x + row * a.cols, c0, a.cols, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
  }

  float rmax[8], cmax[8], csum[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) rmax[i] = cmax[i] = csum[i] = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float m = fabsf(v[i][j]);
      if (ROWS || WHOLE) rmax[i] = max_nan(rmax[i], m);
      if (TRANS && !WHOLE) cmax[j] = max_nan(cmax[j], m);
      csum[j] += v[i][j];
    }

  float row_inv[8], col_inv[8];
  if constexpr (WHOLE) {
    float m = rmax[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max_nan(m, rmax[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (lane == 0) s_col[warp][0] = m;
    __syncthreads();
    m = s_col[0][0];
#pragma unroll
    for (int w = 1; w < 8; ++w) m = max_nan(m, s_col[w][0]);
    const BlockScale b = block_scale(m);
#pragma unroll
    for (int i = 0; i < 8; ++i) row_inv[i] = col_inv[i] = b.inv;
    if (threadIdx.x == 0) {
      if (ROWS) a.scales[size_t(ct) * a.row_tiles + rt] = b.scale;
      if (TRANS) a.scales_t[size_t(rt) * a.col_tiles + ct] = b.scale;
    }
  } else {
    if constexpr (ROWS) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
          rmax[i] = max_nan(rmax[i], __shfl_xor_sync(0xFFFFFFFFu, rmax[i], o));
        const BlockScale b = block_scale(rmax[i]);
        row_inv[i] = b.inv;
        if (l == i && r0 + i < a.rows) a.scales[size_t(ct) * a.rows + r0 + i] = b.scale;
      }
    }
    if constexpr (TRANS) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float m = max_nan(cmax[j], __shfl_xor_sync(0xFFFFFFFFu, cmax[j], 16));
        if (half == 0) s_col[warp][l * 8 + j] = m;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float m = s_col[0][l * 8 + j];
#pragma unroll
        for (int w = 1; w < 8; ++w) m = max_nan(m, s_col[w][l * 8 + j]);
        const BlockScale b = block_scale(m);
        col_inv[j] = b.inv;
        if (warp == 0 && half == 0 && c0 + j < a.cols)
          a.scales_t[size_t(rt) * a.cols + c0 + j] = b.scale;
      }
    }
  }
  if (a.col_sums != nullptr) {  // uniform: the bias gradient of the linear backward
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = csum[j] + __shfl_xor_sync(0xFFFFFFFFu, csum[j], 16);
      if (half == 0) s_sum[warp][l * 8 + j] = s;
    }
    __syncthreads();
    const int c = ct * kFp8Block + int(threadIdx.x);
    if (threadIdx.x < kFp8Block && c < a.cols) {
      float s = s_sum[0][threadIdx.x];
#pragma unroll
      for (int w = 1; w < 8; ++w) s += s_sum[w][threadIdx.x];
      a.col_sums[size_t(rt) * a.cols + c] = s;
    }
  }

  // values behind the last row or column are 0 and give the zero code, which
  // fills the pitch
  if constexpr (ROWS) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (r0 + i < a.rows && c0 < a.pitch &&
          in_range_of(a.error_word, size_t(r0 + i) * a.pitch + c0, 8,
                      size_t(a.rows) * a.pitch)) {
        uint2 w;
        const float s = row_inv[i];
        // behind the last column: zeros even in a block of NaN scale
        float t[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) t[j] = c0 + j < a.cols ? __fmul_rn(v[i][j], s) : 0.f;
        w.x = e4m3x4(t[0], t[1], t[2], t[3]);
        w.y = e4m3x4(t[4], t[5], t[6], t[7]);
        *reinterpret_cast<uint2*>(a.q + size_t(r0 + i) * a.pitch + c0) = w;
      }
    }
  }
  if constexpr (TRANS) {
    const int u = warp * 2 + half;  // the patch's 8-byte unit of a column
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = r0 + i < a.rows ? __fmul_rn(v[i][j], col_inv[j]) : 0.f;
      uint2 w;
      w.x = e4m3x4(t[0], t[1], t[2], t[3]);
      w.y = e4m3x4(t[4], t[5], t[6], t[7]);
      *reinterpret_cast<uint2*>(&s_t[(l * 8 + j) * kFp8Block + ((u ^ l) << 3)]) = w;
    }
    __syncthreads();
    const int m0 = rt * kFp8Block + l * 8;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const int cl = s * 16 + warp * 2 + half;  // column of the tile
      const int c = ct * kFp8Block + cl;
      const uint2 w =
          *reinterpret_cast<const uint2*>(&s_t[cl * kFp8Block + ((l ^ (cl >> 3)) << 3)]);
      if (c < a.cols && m0 < a.pitch_t &&
          in_range_of(a.error_word, size_t(c) * a.pitch_t + m0, 8, size_t(a.cols) * a.pitch_t))
        *reinterpret_cast<uint2*>(a.q_t + size_t(c) * a.pitch_t + m0) = w;
    }
  }
}

// out[c] = sum over the tiles of part[t][c], in a fixed order: 32 columns a CTA,
// 8 threads a column.
__global__ void __launch_bounds__(256) dcn_column_sum_kernel(const float* part, int tiles,
                                                             int cols, float* out) {
  __shared__ float s[8][33];
  const int c = int(blockIdx.x) * 32 + int(threadIdx.x & 31), g = int(threadIdx.x >> 5);
  float v = 0.f;
  if (c < cols)
    for (int t = g; t < tiles; t += 8) v += part[size_t(t) * cols + c];
  s[g][threadIdx.x & 31] = v;
  __syncthreads();
  if (g == 0 && c < cols) {
#pragma unroll
    for (int k = 1; k < 8; ++k) v += s[k][threadIdx.x & 31];
    out[c] = v;
  }
}

}  // namespace dcn
