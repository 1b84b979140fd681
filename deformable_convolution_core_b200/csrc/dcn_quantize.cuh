// Quantiser to block-scaled e4m3 (dcn_fp8.cuh).
#pragma once

#include "dcn_chain.cuh"
#include "dcn_fp8.cuh"
#include "dcn_ptx.cuh"

namespace dcn {

// 8 consecutive values of a row as they lie in memory: 4 words of two 2-byte values or
// 8 of one.  Magnitudes are compared as the integers that their bits are: those order
// as the values do, with infinity and then NaN on top, so a NaN wins every maximum.
template <typename T>
struct Eight {
  static constexpr int kWords = 2 * int(sizeof(T));
  uint32_t w[kWords];

  // Values at or behind column `cols` are 0.  VEC: the row starts on a 16-byte
  // boundary and cols is a multiple of 8.
  template <bool VEC>
  __device__ __forceinline__ void load(const T* row, int col, int cols) {
    if constexpr (VEC) {
#pragma unroll
      for (int h = 0; h < kWords / 4; ++h) {
        const uint4 x = col < cols ? ldg128(row + col + h * (8 / (kWords / 4)))
                                   : make_uint4(0, 0, 0, 0);
        w[4 * h] = x.x; w[4 * h + 1] = x.y; w[4 * h + 2] = x.z; w[4 * h + 3] = x.w;
      }
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = col + j < cols ? __float_as_uint(float(row[col + j])) : 0u;
    } else {
      const unsigned short* r = reinterpret_cast<const unsigned short*>(row);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = col + 2 * j < cols ? r[col + 2 * j] : 0u;
        const uint32_t hi = col + 2 * j + 1 < cols ? r[col + 2 * j + 1] : 0u;
        w[j] = lo | (hi << 16);
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < kWords; ++j) w[j] = 0u;
  }
  __device__ __forceinline__ float2 pair(int j) const {  // values 2 j and 2 j + 1
    if constexpr (sizeof(T) == 4)
      return make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
    else
      return make_float2(Storage<T>::chan(w, 2 * j), Storage<T>::chan(w, 2 * j + 1));
  }
  static __device__ __forceinline__ uint32_t magnitude(uint32_t x) {
    return x & (sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu);
  }
  // Maximum of two words of magnitudes (half by half for 2-byte values).
  static __device__ __forceinline__ uint32_t top(uint32_t x, uint32_t y) {
    if constexpr (sizeof(T) == 4) return max(x, y);
    else return __vmaxu2(x, y);
  }
  // The larger of a word's magnitudes, as a float.
  static __device__ __forceinline__ float single(uint32_t x) {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(x);
    } else {
      const uint32_t y[1] = {max(x & 0xFFFFu, x >> 16)};
      return Storage<T>::chan(y, 0);
    }
  }
};

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
// load of a 2-byte type), and a lane owns 8 consecutive rows, i.e. an 8 x 8 patch.
// Row maxima: the sixteen lanes halve the eight rows among them while they reduce
// (8 shuffles), so that a pair of lanes has one row and divides for it once.  Column
// maxima: over the patch, the other half-warp and, through shared memory, the 8
// warps; one thread a column divides.  For the transpose a patch column packs into 8
// bytes, written to shared memory at unit (u ^ (c / 8)) of column c's 128 bytes: the
// sixteen lanes of a half-warp then meet sixteen different bank pairs, and each
// column leaves as one 128-byte run.  The input is read once and one byte a value
// written for each code tensor: 36,864 x 640 bf16 with the transpose takes 22.5 us
// (4.3 TB/s, 65% of the copy rate) at 60% of the issue slots.
template <typename T, bool VEC, bool WHOLE, bool ROWS, bool TRANS, bool SUMS>
__global__ void __launch_bounds__(kQuantThreads, sizeof(T) == 2 ? 3 : 2)
    dcn_quantize_kernel(const QuantArgs a) {
  chain_release();
  using E = Eight<T>;
  constexpr int kW = E::kWords;
  __shared__ uint32_t s_top[8][16][kW];          // per warp and 8 columns: magnitudes
  __shared__ float s_sum[SUMS ? 8 : 1][kFp8Block];
  __shared__ __align__(16) float s_inv[kFp8Block];
  __shared__ __align__(16) uint8_t s_t[TRANS ? kFp8Block * kFp8Block : 16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int half = lane >> 4, l = lane & 15;
  const int rt = int(blockIdx.x / unsigned(a.col_tiles));
  const int ct = int(blockIdx.x - unsigned(rt) * unsigned(a.col_tiles));
  const int r0 = rt * kFp8Block + warp * 16 + half * 8;  // the patch's first row
  const int c0 = ct * kFp8Block + l * 8;                 // and column
  const T* x = static_cast<const T*>(a.x);
  const size_t total = size_t(a.rows) * a.cols;

  E v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const size_t row = size_t(r0 + i);
    const int n = min(8, a.cols - c0);
    if (r0 + i < a.rows && n > 0 &&
        in_range_of(a.error_word, row * a.cols + c0, size_t(n), total))
      v[i].template load<VEC>(x + row * a.cols, c0, a.cols);
    else
      v[i].zero();
  }

  float row_inv = 0.f;  // of this lane's row (ROWS), or of the tile (WHOLE)
  float col_inv[8];
  if constexpr (WHOLE) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < kW; ++j) m = E::top(m, E::magnitude(v[i].w[j]));
    if constexpr (sizeof(T) == 2) m = max(m & 0xFFFFu, m >> 16);
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if (lane == 0) s_top[warp][0][0] = m;
    __syncthreads();
    m = s_top[0][0][0];
#pragma unroll
    for (int w = 1; w < 8; ++w) m = max(m, s_top[w][0][0]);
    const BlockScale b = block_scale(E::single(m));
    row_inv = b.inv;
#pragma unroll
    for (int j = 0; j < 8; ++j) col_inv[j] = b.inv;
    if (threadIdx.x == 0) {
      if (ROWS) a.scales[size_t(ct) * a.row_tiles + rt] = b.scale;
      if (TRANS) a.scales_t[size_t(rt) * a.col_tiles + ct] = b.scale;
    }
  } else {
    if constexpr (TRANS) {
      uint32_t m[kW];
#pragma unroll
      for (int j = 0; j < kW; ++j) {
        m[j] = E::magnitude(v[0].w[j]);
#pragma unroll
        for (int i = 1; i < 8; ++i) m[j] = E::top(m[j], E::magnitude(v[i].w[j]));
        m[j] = E::top(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], 16));
      }
      if (half == 0)
#pragma unroll
        for (int j = 0; j < kW; ++j) s_top[warp][l][j] = m[j];
    }
    if constexpr (ROWS) {
      uint32_t m[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m[i] = E::magnitude(v[i].w[0]);
#pragma unroll
        for (int j = 1; j < kW; ++j) m[i] = E::top(m[i], E::magnitude(v[i].w[j]));
      }
#pragma unroll
      for (int h = 4; h > 0; h >>= 1) {  // rows kept, and twice the lanes' distance
        const bool up = (l & (2 * h)) != 0;
#pragma unroll
        for (int i = 0; i < h; ++i) {
          const uint32_t mine = up ? m[i + h] : m[i], other = up ? m[i] : m[i + h];
          m[i] = E::top(mine, __shfl_xor_sync(0xFFFFFFFFu, other, 2 * h));
        }
      }
      m[0] = E::top(m[0], __shfl_xor_sync(0xFFFFFFFFu, m[0], 1));
      const BlockScale b = block_scale(E::single(m[0]));
      row_inv = b.inv;
      const int row = r0 + (l >> 1);  // bits 3, 2, 1 of the lane chose the row's bits 2, 1, 0
      if ((l & 1) == 0 && row < a.rows) a.scales[size_t(ct) * a.rows + row] = b.scale;
    }
    if constexpr (TRANS) {
      __syncthreads();
      if (threadIdx.x < kFp8Block) {
        const int g = int(threadIdx.x) >> 3, j = int(threadIdx.x) & 7;
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          if constexpr (sizeof(T) == 4) m = max(m, s_top[w][g][j]);
          else m = max(m, (s_top[w][g][j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
        }
        const BlockScale b = block_scale(E::single(m));
        s_inv[threadIdx.x] = b.inv;
        const int c = ct * kFp8Block + int(threadIdx.x);
        if (c < a.cols) a.scales_t[size_t(rt) * a.cols + c] = b.scale;
      }
      __syncthreads();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 w = *reinterpret_cast<const float4*>(&s_inv[l * 8 + 4 * h]);
        col_inv[4 * h] = w.x; col_inv[4 * h + 1] = w.y;
        col_inv[4 * h + 2] = w.z; col_inv[4 * h + 3] = w.w;
      }
    }
  }
  if constexpr (SUMS) {  // the bias gradient of the linear backward
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float2 s = v[0].pair(j);
#pragma unroll
      for (int i = 1; i < 8; ++i) s = __fadd2_rn(s, v[i].pair(j));
      s.x += __shfl_xor_sync(0xFFFFFFFFu, s.x, 16);
      s.y += __shfl_xor_sync(0xFFFFFFFFu, s.y, 16);
      if (half == 0) *reinterpret_cast<float2*>(&s_sum[warp][l * 8 + 2 * j]) = s;
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

  // Values behind the last row or column are 0 and give the zero code, which fills the
  // pitch; in a block of NaN scale 0 * inv is NaN, and they are set to 0 again.
  if constexpr (ROWS) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = WHOLE ? row_inv : __shfl_sync(0xFFFFFFFFu, row_inv, 2 * i, 16);
      uint2 w;
      uint32_t* wp = &w.x;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float2 p = __fmul2_rn(v[i].pair(2 * h), make_float2(s, s));
        float2 q = __fmul2_rn(v[i].pair(2 * h + 1), make_float2(s, s));
        if (!VEC) {
          const int left = a.cols - c0 - 4 * h;
          if (left < 1) p.x = 0.f;
          if (left < 2) p.y = 0.f;
          if (left < 3) q.x = 0.f;
          if (left < 4) q.y = 0.f;
        }
        wp[h] = e4m3x4(p.x, p.y, q.x, q.y);
      }
      if (VEC && c0 >= a.cols) w = make_uint2(0, 0);
      if (r0 + i < a.rows && c0 < a.pitch &&
          in_range_of(a.error_word, size_t(r0 + i) * a.pitch + c0, 8,
                      size_t(a.rows) * a.pitch))
        *reinterpret_cast<uint2*>(a.q + size_t(r0 + i) * a.pitch + c0) = w;
    }
  }
  if constexpr (TRANS) {
    const int u = warp * 2 + half;  // the patch's 8-byte unit of a column
    const bool ragged = r0 + 8 > a.rows;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 s = make_float2(col_inv[2 * j], col_inv[2 * j + 1]);
      float2 t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        t[i] = __fmul2_rn(v[i].pair(j), s);
        if (ragged && r0 + i >= a.rows) t[i] = make_float2(0.f, 0.f);
      }
      const uint2 p = make_uint2(e4m3x4(t[0].x, t[1].x, t[2].x, t[3].x),
                                 e4m3x4(t[4].x, t[5].x, t[6].x, t[7].x));
      const uint2 q = make_uint2(e4m3x4(t[0].y, t[1].y, t[2].y, t[3].y),
                                 e4m3x4(t[4].y, t[5].y, t[6].y, t[7].y));
      *reinterpret_cast<uint2*>(&s_t[(l * 8 + 2 * j) * kFp8Block + ((u ^ l) << 3)]) = p;
      *reinterpret_cast<uint2*>(&s_t[(l * 8 + 2 * j + 1) * kFp8Block + ((u ^ l) << 3)]) = q;
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
  chain_wait();
  chain_release();
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
