// Shared pieces of the kernels that stage the input in shared memory by TMA
// (sm_100a): the work-item decomposition and the box geometry.
//
// A persistent CTA walks work items (image n, output tile, group g).  For
// each item one TMA tensor copy brings the group's Cg channels of the input
// box the tile can reach into shared memory, zero filled outside the image,
// which is exactly the operator's zero padding.  Every mbarrier wait is
// bounded; on expiry the kernel sets the device error word, waits (bounded)
// for its own copies in flight and returns.
#pragma once

#include <cuda.h>

#include "dcn_common.cuh"
#include "dcn_ptx.cuh"
#include "dcn_tile.cuh"

namespace dcn {

constexpr int kTiledWarps = 15;  // consumer warps: with the producer, 4 warps per SM sub-partition
constexpr int kTiledThreads = (kTiledWarps + 1) * 32;  // + one TMA producer warp
constexpr int kTiledBatch = 32;                       // units per warp batch
constexpr int kTiledMaxTaps = 9;  // the tiled kernels serve 3x3 windows (9 or 8 taps)
constexpr int kTiledMaxBufs = 8;  // input boxes in flight, at most

struct TiledParams {
  int N, H, W, G, Cg, C, stride, pad, dil, Ho, Wo;  // stride/pad/dil: height axis
  int stride_w, pad_w, dil_w;                       // width axis
  float sigma;
  int TH, TW, nTY, nTX, halo, BH, BW;  // BW: the box row pitch in pixels (all of it is loaded)
  int clamp_box;       // 1: box origins are clamped to the image and its one-pixel zero ring
  int nbuf;            // input boxes in flight (2 .. kTiledMaxBufs)
  int items;           // N * nTY * nTX * G
  int inject_stall;    // test knob: 1 = never load the first item's box, so the
                       // bounded waits expire and the error path runs
  int batches;         // warp batches per item: ceil(TH * TW / kTiledBatch)
  uint32_t box_bytes;  // BH * BW * Cg * sizeof(T)
  uint32_t box_stride; // box_bytes rounded up to 1024
  FastDiv fd_G, fd_nTX, fd_tiles, fd_TW;
};

__device__ __forceinline__ void tma_load_box(void* dst, const CUtensorMap* map, uint64_t* bar,
                                             int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
      "r"(smem_addr(bar))
      : "memory");
}

// Item -> (n, ho0, wo0, g); g is the fastest index, so consecutive items of a
// CTA reuse one input neighbourhood (different channels) and one run of
// offset/mask rows.
struct ItemCoord {
  int n, ho0, wo0, g;
};

__device__ __forceinline__ ItemCoord item_coord(const TiledParams& t, int item) {
  ItemCoord c;
  const uint32_t tile = fdiv(uint32_t(item), t.fd_G);
  c.g = item - int(tile) * t.G;
  const uint32_t n = fdiv(tile, t.fd_tiles);
  const uint32_t rem = tile - n * uint32_t(t.nTY * t.nTX);
  const uint32_t ty = fdiv(rem, t.fd_nTX);
  c.n = int(n);
  c.ho0 = int(ty) * t.TH;
  c.wo0 = int(rem - ty * uint32_t(t.nTX)) * t.TW;
  return c;
}

// First input row (or column) of an item's box.  Unclamped it is the tile's
// first sampling row less the halo.  With clamp_box the box is slid to stay
// within the rows that can matter, [-1, extent]: a footprint has rows y0 and
// y0 + 1 with -1 <= y0 < extent for any sample that contributes, and the
// image's zero ring (row -1 or row `extent`) is read as TMA zero fill.  A box
// taller than extent + 2 starts at -1 and covers every such row.
__host__ __device__ __forceinline__ int box_origin(int first, int box, int extent, bool clamp) {
  if (!clamp) return first;
  const int hi = extent + 1 - box;  // last origin whose box still ends at row `extent`
  return first < -1 ? -1 : (first > hi ? (hi < -1 ? -1 : hi) : first);
}

template <typename T>
struct TiledIO;
template <>
struct TiledIO<float> {
  static constexpr int kEpc = 4;  // channels per 16-byte piece
  using Pair = float2;
  using One = float;
  __device__ __forceinline__ static Pair ld_pair(const void* base, size_t i) {
    return __ldg(reinterpret_cast<const float2*>(base) + i);
  }
  __device__ __forceinline__ static One ld_one(const void* base, size_t i) {
    return __ldg(reinterpret_cast<const float*>(base) + i);
  }
  __device__ __forceinline__ static float2 pair(Pair p) { return p; }
  __device__ __forceinline__ static float one(One v) { return v; }
  // acc += w * (the piece's 4 channels), as two packed fp32x2 FMAs.
  __device__ __forceinline__ static void fma16(float2* acc, float2 w, const uint4& v) {
    acc[0] = __ffma2_rn(make_float2(__uint_as_float(v.x), __uint_as_float(v.y)), w, acc[0]);
    acc[1] = __ffma2_rn(make_float2(__uint_as_float(v.z), __uint_as_float(v.w)), w, acc[1]);
  }
};
template <>
struct TiledIO<__nv_bfloat16> {
  static constexpr int kEpc = 8;
  using Pair = uint32_t;
  using One = unsigned short;
  __device__ __forceinline__ static Pair ld_pair(const void* base, size_t i) {
    return __ldg(reinterpret_cast<const unsigned int*>(base) + i);
  }
  __device__ __forceinline__ static One ld_one(const void* base, size_t i) {
    return __ldg(reinterpret_cast<const unsigned short*>(base) + i);
  }
  __device__ __forceinline__ static float2 pair(Pair p) {
    return make_float2(bf16lo_to_f32(p), bf16hi_to_f32(p));
  }
  __device__ __forceinline__ static float one(One v) { return __uint_as_float(uint32_t(v) << 16); }
  // acc += w * (the piece's 8 channels, widened), as four packed fp32x2 FMAs.
  __device__ __forceinline__ static void fma16(float2* acc, float2 w, const uint4& v) {
    acc[0] = __ffma2_rn(make_float2(bf16lo_to_f32(v.x), bf16hi_to_f32(v.x)), w, acc[0]);
    acc[1] = __ffma2_rn(make_float2(bf16lo_to_f32(v.y), bf16hi_to_f32(v.y)), w, acc[1]);
    acc[2] = __ffma2_rn(make_float2(bf16lo_to_f32(v.z), bf16hi_to_f32(v.z)), w, acc[2]);
    acc[3] = __ffma2_rn(make_float2(bf16lo_to_f32(v.w), bf16hi_to_f32(v.w)), w, acc[3]);
  }
};

template <>
struct TiledIO<__half> {
  static constexpr int kEpc = 8;
  using Pair = uint32_t;
  using One = unsigned short;
  __device__ __forceinline__ static Pair ld_pair(const void* base, size_t i) {
    return __ldg(reinterpret_cast<const unsigned int*>(base) + i);
  }
  __device__ __forceinline__ static One ld_one(const void* base, size_t i) {
    return __ldg(reinterpret_cast<const unsigned short*>(base) + i);
  }
  __device__ __forceinline__ static float2 pair(Pair p) { return f16x2_to_f32x2(p); }
  __device__ __forceinline__ static float one(One v) { return __half2float(__ushort_as_half(v)); }
  __device__ __forceinline__ static void fma16(float2* acc, float2 w, const uint4& v) {
    acc[0] = __ffma2_rn(f16x2_to_f32x2(v.x), w, acc[0]);
    acc[1] = __ffma2_rn(f16x2_to_f32x2(v.y), w, acc[1]);
    acc[2] = __ffma2_rn(f16x2_to_f32x2(v.z), w, acc[2]);
    acc[3] = __ffma2_rn(f16x2_to_f32x2(v.w), w, acc[3]);
  }
};

// Output of four fp32 values in storage type T: 16 bytes (fp32) or 8 bytes.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  return pack_bf16x2(lo, hi);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  return pack_f16x2(lo, hi);
}

}  // namespace dcn
