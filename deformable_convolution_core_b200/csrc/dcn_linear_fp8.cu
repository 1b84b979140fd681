// C ABI of the e4m3 quantiser and linear layer: argument validation, the plan of
// a product (kernel, column tile, K splits), launches.  The contract is in
// include/dcn_core.h.
#define DCN_ERROR_WORD_BY_POINTER
#include "dcn_core.h"

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdlib>
#include <cstring>

#include "dcn_chain.cuh"
#include "dcn_fp8.cuh"
#include "dcn_host.h"
#include "dcn_linear_fp8.cuh"
#include "dcn_quantize.cuh"

namespace dcn {
namespace {

int blocks_of(int n) { return int((int64_t(n) + kFp8Block - 1) / kFp8Block); }
int64_t pitch_of(int cols) { return (int64_t(cols) + 15) / 16 * 16; }
size_t round16(size_t n) { return (n + 15) / 16 * 16; }

// Extents up to here: an index may run a tile, or a few K blocks of the row kernel's
// look-ahead, behind the last row or column without leaving 31 bits.
constexpr int kMaxExtent = INT_MAX - 65535;

bool valid_dtype(dcn_dtype d) { return d == DCN_F32 || d == DCN_BF16 || d == DCN_F16; }

dcn_status launched() { return cudaGetLastError() == cudaSuccess ? DCN_OK : DCN_ERR_CUDA; }

// ---------------------------------------------------------------------------
// Quantiser
// ---------------------------------------------------------------------------
template <typename T, bool VEC, bool WHOLE, bool ROWS, bool TRANS>
void launch_quantize(const QuantArgs& a, unsigned grid, cudaStream_t stream) {
  if constexpr (!WHOLE) {
    if (a.col_sums) {
      dcn_quantize_kernel<T, VEC, false, ROWS, TRANS, true><<<grid, kQuantThreads, 0, stream>>>(a);
      return;
    }
  }
  if constexpr (ROWS || TRANS)
    dcn_quantize_kernel<T, VEC, WHOLE, ROWS, TRANS, false><<<grid, kQuantThreads, 0, stream>>>(a);
}

template <typename T, bool VEC, bool WHOLE>
void launch_quantize(const QuantArgs& a, unsigned grid, cudaStream_t stream) {
  const bool rows = a.q != nullptr, trans = a.q_t != nullptr;
  if (rows && trans) launch_quantize<T, VEC, WHOLE, true, true>(a, grid, stream);
  else if (rows) launch_quantize<T, VEC, WHOLE, true, false>(a, grid, stream);
  else if (trans) launch_quantize<T, VEC, WHOLE, false, true>(a, grid, stream);
  else launch_quantize<T, VEC, WHOLE, false, false>(a, grid, stream);  // column sums alone
}

dcn_status quantize(const void* x, dcn_dtype dtype, int rows, int cols, int block_rows, void* q,
                    float* scales, void* q_t, float* scales_t, float* col_sums,
                    unsigned int* error_word, cudaStream_t stream) {
  QuantArgs a;
  a.x = x;
  a.rows = rows;
  a.cols = cols;
  a.pitch = int(pitch_of(cols));
  a.pitch_t = int(pitch_of(rows));
  a.col_tiles = blocks_of(cols);
  a.row_tiles = blocks_of(rows);
  a.q = static_cast<uint8_t*>(q);
  a.scales = scales;
  a.q_t = static_cast<uint8_t*>(q_t);
  a.scales_t = scales_t;
  a.col_sums = col_sums;
  a.error_word = error_word;
  const int64_t tiles = int64_t(a.col_tiles) * a.row_tiles;
  if (tiles > INT_MAX) return DCN_ERR_UNSUPPORTED;
  return with_storage(dtype, [&](auto tag) {
    using T = decltype(tag);
    const bool vec = cols % 8 == 0;
    if (vec && block_rows == 1) launch_quantize<T, true, false>(a, unsigned(tiles), stream);
    else if (vec) launch_quantize<T, true, true>(a, unsigned(tiles), stream);
    else if (block_rows == 1) launch_quantize<T, false, false>(a, unsigned(tiles), stream);
    else launch_quantize<T, false, true>(a, unsigned(tiles), stream);
    return launched();
  });
}

// ---------------------------------------------------------------------------
// Matrix product
// ---------------------------------------------------------------------------
constexpr int kRowsKernelMax = 8;   // rows up to which the weight-streaming kernel is used
constexpr int kMinSplitBlocks = 4;  // K blocks a split has at least
constexpr int kMaxSplits = 32;

struct LinearPlan {
  bool rows;  // the weight-streaming kernel
  int bn, m_tiles, n_tiles, k_blocks, splits, kb_per;
  int part_pitch;  // row pitch of the partial products (values)
};

// What an item costs, in cycles: a K block, and the rest of a tile.  Measured at 18944 x
// 2048 outputs (148 CTAs): K from 2560 to 5120 adds 1100 cycles a block of a 256-column
// tile and 720 of a 128-column one.
struct TileCost {
  int bn, block, tile;
};
constexpr TileCost kTileCosts[2] = {{256, 1100, 2600}, {128, 720, 1500}};
constexpr double kJoinBytesPerCycle = 3000.0, kJoinCycles = 6000.0;  // HBM; a second launch

// The column tile and the number of K splits whose rounds of items over the SMs cost
// least.  Splits pay where there are few tiles and a long inner length (a weight
// gradient): 2560 x 640 over 36864 takes 60 or 100 tiles of 288 blocks on 148 SMs.
LinearPlan linear_plan(int M, int K, int N, bool row_scales, int sms) {
  LinearPlan p;
  p.k_blocks = blocks_of(K);
  p.rows = !row_scales && M <= kRowsKernelMax;
  p.m_tiles = blocks_of(M);
  p.part_pitch = int((int64_t(N) + 3) / 4 * 4);
  if (p.rows) {  // no tiles, no splits
    p.bn = p.n_tiles = 0;
    p.splits = 1;
    p.kb_per = p.k_blocks;
    return p;
  }
  double best = 0;
  for (const TileCost& c : kTileCosts) {
    if (c.bn > 128 && N <= 128) continue;
    const int64_t n_tiles = (int64_t(N) + c.bn - 1) / c.bn;
    const int64_t tiles = int64_t(p.m_tiles) * n_tiles;
    const int most = int(std::min<int64_t>(std::max(1, p.k_blocks / kMinSplitBlocks), kMaxSplits));
    for (int want = 1; want <= most; ++want) {
      const int kb_per = (p.k_blocks + want - 1) / want;
      const int splits = (p.k_blocks + kb_per - 1) / kb_per;
      const double rounds = double((tiles * splits + sms - 1) / sms);
      double cost = rounds * (double(kb_per) * c.block + c.tile);
      if (splits > 1)
        cost += kJoinCycles + double(splits) * M * double(p.part_pitch) * 8 / kJoinBytesPerCycle;
      if (best == 0 || cost < best) {
        best = cost;
        p.bn = c.bn;
        p.n_tiles = int(n_tiles);
        p.splits = splits;
        p.kb_per = kb_per;
      }
      if (tiles * splits >= 4 * int64_t(sms)) break;  // more splits only add to the join
    }
  }
  return p;
}

size_t plan_workspace(const LinearPlan& p, int M) {
  return p.splits > 1 ? size_t(p.splits) * size_t(M) * size_t(p.part_pitch) * sizeof(float) : 0;
}

// Whether a plan's kernel can run: known before anything is enqueued.
bool plan_runs(const LinearPlan& p, const DeviceInfo& dev) {
  return p.rows ||
         (tensor_map_encoder() != nullptr &&
          size_t(dev.smem_optin) >= std::max(LfShape<128>::kSmemBytes, LfShape<256>::kSmemBytes) &&
          int64_t(p.m_tiles) * p.n_tiles * p.splits <= kMaxExtent);
}

// 2-D map of e4m3 codes (inner: values of a row) with a (128, rows) box, 128-byte swizzle.
dcn_status codes_map(CUtensorMap* map, const void* base, int inner, int64_t pitch, int outer,
                     int rows) {
  const cuuint64_t dims[2] = {cuuint64_t(inner), cuuint64_t(outer)};
  const cuuint64_t strides[1] = {cuuint64_t(pitch)};
  const cuuint32_t box[2] = {cuuint32_t(kLfBK), cuuint32_t(rows)};
  const cuuint32_t estr[2] = {1u, 1u};
  const CUresult cr = tensor_map_encoder()(
      map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
      CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return cr == CUDA_SUCCESS ? DCN_OK : DCN_ERR_UNSUPPORTED;
}

// 3-D map (columns, rows, splits) of the output; the box is what an epilogue warp
// stores at once: 32 rows of a quarter of the column tile, 128 bytes at most.
dcn_status out_map(CUtensorMap* map, void* base, dcn_dtype dtype, int N, int pitch, int M,
                   int splits, int bn) {
  const int e = esize(dtype), width = std::min(128 / e, bn / 4);
  const cuuint64_t dims[3] = {cuuint64_t(N), cuuint64_t(M), cuuint64_t(splits)};
  const cuuint64_t strides[2] = {cuuint64_t(pitch) * e, cuuint64_t(pitch) * e * cuuint64_t(M)};
  const cuuint32_t box[3] = {cuuint32_t(width), 32u, 1u};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  const CUresult cr = tensor_map_encoder()(
      map,
      dtype == DCN_BF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
      : dtype == DCN_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
      3, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
      width * e == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
      CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return cr == CUDA_SUCCESS ? DCN_OK : DCN_ERR_UNSUPPORTED;
}

template <typename T, int BN, bool ROWB>
dcn_status launch_linear(const CUtensorMap& amap, const CUtensorMap& bmap, const CUtensorMap& omap,
                         LinearArgs args, int sms, bool follows, cudaStream_t stream) {
  auto k = dcn_linear_fp8_kernel<T, BN, ROWB>;
  constexpr size_t smem = LfShape<BN>::kSmemBytes;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) !=
      cudaSuccess)
    return DCN_ERR_CUDA;
  const int grid = std::min(args.items, sms);
  args.step_n = grid % args.n_tiles;
  args.step_m = grid / args.n_tiles;
  return launch_kernel(k, follows, dim3(unsigned(grid)), kLfThreads, smem, stream, amap, bmap, omap,
                       args);
}

// out (M, N) = A (M, K) B (N, K)^T with the blocks' scales, + bias.  follows: another kernel
// of the call is before it on the stream.
dcn_status linear(const void* a, const float* sa, int M, int K, const void* b, const float* sb,
                  bool row_scales, int N, const float* bias, void* out, dcn_dtype out_dtype,
                  void* workspace, size_t workspace_bytes, const DeviceInfo& dev, bool follows,
                  cudaStream_t stream) {
  const LinearPlan p = linear_plan(M, K, N, row_scales, dev.sms);
  const int64_t pitch = pitch_of(K);
  if (p.rows) {
    LinearRowsArgs r;
    r.M = M; r.N = N; r.K = K;
    r.k_blocks = p.k_blocks;
    r.pitch = int(pitch);
    r.n_blocks = blocks_of(N);
    r.wk = 1;  // so many warps a column group that each has one round of blocks
    while (r.wk < kLrWarps && r.wk * kLrAhead < r.k_blocks) r.wk *= 2;
    r.a = static_cast<const uint8_t*>(a);
    r.b = static_cast<const uint8_t*>(b);
    r.sa = sa; r.sb = sb; r.bias = bias; r.out = out;
    r.error_word = dev.error_word;
    return with_storage(out_dtype, [&](auto tag) {
      using T = decltype(tag);
      const int64_t columns = kLrWarps / r.wk * 8;
      const unsigned grid = unsigned((int64_t(N) + columns - 1) / columns);
      return launch_kernel(dcn_linear_fp8_rows_kernel<T>, follows, dim3(grid), kLrThreads, 0, stream, r);
    });
  }
  const size_t need = plan_workspace(p, M);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return DCN_ERR_INVALID_ARG;
  if (!plan_runs(p, dev)) return DCN_ERR_UNSUPPORTED;
  const int64_t items = int64_t(p.m_tiles) * p.n_tiles * p.splits;
  const bool split = p.splits > 1;
  const dcn_dtype kernel_dtype = split ? DCN_F32 : out_dtype;
  LinearArgs g;
  g.M = M; g.N = N; g.K = K;
  g.k_blocks = p.k_blocks;
  g.m_tiles = p.m_tiles; g.n_tiles = p.n_tiles;
  g.splits = p.splits; g.kb_per = p.kb_per;
  g.items = int(items);
  g.n_blocks = blocks_of(N);
  g.sa = sa; g.sb = sb;
  g.bias = split ? nullptr : bias;
  g.out = split ? workspace : out;
  g.out_pitch = split ? p.part_pitch : N;
  g.tma_out = (int64_t(g.out_pitch) * esize(kernel_dtype)) % 16 == 0;
  const char* stall = std::getenv("DCN_CORE_TEST_STALL");
  g.inject_stall = stall != nullptr && std::atoi(stall) == 1;
  g.error_word = dev.error_word;
  CUtensorMap amap, bmap, omap;
  std::memset(&omap, 0, sizeof(omap));
  dcn_status st;
  if ((st = codes_map(&amap, a, K, pitch, M, kLfBM)) != DCN_OK) return st;
  if ((st = codes_map(&bmap, b, K, pitch, N, p.bn)) != DCN_OK) return st;
  if (g.tma_out && (st = out_map(&omap, g.out, kernel_dtype, N, g.out_pitch, M, p.splits, p.bn)) != DCN_OK)
    return st;
  st = with_storage(kernel_dtype, [&](auto tag) {
    using T = decltype(tag);
    if (row_scales)
      return p.bn == 256 ? launch_linear<T, 256, true>(amap, bmap, omap, g, dev.sms, follows, stream)
                         : launch_linear<T, 128, true>(amap, bmap, omap, g, dev.sms, follows, stream);
    return p.bn == 256 ? launch_linear<T, 256, false>(amap, bmap, omap, g, dev.sms, follows, stream)
                       : launch_linear<T, 128, false>(amap, bmap, omap, g, dev.sms, follows, stream);
  });
  if (st != DCN_OK || !split) return st;
  return with_storage(out_dtype, [&](auto tag) {
    using T = decltype(tag);
    const int64_t grid = std::min<int64_t>((int64_t(M) * N + 255) / 256, int64_t(dev.sms) * 16);
    return launch_kernel(dcn_linear_join_kernel<T>, true, dim3(unsigned(grid)), 256, 0, stream,
                         static_cast<const float*>(workspace), p.splits, M, N, p.part_pitch, bias,
                         static_cast<T*>(out));
  });
}

bool valid_sizes(int M, int K, int N) { return M >= 1 && K >= 1 && N >= 1; }
bool supported_sizes(int M, int K, int N) {
  return M <= kMaxExtent && K <= kMaxExtent && N <= kMaxExtent;
}

// Workspace of the backward, in order (each part 16-byte aligned).
struct BackwardLayout {
  size_t q, scales, q_t, scales_t, col_sums, part, bytes;
};

BackwardLayout backward_layout(int M, int K, int N, int sms) {
  BackwardLayout l;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round16(bytes);
    return here;
  };
  l.q = take(size_t(M) * size_t(pitch_of(N)));
  l.scales = take(size_t(blocks_of(N)) * size_t(M) * 4);
  l.q_t = take(size_t(N) * size_t(pitch_of(M)));
  l.scales_t = take(size_t(blocks_of(M)) * size_t(N) * 4);
  l.col_sums = take(size_t(blocks_of(M)) * size_t(N) * 4);
  // the two products run one after the other and share the partial sums' room
  l.part = take(std::max(plan_workspace(linear_plan(M, N, K, false, sms), M),
                         plan_workspace(linear_plan(N, M, K, true, sms), N)));
  l.bytes = at;
  return l;
}

}  // namespace
}  // namespace dcn

using namespace dcn;

extern "C" {

size_t dcn_core_fp8_pitch(int cols) { return cols < 1 ? 0 : size_t(pitch_of(cols)); }

dcn_status dcn_core_quantize_fp8(const void* input, dcn_dtype dtype, int rows, int cols,
                                 int block_rows, void* q, float* scales, void* q_t,
                                 float* scales_t, cudaStream_t stream) {
  if (!input || rows < 1 || cols < 1 || !valid_dtype(dtype)) return DCN_ERR_INVALID_ARG;
  if (block_rows != 1 && block_rows != kFp8Block) return DCN_ERR_INVALID_ARG;
  if ((q == nullptr) != (scales == nullptr) || (q_t == nullptr) != (scales_t == nullptr) ||
      (!q && !q_t))
    return DCN_ERR_INVALID_ARG;
  if (rows > kMaxExtent || cols > kMaxExtent) return DCN_ERR_UNSUPPORTED;
  if (!aligned(input, 16) || !aligned(q, 16) || !aligned(q_t, 16) || !aligned(scales, 4) ||
      !aligned(scales_t, 4))
    return DCN_ERR_UNSUPPORTED;
  DeviceInfo dev;
  if (device_info(&dev) != DCN_OK) return DCN_ERR_CUDA;
  return quantize(input, dtype, rows, cols, block_rows, q, scales, q_t, scales_t, nullptr,
                  dev.error_word, stream);
}

size_t dcn_core_linear_fp8_workspace(int M, int K, int Nout) {
  DeviceInfo dev;
  if (!valid_sizes(M, K, Nout) || !supported_sizes(M, K, Nout) || device_info(&dev) != DCN_OK)
    return 0;
  return plan_workspace(linear_plan(M, K, Nout, false, dev.sms), M);
}

dcn_status dcn_core_linear_fp8(const void* input, const float* input_scales, int M, int K,
                               const void* weight, const float* weight_scales, int Nout,
                               const float* bias, void* output, dcn_dtype out_dtype,
                               void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!input || !input_scales || !weight || !weight_scales || !output ||
      !valid_sizes(M, K, Nout) || !valid_dtype(out_dtype))
    return DCN_ERR_INVALID_ARG;
  if (!supported_sizes(M, K, Nout)) return DCN_ERR_UNSUPPORTED;
  if (!aligned(input, 16) || !aligned(weight, 16) || !aligned(output, 16) ||
      !aligned(workspace, 16) || !aligned(input_scales, 4) || !aligned(weight_scales, 4) ||
      !aligned(bias, 4))
    return DCN_ERR_UNSUPPORTED;
  DeviceInfo dev;
  if (device_info(&dev) != DCN_OK) return DCN_ERR_CUDA;
  return linear(input, input_scales, M, K, weight, weight_scales, false, Nout, bias, output,
                out_dtype, workspace, workspace_bytes, dev, false, stream);
}

size_t dcn_core_linear_fp8_backward_workspace(int M, int K, int Nout) {
  DeviceInfo dev;
  if (!valid_sizes(M, K, Nout) || !supported_sizes(M, K, Nout) || device_info(&dev) != DCN_OK)
    return 0;
  return backward_layout(M, K, Nout, dev.sms).bytes;
}

dcn_status dcn_core_linear_fp8_backward(const void* grad_out, dcn_dtype dtype, int M, int K,
                                        int Nout, const void* weight_t,
                                        const float* weight_t_scales, const void* input_t,
                                        const float* input_t_scales, void* grad_input,
                                        float* grad_weight, float* grad_bias, void* workspace,
                                        size_t workspace_bytes, cudaStream_t stream) {
  if (!grad_out || !valid_sizes(M, K, Nout) || !valid_dtype(dtype) || !workspace)
    return DCN_ERR_INVALID_ARG;
  if (!grad_input && !grad_weight && !grad_bias) return DCN_ERR_INVALID_ARG;
  if (grad_input && (!weight_t || !weight_t_scales)) return DCN_ERR_INVALID_ARG;
  if (grad_weight && (!input_t || !input_t_scales)) return DCN_ERR_INVALID_ARG;
  if (!supported_sizes(M, K, Nout)) return DCN_ERR_UNSUPPORTED;
  if (!aligned(grad_out, 16) || !aligned(weight_t, 16) || !aligned(input_t, 16) ||
      !aligned(grad_input, 16) || !aligned(grad_weight, 16) || !aligned(workspace, 16) ||
      !aligned(weight_t_scales, 4) || !aligned(input_t_scales, 4) || !aligned(grad_bias, 4))
    return DCN_ERR_UNSUPPORTED;
  DeviceInfo dev;
  if (device_info(&dev) != DCN_OK) return DCN_ERR_CUDA;
  const BackwardLayout l = backward_layout(M, K, Nout, dev.sms);
  if (workspace_bytes < l.bytes) return DCN_ERR_INVALID_ARG;
  if ((grad_input && !plan_runs(linear_plan(M, Nout, K, false, dev.sms), dev)) ||
      (grad_weight && !plan_runs(linear_plan(Nout, M, K, true, dev.sms), dev)) ||
      int64_t(blocks_of(M)) * blocks_of(Nout) > INT_MAX)
    return DCN_ERR_UNSUPPORTED;
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  float* scales = reinterpret_cast<float*>(ws + l.scales);
  float* scales_t = reinterpret_cast<float*>(ws + l.scales_t);
  float* col_sums = reinterpret_cast<float*>(ws + l.col_sums);
  const size_t part_bytes = l.bytes - l.part;
  dcn_status st = quantize(grad_out, dtype, M, Nout, 1, grad_input ? ws + l.q : nullptr,
                           grad_input ? scales : nullptr, grad_weight ? ws + l.q_t : nullptr,
                           grad_weight ? scales_t : nullptr, grad_bias ? col_sums : nullptr,
                           dev.error_word, stream);
  if (st != DCN_OK) return st;
  if (grad_bias &&
      (st = launch_kernel(dcn_column_sum_kernel, true, dim3(unsigned((int64_t(Nout) + 31) / 32)), 256,
                          0, stream, col_sums, blocks_of(M), Nout, grad_bias)) != DCN_OK)
    return st;
  if (grad_input &&
      (st = linear(ws + l.q, scales, M, Nout, weight_t, weight_t_scales, false, K, nullptr,
                   grad_input, dtype, ws + l.part, part_bytes, dev, true, stream)) != DCN_OK)
    return st;
  if (grad_weight &&
      (st = linear(ws + l.q_t, scales_t, Nout, M, input_t, input_t_scales, true, K, nullptr,
                   grad_weight, DCN_F32, ws + l.part, part_bytes, dev, true, stream)) != DCN_OK)
    return st;
  return DCN_OK;
}

}  // extern "C"
