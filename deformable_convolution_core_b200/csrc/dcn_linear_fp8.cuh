// Linear layer on block-scaled e4m3 operands (sm_100a tensor cores).
//
//   out[m, n] = sum_b sa[b, m] * sb[b, n] * (sum_{k in block b} A[m, k] * B[n, k]) + bias[n]
//
// The scales change every 128 products, and they are fp32 numbers, so a block's
// products are summed on the tensor cores into a fresh accumulator in tensor
// memory, and the blocks are added in fp32 registers with one packed FMA for two
// values.  An e4m3 product has at most 8 significant bits, so a block's 128
// products lose nothing but the rounding of their fp32 sum.
//
// Kernel: persistent CTAs over (128-row, BN-column, K split) items, columns
// fastest (the row tile of A stays in L2 while B's column tiles pass).  Warp 0
// streams 128-byte K blocks of A and B into a shared-memory ring by TMA (128-byte
// swizzle); one thread each of warps 1 and 3 issues tcgen05.mma (kind::f8f6f4, K = 32)
// for every other block, into every other one of 512 / BN accumulators (issuing a
// block's four MMAs takes as long as they run, about 550 cycles, and the waits before
// them another 350, which the other thread's MMAs now fill); warp 2 brings the blocks'
// scales into a ring of their own with asynchronous copies; sixteen epilogue warps
// (four lane quarters x four column quarters) read each accumulator back, scale and
// add it, and at an item's end store it by TMA from a swizzled 4 KB buffer each.  The
// sums of a 128 x 256 tile take 64 of the 96 registers of every epilogue thread, and
// four epilogue warps a scheduler hide each other's tensor-memory reads.  (Eight
// warps with 128 sums a thread spill, with or without registers moved to them.)
// What bounds it: a K block's round takes about 1100 cycles, in which its MMAs, its
// scaled additions and the two handshakes between them overlap only in part.  Each part
// alone: MMAs and handshakes 690, loads and additions 730.  9216 x 1280 x 5120 takes
// 75 us (1.6 PFLOP/s) in a short run and 88 under the power cap, 589,824 x 160 x 640,
// whose bytes need 130, 190 and 230.  Weight gradients, whose columns have a scale each,
// need a second packed multiply: 1570 cycles a block.
// Every mbarrier wait is bounded; on expiry the kernel sets the error word, stops
// issuing work, waits (bounded) for what is in flight, frees its tensor memory and
// returns.
#pragma once

#include <cuda.h>

#include "dcn_chain.cuh"
#include "dcn_fp8.cuh"
#include "dcn_ptx.cuh"

namespace dcn {

constexpr int kLfBM = 128;
constexpr int kLfBK = 128;  // values and bytes of a K block: one scale, one swizzle atom
constexpr int kLfFrontWarps = 4;  // TMA, MMA, scales, MMA
constexpr int kLfEpiWarps = 16;
constexpr int kLfThreads = (kLfFrontWarps + kLfEpiWarps) * 32;
constexpr uint32_t kLfTmemCols = 512;
constexpr int kLfStoreBytes = 32 * 128;  // an epilogue warp's buffer: 32 rows of 128 bytes
constexpr int kLfBiasBytes = 64 * 4;     // and its columns' bias
constexpr int kLfScaleSlots = 4;         // K blocks whose scales are in flight

template <int BN>
struct LfShape {
  static constexpr int kStages = BN == 256 ? 3 : 4;
  static constexpr int kAccs = int(kLfTmemCols) / BN;
  // The MMA threads' order of waits needs an accumulator's last block to be no older
  // than a stage's, or both rings to be dealt out evenly to the two threads.
  static_assert(kAccs % 2 == 0 && (kAccs <= kStages || kStages % 2 == 0), "rings of the MMA threads");
  static constexpr uint32_t kStageBytes = uint32_t(kLfBM + BN) * kLfBK;
  static constexpr int kScaleFloats = kLfBM + BN;  // a slot: row scales, column scales
  static constexpr size_t kSmemBytes = 1024 /* alignment slack */ + size_t(kStages) * kStageBytes +
                                       size_t(kLfEpiWarps) * (kLfStoreBytes + kLfBiasBytes) +
                                       size_t(kLfScaleSlots) * kScaleFloats * 4 +
                                       512 /* barriers, TMEM address */;
};

struct LinearArgs {
  int M, N, K;
  int k_blocks;            // ceil(K / 128)
  int m_tiles, n_tiles;
  int splits, kb_per;      // K splits and blocks of each (the last may have fewer)
  int items;               // m_tiles * n_tiles * splits
  int step_n, step_m;      // CTAs % n_tiles and CTAs / n_tiles: from one item of a CTA to its next
  int n_blocks;            // ceil(N / 128): pitch of sb with blocks of 128 rows
  const float* sa;         // (k_blocks, M)
  const float* sb;         // (k_blocks, n_blocks), or (k_blocks, N) with a scale a row
  const float* bias;       // N values, or null
  void* out;               // (splits, M, out_pitch) values of the output type
  int out_pitch;
  int tma_out;             // 1: rows are multiples of 16 bytes, stored by TMA
  int inject_stall;        // test knob: 1 = never load a CTA's first stage, so the waits expire
  unsigned int* error_word;
};

// Instruction descriptor of kind::f8f6f4: e4m3 A and B (K-major), fp32 D, M x N.
__device__ __forceinline__ uint32_t umma_idesc_e4m3_f32(int M, int N) {
  return (1u << 4)                     // D format: fp32 (A and B format 0: e4m3)
         | (uint32_t(N >> 3) << 17)    // N / 8
         | (uint32_t(M >> 4) << 24);   // M / 16
}

__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 16 consecutive fp32 columns of this warp's TMEM lanes, asynchronously: the values
// are there after tmem_wait16 of the same registers.
__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Waits for the thread's TMEM loads; the registers pass through, so that no use of
// them can move in front of the wait.
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// A ring of `N` barriers as one role walks it: the current slot and its phase, without
// a division a step (the roles are single threads or warps whose instructions stand
// in the accumulators' round trip).
template <int N>
struct RingPos {
  uint32_t slot = 0, phase;
  __device__ __forceinline__ explicit RingPos(uint32_t first_phase) : phase(first_phase) {}
  __device__ __forceinline__ void next() {
    if (++slot == uint32_t(N)) {
      slot = 0;
      phase ^= 1;
    }
  }
};

__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

// The part of a wait that did not succeed at once: gives up after 2^31 cycles (about
// a second), or soon after another role has (abort_flag).
__device__ __forceinline__ bool mbar_wait_long(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  const long long t0 = clock64();
#pragma unroll 1
  for (uint32_t i = 1; i < (1u << 28); ++i) {
    if (mbar_try(bar, parity)) return true;
    if ((i & 63u) == 0 && (*abort_flag || clock64() - t0 > (1ll << 31))) return false;
  }
  return false;
}

// Bounded wait of this kernel's roles.
__device__ __forceinline__ bool mbar_wait_watch(uint32_t bar, uint32_t parity,
                                                volatile int* abort_flag) {
  if (mbar_try(bar, parity)) return true;
  return mbar_wait_long(bar, parity, abort_flag);
}

__device__ __forceinline__ void mbar_arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void umma_commit_at(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
               : "memory");
}

// An asynchronous 4-byte copy to shared memory; zero where `in` is false.
__device__ __forceinline__ void cp_async4(float* dst, const float* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(dst)), "l"(src),
               "r"(in ? 4 : 0)
               : "memory");
}
// One arrival on `bar` when all copies of this thread so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}

// Stores a box from shared memory; rows and columns outside the tensor are left out.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int c0,
                                             int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_addr(src)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// The thread's stores have been read from shared memory (read0), or are complete.
__device__ __forceinline__ void bulk_wait_read0() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait0() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// A CTA's items blockIdx.x, blockIdx.x + gridDim.x, ...: column tile fastest, then
// row tile, then K split.  Moving on adds the grid's steps; no division after the first.
template <int BN>
struct LinearItems {
  int item, nt, mt, split;
  int m0, n0, kb0, kb1;
  __device__ __forceinline__ explicit LinearItems(const LinearArgs& a) {
    item = int(blockIdx.x);
    const int r = item / a.n_tiles;
    nt = item - r * a.n_tiles;
    split = r / a.m_tiles;
    mt = r - split * a.m_tiles;
    place(a);
  }
  __device__ __forceinline__ bool valid(const LinearArgs& a) const { return item < a.items; }
  __device__ __forceinline__ void next(const LinearArgs& a) {
    item += int(gridDim.x);
    nt += a.step_n;
    mt += a.step_m;
    if (nt >= a.n_tiles) {
      nt -= a.n_tiles;
      ++mt;
    }
    while (mt >= a.m_tiles) {
      mt -= a.m_tiles;
      ++split;
    }
    place(a);
  }
  __device__ __forceinline__ void place(const LinearArgs& a) {
    m0 = mt * kLfBM;
    n0 = nt * BN;
    kb0 = split * a.kb_per;
    kb1 = min(kb0 + a.kb_per, a.k_blocks);
  }
};

// T: output type.  BN: column tile.  ROWB: sb holds a scale for each row of B (the
// weight gradient), else one for each 128 rows.
template <typename T, int BN, bool ROWB>
__global__ void __launch_bounds__(kLfThreads, 1)
    dcn_linear_fp8_kernel(const __grid_constant__ CUtensorMap amap,
                          const __grid_constant__ CUtensorMap bmap,
                          const __grid_constant__ CUtensorMap omap, const LinearArgs a) {
  using S = LfShape<BN>;
  constexpr int kWide = BN / 4;  // columns of an epilogue warp
  extern __shared__ __align__(1024) unsigned char lf_smem_raw[];
  unsigned char* smem = lf_smem_raw + ((1024u - (smem_addr(lf_smem_raw) & 1023u)) & 1023u);
  unsigned char* stage_a = smem;
  unsigned char* stage_b = smem + size_t(S::kStages) * kLfBM * kLfBK;
  unsigned char* store_buf = smem + size_t(S::kStages) * S::kStageBytes;
  float* bias_buf = reinterpret_cast<float*>(store_buf + kLfEpiWarps * kLfStoreBytes);
  float* scale_ring = bias_buf + kLfEpiWarps * kLfBiasBytes / 4;
  uint64_t* full = reinterpret_cast<uint64_t*>(scale_ring + kLfScaleSlots * S::kScaleFloats);
  uint64_t* empty = full + S::kStages;
  uint64_t* tfull = empty + S::kStages;       // accumulator ready
  uint64_t* tempty = tfull + S::kAccs;    // accumulator read
  uint64_t* sempty = tempty + S::kAccs;       // scales read
  uint64_t* mma_done = sempty + kLfScaleSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 2);
  int* s_abort = reinterpret_cast<int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], 1 + 32);  // the TMA warp's arrival and the scale warp's copies
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kLfScaleSlots; ++s) mbar_init(&sempty[s], kLfEpiWarps);
    for (int b = 0; b < S::kAccs; ++b) {
      // the commit, and an arrival of the issuing thread, which has seen the block's
      // scales land and so hands them on with the accumulator
      mbar_init(&tfull[b], 2);
      mbar_init(&tempty[b], kLfEpiWarps);
    }
    mbar_init(&mma_done[0], 1);
    mbar_init(&mma_done[1], 1);
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(kLfTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  chain_wait();
  chain_release();
  volatile int* abort_flag = s_abort;
  auto give_up = [&]() {
    atomicOr(a.error_word, kErrTimeout);
    *abort_flag = 1;
  };

  const uint32_t full_a = smem_addr(full), empty_a = smem_addr(empty), tfull_a = smem_addr(tfull),
                 tempty_a = smem_addr(tempty), sempty_a = smem_addr(sempty);
  // A wait on the phase before a barrier's first succeeds at once: rings start
  // empty, so whoever fills them starts with phase 1 and whoever drains them with 0.
  if (warp == 0) {
    // ---- TMA producer ----
    if (lane == 0) {
      RingPos<S::kStages> r(1);
      uint32_t issued = 0;
      bool stop = false;
      for (LinearItems<BN> w(a); w.valid(a) && !stop; w.next(a)) {
        for (int kb = w.kb0; kb < w.kb1; ++kb, r.next(), ++issued) {
          if (!mbar_wait_watch(empty_a + 8 * r.slot, r.phase, abort_flag)) {
            give_up();
            stop = true;
            break;
          }
          if (a.inject_stall && issued == 0) continue;  // test knob
          mbar_arrive_expect_tx(&full[r.slot], S::kStageBytes);
          tma_load_2d(stage_a + r.slot * (kLfBM * kLfBK), &amap, &full[r.slot], kb * kLfBK, w.m0);
          tma_load_2d(stage_b + r.slot * (BN * kLfBK), &bmap, &full[r.slot], kb * kLfBK, w.n0);
        }
      }
      // the copies of the last issued stages may still be landing
      for (uint32_t j = issued > uint32_t(S::kStages) ? issued - S::kStages : 0; j < issued; ++j)
        if (!(a.inject_stall && j == 0))
          (void)mbar_wait_bounded(&full[j % S::kStages], (j / S::kStages) & 1);
    }
  } else if (warp == 1 || warp == 3) {
    // ---- MMA issuers: every other K block, one accumulator a block ----
    if (lane == 0) {
      RingPos<S::kStages> r(0);
      RingPos<S::kAccs> t(1);
      const uint64_t a_desc0 = umma_desc_sw128(smem_addr(stage_a));
      const uint64_t b_desc0 = umma_desc_sw128(smem_addr(stage_b));
      bool mine = warp == 1, stop = false;
      for (LinearItems<BN> w(a); w.valid(a) && !stop; w.next(a)) {
        const uint32_t idesc = umma_idesc_e4m3_f32(kLfBM, min(BN, (a.N - w.n0 + 15) / 16 * 16));
        for (int kb = w.kb0; kb < w.kb1; ++kb, r.next(), t.next(), mine = !mine) {
          if (!mine) continue;
          // The accumulator first: once the epilogue, which takes the blocks in order, has
          // read this thread's last one, the block that had this block's stage before,
          // the other thread's perhaps, has long been multiplied.  So the stage's barrier
          // is at this block's phase, and the parity of an older one cannot be taken for it.
          if (!mbar_wait_watch(tempty_a + 8 * t.slot, t.phase, abort_flag) ||
              !mbar_wait_watch(full_a + 8 * r.slot, r.phase, abort_flag)) {
            give_up();
            stop = true;
            break;
          }
          tc_fence_after();
          // 32 bytes of K an instruction (2 units of 16 in a descriptor's address)
          const uint64_t ad = a_desc0 + r.slot * (kLfBM * kLfBK / 16);
          const uint64_t bd = b_desc0 + r.slot * (BN * kLfBK / 16);
          const uint32_t d = tmem_base + t.slot * BN;
          umma_e4m3(d, ad, bd, idesc, 0);
          const int left = a.K - kb * kLfBK;  // bytes behind K are zeros: no need to multiply them
          if (left > 32) umma_e4m3(d, ad + 2, bd + 2, idesc, 1);
          if (left > 64) umma_e4m3(d, ad + 4, bd + 4, idesc, 1);
          if (left > 96) umma_e4m3(d, ad + 6, bd + 6, idesc, 1);
          umma_commit_at(tfull_a + 8 * t.slot);
          mbar_arrive_at(tfull_a + 8 * t.slot);
          umma_commit_at(empty_a + 8 * r.slot);
        }
      }
      // every MMA this thread issued has retired before the accumulators are freed
      umma_commit(&mma_done[warp >> 1]);
      (void)mbar_wait_bounded(&mma_done[warp >> 1], 0);
    }
  } else if (warp == 2) {
    // ---- scales ----
    RingPos<kLfScaleSlots> r(1);
    RingPos<S::kStages> st(1);
    bool stop = false;
    for (LinearItems<BN> w(a); w.valid(a) && !stop; w.next(a)) {
      for (int kb = w.kb0; kb < w.kb1; ++kb, r.next(), st.next()) {
        // a free slot, and the block's stage free too: its barrier's phase is this block's
        if (!mbar_wait_watch(sempty_a + 8 * r.slot, r.phase, abort_flag) ||
            !mbar_wait_watch(empty_a + 8 * st.slot, st.phase, abort_flag)) {
          give_up();
          stop = true;
          break;
        }
        float* slot = scale_ring + r.slot * S::kScaleFloats;
        const float* sa = a.sa + size_t(kb) * a.M;
#pragma unroll
        for (int i = lane; i < kLfBM; i += 32)
          cp_async4(slot + i, w.m0 + i < a.M ? sa + w.m0 + i : sa, w.m0 + i < a.M);
        if constexpr (ROWB) {
          const float* sb = a.sb + size_t(kb) * a.N;
#pragma unroll
          for (int i = lane; i < BN; i += 32)
            cp_async4(slot + kLfBM + i, w.n0 + i < a.N ? sb + w.n0 + i : sb, w.n0 + i < a.N);
        } else if (lane < BN / kFp8Block) {
          const float* sb = a.sb + size_t(kb) * a.n_blocks;
          const int n = w.n0 / kFp8Block + lane;
          cp_async4(slot + kLfBM + lane, n < a.n_blocks ? sb + n : sb, n < a.n_blocks);
        }
        cp_async_arrive(&full[st.slot]);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= kLfFrontWarps) {
    // ---- epilogue warps: TMEM lanes 32 (warp % 4) .. + 31, column quarter h ----
    const int ew = warp - kLfFrontWarps, q = warp & 3, h = ew >> 2;
    unsigned char* buf = store_buf + ew * kLfStoreBytes;
    float* bias_w = bias_buf + ew * kLfBiasBytes / 4;
    const uint32_t tq = tmem_base + (uint32_t(q * 32) << 16) + uint32_t(h * kWide);
    const float* row_scale = scale_ring + q * 32 + lane;
    const float* col_scale = scale_ring + kLfBM + (ROWB ? h * kWide : h * kWide / kFp8Block);
    constexpr int kLanes = kWide / 32;  // columns of a lane when the bias is fetched
    float bias[kLanes];
    LinearItems<BN> w(a);
    auto fetch_bias = [&]() {
      if (a.bias == nullptr || !w.valid(a)) return;
#pragma unroll
      for (int i = 0; i < kLanes; ++i) {
        const int c = w.n0 + h * kWide + i * 32 + lane;
        bias[i] = c < a.N ? __ldg(a.bias + c) : 0.f;
      }
    };
    fetch_bias();
    RingPos<S::kAccs> t(0);
    RingPos<kLfScaleSlots> sr(0);
    bool stop = false;
    while (w.valid(a) && !stop) {
      const int col0 = w.n0 + h * kWide;
      const int cols = min(kWide, a.N - col0);  // columns of this warp inside the tensor
      const int r0 = w.m0 + q * 32, split = w.split;
      const int kbs = w.kb1 - w.kb0;
      // the sums start from the bias, spread over the lanes through shared memory
      float2 acc[kWide / 2];
      if (a.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < kLanes; ++i) bias_w[i * 32 + lane] = bias[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kWide / 4; ++i) {
          const float4 b = *reinterpret_cast<const float4*>(bias_w + 4 * i);
          acc[2 * i] = make_float2(b.x, b.y);
          acc[2 * i + 1] = make_float2(b.z, b.w);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kWide / 2; ++i) acc[i] = make_float2(0.f, 0.f);
      }
      w.next(a);
      fetch_bias();
      if (cols <= 0) {  // a last column tile that ends before this warp's columns
        for (int kb = 0; kb < kbs; ++kb, t.next(), sr.next()) {
          if (!mbar_wait_watch(tfull_a + 8 * t.slot, t.phase, abort_flag)) {
            give_up();
            stop = true;
            break;
          }
          if (lane == 0) {
            mbar_arrive_at(tempty_a + 8 * t.slot);
            mbar_arrive_at(sempty_a + 8 * sr.slot);
          }
        }
        continue;
      }
      for (int kb = 0; kb < kbs; ++kb, t.next(), sr.next()) {
        const float* s_col = col_scale + sr.slot * S::kScaleFloats;
        const uint32_t s_done = sempty_a + 8 * sr.slot;
        if (!mbar_wait_watch(tfull_a + 8 * t.slot, t.phase, abort_flag)) {
          give_up();
          stop = true;
          break;
        }
        tc_fence_after();
        // chunks of 16 columns; the next one's load runs under this one's additions
        // (columns behind the tensor's last are never stored)
        uint32_t v[2][16];
        tmem_ld16_async(tq + t.slot * BN, v[0]);
        float s_row = row_scale[sr.slot * S::kScaleFloats];
        if (!ROWB) s_row *= *s_col;
        const float2 s2 = make_float2(s_row, s_row);
#pragma unroll
        for (int c = 0; c < kWide / 16; ++c) {
          tmem_wait16(v[c & 1]);
          if (c + 1 < kWide / 16) {
            tmem_ld16_async(tq + t.slot * BN + (c + 1) * 16, v[(c + 1) & 1]);
          } else {  // all read: the accumulator may be overwritten
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive_at(tempty_a + 8 * t.slot);
              if (!ROWB) mbar_arrive_at(s_done);
            }
          }
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            float2 sc[2] = {s2, s2};
            if constexpr (ROWB) {  // the same four columns' scales for every lane: one read
              const float4 cs = *reinterpret_cast<const float4*>(s_col + c * 16 + 2 * i);
              sc[0] = __fmul2_rn(s2, make_float2(cs.x, cs.y));
              sc[1] = __fmul2_rn(s2, make_float2(cs.z, cs.w));
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
              acc[c * 8 + i + k] =
                  __ffma2_rn(make_float2(__uint_as_float(v[c & 1][2 * (i + k)]),
                                         __uint_as_float(v[c & 1][2 * (i + k) + 1])),
                             sc[k], acc[c * 8 + i + k]);
          }
        }
        if (ROWB) {
          __syncwarp();
          if (lane == 0) mbar_arrive_at(s_done);
        }
      }
      if (stop) break;
      // ---- the item's output: 32 rows of up to 128 bytes at a time ----
      constexpr int kCols = 128 / int(sizeof(T)) < kWide ? 128 / int(sizeof(T)) : kWide;
      constexpr int kPer = 16 / int(sizeof(T));
      constexpr int kUnits = kCols / kPer;      // 16-byte units of a row: 8, or 4
      constexpr int kRowBytes = kUnits * 16;
      // the 128- or 64-byte swizzle of the output's tensor map
      auto unit_at = [](int r, int g) {
        return r * kRowBytes + ((kUnits == 8 ? g ^ (r & 7) : g ^ ((r >> 1) & 3)) << 4);
      };
      const int rows = min(32, a.M - r0);
#pragma unroll
      for (int c = 0; c < kWide / kCols; ++c) {
        if (lane == 0) bulk_wait_read0();  // the buffer's last store has been read
        __syncwarp();
#pragma unroll
        for (int g = 0; g < kUnits; ++g) {
          float f[kPer];
#pragma unroll
          for (int i = 0; i < kPer; i += 2) {
            f[i] = acc[(c * kCols + g * kPer + i) / 2].x;
            f[i + 1] = acc[(c * kCols + g * kPer + i) / 2].y;
          }
          uint32_t p[4];
          Storage<T>::pack(p, f);
          *reinterpret_cast<uint4*>(buf + unit_at(lane, g)) = make_uint4(p[0], p[1], p[2], p[3]);
        }
        if (a.tma_out) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && rows > 0 && c * kCols < cols) {
            tma_store_3d(&omap, buf, col0 + c * kCols, r0, split);
            bulk_commit();
          }
        } else {
          __syncwarp();
          // rows that no vector or TMA store can start: a lane's columns of one row after
          // the other, so that a warp's stores are one run of the row
          size_t o = (size_t(split) * a.M + size_t(r0)) * a.out_pitch + col0 + c * kCols + lane;
          const size_t total = size_t(a.splits) * a.M * a.out_pitch;
          constexpr int kLaneCols = kCols / 32;
          const int left = cols - c * kCols - lane;
#pragma unroll 8
          for (int r = 0; r < 32; ++r, o += a.out_pitch) {
#pragma unroll
            for (int k = 0; k < kLaneCols; ++k) {
              const int byte = (lane + 32 * k) * int(sizeof(T));
              const T x = *reinterpret_cast<const T*>(buf + unit_at(r, byte >> 4) + (byte & 15));
              if (r < rows && 32 * k < left && in_range_of(a.error_word, o + 32 * k, 1, total))
                static_cast<T*>(a.out)[o + 32 * k] = x;
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait0();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base),
                 "r"(kLfTmemCols)
                 : "memory");
  }
}

// out[m, n] = sum over the splits of part[s][m][n], in order, + bias[n].
template <typename T>
__global__ void __launch_bounds__(256)
    dcn_linear_join_kernel(const float* part, int splits, int M, int N, int pitch,
                           const float* bias, T* out) {
  chain_wait();
  chain_release();
  const size_t plane = size_t(M) * pitch, n = size_t(M) * N;
  for (size_t i = size_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += size_t(gridDim.x) * 256) {
    const size_t m = i / unsigned(N);
    const int c = int(i - m * unsigned(N));
    const float* p = part + m * pitch + c;
    float v = p[0];
    for (int s = 1; s < splits; ++s) v += p[s * plane];
    if (bias) v += __ldg(bias + c);
    Storage<T>::store_float(out + i, v);
  }
}

// ---------------------------------------------------------------------------
// Few rows.  The weight is read once and nothing else matters, so the work is spread
// over many warps instead of 128-row tiles: a warp owns 8 output columns and every
// `wk`-th K block, five blocks in flight at a time, and mma.sync m16n8k32 multiplies the
// rows (its first eight) by the 8 columns (rows that are not there cost no traffic).  A lane
// reads 32 contiguous bytes of its weight row a block, two 16-byte loads; the order of
// the 128 products is permuted the same way in both operands, so no shuffle is needed.
// The `wk` warps of a column group are joined in shared memory in a fixed order.  Bound
// by latency: 1 to 8 rows of 5120 x 1280 take 5.3 to 5.5 us from launch to launch (the
// tile kernel 8.6, the weight's 6.6 MB alone 1.0), of 1280 x 5120 5.5 to 5.8 (7.7).  With
// rows in the MMA's upper half too, 9 to 16 took 10 to 11: the tile kernel has those.
struct LinearRowsArgs {
  int M, N, K, k_blocks, pitch, n_blocks;
  int wk;  // warps that share a column group: a power of two up to kLrWarps
  const uint8_t* a;
  const uint8_t* b;
  const float* sa;
  const float* sb;
  const float* bias;
  void* out;
  unsigned int* error_word;
};

constexpr int kLrWarps = 8;
constexpr int kLrThreads = kLrWarps * 32;
constexpr int kLrAhead = 5;  // K blocks in flight a warp

__device__ __forceinline__ void mma_e4m3_16x8x32(float (&d)[4], uint32_t a0, uint32_t a1,
                                                 uint32_t a2, uint32_t a3, uint32_t b0,
                                                 uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 32 bytes of a row of codes at byte k; bytes at or behind K are zeros.
__device__ __forceinline__ void load_codes(const uint8_t* row, bool in, int k, int K, int pitch,
                                           uint32_t (&w)[8]) {
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    uint4 x = make_uint4(0, 0, 0, 0);
    const int k0 = k + 16 * v;
    if (in && k0 < pitch) x = ldg128(row + k0);
    w[4 * v] = x.x; w[4 * v + 1] = x.y; w[4 * v + 2] = x.z; w[4 * v + 3] = x.w;
    if (k0 + 16 > K) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int left = K - (k0 + 4 * i);  // bytes of this word inside the row
        if (left < 4) w[4 * v + i] &= left <= 0 ? 0u : (1u << (8 * left)) - 1u;
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kLrThreads)
    dcn_linear_fp8_rows_kernel(const LinearRowsArgs a) {
  chain_wait();
  chain_release();
  __shared__ float red[kLrWarps][8][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int groups = kLrWarps / a.wk;  // column groups of the CTA
  const int n_cta = int(blockIdx.x) * groups * 8;
  const int n0 = n_cta + warp / a.wk * 8;
  const bool col = n0 + g < a.N;
  const uint8_t* brow = a.b + size_t(min(n0 + g, a.N - 1)) * a.pitch;
  float acc[2] = {0.f, 0.f};  // row g, columns 2 t and 2 t + 1
  for (int kb0 = warp & (a.wk - 1); kb0 < a.k_blocks; kb0 += a.wk * kLrAhead) {
    uint32_t wb[kLrAhead][8], wa[kLrAhead][8];
    float s[kLrAhead];
#pragma unroll
    for (int u = 0; u < kLrAhead; ++u) {
      const int kb = kb0 + u * a.wk, k = kb * kFp8Block + 32 * t;
      const bool in = kb < a.k_blocks && n0 < a.N;
      load_codes(brow, in && col, k, a.K, a.pitch, wb[u]);
      load_codes(a.a + size_t(g) * a.pitch, in && g < a.M, k, a.K, a.pitch, wa[u]);
      const float sb = in ? __ldg(a.sb + size_t(kb) * a.n_blocks + n0 / kFp8Block) : 0.f;
      s[u] = in && g < a.M ? sb * __ldg(a.sa + size_t(kb) * a.M + g) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kLrAhead; ++u) {
      if (kb0 + u * a.wk >= a.k_blocks) break;
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        mma_e4m3_16x8x32(d, wa[u][2 * k], 0u, wa[u][2 * k + 1], 0u, wb[u][2 * k], wb[u][2 * k + 1]);
      acc[0] = fmaf(d[0], s[u], acc[0]);
      acc[1] = fmaf(d[1], s[u], acc[1]);
    }
  }
  *reinterpret_cast<float2*>(&red[warp][g][2 * t]) = make_float2(acc[0], acc[1]);
  __syncthreads();
  for (int e = int(threadIdx.x); e < groups * 64; e += kLrThreads) {
    const int m = (e >> 3) & 7, c = e & 7, grp = e >> 6;
    const int n = n_cta + grp * 8 + c;
    if (m >= a.M || n >= a.N) continue;
    float v = red[grp * a.wk][m][c];
    for (int w = 1; w < a.wk; ++w) v += red[grp * a.wk + w][m][c];
    if (a.bias) v += __ldg(a.bias + n);
    const size_t o = size_t(m) * a.N + n;
    if (in_range_of(a.error_word, o, 1, size_t(a.M) * a.N))
      Storage<T>::store_float(static_cast<T*>(a.out) + o, v);
  }
}

}  // namespace dcn
