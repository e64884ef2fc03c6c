// Grouped products on the tensor cores (bf16 operands, fp32 accumulation in
// TMEM), for every size the library takes. Persistent, warp-specialised
// kernels for sm_100a, on single CTAs or on CTA pairs (cta_group::2):
//   warp 0      TMA producer: operand tiles -> shared-memory ring
//   warp 1      MMA issuer: tcgen05.mma into TMEM, tcgen05.commit
//   warps 2..9  epilogue: tcgen05.ld, conversion, stores
//
// Row products (row_gemm_kernel), out[r, c] for the rows of each segment. The
// weights fill the MMA's M (128 output columns per CTA) and up to BN rows of
// the segment are its N, so a segment of a few rows is not padded to 128:
//   y  = x W^T   contraction over n_in: W's rows are K-major, as x's are
//   dx = dy W    contraction over n_out: W is read as it lies and its tile is
//                MN-major (the output direction is contiguous); a second pair
//                (dy2, W2) may extend the contraction
//   the SwiGLU backward: gate and up accumulators of the same tile, and an
//                epilogue that turns them and dh into h, da and du
// Weight gradients (dw_gemm_kernel), dw[e] = dy^T x: contraction over the
// segment's rows, both operands MN-major as they lie. The last rows of a
// segment come by gather4 in groups of four, with a row outside the tensor
// (zeros) for what lies behind the segment's end, in both operands: nothing of
// the next segment, nor of what lies behind the last one, enters a product.
//
// Ragged sizes need no special code in the main loop: weights are 3-D tensors
// (columns, rows, group), so a tile that reaches past a matrix reads zeros
// there instead of the next group's values, and so do activations past their
// columns. Stores are clipped by the epilogue or by the TMA store.
//
// Every mbarrier wait is bounded (about 2 s); on expiry the kernel records an
// error code, the other roles stop, copies and MMAs in flight are waited for
// (again bounded), TMEM is freed and the kernel returns.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "grouped.cuh"
#include "sm100_ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 320;
constexpr int kEpiWarps = 8;
constexpr int BM = 128;  // output columns (row products) or rows (dw) per CTA
constexpr int BK = 64;   // contraction elements per stage
constexpr uint32_t kTileBytes = BM * BK * 2;
constexpr uint32_t kBlockBytes = 64 * 128;  // 64 x 64 bf16 block of an MN-major tile
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kAccStride = 256;
constexpr uint64_t kWaitLimitNs = 2000000000ull;

// --------------------------------------------------------------- PTX forms --
__device__ __forceinline__ void tma_load_3d(const CUtensorMap* map, uint32_t dst, uint32_t bar,
                                            int32_t x, int32_t y, int32_t z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::"
      "bytes.L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(const CUtensorMap* map, uint32_t dst,
                                                 uint32_t leader_bar, int32_t x, int32_t y,
                                                 int32_t z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::"
      "complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(leader_bar), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_gather4_2d_pair(const CUtensorMap* map, uint32_t dst,
                                                    uint32_t leader_bar, int32_t x, int32_t y0,
                                                    int32_t y1, int32_t y2, int32_t y3,
                                                    uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::"
      "bytes.cta_group::2.L2::cache_hint [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(leader_bar), "r"(x), "r"(y0), "r"(y1), "r"(y2),
      "r"(y3), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t src, int32_t x,
                                             int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(src), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void store_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// At most N of this thread's store groups still read shared memory.
template <int N>
__device__ __forceinline__ void store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void store_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

// Shared-memory descriptor of an MN-major tile with 128-byte swizzling: blocks
// of 64 (MN) x 64 (contraction) elements, contraction rows of 128 bytes. Eight
// rows are 1024 bytes (stride byte offset), the next 64 MN elements lie
// kBlockBytes further (leading byte offset). A step of 16 along the
// contraction moves the start by 2048 bytes.
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(kBlockBytes >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
// Instruction descriptor bits: operand A, operand B is MN-major.
constexpr uint32_t kAMn = 1u << 15, kBMn = 1u << 16;

// The same operations on one CTA or, from the leader, on a CTA pair. Copies of
// a pair complete on the leader's barrier; commits arrive in both CTAs.
template <bool PAIR>
struct Cg;
template <>
struct Cg<false> {
  __device__ static void load_2d(const CUtensorMap* m, uint32_t dst, uint32_t bar, int32_t x,
                                 int32_t y, uint64_t pol) {
    ptx::tma_load_2d(m, dst, bar, x, y, pol);
  }
  __device__ static void load_3d(const CUtensorMap* m, uint32_t dst, uint32_t bar, int32_t x,
                                 int32_t y, int32_t z, uint64_t pol) {
    tma_load_3d(m, dst, bar, x, y, z, pol);
  }
  __device__ static void gather4(const CUtensorMap* m, uint32_t dst, uint32_t bar, int32_t x,
                                 int32_t y0, int32_t y1, int32_t y2, int32_t y3, uint64_t pol) {
    ptx::tma_gather4_2d(m, dst, bar, x, y0, y1, y2, y3, pol);
  }
  __device__ static void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    ptx::mma_bf16(d, a, b, idesc, acc);
  }
  __device__ static void commit(uint32_t bar) { ptx::mma_commit(bar); }
  __device__ static void alloc(uint32_t slot) {
    ptx::tmem_alloc(slot, kTmemCols);
    ptx::tmem_relinquish();
  }
  __device__ static void dealloc(uint32_t t) { ptx::tmem_dealloc(t, kTmemCols); }
  __device__ static uint32_t rank() { return 0; }
  __device__ static uint32_t at_leader(uint32_t bar) { return bar; }
  __device__ static void sync_all() {}
};
template <>
struct Cg<true> {
  __device__ static void load_2d(const CUtensorMap* m, uint32_t dst, uint32_t bar, int32_t x,
                                 int32_t y, uint64_t pol) {
    ptx::tma_load_2d_pair(m, dst, bar, x, y, pol);
  }
  __device__ static void load_3d(const CUtensorMap* m, uint32_t dst, uint32_t bar, int32_t x,
                                 int32_t y, int32_t z, uint64_t pol) {
    tma_load_3d_pair(m, dst, bar, x, y, z, pol);
  }
  __device__ static void gather4(const CUtensorMap* m, uint32_t dst, uint32_t bar, int32_t x,
                                 int32_t y0, int32_t y1, int32_t y2, int32_t y3, uint64_t pol) {
    tma_gather4_2d_pair(m, dst, bar, x, y0, y1, y2, y3, pol);
  }
  __device__ static void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    ptx::mma_bf16_pair(d, a, b, idesc, acc);
  }
  __device__ static void commit(uint32_t bar) { ptx::mma_commit_pair(bar); }
  __device__ static void alloc(uint32_t slot) {
    ptx::tmem_alloc_pair(slot, kTmemCols);
    ptx::tmem_relinquish_pair();
  }
  __device__ static void dealloc(uint32_t t) { ptx::tmem_dealloc_pair(t, kTmemCols); }
  __device__ static uint32_t rank() { return ptx::cluster_ctarank(); }
  __device__ static uint32_t at_leader(uint32_t bar) { return ptx::map_to_rank(bar, 0); }
  __device__ static void sync_all() { ptx::cluster_sync(); }
};

// Bounded wait on an mbarrier phase. False when the CTA was told to stop, or
// when the limit ran out (then it tells the CTA to stop and records the error).
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity,
                                             volatile int* abort_flag, int32_t* err) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::global_timer_ns();
  while (true) {
    for (int i = 0; i < 64; ++i)
      if (ptx::mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (ptx::global_timer_ns() - t0 > kWaitLimitNs) {
      *abort_flag = 1;
      atomicCAS(err, 0, kErrWaitTimeout);
      return false;
    }
  }
}

// Bounded wait that ignores the stop flag (used while cleaning up).
__device__ __forceinline__ void wait_cleanup(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = ptx::global_timer_ns();
  while (!ptx::mbar_try_wait(bar, parity))
    if (ptx::global_timer_ns() - t0 > kWaitLimitNs) return;
}
__device__ __forceinline__ void settle_ns(uint64_t ns) {
  const uint64_t t0 = ptx::global_timer_ns();
  while (ptx::global_timer_ns() - t0 < ns) {
  }
}

// The barriers and small state behind the ring, common to both kernels.
template <int S, bool PAIR>
struct Control {
  uint32_t bars;
  volatile int* abort_flag;
  uint32_t* tmem_slot;
  __device__ uint32_t full(int s) const { return bars + 8u * s; }
  __device__ uint32_t empty(int s) const { return bars + 8u * (S + s); }
  __device__ uint32_t tfull(int b) const { return bars + 8u * (2 * S + b); }
  __device__ uint32_t tempty(int b) const { return bars + 8u * (2 * S + 2 + b); }
  __device__ uint32_t mma_done() const { return bars + 8u * (2 * S + 4); }
  __device__ void init(uint8_t* smem, uint32_t sbase, uint32_t bar_off) {
    static_assert(8 * (2 * S + 5) + 8 <= 256, "barriers fit their 256 bytes");
    bars = sbase + bar_off;
    tmem_slot = reinterpret_cast<uint32_t*>(smem + bar_off + 8 * (2 * S + 5));
    abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    if (threadIdx.x == 0) {
      for (int s = 0; s < S; ++s) {
        ptx::mbar_init(full(s), 1);
        ptx::mbar_init(empty(s), 1);
      }
      for (int b = 0; b < 2; ++b) {
        ptx::mbar_init(tfull(b), 1);
        ptx::mbar_init(tempty(b), PAIR ? 2 * kEpiWarps : kEpiWarps);
      }
      ptx::mbar_init(mma_done(), 1);
      *abort_flag = 0;
      ptx::fence_mbar_init();
    }
    if ((threadIdx.x >> 5) == 1) Cg<PAIR>::alloc(ptx::smem_addr(tmem_slot));
  }
  // An epilogue warp is done with accumulator b.
  __device__ void release(int b, int lane) const {
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      if (PAIR)
        ptx::mbar_arrive_remote(ptx::map_to_rank(tempty(b), 0));
      else
        ptx::mbar_arrive(tempty(b));
    }
  }
  // After an abort: let the copies that were issued land before the CTA goes.
  // The leader sees them on its full barriers; the peer's complete there too.
  __device__ void settle_loads(uint32_t armed, uint32_t par) const {
    if (!PAIR || Cg<PAIR>::rank() == 0) {
      for (int s = 0; s < S; ++s)
        if ((armed >> s) & 1u) wait_cleanup(full(s), (par >> s) & 1u);
    } else if (armed) {
      settle_ns(2000000);
    }
  }
  __device__ void finish(uint32_t tmem_base) const {
    ptx::tc_fence_before();
    __syncthreads();
    Cg<PAIR>::sync_all();  // neither CTA frees TMEM or exits while the pair works
    if ((threadIdx.x >> 5) == 1) {
      ptx::tc_fence_after();
      Cg<PAIR>::dealloc(tmem_base);
    }
  }
};

// ------------------------------------------------------------ row products --
enum class Mode : int { kFwd = 0, kDx = 1, kGateUp = 2 };

struct RowArgs {
  const int32_t* offsets;
  int32_t* err;
  int64_t rows;
  int groups;
  int cols;      // output columns
  int k_blocks;  // per source
  int sources;   // 2: a second (weights, rows) pair extends the contraction
  void* out;     // bf16 or float rows; kGateUp: h
  bool out_f32;
  // kGateUp only
  const float* dh;
  __nv_bfloat16* da;
  __nv_bfloat16* du;
};

struct RowMaps {
  CUtensorMap w[2];     // weights (kGateUp: gate, up; kDx: the two sources)
  CUtensorMap r16[2];   // rows, 16 per box
  CUtensorMap r128[2];  // rows, 128 per box
};

template <Mode MODE, int BN_, bool PAIR_>
struct RowCfg {
  static constexpr bool PAIR = PAIR_;
  static constexpr int kCtas = PAIR ? 2 : 1;
  static constexpr int BN = BN_;
  static constexpr int BNH = BN / kCtas;  // rows one CTA loads
  static constexpr int kNumA = MODE == Mode::kGateUp ? 2 : 1;
  static_assert(BN <= 256 && BN % (16 * kCtas) == 0 && BNH <= 128 + 128 * (1 - (kCtas - 1)), "");
  static constexpr uint32_t kAccCols = kNumA * BN;
  static constexpr int kAccBufs = kAccCols <= kAccStride ? 2 : 1;
  static constexpr uint32_t kStageBytes = kNumA * kTileBytes + BNH * BK * 2;
  static constexpr int kStages = 204800 / kStageBytes > 8 ? 8 : (int)(204800 / kStageBytes);
  static constexpr uint32_t kBarOff = kStages * kStageBytes;
  static constexpr uint32_t kTabOff = kBarOff + 256;
  static constexpr uint32_t kSmemBytes = 1024 + kTabOff + 2 * 4 * (kMaxExperts + 1) + 128;
};

struct RowUnit {
  int e, m, row0, n_valid, n_mma, ntiles;
};

template <int BN, int STEP>
__device__ __forceinline__ RowUnit row_unit(int u, const int32_t* s_tile, const int32_t* s_off,
                                            int groups, int m_tiles) {
  int lo = 0, hi = groups - 1;  // largest e with m_tiles * s_tile[e] <= u
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (m_tiles * s_tile[mid] <= u)
      lo = mid;
    else
      hi = mid - 1;
  }
  RowUnit un;
  un.e = lo;
  un.ntiles = s_tile[lo + 1] - s_tile[lo];
  const int local = u - m_tiles * s_tile[lo];
  un.m = local / un.ntiles;
  const int tt = local - un.m * un.ntiles;
  un.row0 = s_off[lo] + tt * BN;
  const int rem = s_off[lo + 1] - un.row0;
  un.n_valid = rem < BN ? rem : BN;
  un.n_mma = (un.n_valid + STEP - 1) / STEP * STEP;
  return un;
}

// 1 / (1 + e^-z), with the fast exponential and divide: their error is far
// below the bf16 rounding of h, da and du that follows (e^-z = infinity gives
// the limit 0).
__device__ __forceinline__ float sigmoid_f(float z) {
  return __fdividef(1.0f, 1.0f + __expf(-z));
}

template <Mode MODE, int BN_, bool PAIR_>
__global__ void __launch_bounds__(kThreads, 1)
    row_gemm_kernel(const __grid_constant__ RowMaps maps, const RowArgs args) {
  using C = RowCfg<MODE, BN_, PAIR_>;
  using G = Cg<PAIR_>;
  constexpr bool PAIR = PAIR_;
  constexpr int S = C::kStages, BN = C::BN, STEP = 16 * C::kCtas;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = ptx::smem_addr(smem);
  int32_t* s_tile = reinterpret_cast<int32_t*>(smem + C::kTabOff);
  int32_t* s_off = s_tile + (kMaxExperts + 1);
  int32_t* s_warp = s_off + (kMaxExperts + 1);
  Control<S, PAIR> ctl;
  ctl.init(smem, sbase, C::kBarOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = G::rank();
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tensormap(&maps.w[0]);
    ptx::prefetch_tensormap(&maps.r16[0]);
    ptx::prefetch_tensormap(&maps.r128[0]);
  }
  // everything above overlaps the previous kernel's tail
  griddep_wait();
  griddep_launch_dependents();
  segment_table<kThreads>(args.offsets, args.groups, args.rows, BN, s_off, s_tile, s_warp);
  ptx::tc_fence_before();
  __syncthreads();
  G::sync_all();  // both CTAs' barriers exist before any remote arrive
  ptx::tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(ctl.tmem_slot);
  const int m_tiles = (args.cols + BM * C::kCtas - 1) / (BM * C::kCtas);
  const int total = s_tile[args.groups] * m_tiles;
  const int first = (int)blockIdx.x / C::kCtas, stride = (int)gridDim.x / C::kCtas;
  const int n_kb = args.k_blocks * args.sources;

  if (warp == 0) {
    // ---------------------------------------------------- TMA producer --
    if (lane == 0) {
      const uint64_t pol_first = ptx::policy_evict_first();
      const uint64_t pol_normal = ptx::policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_par = 0;
      bool ok = true;
      for (int u = first; u < total && ok; u += stride) {
        const RowUnit un = row_unit<BN, STEP>(u, s_tile, s_off, args.groups, m_tiles);
        const int half = un.n_mma / C::kCtas;
        const int col0 = (un.m * C::kCtas + (int)rank) * BM;
        const int brow = un.row0 + (int)rank * half;
        const uint32_t bytes =
            (uint32_t)C::kCtas * (C::kNumA * kTileBytes + (uint32_t)half * 128u);
        // weights that only this unit reads (one row tile) are streamed
        const uint64_t pol_w = un.ntiles == 1 ? pol_first : pol_normal;
        for (int kb = 0; kb < n_kb; ++kb) {
          if (!wait_bounded(ctl.empty(stage), phase ^ 1u, ctl.abort_flag, args.err)) {
            ok = false;
            break;
          }
          const int src = kb >= args.k_blocks ? 1 : 0;
          const int k0 = (kb - src * args.k_blocks) * BK;
          if (rank == 0) ptx::mbar_arrive_expect_tx(ctl.full(stage), bytes);
          const uint32_t fb = G::at_leader(ctl.full(stage));
          const uint32_t a0 = sbase + stage * C::kStageBytes;
          if (MODE == Mode::kDx) {
            G::load_3d(&maps.w[src], a0, fb, col0, k0, un.e, pol_w);
            G::load_3d(&maps.w[src], a0 + kBlockBytes, fb, col0 + 64, k0, un.e, pol_w);
          } else {
            G::load_3d(&maps.w[0], a0, fb, k0, col0, un.e, pol_w);
            if (MODE == Mode::kGateUp)
              G::load_3d(&maps.w[1], a0 + kTileBytes, fb, k0, col0, un.e, pol_w);
          }
          const uint32_t b0 = a0 + C::kNumA * kTileBytes;
          int j = 0;
          for (; j + 128 <= half; j += 128)
            G::load_2d(&maps.r128[src], b0 + j * 128u, fb, k0, brow + j, pol_normal);
          for (; j < half; j += 16)
            G::load_2d(&maps.r16[src], b0 + j * 128u, fb, k0, brow + j, pol_normal);
          armed |= 1u << stage;
          armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) ctl.settle_loads(armed, armed_par);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA issuer --
    if (lane == 0 && rank == 0) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true, issued = false;
      for (int u = first; u < total && ok; u += stride) {
        const RowUnit un = row_unit<BN, STEP>(u, s_tile, s_off, args.groups, m_tiles);
        if (!wait_bounded(ctl.tempty(acc), acc_phase ^ 1u, ctl.abort_flag, args.err)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t idesc = ptx::idesc_bf16_f32(BM * C::kCtas, un.n_mma) |
                               (MODE == Mode::kDx ? kAMn : 0u);
        const uint32_t d0 = tmem_base + (uint32_t)acc * kAccStride;
        for (int kb = 0; kb < n_kb; ++kb) {
          if (!wait_bounded(ctl.full(stage), phase, ctl.abort_flag, args.err)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t a0 = sbase + stage * C::kStageBytes;
          const uint32_t b0 = a0 + C::kNumA * kTileBytes;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            const uint64_t bdesc = ptx::desc_k_sw128(b0 + kk * 32);
            const uint64_t adesc = MODE == Mode::kDx ? desc_mn_sw128(a0 + kk * 2048)
                                                     : ptx::desc_k_sw128(a0 + kk * 32);
            const uint32_t accum = (kb | kk) != 0 ? 1u : 0u;
            G::mma(d0, adesc, bdesc, idesc, accum);
            if (MODE == Mode::kGateUp)
              G::mma(d0 + BN, ptx::desc_k_sw128(a0 + kTileBytes + kk * 32), bdesc, idesc, accum);
          }
          issued = true;
          G::commit(ctl.empty(stage));
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        G::commit(ctl.tfull(acc));
        if (++acc == C::kAccBufs) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (!ok && issued) {  // MMAs already issued must finish before TMEM is freed
        G::commit(ctl.mma_done());
        wait_cleanup(ctl.mma_done(), 0);
      }
    }
  } else {
    // -------------------------------------------------------- epilogue --
    const int ew = warp & 3;         // TMEM lane quarter this warp may access
    const int eh = (warp - 2) >> 2;  // which half of the column chunks
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int u = first; u < total; u += stride) {
      const RowUnit un = row_unit<BN, STEP>(u, s_tile, s_off, args.groups, m_tiles);
      const bool ok = wait_bounded(ctl.tfull(acc), acc_phase, ctl.abort_flag, args.err);
      if (!__all_sync(0xffffffffu, ok)) break;
      ptx::tc_fence_after();
      const uint32_t tb =
          tmem_base + (static_cast<uint32_t>(ew * 32) << 16) + (uint32_t)acc * kAccStride;
      const int col = (un.m * C::kCtas + (int)rank) * BM + ew * 32 + lane;
      const bool col_ok = col < args.cols;
      const int64_t obase = (int64_t)un.row0 * args.cols + col;
      // 32-row chunks, alternating between the two warps of this quarter
      for (int c0 = 32 * eh; c0 < un.n_mma; c0 += 64) {
        if (MODE == Mode::kGateUp) {
          float a[32], v[32], g[32];
#pragma unroll
          for (int c = 0; c < 32; ++c)
            g[c] = col_ok && c0 + c < un.n_valid
                       ? __ldg(args.dh + obase + (int64_t)(c0 + c) * args.cols)
                       : 0.f;
          ptx::tmem_ld32x2(tb + c0, tb + BN + c0, a, v);
          __nv_bfloat16* h = static_cast<__nv_bfloat16*>(args.out) + obase;
          __nv_bfloat16* da = args.da + obase;
          __nv_bfloat16* du = args.du + obase;
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            if (col_ok && c0 + c < un.n_valid) {
              const int64_t at = (int64_t)(c0 + c) * args.cols;
              const float sig = sigmoid_f(a[c]);
              const float silu = a[c] * sig;
              h[at] = __float2bfloat16_rn(silu * v[c]);
              da[at] = __float2bfloat16_rn(g[c] * v[c] * (sig + silu * (1.0f - sig)));
              du[at] = __float2bfloat16_rn(g[c] * silu);
            }
          }
        } else {
          float g[32];
          ptx::tmem_ld32(tb + c0, g);
          if (args.out_f32) {
            float* o = static_cast<float*>(args.out) + obase;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (col_ok && c0 + c < un.n_valid) o[(int64_t)(c0 + c) * args.cols] = g[c];
          } else {
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(args.out) + obase;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (col_ok && c0 + c < un.n_valid)
                o[(int64_t)(c0 + c) * args.cols] = __float2bfloat16_rn(g[c]);
          }
        }
      }
      ctl.release(acc, lane);
      if (++acc == C::kAccBufs) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
  }
  ctl.finish(tmem_base);
}

// -------------------------------------------------------- weight gradients --
struct DwJob {
  CUtensorMap a64, a16, a1;  // dy: 64-, 16- and 1-row boxes of 64 columns
  CUtensorMap b64, b16, b1;  // x
  CUtensorMap out;           // dw: 32 rows of 128 bytes
  int n_out, n_in;
};
struct DwMaps {
  DwJob job[kMaxJobs];
};
struct DwArgs {
  const int32_t* offsets;
  int32_t* err;
  int64_t rows;
  int groups;
  int n_jobs;
  bool out_f32;
};

// Tile: 128 rows of dw per CTA x 256 columns; TMEM holds two accumulators.
template <bool PAIR_>
struct DwCfg {
  static constexpr bool PAIR = PAIR_;
  static constexpr int kCtas = PAIR ? 2 : 1;
  static constexpr int BN = 256;
  static constexpr int kABlocks = 2, kBBlocks = BN / 64 / kCtas;  // 64-column blocks per CTA
  static constexpr uint32_t kStageBytes = (kABlocks + kBBlocks) * kBlockBytes;
  static constexpr int kStages = PAIR ? 4 : 3;
  static constexpr uint32_t kStageBuf = 4096;  // one warp's 32 rows x 128 bytes
  static constexpr uint32_t kOutOff = kStages * kStageBytes;
  static constexpr uint32_t kBarOff = kOutOff + kEpiWarps * 2 * kStageBuf;
  static constexpr uint32_t kOffOff = kBarOff + 256;
  static constexpr uint32_t kSmemBytes = 1024 + kOffOff + 4 * (kMaxExperts + 1);
};

struct DwUnit {
  int job, e, it, jt, row0, n_rows;
};

template <int CTAS>
__device__ __forceinline__ DwUnit dw_unit(int u, const int* first, const DwMaps& maps,
                                          const int32_t* s_off) {
  DwUnit un;
  un.job = u >= first[2] ? 2 : (u >= first[1] ? 1 : 0);
  const DwJob& j = maps.job[un.job];
  const int v = u - first[un.job];
  const int nj = (j.n_in + 255) / 256, ni = (j.n_out + BM * CTAS - 1) / (BM * CTAS);
  un.jt = v % nj;
  un.it = (v / nj) % ni;
  un.e = v / nj / ni;
  un.row0 = s_off[un.e];
  const int n = s_off[un.e + 1] - un.row0;
  un.n_rows = n > 0 ? n : 0;
  return un;
}

template <bool PAIR_>
__global__ void __launch_bounds__(kThreads, 1)
    dw_gemm_kernel(const __grid_constant__ DwMaps maps, const DwArgs args) {
  using C = DwCfg<PAIR_>;
  using G = Cg<PAIR_>;
  constexpr bool PAIR = PAIR_;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = ptx::smem_addr(smem);
  int32_t* s_off = reinterpret_cast<int32_t*>(smem + C::kOffOff);
  Control<S, PAIR> ctl;
  ctl.init(smem, sbase, C::kBarOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = G::rank();
  griddep_wait();
  griddep_launch_dependents();
  for (int i = threadIdx.x; i <= args.groups; i += kThreads) {
    const int32_t o = args.offsets[i];
    s_off[i] = o < 0 ? 0 : (o > args.rows ? (int32_t)args.rows : o);
  }
  ptx::tc_fence_before();
  __syncthreads();
  G::sync_all();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(ctl.tmem_slot);
  int first_unit[kMaxJobs + 1];
  first_unit[0] = 0;
#pragma unroll
  for (int q = 0; q < kMaxJobs; ++q) {
    int n = 0;
    if (q < args.n_jobs)
      n = args.groups * ((maps.job[q].n_out + BM * C::kCtas - 1) / (BM * C::kCtas)) *
          ((maps.job[q].n_in + 255) / 256);
    first_unit[q + 1] = first_unit[q] + n;
  }
  const int total = first_unit[kMaxJobs];
  const int first = (int)blockIdx.x / C::kCtas, stride = (int)gridDim.x / C::kCtas;

  if (warp == 0) {
    // ---------------------------------------------------- TMA producer --
    if (lane == 0) {
      const uint64_t pol = ptx::policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_par = 0;
      bool ok = true;
      for (int u = first; u < total && ok; u += stride) {
        const DwUnit un = dw_unit<C::kCtas>(u, first_unit, maps, s_off);
        const DwJob& job = maps.job[un.job];
        const int acol = (un.it * C::kCtas + (int)rank) * BM;
        const int bcol = un.jt * 256 + (int)rank * (C::kBBlocks * 64);
        for (int k0 = 0; k0 < un.n_rows; k0 += BK) {
          if (!wait_bounded(ctl.empty(stage), phase ^ 1u, ctl.abort_flag, args.err)) {
            ok = false;
            break;
          }
          const int left = un.n_rows - k0;
          const int n = left < BK ? left : BK;       // rows of this block
          const int n16 = (n + 15) & ~15;            // rows the MMAs read
          if (rank == 0)
            ptx::mbar_arrive_expect_tx(
                ctl.full(stage),
                (uint32_t)(C::kCtas * (C::kABlocks + C::kBBlocks)) * (uint32_t)n16 * 128u);
          const uint32_t fb = G::at_leader(ctl.full(stage));
          const uint32_t s0 = sbase + stage * C::kStageBytes;
          const int r0 = un.row0 + k0;
          const int oob = (int)args.rows;  // a row outside the tensors: zeros
#pragma unroll
          for (int b = 0; b < C::kABlocks + C::kBBlocks; ++b) {
            const bool is_a = b < C::kABlocks;
            const int x = is_a ? acol + 64 * b : bcol + 64 * (b - C::kABlocks);
            const uint32_t dst = s0 + b * kBlockBytes;
            if (n == BK) {
              G::load_2d(is_a ? &job.a64 : &job.b64, dst, fb, x, r0, pol);
            } else {
              int j = 0;
              for (; j + 16 <= n; j += 16)
                G::load_2d(is_a ? &job.a16 : &job.b16, dst + j * 128u, fb, x, r0 + j, pol);
              for (; j < n16; j += 4)
                G::gather4(is_a ? &job.a1 : &job.b1, dst + j * 128u, fb, x,
                           j < n ? r0 + j : oob, j + 1 < n ? r0 + j + 1 : oob,
                           j + 2 < n ? r0 + j + 2 : oob, j + 3 < n ? r0 + j + 3 : oob, pol);
            }
          }
          armed |= 1u << stage;
          armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) ctl.settle_loads(armed, armed_par);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA issuer --
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = ptx::idesc_bf16_f32(BM * C::kCtas, C::BN) | kAMn | kBMn;
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true, issued = false;
      for (int u = first; u < total && ok; u += stride) {
        const DwUnit un = dw_unit<C::kCtas>(u, first_unit, maps, s_off);
        if (un.n_rows == 0) continue;  // the epilogue writes zeros by itself
        if (!wait_bounded(ctl.tempty(acc), acc_phase ^ 1u, ctl.abort_flag, args.err)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t d0 = tmem_base + (uint32_t)acc * kAccStride;
        for (int k0 = 0; k0 < un.n_rows; k0 += BK) {
          if (!wait_bounded(ctl.full(stage), phase, ctl.abort_flag, args.err)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const int left = un.n_rows - k0;
          const int steps = left >= BK ? BK / 16 : (left + 15) / 16;
          const uint32_t a0 = sbase + stage * C::kStageBytes;
          const uint32_t b0 = a0 + C::kABlocks * kBlockBytes;
          for (int kk = 0; kk < steps; ++kk)
            G::mma(d0, desc_mn_sw128(a0 + kk * 2048), desc_mn_sw128(b0 + kk * 2048), idesc,
                   (k0 | kk) != 0 ? 1u : 0u);
          issued = true;
          G::commit(ctl.empty(stage));
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        G::commit(ctl.tfull(acc));
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (!ok && issued) {
        G::commit(ctl.mma_done());
        wait_cleanup(ctl.mma_done(), 0);
      }
    }
  } else {
    // -------------------------------------------------------- epilogue --
    // A warp owns 32 rows (its TMEM lanes) and half of the 256 columns. Each
    // 128-byte-wide piece (64 bf16 or 32 float columns) is laid out swizzled in
    // shared memory and stored by TMA, which clips it to the matrix.
    const int ew = warp & 3, eh = (warp - 2) >> 2;
    const uint32_t buf0 = sbase + C::kOutOff + (uint32_t)(warp - 2) * 2 * C::kStageBuf;
    int acc = 0, piece = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int u = first; u < total && ok; u += stride) {
      const DwUnit un = dw_unit<C::kCtas>(u, first_unit, maps, s_off);
      const DwJob& job = maps.job[un.job];
      const bool some = un.n_rows > 0;
      if (some) {
        ok = __all_sync(0xffffffffu,
                        wait_bounded(ctl.tfull(acc), acc_phase, ctl.abort_flag, args.err));
        if (!ok) break;
        ptx::tc_fence_after();
      }
      const uint32_t tb =
          tmem_base + (static_cast<uint32_t>(ew * 32) << 16) + (uint32_t)acc * kAccStride;
      const int row = (un.it * C::kCtas + (int)rank) * BM + ew * 32;
      const int width = args.out_f32 ? 32 : 64;
      const bool rows_in = row < job.n_out;
      for (int c0 = eh * 128; c0 < eh * 128 + 128; c0 += width) {
        const int col = un.jt * 256 + c0;
        if (!rows_in || col >= job.n_in) continue;  // warp-uniform
        const uint32_t buf = buf0 + (uint32_t)(piece & 1) * C::kStageBuf;
        uint32_t w[32];
        if (args.out_f32) {
          float g[32];
          if (some) ptx::tmem_ld32(tb + c0, g);
#pragma unroll
          for (int c = 0; c < 32; ++c) w[c] = some ? __float_as_uint(g[c]) : 0u;
        } else {
          float g[32], v[32];
          if (some) ptx::tmem_ld32x2(tb + c0, tb + c0 + 32, g, v);
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(g[2 * c], g[2 * c + 1]);
            const __nv_bfloat162 q = __floats2bfloat162_rn(v[2 * c], v[2 * c + 1]);
            w[c] = some ? *reinterpret_cast<const uint32_t*>(&p) : 0u;
            w[16 + c] = some ? *reinterpret_cast<const uint32_t*>(&q) : 0u;
          }
        }
        if (lane == 0) store_wait_read<1>();  // this buffer's last store has read it
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c)
          st_shared_v4(buf + lane * 128u + (uint32_t)((c ^ (lane & 7)) << 4), w[4 * c],
                       w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(&job.out, buf, col, row, un.e);
          store_commit();
        }
        ++piece;
      }
      if (some) {
        ctl.release(acc, lane);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
    }
    if (lane == 0) store_wait_all();
  }
  ctl.finish(tmem_base);
}

// -------------------------------------------------------------------- host --
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
  if (!fn.load()) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn.store(reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p));
  }
  return fn.load();
}

bool encode(CUtensorMap* map, bool f32, int rank, const void* base, const uint64_t* dims,
            const uint32_t* box) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  const uint64_t es = f32 ? 4 : 2;
  cuuint64_t d[3], strides[2];
  cuuint32_t b[3], one[3] = {1, 1, 1};
  uint64_t bytes = es;
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    bytes *= dims[i];
    if (i + 1 < rank) strides[i] = bytes;
  }
  return enc(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
             (cuuint32_t)rank, const_cast<void*>(base), d, strides, b, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Row-major bf16 [rows, cols], box of 64 columns x box_rows.
bool rows_map(CUtensorMap* map, const void* base, int64_t rows, int cols, uint32_t box_rows) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
  const uint32_t box[2] = {64, box_rows};
  return encode(map, false, 2, base, dims, box);
}
// [groups, n_out, n_in], box of box_cols columns x box_rows rows of one group.
bool group_map(CUtensorMap* map, bool f32, const void* base, int groups, int n_out, int n_in,
               uint32_t box_cols, uint32_t box_rows) {
  const uint64_t dims[3] = {(uint64_t)n_in, (uint64_t)n_out, (uint64_t)groups};
  const uint32_t box[3] = {box_cols, box_rows, 1};
  return encode(map, f32, 3, base, dims, box);
}

// Persistent launch: one CTA per SM, or as many pairs as can be resident.
template <bool PAIR, typename... KArgs, typename... Args>
cudaError_t launch_persistent(void (*kernel)(KArgs...), uint32_t smem,
                              std::atomic<uint64_t>& attr_set, std::atomic<int>* grids,
                              cudaStream_t st, Args&&... args) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = raise_smem_once(attr_set, kernel, (int)smem);
  if (e != cudaSuccess) return e;
  if (!PAIR)
    return launch_pdl(kernel, dim3(num_sms()), dim3(kThreads), smem, st,
                      std::forward<Args>(args)...);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  int grid = grids[dev & 63].load();
  if (grid == 0) {
    cfg.gridDim = dim3(num_sms());
    cfg.numAttrs = 1;
    int clusters = 0;
    e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (clusters < 1) return cudaErrorInvalidConfiguration;
    const int most = num_sms() / 2;
    grid = 2 * (clusters < most ? clusters : most);
    grids[dev & 63].store(grid);
  }
  cfg.gridDim = dim3(grid);
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <Mode MODE, int BN, bool PAIR>
cudaError_t run_rows(const RowMaps& maps, const RowArgs& args, cudaStream_t st) {
  using C = RowCfg<MODE, BN, PAIR>;
  static std::atomic<uint64_t> attr_set{0};
  static std::atomic<int> grids[64];
  return launch_persistent<PAIR>(row_gemm_kernel<MODE, BN, PAIR>, C::kSmemBytes, attr_set, grids,
                                 st, maps, args);
}

template <Mode MODE>
cudaError_t run_rows_sized(const RowMaps& maps, const RowArgs& args, cudaStream_t st) {
  // rows per group if they were spread evenly: few rows want small row tiles
  // (deeper rings while weights stream), many rows want CTA pairs
  const int64_t avg = args.rows / args.groups;
  if (avg <= 32) return run_rows<MODE, 64, false>(maps, args, st);
  if (avg <= 128) return run_rows<MODE, 128, false>(maps, args, st);
  return run_rows<MODE, 256, true>(maps, args, st);
}

}  // namespace

cudaError_t launch_grouped_rows_tc(const GroupedShape& g, const GroupedJob& job,
                                   const int32_t* offsets, int32_t* err, cudaStream_t st) {
  RowMaps maps;
  const bool fwd = job.form == Form::kFwd;
  const int k = fwd ? job.n_in : job.n_out;
  const void* w[2] = {job.b, job.b2 ? job.b2 : job.b};
  const void* r[2] = {job.a, job.a2 ? job.a2 : job.a};
  bool ok = true;
  for (int q = 0; q < 2; ++q)
    ok = ok && group_map(&maps.w[q], false, w[q], g.groups, job.n_out, job.n_in, 64,
                         fwd ? 128 : 64) &&
         rows_map(&maps.r16[q], r[q], g.rows, k, 16) &&
         rows_map(&maps.r128[q], r[q], g.rows, k, 128);
  if (!ok) return cudaErrorInvalidValue;
  RowArgs a = {};
  a.offsets = offsets;
  a.err = err;
  a.rows = g.rows;
  a.groups = g.groups;
  a.cols = fwd ? job.n_out : job.n_in;
  a.k_blocks = (k + BK - 1) / BK;
  a.sources = job.a2 ? 2 : 1;
  a.out = job.out;
  a.out_f32 = job.out_f32;
  return fwd ? run_rows_sized<Mode::kFwd>(maps, a, st) : run_rows_sized<Mode::kDx>(maps, a, st);
}

cudaError_t launch_swiglu_backward_tc(const GroupedShape& g, const void* x, const void* w_gate,
                                      const void* w_up, const float* dh, void* h, void* da,
                                      void* du, int d, int F, const int32_t* offsets,
                                      int32_t* err, cudaStream_t st) {
  RowMaps maps;
  const void* w[2] = {w_gate, w_up};
  bool ok = true;
  for (int q = 0; q < 2; ++q)
    ok = ok && group_map(&maps.w[q], false, w[q], g.groups, F, d, 64, 128) &&
         rows_map(&maps.r16[q], x, g.rows, d, 16) && rows_map(&maps.r128[q], x, g.rows, d, 128);
  if (!ok) return cudaErrorInvalidValue;
  RowArgs a = {};
  a.offsets = offsets;
  a.err = err;
  a.rows = g.rows;
  a.groups = g.groups;
  a.cols = F;
  a.k_blocks = (d + BK - 1) / BK;
  a.sources = 1;
  a.out = h;
  a.dh = dh;
  a.da = static_cast<__nv_bfloat16*>(da);
  a.du = static_cast<__nv_bfloat16*>(du);
  return run_rows_sized<Mode::kGateUp>(maps, a, st);
}

cudaError_t launch_grouped_dw_tc(const GroupedShape& g, const GroupedJob* jobs, int n_jobs,
                                 const int32_t* offsets, int32_t* err, cudaStream_t st) {
  DwMaps maps = {};
  for (int q = 0; q < n_jobs; ++q) {
    const GroupedJob& j = jobs[q];
    DwJob& m = maps.job[q];
    m.n_out = j.n_out;
    m.n_in = j.n_in;
    const bool ok = rows_map(&m.a64, j.a, g.rows, j.n_out, 64) &&
                    rows_map(&m.a16, j.a, g.rows, j.n_out, 16) &&
                    rows_map(&m.a1, j.a, g.rows, j.n_out, 1) &&
                    rows_map(&m.b64, j.b, g.rows, j.n_in, 64) &&
                    rows_map(&m.b16, j.b, g.rows, j.n_in, 16) &&
                    rows_map(&m.b1, j.b, g.rows, j.n_in, 1) &&
                    group_map(&m.out, j.out_f32, j.out, g.groups, j.n_out, j.n_in,
                              j.out_f32 ? 32 : 64, 32);
    if (!ok) return cudaErrorInvalidValue;
  }
  DwArgs a = {};
  a.offsets = offsets;
  a.err = err;
  a.rows = g.rows;
  a.groups = g.groups;
  a.n_jobs = n_jobs;
  a.out_f32 = jobs[0].out_f32;
  static std::atomic<uint64_t> attr_set{0};
  static std::atomic<int> grids[64];
  return launch_persistent<true>(dw_gemm_kernel<true>, DwCfg<true>::kSmemBytes, attr_set, grids,
                                 st, maps, a);
}

}  // namespace moe
