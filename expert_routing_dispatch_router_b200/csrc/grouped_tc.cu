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
//   the experts' backward takes the pre-activations a = x W_gate^T and
//                u = x W_up^T in float (one launch), and then dh = dy W_down with
//                an epilogue that turns it, a and u into h, da and du
// On CTA pairs a segment's last rows, up to kMerge of them behind a full tile of
// 256, join that tile as a second MMA into the second accumulator: a unit of
// their own would load the weight tile again, and operands from L2 (about 75
// GB/s per SM) bound it.
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
constexpr int kDwThreads = 352;  // weight gradients: warp 10 loads the second operand
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
__device__ __forceinline__ void tma_load_4d(const CUtensorMap* map, uint32_t dst, uint32_t bar,
                                            int32_t x, int32_t y, int32_t z, int32_t w,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::"
      "bytes.L2::cache_hint [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d_pair(const CUtensorMap* map, uint32_t dst,
                                                 uint32_t leader_bar, int32_t x, int32_t y,
                                                 int32_t z, int32_t w, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::"
      "complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(leader_bar), "r"(x), "r"(y), "r"(z), "r"(w),
      "l"(policy)
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

// True in one lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p)::"memory");
  return p != 0;
}

// Four MMAs over one stage (64 contraction elements): descriptors a and b move
// on by ASTEP and BSTEP (in 16-byte units) from one to the next. accum is 0 for
// the first MMA of an accumulator. One statement, so the operands are set up
// once: an MMA issued by itself took about 90 cycles, whatever its N, and with
// the commit four of them took as long as the tensor core needs for N = 256.
template <bool PAIR, int ASTEP, int BSTEP>
__device__ __forceinline__ void mma_stage(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accum) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "setp.eq.b32 p, 0, 0;\n\t"
        "add.s64 a, %1, %5;\n\tadd.s64 b, %2, %6;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t"
        "add.s64 a, a, %5;\n\tadd.s64 b, b, %6;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t"
        "add.s64 a, a, %5;\n\tadd.s64 b, b, %6;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accum), "n"(ASTEP), "n"(BSTEP)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "setp.eq.b32 p, 0, 0;\n\t"
        "add.s64 a, %1, %5;\n\tadd.s64 b, %2, %6;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
        "add.s64 a, a, %5;\n\tadd.s64 b, b, %6;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t"
        "add.s64 a, a, %5;\n\tadd.s64 b, b, %6;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accum), "n"(ASTEP), "n"(BSTEP)
        : "memory");
}

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
  __device__ static void load_4d(const CUtensorMap* m, uint32_t dst, uint32_t bar, int32_t x,
                                 int32_t y, int32_t z, int32_t w, uint64_t pol) {
    tma_load_4d(m, dst, bar, x, y, z, w, pol);
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
  __device__ static void load_4d(const CUtensorMap* m, uint32_t dst, uint32_t bar, int32_t x,
                                 int32_t y, int32_t z, int32_t w, uint64_t pol) {
    tma_load_4d_pair(m, dst, bar, x, y, z, w, pol);
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
// In a CTA pair (PAIR) with acquire at cluster scope: the other CTA takes part in
// most phases, by arrivals, commits or copies, and what it did before is ordered
// before what follows here. (CTA scope for those that it does not: no faster.)
template <bool PAIR>
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  return PAIR ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity);
}
template <bool PAIR>
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity,
                                             volatile int* abort_flag, int32_t* err) {
  if (try_wait<PAIR>(bar, parity)) return true;
  const uint64_t t0 = ptx::global_timer_ns();
  while (true) {
    for (int i = 0; i < 64; ++i)
      if (try_wait<PAIR>(bar, parity)) return true;
    if (*abort_flag) return false;
    if (ptx::global_timer_ns() - t0 > kWaitLimitNs) {
      *abort_flag = 1;
      atomicCAS(err, 0, kErrWaitTimeout);
      return false;
    }
  }
}

// The same by a whole warp; every lane gets the same answer.
template <bool PAIR>
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                          int32_t* err) {
  return __all_sync(0xffffffffu, wait_bounded<PAIR>(bar, parity, abort_flag, err));
}

// Whether an mbarrier phase is complete, without waiting.
__device__ __forceinline__ bool phase_done(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
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

constexpr int kRing = 4;  // units handed out ahead
constexpr uint32_t kCtlBytes = 320;

// The barriers and small state behind the ring of operand tiles, and the hand
// -out of work units, common to both kernels. Units are taken in order from a
// counter in the workspace, so CTAs whose units were short take more of them.
// The (leader's) producer publishes each unit id, -1 at the end, in a ring of
// kRing slots in its own and its peer's shared memory; the other roles read
// their units from there and arrive on the ring_empty barrier of their own CTA:
// the MMA warp, the epilogue warps, a second producer if there is one (TWO), and
// in the peer its producers and epilogue warps. The epilogue warps of both CTAs
// arrive on the tempty barriers of their own CTA once they have read an
// accumulator. A thread of the peer's otherwise idle warp 1 passes both on to the
// leader with release at cluster scope, so a slot is stored to, and an accumulator
// written, only after everyone has read it. (Each reader could arrive there
// itself; at cluster scope it would first wait for its stores in flight, 1700 to
// 2600 cycles, and at a narrower one its reads would not be ordered before what
// the leader does next.) The last CTA (pair) to finish returns the counters to
// zero.
template <int S, bool PAIR, bool TWO>
struct Control {
  uint32_t bars;
  volatile int* abort_flag;
  uint32_t* tmem_slot;
  volatile int* ring;
  static constexpr uint32_t kRingOff = 8 * (2 * S + 6);  // behind the barriers and tmem_slot
  __device__ uint32_t ring_full(int r) const { return bars + kRingOff + 8u * r; }
  __device__ uint32_t ring_empty(int r) const { return bars + kRingOff + 32u + 8u * r; }
  // counters: [0] next unit, [1] CTAs (pairs) that have finished
  __device__ bool publish(int seq, int u, int32_t* err) const {
    const int r = seq % kRing;
    const uint32_t par = (uint32_t)(seq / kRing) & 1u;
    if (!wait_bounded<PAIR>(ring_empty(r), par ^ 1u, abort_flag, err)) return false;
    ring[r] = u;
    if (PAIR) {
      ptx::st_shared_cluster_u32(
          ptx::map_to_rank(ptx::smem_addr(const_cast<const int*>(ring + r)), 1), (uint32_t)u);
      ptx::mbar_arrive_remote(ptx::map_to_rank(ring_full(r), 1));
    }
    ptx::mbar_arrive(ring_full(r));
    return true;
  }
  __device__ bool take(int seq, int* u, int32_t* err) const {
    const int r = seq % kRing;
    const uint32_t par = (uint32_t)(seq / kRing) & 1u;
    if (!wait_bounded<PAIR>(ring_full(r), par, abort_flag, err)) return false;
    *u = ring[r];
    ptx::mbar_arrive(ring_empty(r));
    return true;
  }
  // The peer's warp 1 (one lane): once all of the peer has taken a unit, or has
  // read an accumulator, say so to the leader. It waits for three barriers at
  // once, so it asks them in turn. After the last take no accumulator is waited
  // for any more: the peer's epilogue takes it when its last unit is done.
  __device__ void relay(int32_t* err) const {
    int seq = 0, u = 0;
    bool published = false;  // unit seq is here, and not yet taken by all
    uint32_t acc_par = 0;    // bit b: the phase of tempty(b) to come
    uint64_t t0 = ptx::global_timer_ns();
    for (int idle = 0;; ++idle) {
      const int r = seq % kRing;
      const uint32_t par = (uint32_t)(seq / kRing) & 1u;
#pragma unroll
      for (int b = 0; b < 2; ++b)
        if (phase_done(tempty(b), (acc_par >> b) & 1u)) {
          ptx::mbar_arrive_remote(ptx::map_to_rank(tempty(b), 0));
          acc_par ^= 1u << b;
          idle = 0;
        }
      if (!published) {
        if (phase_done(ring_full(r), par)) {
          u = ring[r];
          published = true;
          idle = 0;
        }
      } else if (phase_done(ring_empty(r), par)) {
        ptx::mbar_arrive_remote(ptx::map_to_rank(ring_empty(r), 0));
        if (u < 0) return;
        published = false;
        ++seq;
        idle = 0;
      }
      if (idle == 0) t0 = ptx::global_timer_ns();
      if ((idle & 63) == 63) {
        if (*abort_flag) return;
        if (ptx::global_timer_ns() - t0 > kWaitLimitNs) {
          *abort_flag = 1;
          atomicCAS(err, 0, kErrWaitTimeout);
          return;
        }
      }
    }
  }
  // A warp's wait for a phase.
  __device__ bool wait(uint32_t bar, uint32_t parity, int32_t* err) const {
    return wait_warp<PAIR>(bar, parity, abort_flag, err);
  }
  // Next unit for the producer warp: the leader publishes the one it claimed
  // before, then claims another (after the arrivals, which would wait for the
  // atomic's return); the peer reads it.
  __device__ bool next(int seq, int total, int32_t* counters, int* claimed, int* u,
                       int32_t* err) const {
    if (PAIR && Cg<PAIR>::rank() != 0) return take_warp(seq, u, err);
    int v = -1;
    bool ok = true;
    if ((threadIdx.x & 31) == 0) {
      v = seq == 0 ? atomicAdd(counters, 1) : *claimed;
      if (v >= total) v = -1;
      ok = publish(seq, v, err);
      if (v >= 0) *claimed = atomicAdd(counters, 1);
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
    *u = __shfl_sync(0xffffffffu, v, 0);
    return ok;
  }
  // The same for a whole warp: lane 0 reads, all lanes get it.
  __device__ bool take_warp(int seq, int* u, int32_t* err) const {
    int v = -1;
    bool ok = true;
    if ((threadIdx.x & 31) == 0) ok = take(seq, &v, err);
    ok = __shfl_sync(0xffffffffu, ok, 0);
    *u = __shfl_sync(0xffffffffu, v, 0);
    return ok;
  }
  __device__ uint32_t full(int s) const { return bars + 8u * s; }
  __device__ uint32_t empty(int s) const { return bars + 8u * (S + s); }
  __device__ uint32_t tfull(int b) const { return bars + 8u * (2 * S + b); }
  __device__ uint32_t tempty(int b) const { return bars + 8u * (2 * S + 2 + b); }
  __device__ uint32_t mma_done() const { return bars + 8u * (2 * S + 4); }
  __device__ void init(uint8_t* smem, uint32_t sbase, uint32_t bar_off) {
    static_assert(kRing == 4 && kRingOff + 80 <= kCtlBytes, "barriers fit their bytes");
    bars = sbase + bar_off;
    tmem_slot = reinterpret_cast<uint32_t*>(smem + bar_off + 8 * (2 * S + 5));
    abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    ring = reinterpret_cast<volatile int*>(smem + bar_off + kRingOff + 64);
    if (threadIdx.x == 0) {
      for (int s = 0; s < S; ++s) {
        ptx::mbar_init(full(s), 1);
        ptx::mbar_init(empty(s), 1);
      }
      for (int b = 0; b < 2; ++b) {
        ptx::mbar_init(tfull(b), 1);
        // the epilogue; in the leader also the relay
        ptx::mbar_init(tempty(b), kEpiWarps + (PAIR && Cg<PAIR>::rank() == 0 ? 1 : 0));
      }
      ptx::mbar_init(mma_done(), 1);
      for (int r = 0; r < kRing; ++r) {
        ptx::mbar_init(ring_full(r), 1);
        // leader: MMA warp, epilogue, second producer, relay; peer: producer,
        // epilogue, second producer
        ptx::mbar_init(ring_empty(r),
                       1 + kEpiWarps + TWO + (PAIR && Cg<PAIR>::rank() == 0 ? 1 : 0));
      }
      *abort_flag = 0;
      ptx::fence_mbar_init();
    }
    if ((threadIdx.x >> 5) == 1) Cg<PAIR>::alloc(ptx::smem_addr(tmem_slot));
  }
  // An epilogue warp is done with accumulator b.
  __device__ void release(int b, int lane) const {
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(tempty(b));
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
  __device__ void finish(uint32_t tmem_base, int32_t* counters) const {
    ptx::tc_fence_before();
    __syncthreads();
    Cg<PAIR>::sync_all();  // neither CTA frees TMEM or exits while the pair works
    if (threadIdx.x == 0 && Cg<PAIR>::rank() == 0) {
      const int teams = (int)gridDim.x / (PAIR ? 2 : 1);
      if (atomicAdd(counters + 1, 1) == teams - 1) {  // nobody claims units any more
        counters[0] = 0;
        counters[1] = 0;
      }
    }
    if ((threadIdx.x >> 5) == 1) {
      ptx::tc_fence_after();
      Cg<PAIR>::dealloc(tmem_base);
    }
  }
};

// ------------------------------------------------------------ row products --
enum class Mode : int {
  kFwd,     // y, bf16
  kFwdF32,  // two weights for the same rows, float: a and u
  kDx,      // dx, bf16
  kSwiglu   // dh, turned into h, da and du
};
__host__ __device__ constexpr bool is_dx(Mode m) { return m == Mode::kDx || m == Mode::kSwiglu; }

struct RowArgs {
  const int32_t* offsets;
  int32_t* err;
  int32_t* counters;  // two, zero between launches
  int64_t rows;
  int groups;
  int cols;      // output columns
  int k_blocks;  // per source
  bool wide_w;   // kDx, kSwiglu: both 64-column blocks of a weight tile come in one copy
  int sources;   // 2: a second (weights, rows) pair extends the contraction
  // kFwd, kDx: out[0] bf16. kFwdF32: out[0] a, out[1] u. kSwiglu: out[0] h,
  // out[1] da, out[2] du, all bf16, from pre[0] a and pre[1] u.
  void* out[3];
  const float* pre[2];
};

constexpr int kRowBoxes = 4;  // boxes of 128, 64, 32 and 16 rows
struct RowMaps {
  CUtensorMap w[2];  // weights (kFwdF32: gate, up; kDx: the two sources)
  CUtensorMap r[2][kRowBoxes];
};

template <int BN_, bool PAIR_>
struct RowCfg {
  static constexpr bool PAIR = PAIR_;
  static constexpr int kCtas = PAIR ? 2 : 1;
  static constexpr int BN = BN_;                    // rows of a tile
  // rows that may join the last one (16 groups of 2048 x 6144, y and dx: 270 rows
  // 105 and 112-127 us with, 129 and 141-146 without; 256 and from 330 rows on the
  // same within 5 %)
  static constexpr int kMerge = PAIR ? 64 : 0;
  static constexpr int BNH = BN / kCtas;            // rows one CTA loads, and of those
  static constexpr int kMergeH = kMerge / kCtas;    // that join
  static_assert(BNH <= 128 && BN % (16 * kCtas) == 0, "rows of a unit");
  static constexpr uint32_t kStageBytes = kTileBytes + (BNH + kMergeH) * BK * 2;
  static constexpr int kStages = 221184 / kStageBytes > 8 ? 8 : (int)(221184 / kStageBytes);
  static constexpr uint32_t kBarOff = kStages * kStageBytes;
  static constexpr uint32_t kTabOff = kBarOff + kCtlBytes;
  static constexpr uint32_t kSmemBytes = 1024 + kTabOff + 2 * 4 * (kMaxExperts + 1) + 128;
  static_assert(kSmemBytes <= 232448, "shared memory of a CTA");
};

struct RowUnit {
  int e, m, row0, n, ntiles;  // n rows: the first BN, then those that join them
};

template <int BN>
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
  un.n = tt + 1 < un.ntiles ? BN : s_off[lo + 1] - un.row0;
  return un;
}

// 1 / (1 + e^-z), with the fast exponential and divide: their error is far
// below the bf16 rounding of h, da and du that follows (e^-z = infinity gives
// the limit 0).
__device__ __forceinline__ float sigmoid_f(float z) {
  return __fdividef(1.0f, 1.0f + __expf(-z));
}

// Stores 2 N rows of one column per lane: w[i] holds rows 2 i (low half) and
// 2 i + 1 of the lane's column. Lanes exchange halves in pairs, so that an even
// lane has row 2 i of two columns and an odd lane row 2 i + 1, and one 4-byte
// store per pair of rows writes both. out points at row 0 of the lane's column;
// rows from n on are not written (n differs between lanes of columns that exist
// and lanes of columns that do not, never within a pair).
template <int N>
__device__ __forceinline__ void store_row_pairs(const uint32_t (&w)[N], uint16_t* out,
                                                int64_t cols, int n) {
  const int odd = threadIdx.x & 1;
  uint16_t* p = out - odd + odd * cols;
  const uint32_t pick = odd ? 0x3276 : 0x5410;  // (other hi, own hi) or (own lo, other lo)
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, w[i], 1);
    const uint32_t v = __byte_perm(w[i], other, pick);
    if (2 * i + odd < n) *reinterpret_cast<uint32_t*>(p) = v;
    p += 2 * cols;
  }
}

template <Mode MODE, int BN_, bool PAIR_>
__global__ void __launch_bounds__(kThreads, 1)
    row_gemm_kernel(const __grid_constant__ RowMaps maps, const RowArgs args) {
  using C = RowCfg<BN_, PAIR_>;
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
  Control<S, PAIR, false> ctl;
  ctl.init(smem, sbase, C::kBarOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = G::rank();
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tensormap(&maps.w[0]);
    ptx::prefetch_tensormap(&maps.r[0][0]);
    ptx::prefetch_tensormap(&maps.r[0][kRowBoxes - 1]);
  }
  // everything above overlaps the previous kernel's tail
  griddep_wait();
  griddep_launch_dependents();
  segment_table<kThreads>(args.offsets, args.groups, args.rows, BN, C::kMerge, s_off, s_tile,
                          s_warp);
  ptx::tc_fence_before();
  __syncthreads();
  G::sync_all();  // both CTAs' barriers exist before any remote arrive
  ptx::tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(ctl.tmem_slot);
  // column tiles of one weight matrix, and of a unit row (kFwdF32: gate's, then
  // up's)
  const int tiles = (args.cols + BM * C::kCtas - 1) / (BM * C::kCtas);
  const int m_tiles = MODE == Mode::kFwdF32 ? 2 * tiles : tiles;
  const int total = s_tile[args.groups] * m_tiles;
  const int n_kb = args.k_blocks * args.sources;
  // rows of a unit's two MMAs, rounded up to what an MMA takes
  auto mma_rows = [](int n, int q) -> int {
    const int r = q == 0 ? (n < BN ? n : BN) : n - BN;
    return r > 0 ? (r + STEP - 1) / STEP * STEP : 0;
  };

  if (warp == 0) {
    // ---------------------------------------------------- TMA producer --
    // The warp stays converged and one lane issues.
    const bool elected = elect_one();
    const uint64_t pol_first = ptx::policy_evict_first();
    const uint64_t pol_normal = ptx::policy_evict_normal();
    const uint32_t full0 = G::at_leader(ctl.full(0));
    int stage = 0, claimed = 0;
    uint32_t phase = 0, armed = 0, armed_par = 0;
    bool ok = true;
    for (int seq = 0, u; ok; ++seq) {
      ok = ctl.next(seq, total, args.counters, &claimed, &u, args.err);
      if (!ok || u < 0) break;
      const RowUnit un = row_unit<BN>(u, s_tile, s_off, args.groups, m_tiles);
      const int half = mma_rows(un.n, 0) / C::kCtas;
      const int more = PAIR ? mma_rows(un.n, 1) / C::kCtas : 0;
      const int job = MODE == Mode::kFwdF32 && un.m >= tiles ? 1 : 0;
      const int col0 = ((un.m - job * tiles) * C::kCtas + (int)rank) * BM;
      const int brow = un.row0 + (int)rank * half;
      const uint32_t bytes = (uint32_t)C::kCtas * (kTileBytes + (uint32_t)(half + more) * 128u);
      // weights that only this unit reads (one row tile) are streamed
      const uint64_t pol_w = un.ntiles == 1 ? pol_first : pol_normal;
      for (int kb = 0; kb < n_kb; ++kb) {
        if (!(ok = ctl.wait(ctl.empty(stage), phase ^ 1u, args.err))) break;
        const int src = kb >= args.k_blocks ? 1 : 0;
        const int k0 = (kb - src * args.k_blocks) * BK;
        if (elected) {
          if (rank == 0) ptx::mbar_arrive_expect_tx(ctl.full(stage), bytes);
          const uint32_t fb = full0 + 8u * stage;
          const uint32_t a0 = sbase + stage * C::kStageBytes;
          if (!is_dx(MODE)) {
            G::load_3d(&maps.w[job], a0, fb, k0, col0, un.e, pol_w);
          } else if (args.wide_w) {
            G::load_4d(&maps.w[src], a0, fb, 0, k0, col0 / 64, un.e, pol_w);
          } else {
            G::load_3d(&maps.w[src], a0, fb, col0, k0, un.e, pol_w);
            G::load_3d(&maps.w[src], a0 + kBlockBytes, fb, col0 + 64, k0, un.e, pol_w);
          }
          uint32_t b0 = a0 + kTileBytes;
          int j = brow;
#pragma unroll
          for (int q = 0; q < kRowBoxes; ++q) {
            const int h = 128 >> q;
            if (half & h) {
              G::load_2d(&maps.r[src][q], b0, fb, k0, j, pol_normal);
              b0 += h * 128u;
              j += h;
            }
          }
          if (PAIR && more > 0)  // 16 or 32 rows
            G::load_2d(&maps.r[src][more == 32 ? 2 : 3], a0 + kTileBytes + C::BNH * 128u, fb, k0,
                       un.row0 + BN + (int)rank * more, pol_normal);
        }
        armed |= 1u << stage;
        armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && elected) ctl.settle_loads(armed, armed_par);
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA issuer --
    // Accumulators alternate: MMA number `slot` (a unit has one or two) uses
    // accumulator slot & 1.
    if (rank == 0) {
      const bool elected = elect_one();
      const uint64_t hi_k = ptx::desc_k_sw128(0), hi_mn = desc_mn_sw128(0);
      constexpr int kAStep = is_dx(MODE) ? 2048 / 16 : 32 / 16;
      constexpr uint32_t kFlags = is_dx(MODE) ? kAMn : 0u;
      int stage = 0;
      uint32_t phase = 0, slot = 0;
      bool ok = true, issued = false;
      for (int seq = 0, u; ok; ++seq) {
        ok = ctl.take_warp(seq, &u, args.err);
        if (!ok || u < 0) break;
        const RowUnit un = row_unit<BN>(u, s_tile, s_off, args.groups, m_tiles);
        const int n0 = mma_rows(un.n, 0), n1 = PAIR ? mma_rows(un.n, 1) : 0;
        if (!(ok = ctl.wait(ctl.tempty(slot & 1), ((slot >> 1) & 1u) ^ 1u, args.err))) break;
        if (n1 > 0 && !(ok = ctl.wait(ctl.tempty((slot + 1) & 1),
                                      (((slot + 1) >> 1) & 1u) ^ 1u, args.err)))
          break;
        ptx::tc_fence_after();
        const uint32_t i0 = ptx::idesc_bf16_f32(BM * C::kCtas, n0) | kFlags;
        const uint32_t i1 = ptx::idesc_bf16_f32(BM * C::kCtas, n1) | kFlags;
        const uint32_t d0 = tmem_base + (slot & 1) * kAccStride;
        const uint32_t d1 = tmem_base + ((slot + 1) & 1) * kAccStride;
        for (int kb = 0; kb < n_kb; ++kb) {
          if (!(ok = ctl.wait(ctl.full(stage), phase, args.err))) break;
          ptx::tc_fence_after();
          if (elected) {
            const uint32_t a0 = sbase + stage * C::kStageBytes;
            const uint64_t a = (is_dx(MODE) ? hi_mn : hi_k) | (a0 >> 4);
            const uint64_t b = hi_k | ((a0 + kTileBytes) >> 4);
            const uint32_t accum = kb != 0 ? 1u : 0u;
            mma_stage<PAIR, kAStep, 2>(d0, a, b, i0, accum);
            if (PAIR && n1 > 0)
              mma_stage<PAIR, kAStep, 2>(d1, a, b + (C::BNH * 128 >> 4), i1, accum);
            G::commit(ctl.empty(stage));
          }
          issued = true;
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (elected) {
          G::commit(ctl.tfull(slot & 1));
          if (n1 > 0) G::commit(ctl.tfull((slot + 1) & 1));
        }
        slot += n1 > 0 ? 2 : 1;
      }
      if (!ok && issued && elected) {  // MMAs already issued finish before TMEM is freed
        G::commit(ctl.mma_done());
        wait_cleanup(ctl.mma_done(), 0);
      }
      __syncwarp();
    } else {
      if (lane == 0) ctl.relay(args.err);
      __syncwarp();
    }
  } else {
    // -------------------------------------------------------- epilogue --
    const int ew = warp & 3;         // TMEM lane quarter this warp may access
    const int eh = (warp - 2) >> 2;  // which half of the 32-row chunks
    uint32_t next_slot = 0;
    bool ok = true;
    for (int seq = 0, u; ok && ctl.take_warp(seq, &u, args.err) && u >= 0; ++seq) {
      const RowUnit un = row_unit<BN>(u, s_tile, s_off, args.groups, m_tiles);
      const int job = MODE == Mode::kFwdF32 && un.m >= tiles ? 1 : 0;
      const int col = ((un.m - job * tiles) * C::kCtas + (int)rank) * BM + ew * 32 + lane;
      const int parts = PAIR && un.n > BN ? 2 : 1;
      // the rows that joined come first: they are few, and the next unit's
      // products wait for both accumulators
      for (int part = parts - 1; part >= 0; --part) {
        const uint32_t slot = next_slot + part;
        const int64_t obase = (int64_t)(un.row0 + part * BN) * args.cols + col;
        const int n_rows = part == 0 ? (un.n < BN ? un.n : BN) : un.n - BN;
        const int n_out = col < args.cols ? n_rows : 0;  // rows this lane stores
        // 32-row chunks, alternating between the two warps of this quarter:
        // chunk q covers rows 64 q + r0 ..
        const int r0 = 32 * eh;
        const uint32_t tb = tmem_base + (static_cast<uint32_t>(ew * 32) << 16) +
                            (slot & 1) * kAccStride + (uint32_t)r0;
        // kSwiglu takes half chunks of 16 rows (i -> row half_row(i)), whose
        // pre-activations are fetched one ahead
        auto half_row = [&](int i) { return 64 * (i >> 1) + r0 + 16 * (i & 1); };
        float a[16], v[16];
        auto fetch = [&](int i) {
          const int left = n_out - half_row(i);
          const float* pa = args.pre[0] + obase + (int64_t)half_row(i) * args.cols;
          const float* pv = args.pre[1] + obase + (int64_t)half_row(i) * args.cols;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            a[c] = c < left ? __ldg(pa) : 0.f;
            v[c] = c < left ? __ldg(pv) : 0.f;
            pa += args.cols;
            pv += args.cols;
          }
        };
        if (MODE == Mode::kSwiglu) fetch(0);  // while the unit's products still run
        ok = ctl.wait(ctl.tfull(slot & 1), (slot >> 1) & 1u, args.err);
        if (!ok) break;
        ptx::tc_fence_after();
        if (MODE == Mode::kSwiglu) {
          // the accumulator goes back as soon as its last rows have left TMEM
          const int halves = n_rows > r0 ? 2 * ((n_rows - r0 + 63) / 64) : 0;  // warp-uniform
          if (halves == 0) ctl.release(slot & 1, lane);
#pragma unroll 1
          for (int i = 0; i < halves; ++i) {
            uint32_t h2[8], da2[8], du2[8];
            float g[16];
            ptx::tmem_ld16(tb - r0 + half_row(i), g);
            if (i == halves - 1) ctl.release(slot & 1, lane);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              float x[2], y[2], z[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int n = 2 * c + k;
                const float sig = sigmoid_f(a[n]);
                const float silu = a[n] * sig;
                x[k] = silu * v[n];
                y[k] = g[n] * v[n] * (sig + silu * (1.0f - sig));
                z[k] = g[n] * silu;
              }
              const __nv_bfloat162 xb = __floats2bfloat162_rn(x[0], x[1]);
              const __nv_bfloat162 yb = __floats2bfloat162_rn(y[0], y[1]);
              const __nv_bfloat162 zb = __floats2bfloat162_rn(z[0], z[1]);
              h2[c] = *reinterpret_cast<const uint32_t*>(&xb);
              da2[c] = *reinterpret_cast<const uint32_t*>(&yb);
              du2[c] = *reinterpret_cast<const uint32_t*>(&zb);
            }
            if (i + 1 < halves) fetch(i + 1);
            const int64_t at = obase + (int64_t)half_row(i) * args.cols;
            const int left = n_out - half_row(i);
            store_row_pairs(h2, static_cast<uint16_t*>(args.out[0]) + at, args.cols, left);
            store_row_pairs(da2, static_cast<uint16_t*>(args.out[1]) + at, args.cols, left);
            store_row_pairs(du2, static_cast<uint16_t*>(args.out[2]) + at, args.cols, left);
          }
        } else {
          // the whole share leaves TMEM before anything is stored, so the next
          // unit's products wait for no store
          constexpr bool F32 = MODE == Mode::kFwdF32;
          constexpr int NQ = BN / 64, kPer = F32 ? 32 : 16;
          uint32_t w[NQ][kPer];
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            if (64 * q + r0 < n_rows) {  // warp-uniform
              float g[32];
              ptx::tmem_ld32(tb + 64 * q, g);
#pragma unroll
              for (int c = 0; c < kPer; ++c) {
                if (F32) {
                  w[q][c] = __float_as_uint(g[c]);
                } else {
                  const __nv_bfloat162 p = __floats2bfloat162_rn(g[2 * c % 32], g[(2 * c + 1) % 32]);
                  w[q][c] = *reinterpret_cast<const uint32_t*>(&p);
                }
              }
            }
          }
          ctl.release(slot & 1, lane);
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            if (64 * q + r0 < n_rows) {
              const int64_t at = obase + (int64_t)(64 * q + r0) * args.cols;
              const int left = n_out - 64 * q - r0;
              if (F32) {
                uint32_t* p = static_cast<uint32_t*>(job ? args.out[1] : args.out[0]) + at;
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                  if (c < left) *p = w[q][c % kPer];
                  p += args.cols;
                }
              } else {
                store_row_pairs(w[q], static_cast<uint16_t*>(args.out[0]) + at, args.cols, left);
              }
            }
          }
        }
      }
      next_slot += parts;
    }
  }
  ctl.finish(tmem_base, args.counters);
}

// -------------------------------------------------------- weight gradients --
constexpr int kBoxes = 4;  // boxes of 64, 16, 8 and 4 rows, then single rows
struct DwJob {
  CUtensorMap a[kBoxes + 1];  // dy, 64 columns wide (a[0]: 2 x 64 if n_out is a
                              // multiple of 64)
  CUtensorMap b[kBoxes + 1];  // x
  CUtensorMap out;            // dw: 32 rows of 128 bytes
  int n_out, n_in;
};
struct DwMaps {
  DwJob job[kMaxJobs];
};
struct DwArgs {
  const int32_t* offsets;
  int32_t* err;
  int32_t* counters;  // two, zero between launches
  int64_t rows;
  int groups;
  int n_jobs;
};

// A CTA pair computes tiles of 256 x 256: each CTA has 128 rows of dw (its own
// dy columns) and all 256 columns (half of the x columns in its own shared
// memory); TMEM holds two accumulators. A unit is a run of up to kRun tiles of
// one row of tiles. A segment of at most kASlots blocks of 64 rows keeps its dy
// panel in shared memory for the whole run, so only x streams: half the
// operand bytes of loading both, which is what bounds short segments (their
// operands come from L2 at about 64 bytes a clock and SM).
// The tensor cores cut where they add to an accumulator, so a chain over all rows
// of a long segment drifts when its terms have one sign: 5e-4 of the sum at 400000
// rows. A tile therefore starts a new accumulator every kChain rows (64 additions
// of 16 rows), and the epilogue adds them in registers, in order and rounding. It
// does so under the next chain's products.
struct DwCfg {
  static constexpr int kChain = 1024;
  static constexpr int kRun = 8;
  // Slots of dy and of x, of which shared memory holds twelve. 16 groups of 2048 x
  // 6144 in bf16, with 4 + 8 / 5 + 7 / 6 + 6: 100 and 500 rows within 3 % of each
  // other; 200 rows 111 / 111 / 114 us, 270 to 320 rows 142 / 123-128 / 128-131,
  // 330 to 380 rows 158-176 / 153-172 / 140-150, 400 rows 168 / 163 / 166.
  static constexpr int kASlots = 5, kBSlots = 7;
  static constexpr uint32_t kSlotBytes = 2 * kBlockBytes;  // 128 columns x 64 rows
  static constexpr uint32_t kOutBuf = 4096;  // one warp's 32 rows x 128 bytes
  static constexpr uint32_t kBOff = kASlots * kSlotBytes;
  static constexpr uint32_t kOutOff = kBOff + kBSlots * kSlotBytes;
  static constexpr uint32_t kBarOff = kOutOff + kEpiWarps * kOutBuf;
  static constexpr uint32_t kSmemBytes = 1024 + kBarOff + kCtlBytes;
  static_assert(kSmemBytes <= 232448, "shared memory of a CTA");
  static_assert(kChain % BK == 0 && kASlots * BK <= kChain, "a kept panel is one chain");
};

struct DwUnit {
  int job, e, it, jt0, jt1, row0, n_rows;
};

// Runs per row of tiles, of about equal length.
__host__ __device__ __forceinline__ int dw_runs(int n_in) {
  const int nj = (n_in + 255) / 256;
  return (nj + DwCfg::kRun - 1) / DwCfg::kRun;
}

// The offsets are read where a unit is taken up (shared memory is all operand
// slots), clamped and by their running maximum as in segment_table. That needs
// the offsets before only where they do not ascend anyway (!ascending).
__device__ __forceinline__ DwUnit dw_unit(int u, const int* first, const DwMaps& maps,
                                          const DwArgs& args, bool ascending) {
  DwUnit un;
  un.job = u >= first[2] ? 2 : (u >= first[1] ? 1 : 0);
  const DwJob& j = maps.job[un.job];
  const int v = u - first[un.job];
  const int nj = (j.n_in + 255) / 256, ni = (j.n_out + 255) / 256, runs = dw_runs(j.n_in);
  const int run = v % runs;
  un.it = (v / runs) % ni;
  un.e = v / runs / ni;
  un.jt0 = nj * run / runs;
  un.jt1 = nj * (run + 1) / runs;
  un.row0 = clamp_offset(__ldg(args.offsets + un.e), args.rows);
  if (!ascending)
    for (int i = 0; i < un.e; ++i)
      un.row0 = max(un.row0, clamp_offset(__ldg(args.offsets + i), args.rows));
  const int end = clamp_offset(__ldg(args.offsets + un.e + 1), args.rows);
  un.n_rows = end > un.row0 ? end - un.row0 : 0;
  return un;
}

// 128 columns (from x) of the n rows from r0, rounded up to 16 rows, into two
// 64-column blocks. Whole boxes where the rows are the segment's own; the last
// one to three rows by gather4 with row `oob` (outside the tensor: zeros), and
// boxes there for the rest of the 16.
__device__ __forceinline__ void dw_load(const CUtensorMap* maps, bool wide, uint32_t dst,
                                        uint32_t fb, int x, int r0, int n, int oob,
                                        uint64_t pol) {
  using G = Cg<true>;
  if (wide && n == BK) {  // maps[0] is 3-D: both blocks in one copy
    G::load_3d(maps, dst, fb, 0, r0, x / 64, pol);
    return;
  }
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int xb = x + 64 * b;
    const uint32_t d = dst + b * kBlockBytes;
    if (n == BK) {  // not wide
      G::load_2d(maps, d, fb, xb, r0, pol);
      continue;
    }
    int j = 0;
    for (; j + 16 <= n; j += 16) G::load_2d(maps + 1, d + j * 128u, fb, xb, r0 + j, pol);
    if (j + 8 <= n) {
      G::load_2d(maps + 2, d + j * 128u, fb, xb, r0 + j, pol);
      j += 8;
    }
    if (j + 4 <= n) {
      G::load_2d(maps + 3, d + j * 128u, fb, xb, r0 + j, pol);
      j += 4;
    }
    if (j < n) {
      G::gather4(maps + 4, d + j * 128u, fb, xb, r0 + j, j + 1 < n ? r0 + j + 1 : oob,
                 j + 2 < n ? r0 + j + 2 : oob, oob, pol);
      j += 4;
    }
    if (j & 4) {
      G::load_2d(maps + 3, d + j * 128u, fb, xb, oob, pol);
      j += 4;
    }
    if (j & 8) G::load_2d(maps + 2, d + j * 128u, fb, xb, oob, pol);
  }
}

template <bool OUT_F32>
__global__ void __launch_bounds__(kDwThreads, 1)
    dw_gemm_kernel(const __grid_constant__ DwMaps maps, const DwArgs args) {
  using C = DwCfg;
  using G = Cg<true>;
  constexpr int SA = C::kASlots, SB = C::kBSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = ptx::smem_addr(smem);
  // slots 0..SA-1 hold dy, SA..SA+SB-1 hold x; one pair of barriers each
  Control<SA + SB, true, true> ctl;
  ctl.init(smem, sbase, C::kBarOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = G::rank();
  griddep_wait();
  griddep_launch_dependents();
  bool falls = false;
  for (int i = threadIdx.x; i < args.groups; i += kDwThreads)
    falls |= clamp_offset(__ldg(args.offsets + i + 1), args.rows) <
             clamp_offset(__ldg(args.offsets + i), args.rows);
  ptx::tc_fence_before();
  const bool ascending = !__syncthreads_or(falls);
  G::sync_all();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(ctl.tmem_slot);
  int first_unit[kMaxJobs + 1];
  first_unit[0] = 0;
#pragma unroll
  for (int q = 0; q < kMaxJobs; ++q) {
    int n = 0;
    if (q < args.n_jobs)
      n = args.groups * ((maps.job[q].n_out + 255) / 256) * dw_runs(maps.job[q].n_in);
    first_unit[q + 1] = first_unit[q] + n;
  }
  const int total = first_unit[kMaxJobs];

  if (warp == 0 || warp == 10) {
    // --------------------------------------------------- TMA producers --
    // Warp 0 loads dy and hands out the units, warp 10 loads x: a slot costs its
    // producer about 380 cycles (wait, arm, copy, loop), and one warp for both
    // took longer than the products of a 64-row block, 512.
    const bool load_b = warp == 10;
    const bool elected = elect_one();
    const uint64_t pol = ptx::policy_evict_normal();
    const uint32_t full0 = G::at_leader(ctl.full(0));
    const int oob = (int)args.rows;
    const int base = load_b ? SA : 0, slots = load_b ? SB : SA;
    int slot = 0, claimed = 0;
    uint32_t phase = 0, armed = 0, armed_par = 0;
    bool ok = true;
    for (int seq = 0, u; ok; ++seq) {
      ok = load_b ? ctl.take_warp(seq, &u, args.err)
                  : ctl.next(seq, total, args.counters, &claimed, &u, args.err);
      if (!ok || u < 0) break;
      const DwUnit un = dw_unit(u, first_unit, maps, args, ascending);
      const DwJob& job = maps.job[un.job];
      const CUtensorMap* m = load_b ? job.b : job.a;
      const bool wide = (load_b ? job.n_in : job.n_out) % 64 == 0;
      // a dy panel that is kept is loaded once, for the first tile of the run
      const int jt1 = load_b || un.n_rows > SA * BK ? un.jt1 : un.jt0 + 1;
      for (int jt = un.jt0; jt < jt1 && ok; ++jt) {
        const int x = load_b ? jt * 256 + (int)rank * 128 : (un.it * 2 + (int)rank) * BM;
        for (int k0 = 0; k0 < un.n_rows; k0 += BK) {
          const int n = un.n_rows - k0 < BK ? un.n_rows - k0 : BK;
          const int at = base + slot;
          if (!(ok = ctl.wait(ctl.empty(at), phase ^ 1u, args.err))) break;
          if (elected) {
            if (rank == 0)
              ptx::mbar_arrive_expect_tx(ctl.full(at),
                                         2u * 2u * 128u * (uint32_t)((n + 15) & ~15));
            dw_load(m, wide, sbase + at * C::kSlotBytes, full0 + 8u * at, x, un.row0 + k0, n, oob,
                    pol);
          }
          armed |= 1u << at;
          armed_par = (armed_par & ~(1u << at)) | (phase << at);
          if (++slot == slots) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
    }
    if (!ok && elected) ctl.settle_loads(armed, armed_par);
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA issuer --
    if (rank == 0) {
      const bool elected = elect_one();
      const uint64_t hi = desc_mn_sw128(0);
      const uint32_t idesc = ptx::idesc_bf16_f32(256, 256) | kAMn | kBMn;
      int sa = 0, sb = 0, acc = 0;
      uint32_t pa = 0, pb = 0, acc_phase = 0;
      bool ok = true, issued = false;
      for (int seq = 0, u; ok; ++seq) {
        ok = ctl.take_warp(seq, &u, args.err);
        if (!ok || u < 0) break;
        const DwUnit un = dw_unit(u, first_unit, maps, args, ascending);
        if (un.n_rows == 0) continue;  // the epilogue writes zeros by itself
        const bool keep = un.n_rows <= SA * BK;
        const int sa0 = sa;
        const uint32_t pa0 = pa;
        for (int jt = un.jt0; jt < un.jt1 && ok; ++jt) {
          const bool load_a = jt == un.jt0 || !keep;
          const bool free_a = jt == un.jt1 - 1 || !keep;
          if (keep) {  // each tile of the run reads the same slots
            sa = sa0;
            pa = pa0;
          }
          for (int c0 = 0; c0 < un.n_rows && ok; c0 += C::kChain) {
            if (!(ok = ctl.wait(ctl.tempty(acc), acc_phase ^ 1u, args.err))) break;
            ptx::tc_fence_after();
            const uint32_t d0 = tmem_base + (uint32_t)acc * kAccStride;
            const int rows = un.n_rows - c0 < C::kChain ? un.n_rows - c0 : C::kChain;
            for (int k0 = 0; k0 < rows; k0 += BK) {
              if (load_a && !(ok = ctl.wait(ctl.full(sa), pa, args.err))) break;
              if (!(ok = ctl.wait(ctl.full(SA + sb), pb, args.err))) break;
              ptx::tc_fence_after();
              const int left = rows - k0;
              if (elected) {
                const uint64_t a = hi | ((sbase + sa * C::kSlotBytes) >> 4);
                const uint64_t b = hi | ((sbase + C::kBOff + sb * C::kSlotBytes) >> 4);
                if (left > BK - 16) {
                  mma_stage<true, 128, 128>(d0, a, b, idesc, k0 != 0 ? 1u : 0u);
                } else {
                  for (int kk = 0; kk * 16 < left; ++kk)
                    G::mma(d0, a + kk * 128, b + kk * 128, idesc, (k0 | kk) != 0 ? 1u : 0u);
                }
                G::commit(ctl.empty(SA + sb));
                if (free_a) G::commit(ctl.empty(sa));
              }
              issued = true;
              if (++sa == SA) {
                sa = 0;
                pa ^= 1u;
              }
              if (++sb == SB) {
                sb = 0;
                pb ^= 1u;
              }
            }
            if (!ok) break;
            if (elected) G::commit(ctl.tfull(acc));
            if (++acc == 2) {
              acc = 0;
              acc_phase ^= 1u;
            }
          }
        }
      }
      if (!ok && issued && elected) {
        G::commit(ctl.mma_done());
        wait_cleanup(ctl.mma_done(), 0);
      }
      __syncwarp();
    } else {
      if (lane == 0) ctl.relay(args.err);
      __syncwarp();
    }
  } else {
    // -------------------------------------------------------- epilogue --
    // A warp owns 32 rows (its TMEM lanes) and half of the 256 columns. It takes
    // its whole share out of TMEM and hands the accumulator back before it
    // stores anything. Each 128-byte-wide piece (64 bf16 or 32 float columns) is
    // laid out swizzled in shared memory and stored by TMA, which clips it to
    // the matrix.
    const int ew = warp & 3, eh = (warp - 2) >> 2;
    const uint32_t buf = sbase + C::kOutOff + (uint32_t)(warp - 2) * C::kOutBuf;
    constexpr int kWidth = OUT_F32 ? 32 : 64, kPieces = 128 / kWidth;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int seq = 0, u; ok && ctl.take_warp(seq, &u, args.err) && u >= 0; ++seq) {
      const DwUnit un = dw_unit(u, first_unit, maps, args, ascending);
      const DwJob& job = maps.job[un.job];
      const int n_out = job.n_out, n_in = job.n_in;
      const int row = (un.it * 2 + (int)rank) * BM + ew * 32;
      for (int jt = un.jt0; jt < un.jt1; ++jt) {
        float sum[4][32];  // this lane's row, 128 columns
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int c = 0; c < 32; ++c) sum[q][c] = 0.f;
        for (int c0 = 0; c0 < un.n_rows; c0 += C::kChain) {
          ok = ctl.wait(ctl.tfull(acc), acc_phase, args.err);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t tb = tmem_base + (static_cast<uint32_t>(ew * 32) << 16) +
                              (uint32_t)acc * kAccStride + (uint32_t)eh * 128u;
          if (c0 == 0) {
            ptx::tmem_ld32x2(tb, tb + 32, sum[0], sum[1]);
            ptx::tmem_ld32x2(tb + 64, tb + 96, sum[2], sum[3]);
          } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              float g[16];
              ptx::tmem_ld16(tb + 16 * q, g);
#pragma unroll
              for (int c = 0; c < 16; ++c) sum[q >> 1][16 * (q & 1) + c] += g[c];
            }
          }
          ctl.release(acc, lane);
          if (++acc == 2) {
            acc = 0;
            acc_phase ^= 1u;
          }
        }
        if (!ok) break;
#pragma unroll
        for (int q = 0; q < kPieces; ++q) {
          const int col = jt * 256 + eh * 128 + q * kWidth;
          if (row >= n_out || col >= n_in) continue;  // warp-uniform
          if (lane == 0) store_wait_read<0>();  // the last store has read the buffer
          __syncwarp();
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (OUT_F32) {
                w[i] = __float_as_uint(sum[q][4 * c + i]);
              } else {
                const int at = 64 * q + 8 * c + 2 * i;
                const __nv_bfloat162 p =
                    __floats2bfloat162_rn(sum[at >> 5][at & 31], sum[at >> 5][(at & 31) + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&p);
              }
            }
            st_shared_v4(buf + lane * 128u + (uint32_t)((c ^ (lane & 7)) << 4), w[0], w[1], w[2],
                         w[3]);
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&job.out, buf, col, row, un.e);
            store_commit();
          }
        }
      }
    }
    if (lane == 0) store_wait_all();
  }
  ctl.finish(tmem_base, args.counters);
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
            const uint64_t* strides, const uint32_t* box) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t d[4], st[4];
  cuuint32_t b[4], one[4] = {1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    if (i + 1 < rank) st[i] = strides[i];
  }
  return enc(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
             (cuuint32_t)rank, const_cast<void*>(base), d, st, b, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Row-major bf16 [rows, cols], box of 64 columns x box_rows.
bool rows_map(CUtensorMap* map, const void* base, int64_t rows, int cols, uint32_t box_rows) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
  const uint64_t strides[1] = {(uint64_t)cols * 2};
  const uint32_t box[2] = {64, box_rows};
  return encode(map, false, 2, base, dims, strides, box);
}
// The same as [cols / 64][rows][64], box of two 64-column blocks x 64 rows.
bool wide_rows_map(CUtensorMap* map, const void* base, int64_t rows, int cols) {
  const uint64_t dims[3] = {64, (uint64_t)rows, (uint64_t)cols / 64};
  const uint64_t strides[2] = {(uint64_t)cols * 2, 128};
  const uint32_t box[3] = {64, 64, 2};
  return encode(map, false, 3, base, dims, strides, box);
}
// [groups, n_out, n_in], box of box_cols columns x box_rows rows of one group.
bool group_map(CUtensorMap* map, bool f32, const void* base, int groups, int n_out, int n_in,
               uint32_t box_cols, uint32_t box_rows) {
  const uint64_t es = f32 ? 4 : 2;
  const uint64_t dims[3] = {(uint64_t)n_in, (uint64_t)n_out, (uint64_t)groups};
  const uint64_t strides[2] = {n_in * es, (uint64_t)n_out * n_in * es};
  const uint32_t box[3] = {box_cols, box_rows, 1};
  return encode(map, f32, 3, base, dims, strides, box);
}
// The same as [groups][n_in / 64][n_out][64], box of two blocks x 64 rows.
bool wide_group_map(CUtensorMap* map, const void* base, int groups, int n_out, int n_in) {
  const uint64_t dims[4] = {64, (uint64_t)n_out, (uint64_t)n_in / 64, (uint64_t)groups};
  const uint64_t strides[3] = {(uint64_t)n_in * 2, 128, (uint64_t)n_out * n_in * 2};
  const uint32_t box[4] = {64, 64, 2, 1};
  return encode(map, false, 4, base, dims, strides, box);
}

// Persistent launch: one CTA per SM, or as many pairs as can be resident.
template <bool PAIR, typename... KArgs, typename... Args>
cudaError_t launch_persistent(void (*kernel)(KArgs...), int threads, uint32_t smem,
                              std::atomic<uint64_t>& attr_set, std::atomic<int>* grids,
                              cudaStream_t st, Args&&... args) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = raise_smem_once(attr_set, kernel, (int)smem);
  if (e != cudaSuccess) return e;
  if (!PAIR)
    return launch_pdl(kernel, dim3(num_sms()), dim3(threads), smem, st,
                      std::forward<Args>(args)...);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(threads);
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
  using C = RowCfg<BN, PAIR>;
  static std::atomic<uint64_t> attr_set{0};
  static std::atomic<int> grids[64];
  return launch_persistent<PAIR>(row_gemm_kernel<MODE, BN, PAIR>, kThreads, C::kSmemBytes,
                                 attr_set, grids, st, maps, args);
}

template <Mode MODE>
cudaError_t run_rows_sized(const RowMaps& maps, const RowArgs& args, cudaStream_t st) {
  // Rows per group if the capacity were used and spread evenly (how many there
  // are is known on the device only). 32 groups of 1024 x 4096, y and dx, with
  // 64-row tiles / 128-row tiles / pairs of 256:
  //   32 rows    45, 43 /  46,  44 / 49, 51 us: a smaller tile, a deeper ring
  //   64 rows    47, 44 /  47,  45 / 50, 52
  //   65 rows    66, 75 /  49,  47 / 51, 53: a second tile loads the weights again
  //   128 rows   69, 78 /  52,  51 / 53, 56
  //   129 rows   94, 110 / 74,  80 / 55, 57
  // At an average of 32 hardly a group has more than 64 rows; at 128 half of
  // them have more, but few of those more than twice that.
  const int64_t avg = args.rows / args.groups;
  if (avg <= 32) return run_rows<MODE, 64, false>(maps, args, st);
  if (avg <= 128) return run_rows<MODE, 128, false>(maps, args, st);
  return run_rows<MODE, 256, true>(maps, args, st);
}

template <bool OUT_F32>
cudaError_t run_dw(const DwMaps& maps, const DwArgs& args, cudaStream_t st) {
  static std::atomic<uint64_t> attr_set{0};
  static std::atomic<int> grids[64];
  return launch_persistent<true>(dw_gemm_kernel<OUT_F32>, kDwThreads, DwCfg::kSmemBytes,
                                 attr_set, grids, st, maps, args);
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
  const bool wide = !fwd && job.n_in % 64 == 0;
  for (int q = 0; q < 2; ++q) {
    ok = ok && (wide ? wide_group_map(&maps.w[q], w[q], g.groups, job.n_out, job.n_in)
                     : group_map(&maps.w[q], false, w[q], g.groups, job.n_out, job.n_in, 64,
                                 fwd ? 128 : 64));
    for (int i = 0; i < kRowBoxes; ++i)
      ok = ok && rows_map(&maps.r[q][i], r[q], g.rows, k, 128u >> i);
  }
  if (!ok) return cudaErrorInvalidValue;
  RowArgs a = {};
  a.offsets = offsets;
  a.err = err;
  a.counters = err + kUnitCounter;
  a.rows = g.rows;
  a.groups = g.groups;
  a.cols = fwd ? job.n_out : job.n_in;
  a.k_blocks = (k + BK - 1) / BK;
  a.wide_w = wide;
  a.sources = job.a2 ? 2 : 1;
  a.out[0] = job.out;
  return fwd ? run_rows_sized<Mode::kFwd>(maps, a, st) : run_rows_sized<Mode::kDx>(maps, a, st);
}

cudaError_t launch_swiglu_backward_tc(const GroupedShape& g, const void* x, const void* w_gate,
                                      const void* w_up, const void* dy, const void* w_down,
                                      float* pre_a, float* pre_u, void* h, void* da, void* du,
                                      int d, int F, const int32_t* offsets, int32_t* err,
                                      cudaStream_t st) {
  RowMaps up, down;
  const void* w[2] = {w_gate, w_up};
  const bool wide = F % 64 == 0;
  bool ok = true;
  for (int q = 0; q < 2; ++q) {
    ok = ok && group_map(&up.w[q], false, w[q], g.groups, F, d, 64, 128) &&
         (wide ? wide_group_map(&down.w[q], w_down, g.groups, d, F)
               : group_map(&down.w[q], false, w_down, g.groups, d, F, 64, 64));
    for (int i = 0; i < kRowBoxes; ++i)
      ok = ok && rows_map(&up.r[q][i], x, g.rows, d, 128u >> i) &&
           rows_map(&down.r[q][i], dy, g.rows, d, 128u >> i);
  }
  if (!ok) return cudaErrorInvalidValue;
  RowArgs a = {};
  a.offsets = offsets;
  a.err = err;
  a.counters = err + kUnitCounter;
  a.rows = g.rows;
  a.groups = g.groups;
  a.cols = F;
  a.k_blocks = (d + BK - 1) / BK;
  a.sources = 1;
  a.out[0] = pre_a;
  a.out[1] = pre_u;
  const cudaError_t e = run_rows_sized<Mode::kFwdF32>(up, a, st);
  if (e != cudaSuccess) return e;
  a.wide_w = wide;
  a.pre[0] = pre_a;
  a.pre[1] = pre_u;
  a.out[0] = h;
  a.out[1] = da;
  a.out[2] = du;
  return run_rows_sized<Mode::kSwiglu>(down, a, st);
}

cudaError_t launch_grouped_dw_tc(const GroupedShape& g, const GroupedJob* jobs, int n_jobs,
                                 const int32_t* offsets, int32_t* err, cudaStream_t st) {
  DwMaps maps = {};
  for (int q = 0; q < n_jobs; ++q) {
    const GroupedJob& j = jobs[q];
    DwJob& m = maps.job[q];
    m.n_out = j.n_out;
    m.n_in = j.n_in;
    const uint32_t box[kBoxes + 1] = {64, 16, 8, 4, 1};
    bool ok = group_map(&m.out, j.out_f32, j.out, g.groups, j.n_out, j.n_in,
                        j.out_f32 ? 32 : 64, 32);
    for (int i = 0; i <= kBoxes; ++i)
      ok = ok &&
           (i == 0 && j.n_out % 64 == 0 ? wide_rows_map(&m.a[i], j.a, g.rows, j.n_out)
                                        : rows_map(&m.a[i], j.a, g.rows, j.n_out, box[i])) &&
           (i == 0 && j.n_in % 64 == 0 ? wide_rows_map(&m.b[i], j.b, g.rows, j.n_in)
                                       : rows_map(&m.b[i], j.b, g.rows, j.n_in, box[i]));
    if (!ok) return cudaErrorInvalidValue;
  }
  DwArgs a = {};
  a.offsets = offsets;
  a.err = err;
  a.counters = err + kUnitCounter;
  a.rows = g.rows;
  a.groups = g.groups;
  a.n_jobs = n_jobs;
  return jobs[0].out_f32 ? run_dw<true>(maps, a, st) : run_dw<false>(maps, a, st);
}

}  // namespace moe
