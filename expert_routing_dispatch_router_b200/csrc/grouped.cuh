// Internal declarations of the training operators: grouped products in three
// directions, the experts' backward pass, and the gradients of the combine and
// of the layer input.
#pragma once

#include "moe_internal.cuh"

namespace moe {

// Direction of a grouped product over the row segments of `groups` weight
// matrices w[e] of [n_out, n_in]:
//   kFwd  y[r, o]     = sum_i x[r, i] w[e][o, i]
//   kDx   dx[r, i]    = sum_o dy[r, o] w[e][o, i]
//   kDw   dw[e][o, i] = sum_{r of e} dy[r, o] x[r, i]
enum class Form : int { kFwd = 0, kDx = 1, kDw = 2 };

// One product. a holds the rows (x, dy, dy), b the weights (w, w, x). A
// second pair (kDx only) adds a2 w2 to the same output: the input gradient of
// two projections that share their input.
struct GroupedJob {
  Form form;
  const void* a;
  const void* b;
  const void* a2;
  const void* b2;
  void* out;
  int n_in, n_out;
  bool out_f32;  // out in float; else in the activation type
};
constexpr int kMaxJobs = 3;

// Workspace header of these calls (int32 words): [0] error code, and the
// tensor-core kernels' unit counters, which every launch returns to zero.
constexpr int kUnitCounter = 2;

struct GroupedShape {
  int64_t rows;  // capacity of the row buffers
  int groups;
  bool bf16;
};

// Runs independent products over the same segments, either all weight gradients
// or none: bf16 on the tensor cores, float on the CUDA cores. err: the workspace
// error word (bounded waits of the tensor-core kernels).
cudaError_t launch_grouped_jobs(const GroupedShape& g, const GroupedJob* jobs, int n_jobs,
                                const int32_t* offsets, int32_t* err, cudaStream_t st);
// Its tensor-core parts, and the first half of the experts' backward pass: from
// x, dy and the weights to h, da and du, with the pre-activations in float on
// the way.
cudaError_t launch_grouped_rows_tc(const GroupedShape& g, const GroupedJob& job,
                                   const int32_t* offsets, int32_t* err, cudaStream_t st);
cudaError_t launch_grouped_dw_tc(const GroupedShape& g, const GroupedJob* jobs, int n_jobs,
                                 const int32_t* offsets, int32_t* err, cudaStream_t st);
cudaError_t launch_swiglu_backward_tc(const GroupedShape& g, const void* x, const void* w_gate,
                                      const void* w_up, const void* dy, const void* w_down,
                                      float* pre_a, float* pre_u, void* h, void* da, void* du,
                                      int d, int F, const int32_t* offsets, int32_t* err,
                                      cudaStream_t st);
// Rows of a call. One work unit of the weight gradients is up to eight tiles over
// all rows of a segment, about 40 ns a row; at this limit that is a third of the
// time after which a wait for the next unit gives up.
constexpr int64_t kMaxGroupedRows = 1ll << 24;
// Sizes of a matrix. A row product is one chain of sums over its contraction,
// which drifts where the tensor cores cut: 1.3e-3 of a sum of terms of one sign at
// this limit, a third of bf16's half step. A unit of it also stays far inside the
// wait's bound, and the numbers of column tiles within 32 bits when multiplied.
constexpr int64_t kMaxGroupedDim = 1ll << 20;
// Whether a product keeps to that, and its unit numbers to 32 bits.
bool grouped_fits(int64_t rows, int64_t groups, int64_t n_in, int64_t n_out);

// ---- the experts' backward pass and the layer's other gradients ----
struct BackwardWs {   // byte offsets from the workspace's base
  size_t header;      // int32[64]: [0] error code
  size_t pre_a, pre_u;  // float [T*k, F]: the pre-activations (float layers:
                        // then their gradients da and du)
  size_t dh;          // float [T*k, F]: gradient of h (float layers)
  size_t h;           // act [T*k, F]
  size_t da, du;      // bf16 [T*k, F]: the pre-activations' gradients (bf16 layers)
  size_t dy_perm;     // act [T*k, d]  (whole-layer call)
  size_t dx_perm;     // act [T*k, d]  (whole-layer call)
  size_t dgate;       // float [T, k]  (whole-layer call)
  size_t dl_row;      // float [T*k]: the logits' gradients in the slot list's order
  size_t chunk_base;  // int32 [nchunks, E]
  size_t counts;      // int32 [E + 1]: slot counts, then the first chunk per expert
  size_t offsets;     // int32 [E + 1]: slots per expert, zero experts included
  size_t row_token;   // int32 [T*k]
  size_t slot_row;    // int32 [T*k]
  size_t dw_part;     // float [chunks, d] partial router-weight gradients
  size_t total;
};
BackwardWs backward_ws(const Shape& sh);

cudaError_t launch_expert_ffn_backward(const Shape& sh, const void* x_perm,
                                       const int32_t* offsets, const void* w_gate,
                                       const void* w_up, const void* w_down,
                                       const void* dy_perm, void* dx_perm, void* dw_gate,
                                       void* dw_up, void* dw_down, bool dw_f32, void* ws,
                                       cudaStream_t st);
cudaError_t launch_combine_backward(const Shape& sh, const void* dout, const void* x,
                                    const void* y_perm, const int32_t* idx, const float* gate,
                                    const int32_t* slot_row, void* dy_perm, float* dgate,
                                    cudaStream_t st);
cudaError_t launch_input_backward(const Shape& sh, const void* dout, const void* x,
                                  const float* w_router, const int32_t* idx, const float* gate,
                                  const int32_t* slot_row, const float* dgate,
                                  const void* dx_perm, void* dx, float* dw_router, void* ws,
                                  cudaStream_t st);

// ---- host helpers of the entry points ----
// A buffer of a call: outputs may share no byte with any other buffer.
struct Span {
  const void* p;
  size_t bytes;
  bool out;
};
template <int N>
bool disjoint(const Span (&s)[N]) {
  for (int i = 0; i < N; ++i)
    for (int j = i + 1; j < N; ++j) {
      if (!s[i].out && !s[j].out) continue;
      const uintptr_t a = reinterpret_cast<uintptr_t>(s[i].p);
      const uintptr_t b = reinterpret_cast<uintptr_t>(s[j].p);
      if (s[i].bytes && s[j].bytes && a < b + s[j].bytes && b < a + s[i].bytes) return false;
    }
  return true;
}

// ---- device helpers ----
// An offset within the row buffers.
__device__ __forceinline__ int32_t clamp_offset(int32_t o, int64_t rows) {
  return o < 0 ? 0 : (o > rows ? (int32_t)rows : o);
}
// Segment table of a block in shared memory: s_off[0..n] the row offsets,
// s_tile[0..n] the prefix sums of the segments' tiles of `tile` rows, where up
// to `slack` rows behind the last full tile count as part of it. Offsets are
// clamped to [0, rows] and replaced by their running maximum, so no table sends a
// kernel outside its buffers, gives a row to two segments, or has more tiles than
// the rows do (ASCENDING: they come from a sort and do not fall). All THREADS
// threads call it; s_warp holds 32 ints. Each thread takes `per` consecutive
// segments.
__device__ __forceinline__ int32_t segment_tiles(int32_t rows, int tile, int slack) {
  if (rows <= 0) return 0;
  return rows <= tile + slack ? 1 : (rows - slack + tile - 1) / tile;
}
// The table of offsets that fall, by one thread. Looking whether any falls takes
// the CUDA-core kernels up to 1 us, the others nothing that shows.
static __device__ __noinline__ void raise_segments(int n, int tile, int slack, int32_t* s_off,
                                                   int32_t* s_tile) {
  if (threadIdx.x == 0) {
    s_tile[0] = 0;
    for (int e = 0; e < n; ++e) {
      s_off[e + 1] = max(s_off[e + 1], s_off[e]);
      s_tile[e + 1] = s_tile[e] + segment_tiles(s_off[e + 1] - s_off[e], tile, slack);
    }
  }
  __syncthreads();
}
template <int THREADS, bool ASCENDING = false>
__device__ __forceinline__ void segment_table(const int32_t* __restrict__ offsets, int n,
                                              int64_t rows, int tile, int slack, int32_t* s_off,
                                              int32_t* s_tile, int32_t* s_warp) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int per = (n + THREADS - 1) / THREADS;
  for (int i = threadIdx.x; i <= n; i += THREADS) s_off[i] = clamp_offset(offsets[i], rows);
  __syncthreads();
  int32_t sum = 0;
  bool falls = false;
  for (int q = 0; q < per; ++q) {
    const int e = threadIdx.x * per + q;
    if (e < n) {
      const int32_t len = s_off[e + 1] - s_off[e];
      falls |= len < 0;
      sum += segment_tiles(len, tile, slack);
    }
  }
  int32_t incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int32_t o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) s_warp[wid] = incl;
  if (ASCENDING) {
    __syncthreads();
  } else if (__syncthreads_or(falls)) {
    raise_segments(n, tile, slack, s_off, s_tile);
    return;
  }
  int32_t before = incl - sum;
  for (int w = 0; w < wid; ++w) before += s_warp[w];
  for (int q = 0; q < per; ++q) {
    const int e = threadIdx.x * per + q;
    if (e < n) {
      s_tile[e] = before;
      before += segment_tiles(s_off[e + 1] - s_off[e], tile, slack);
      if (e == n - 1) s_tile[n] = before;
    }
  }
  __syncthreads();
}

// Largest e in [0, n) with s[e] <= v (s non-decreasing, s[0] <= v).
__device__ __forceinline__ int segment_of(const int32_t* s, int n, int v) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s[mid] <= v)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Four consecutive elements (8- or 16-byte aligned) widened to fp32.
__device__ __forceinline__ float4 load4(const float* p) {
  return __ldg(reinterpret_cast<const float4*>(p));
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, float4 v) {
  *reinterpret_cast<float4*>(p) = v;
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y);
  const __nv_bfloat162 b = __floats2bfloat162_rn(v.z, v.w);
  uint2 o;
  o.x = *reinterpret_cast<const uint32_t*>(&a);
  o.y = *reinterpret_cast<const uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p) = o;
}

}  // namespace moe
