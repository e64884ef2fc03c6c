// Gradients of the layer around its grouped products: the combine's, the
// SwiGLU's, and those of the layer input and the router.
//
// With out = s sum_{routed} g_j y_j + sum_{zero} g_j x (the combine) and
// g = softmax of the selected logits l_j = x . w_router[e_j]:
//   dy_perm[row(t, j)] = s g_j dout_t
//   dg_j   = s <dout_t, y_j> for a routed slot, <dout_t, x_t> for a zero one
//   dl_j   = g_j (dg_j - sum_i g_i dg_i)
//   dx_t   = sum_{routed} dx_perm[row(t, j)] + (sum_{zero} g_j) dout_t
//            + sum_j dl_j w_router[e_j]
//   dw_router[e] = sum_{t that chose e} dl x_t
// The selection itself has no gradient, and so neither has the bias. All sums
// run in fp32 in a fixed order (slots j = 0..k-1, tokens in ascending order in
// fixed chunks), and activations are rounded once when they are stored.
#include "grouped.cuh"

namespace moe {
namespace {

// Two floats in one 64-bit register, and the operations on both at once: each
// half is rounded as the single operation would, at half the instructions.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ ulonglong2 load_pairs(const float* p) {
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
  return make_ulonglong2((uint64_t)u.y << 32 | u.x, (uint64_t)u.w << 32 | u.z);
}

// Element `at` of row `row`; rows are shorter than 2^32 elements, so one wide
// multiply has the offset.
template <typename T>
__device__ __forceinline__ const T* in_row(const T* p, int row, uint32_t d, int64_t col) {
  return p + col + (uint64_t)(uint32_t)row * d;
}

// 16 bytes of activations along d.
template <typename AT>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
  static constexpr int n = 8;
  uint4 u;
  __device__ void load(const __nv_bfloat16* p) { u = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ void load_any(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ float get(int i) const {
    const uint32_t w = i < 2 ? u.x : (i < 4 ? u.y : (i < 6 ? u.z : u.w));
    return (i & 1) ? __uint_as_float(w & 0xffff0000u) : __uint_as_float(w << 16);
  }
  __device__ uint64_t pair(int i) const { return pack2(get(2 * i), get(2 * i + 1)); }
  __device__ static void store(__nv_bfloat16* p, const float* v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Chunk<float> {
  static constexpr int n = 4;
  float4 f;
  __device__ void load(const float* p) { f = __ldg(reinterpret_cast<const float4*>(p)); }
  __device__ void load_any(const float* p) { f = *reinterpret_cast<const float4*>(p); }
  __device__ void zero() { f = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ float get(int i) const {
    return i == 0 ? f.x : (i == 1 ? f.y : (i == 2 ? f.z : f.w));
  }
  __device__ uint64_t pair(int i) const { return pack2(get(2 * i), get(2 * i + 1)); }
  __device__ static void store(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};

__device__ __forceinline__ float sum_warp(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// ------------------------------------------------------- combine backward --
constexpr int kSlotGroup = 8;  // 16-byte loads in flight together
constexpr int kCbThreads = 128;
constexpr size_t kCbStage = 40 * 1024;  // dout rows up to this size are staged

// One block per token, one warp per slot at a time: the warp reads the slot's
// expert output once, multiplies it into dout and writes dout times the gate.
// The token's dout row is staged in shared memory (STAGE; longer rows are read
// again from L2). Bound by HBM: y in, dy out. A slot whose id or row is outside
// the buffers gets a zero gate gradient; all zero-expert slots of a token share
// one sum.
template <typename AT, bool STAGE>
__global__ void __launch_bounds__(kCbThreads)
    combine_backward_kernel(const AT* __restrict__ dout, const AT* __restrict__ x,
                            const AT* __restrict__ y, const int32_t* __restrict__ idx,
                            const float* __restrict__ gate,
                            const int32_t* __restrict__ slot_row, AT* __restrict__ dy,
                            float* __restrict__ dgate, int64_t d, int N, int E, int k, float s,
                            int64_t rows) {
  constexpr int V = Chunk<AT>::n, W = kCbThreads / 32;
  extern __shared__ __align__(16) uint8_t s_raw[];
  AT* s_dout = reinterpret_cast<AT*>(s_raw);
  __shared__ int32_t s_row[kMaxTopK];  // row, -1: zero expert, -2: nothing
  __shared__ float s_gate[kMaxTopK];
  __shared__ float s_zero;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((int)threadIdx.x < k) {
    const int e = idx[t * k + threadIdx.x];
    const int r = slot_row[t * k + threadIdx.x];
    s_row[threadIdx.x] = e < 0 || e >= E ? -2 : (e >= N ? -1 : (r < 0 || r >= rows ? -2 : r));
    s_gate[threadIdx.x] = s * gate[t * k + threadIdx.x];
  }
  if (STAGE) {
    const uint4* src = reinterpret_cast<const uint4*>(dout + t * d);
    uint4* dst = reinterpret_cast<uint4*>(s_dout);
    for (int i = threadIdx.x; i < (int)(d / V); i += kCbThreads) dst[i] = __ldg(src + i);
  }
  __syncthreads();
  const AT* row = STAGE ? s_dout : dout + t * d;
  int first_zero = -1;
  for (int j = 0; j < k; ++j)
    if (first_zero < 0 && s_row[j] == -1) first_zero = j;
  // warp w takes the routed slots and, once, the zero experts' sum, in turn
  int turn = 0;
  for (int j = 0; j < k; ++j) {
    const int r = s_row[j];
    if (r < 0 && j != first_zero) continue;
    if (turn++ % W != warp) continue;
    const bool routed = r >= 0;
    const AT* in = routed ? y + (int64_t)r * d : x + t * d;
    AT* out = dy + (int64_t)(routed ? r : 0) * d;
    const float g = s_gate[j];
    float acc = 0.f;
    for (int64_t c0 = (int64_t)lane * V; c0 < d; c0 += 32 * V * kSlotGroup) {
      Chunk<AT> v[kSlotGroup];
#pragma unroll
      for (int q = 0; q < kSlotGroup; ++q) {
        const int64_t c = c0 + q * 32 * V;
        if (c < d)
          v[q].load(in + c);
        else
          v[q].zero();
      }
#pragma unroll
      for (int q = 0; q < kSlotGroup; ++q) {
        const int64_t c = c0 + q * 32 * V;
        if (c >= d) continue;
        Chunk<AT> b;
        b.load_any(row + c);
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          acc = fmaf(b.get(i), v[q].get(i), acc);
          o[i] = g * b.get(i);
        }
        if (routed) Chunk<AT>::store(out + c, o);
      }
    }
    acc = sum_warp(acc);
    if (lane == 0) {
      if (routed)
        dgate[t * k + j] = s * acc;
      else
        s_zero = acc;
    }
  }
  __syncthreads();
  if ((int)threadIdx.x < k && s_row[threadIdx.x] < 0)
    dgate[t * k + threadIdx.x] = s_row[threadIdx.x] == -1 ? s_zero : 0.f;
}

template <typename AT>
cudaError_t combine_backward(const Shape& sh, const void* dout, const void* x, const void* y,
                             const int32_t* idx, const float* gate, const int32_t* slot_row,
                             void* dy, float* dgate, cudaStream_t st) {
  const size_t bytes = (size_t)sh.d * sizeof(AT);
  const bool stage = bytes <= kCbStage;
  return launch_pdl(stage ? combine_backward_kernel<AT, true> : combine_backward_kernel<AT, false>,
                    dim3((unsigned)sh.T), dim3(kCbThreads), stage ? bytes : 0, st,
                    static_cast<const AT*>(dout), static_cast<const AT*>(x),
                    static_cast<const AT*>(y), idx, gate, slot_row, static_cast<AT*>(dy), dgate,
                    sh.d, (int)sh.N, (int)sh.E, (int)sh.k, sh.s, sh.T * sh.k);
}

// -------------------------------------------------------- SwiGLU backward --
// The float layers' SwiGLU backward, for routed rows: da and du hold the
// pre-activations a and u and are replaced,
//   h = silu(a) u, da = dh u sig(a) (1 + a (1 - sig(a))), du = dh silu(a).
__global__ void __launch_bounds__(256)
    swiglu_backward_kernel(const float* __restrict__ dh, const int32_t* __restrict__ offsets,
                           int N, int64_t rows, int64_t F, float* __restrict__ h, float* da,
                           float* du) {
  griddep_wait();
  griddep_launch_dependents();
  // the rows end at the largest offset (segment_table's running maximum)
  int32_t end = 0;
  for (int i = threadIdx.x & 31; i <= N; i += 32) end = max(end, clamp_offset(offsets[i], rows));
  const int64_t R = __reduce_max_sync(0xffffffffu, end);
  for (int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 4; i < R * F;
       i += (int64_t)gridDim.x * blockDim.x * 4) {
    const float4 av = *reinterpret_cast<const float4*>(da + i);
    const float4 uv = *reinterpret_cast<const float4*>(du + i);
    const float4 gv = *reinterpret_cast<const float4*>(dh + i);
    const float as[4] = {av.x, av.y, av.z, av.w}, us[4] = {uv.x, uv.y, uv.z, uv.w};
    const float gs[4] = {gv.x, gv.y, gv.z, gv.w};
    float hh[4], dd[4], ee[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float sig = 1.0f / (1.0f + expf(-as[q]));
      const float silu = as[q] * sig;
      hh[q] = silu * us[q];
      dd[q] = gs[q] * us[q] * (sig + silu * (1.0f - sig));
      ee[q] = gs[q] * silu;
    }
    store4(h + i, make_float4(hh[0], hh[1], hh[2], hh[3]));
    store4(da + i, make_float4(dd[0], dd[1], dd[2], dd[3]));
    store4(du + i, make_float4(ee[0], ee[1], ee[2], ee[3]));
  }
}

// --------------------------------------------------- input and router grads --
// A token's slots, one per lane (lanes < k): the row of dx_perm (-1: none), the
// router row, the gate of a zero-expert slot (else 0), and the gradient of the
// slot's logit, dl = gate (dgate - sum gate dgate). A slot with an id outside
// [0, E) has none of them (e is -1).
struct Slot {
  int row, e;
  float zero, dl;
};
__device__ __forceinline__ Slot load_slot(const int32_t* __restrict__ idx,
                                          const float* __restrict__ gate,
                                          const float* __restrict__ dgate,
                                          const int32_t* __restrict__ slot_row, int64_t t, int N,
                                          int E, int k, int64_t rows) {
  const int lane = threadIdx.x & 31;
  Slot s{-1, -1, 0.f, 0.f};
  float g = 0.f, dg = 0.f;
  int e = -1, r = -1;
  if (lane < k) {
    e = idx[t * k + lane];
    r = slot_row[t * k + lane];
    g = gate[t * k + lane];
    dg = dgate[t * k + lane];
  }
  const float mean = sum_warp(g * dg);
  if (e >= 0 && e < E) {
    s.e = e;
    s.dl = g * (dg - mean);
    if (e >= N)
      s.zero = g;
    else if (r >= 0 && r < rows)
      s.row = r;
  }
  return s;
}

constexpr int kDwChunk = 128;   // slots per partial sum of the router gradient
constexpr int kDwThreads = 128;

// part[c, :] = sum over the slots of chunk c (of one expert) of dl x[token].
// chunk_start[e] is the first chunk of expert e (block 0 writes it).
template <typename AT>
__global__ void __launch_bounds__(kDwThreads)
    router_dw_part_kernel(const AT* __restrict__ x, const int32_t* __restrict__ offsets,
                          const int32_t* __restrict__ row_token,
                          const float* __restrict__ dl_row, int E, int64_t slots, int64_t d,
                          float* __restrict__ part, int32_t* __restrict__ chunk_start) {
  constexpr int V = Chunk<AT>::n;
  __shared__ int32_t s_off[kMaxExperts + 1], s_tile[kMaxExperts + 1], s_warp[32];
  __shared__ int32_t s_tok[kDwChunk];
  __shared__ float s_dl[kDwChunk];
  griddep_wait();
  griddep_launch_dependents();
  segment_table<kDwThreads, true>(offsets, E, slots, kDwChunk, 0, s_off, s_tile, s_warp);
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= E; i += kDwThreads) chunk_start[i] = s_tile[i];
  const int cb = (int)((d + kDwThreads * V - 1) / (kDwThreads * V));
  const int64_t units = (int64_t)s_tile[E] * cb;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int c = (int)(u / cb);
    const int64_t col = ((int64_t)(u % cb) * kDwThreads + threadIdx.x) * V;
    const int e = segment_of(s_tile, E, c);
    const int r0 = s_off[e] + (c - s_tile[e]) * kDwChunk;
    int n = s_off[e + 1] - r0;
    if (n > kDwChunk) n = kDwChunk;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kDwThreads) {
      s_tok[i] = row_token[r0 + i];
      s_dl[i] = dl_row[r0 + i];
    }
    __syncthreads();
    if (col < d) {
      uint64_t acc[V / 2];
#pragma unroll
      for (int i = 0; i < V / 2; ++i) acc[i] = 0;
      for (int r = 0; r < n; r += 8) {
        Chunk<AT> xv[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          if (r + q < n)
            xv[q].load(in_row(x, s_tok[r + q], (uint32_t)d, col));
          else
            xv[q].zero();
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          if (r + q >= n) continue;
          const uint64_t w = pack2(s_dl[r + q], s_dl[r + q]);
#pragma unroll
          for (int i = 0; i < V / 2; ++i) acc[i] = fma2(w, xv[q].pair(i), acc[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < V / 2; i += 2) {
        const float2 lo = unpack2(acc[i]), hi = unpack2(acc[i + 1]);
        store4(part + (int64_t)c * d + col + 2 * i, make_float4(lo.x, lo.y, hi.x, hi.y));
      }
    }
  }
}

// dw_router[e, :] = sum of e's chunks in order (zeros without any).
__global__ void __launch_bounds__(256)
    router_dw_sum_kernel(const float* __restrict__ part,
                         const int32_t* __restrict__ chunk_start, int64_t d,
                         float* __restrict__ dw) {
  griddep_wait();
  griddep_launch_dependents();
  const int e = blockIdx.x;
  const int64_t col = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * 4;
  if (col >= d) return;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  const int c1 = chunk_start[e + 1];
  for (int c = chunk_start[e]; c < c1; ++c) {
    const float4 p = *reinterpret_cast<const float4*>(part + (int64_t)c * d + col);
    v.x += p.x;
    v.y += p.y;
    v.z += p.z;
    v.w += p.w;
  }
  store4(dw + (int64_t)e * d + col, v);
}

// dx[t, :], one block per token and 128 vectors of columns. The first block of a
// token also puts the slots' dl into the order of the slot list.
template <typename AT>
__global__ void __launch_bounds__(128)
    input_dx_kernel(const AT* __restrict__ dout, const AT* __restrict__ dx_perm,
                    const float* __restrict__ w_router, const int32_t* __restrict__ idx,
                    const float* __restrict__ gate, const float* __restrict__ dgate,
                    const int32_t* __restrict__ slot_row, const int32_t* __restrict__ list_row,
                    float* __restrict__ dl_row, AT* __restrict__ dx, int64_t d, int N, int E,
                    int k, int64_t rows) {
  constexpr int V = Chunk<AT>::n;
  __shared__ int32_t s_row[kMaxTopK], s_e[kMaxTopK];
  __shared__ float s_dl[kMaxTopK], s_zero[kMaxTopK];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t t = blockIdx.x;
  const int64_t col = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * V;
  if (threadIdx.x < 32) {
    const Slot s = load_slot(idx, gate, dgate, slot_row, t, N, E, k, rows);
    if ((int)threadIdx.x < k) {
      s_row[threadIdx.x] = s.row;
      s_e[threadIdx.x] = s.e;
      s_dl[threadIdx.x] = s.dl;
      s_zero[threadIdx.x] = s.zero;
      const int r = blockIdx.y == 0 ? list_row[t * k + threadIdx.x] : -1;
      if (r >= 0 && r < rows) dl_row[r] = s.dl;
    }
  }
  Chunk<AT> g;
  if (col < d)
    g.load(dout + t * d + col);
  else
    g.zero();
  __syncthreads();
  if (col >= d) return;
  uint64_t acc[V / 2], r[V / 2];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) acc[i] = r[i] = 0;
  for (int j0 = 0; j0 < k; j0 += kSlotGroup) {
    Chunk<AT> v[kSlotGroup];
#pragma unroll
    for (int q = 0; q < kSlotGroup; ++q) {
      const int j = j0 + q;
      if (j < k && s_row[j] >= 0)
        v[q].load(in_row(dx_perm, s_row[j], (uint32_t)d, col));
      else
        v[q].zero();
    }
#pragma unroll
    for (int q = 0; q < kSlotGroup; ++q)
#pragma unroll
      for (int i = 0; i < V / 2; ++i) acc[i] = add2(acc[i], v[q].pair(i));
  }
  float zero = 0.f;
  bool any_zero = false;
  for (int j = 0; j < k; ++j) {
    zero += s_zero[j];
    any_zero |= s_e[j] >= N;
  }
  if (any_zero) {  // a token without zero experts does not see dout here
#pragma unroll
    for (int i = 0; i < V / 2; ++i) acc[i] = fma2(pack2(zero, zero), g.pair(i), acc[i]);
  }
  for (int j0 = 0; j0 < k; j0 += 4) {
    ulonglong2 w[4][V / 4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int i = 0; i < V / 4; ++i)
        w[q][i] = j0 + q < k && s_e[j0 + q] >= 0
                      ? load_pairs(in_row(w_router, s_e[j0 + q], (uint32_t)d, col) + 4 * i)
                      : make_ulonglong2(0, 0);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float dl = j0 + q < k ? s_dl[j0 + q] : 0.f;
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        r[2 * i] = fma2(pack2(dl, dl), w[q][i].x, r[2 * i]);
        r[2 * i + 1] = fma2(pack2(dl, dl), w[q][i].y, r[2 * i + 1]);
      }
    }
  }
  float out[V];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    const float2 o = unpack2(add2(acc[i], r[i]));
    out[2 * i] = o.x;
    out[2 * i + 1] = o.y;
  }
  Chunk<AT>::store(dx + t * d + col, out);
}

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off);
}

int64_t router_dw_chunks(const Shape& sh) { return sh.T * sh.k / kDwChunk + sh.E; }

// Slots up to which the list is sorted by one block in one launch instead of three
// kernels. The whole call (d = 2048) with one block / three kernels:
//   8 experts    2048 slots 39 / 39 us, 4096 slots 49 / 45, 6144 slots 58 / 51
//   40 experts   2048 slots 26 / 28, 4096 slots 46 / 41, 6144 slots 48 / 44
//   160 experts  2048 slots 19 / 24, 4096 slots 28 / 28, 6144 slots 35 / 34
//   320 experts  2048 slots 19 / 26, 4096 slots 25 / 30, 6144 slots 35 / 33
//   1024 experts 2048 slots 31 / 45, 4096 slots 38 / 50, more do not fit one block
constexpr int64_t kListOneBlock = 4096;

template <typename AT>
cudaError_t input_backward(const Shape& sh, const BackwardWs& L, const void* dout,
                           const void* x, const float* w_router, const int32_t* idx,
                           const float* gate, const int32_t* slot_row, const float* dgate,
                           const void* dx_perm, void* dx, float* dw_router, void* ws,
                           cudaStream_t st) {
  constexpr int V = Chunk<AT>::n;
  // the slot list of every expert: the dispatch's sort with no zero experts
  Shape all = sh;
  all.N = sh.E;
  all.Z = 0;
  int32_t* offsets = at<int32_t>(ws, L.offsets);
  int32_t* list_row = at<int32_t>(ws, L.slot_row);
  int32_t* token = at<int32_t>(ws, L.row_token);
  float* dl_row = at<float>(ws, L.dl_row);
  float* part = at<float>(ws, L.dw_part);
  int32_t* counts = at<int32_t>(ws, L.counts);
  cudaError_t e =
      launch_dispatch(all, x, idx, at<int32_t>(ws, L.chunk_base), counts, offsets, token,
                      list_row, nullptr, at<int32_t>(ws, L.header), st, nullptr, 0, 0,
                      sh.T * sh.k > kListOneBlock);
  if (e != cudaSuccess) return e;
  const AT *go = static_cast<const AT*>(dout), *gp = static_cast<const AT*>(dx_perm);
  AT* gx = static_cast<AT*>(dx);
  const int64_t slots = sh.T * sh.k;
  e = launch_pdl(input_dx_kernel<AT>,
                 dim3((unsigned)sh.T, (unsigned)((sh.d + 128 * V - 1) / (128 * V))), dim3(128),
                 0, st, go, gp, w_router, idx, gate, dgate, slot_row,
                 static_cast<const int32_t*>(list_row), dl_row, gx, sh.d, (int)sh.N, (int)sh.E,
                 (int)sh.k, slots);
  if (e != cudaSuccess) return e;
  const int64_t cb = (sh.d + kDwThreads * V - 1) / (kDwThreads * V);
  int64_t blocks = router_dw_chunks(sh) * cb;
  const int64_t cap = (int64_t)num_sms() * 12;
  if (blocks > cap) blocks = cap;
  e = launch_pdl(router_dw_part_kernel<AT>, dim3((unsigned)blocks), dim3(kDwThreads), 0, st,
                 static_cast<const AT*>(x), static_cast<const int32_t*>(offsets),
                 static_cast<const int32_t*>(token), static_cast<const float*>(dl_row),
                 (int)sh.E, sh.T * sh.k, sh.d, part, counts);
  if (e != cudaSuccess) return e;
  return launch_pdl(router_dw_sum_kernel,
                    dim3((unsigned)sh.E, (unsigned)((sh.d + 1023) / 1024)), dim3(256), 0, st,
                    static_cast<const float*>(part), static_cast<const int32_t*>(counts), sh.d,
                    dw_router);
}

cudaError_t swiglu_backward(const Shape& sh, const float* dh, const int32_t* offsets, void* h,
                            void* da, void* du, cudaStream_t st) {
  int64_t blocks = (sh.T * sh.k * sh.F / 4 + 255) / 256;
  const int64_t cap = (int64_t)num_sms() * 8;
  if (blocks > cap) blocks = cap;
  return launch_pdl(swiglu_backward_kernel, dim3((unsigned)blocks), dim3(256), 0, st, dh,
                    offsets, (int)sh.N, sh.T * sh.k, sh.F, static_cast<float*>(h),
                    static_cast<float*>(da), static_cast<float*>(du));
}

}  // namespace

BackwardWs backward_ws(const Shape& sh) {
  BackwardWs L;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t p = off;
    off = (off + bytes + kWsAlign - 1) / kWsAlign * kWsAlign;
    return p;
  };
  const size_t Tk = (size_t)(sh.T * sh.k), act = (size_t)sh.es;
  const bool routed = sh.N > 0;
  L.header = take(256);
  L.pre_a = take(routed ? Tk * sh.F * 4 : 0);
  L.pre_u = take(routed ? Tk * sh.F * 4 : 0);
  L.dh = take(routed && !sh.bf16 ? Tk * sh.F * 4 : 0);
  L.h = take(routed ? Tk * sh.F * act : 0);
  L.da = take(routed && sh.bf16 ? Tk * sh.F * 2 : 0);
  L.du = take(routed && sh.bf16 ? Tk * sh.F * 2 : 0);
  L.dy_perm = take(routed ? Tk * sh.d * act : 0);
  L.dx_perm = take(routed ? Tk * sh.d * act : 0);
  L.dgate = take(Tk * 4);
  L.dl_row = take(Tk * 4);
  L.chunk_base = take((size_t)sh.nchunks * sh.E * 4);
  L.counts = take((size_t)(sh.E + 1) * 4);
  L.offsets = take((size_t)(sh.E + 1) * 4);
  L.row_token = take(Tk * 4);
  L.slot_row = take(Tk * 4);
  L.dw_part = take((size_t)router_dw_chunks(sh) * sh.d * 4);
  L.total = off;
  return L;
}

cudaError_t launch_combine_backward(const Shape& sh, const void* dout, const void* x,
                                    const void* y_perm, const int32_t* idx, const float* gate,
                                    const int32_t* slot_row, void* dy_perm, float* dgate,
                                    cudaStream_t st) {
  return sh.bf16 ? combine_backward<__nv_bfloat16>(sh, dout, x, y_perm, idx, gate, slot_row,
                                                   dy_perm, dgate, st)
                 : combine_backward<float>(sh, dout, x, y_perm, idx, gate, slot_row, dy_perm,
                                           dgate, st);
}

cudaError_t launch_input_backward(const Shape& sh, const void* dout, const void* x,
                                  const float* w_router, const int32_t* idx, const float* gate,
                                  const int32_t* slot_row, const float* dgate,
                                  const void* dx_perm, void* dx, float* dw_router, void* ws,
                                  cudaStream_t st) {
  const BackwardWs L = backward_ws(sh);
  return sh.bf16 ? input_backward<__nv_bfloat16>(sh, L, dout, x, w_router, idx, gate, slot_row,
                                                 dgate, dx_perm, dx, dw_router, ws, st)
                 : input_backward<float>(sh, L, dout, x, w_router, idx, gate, slot_row, dgate,
                                         dx_perm, dx, dw_router, ws, st);
}

cudaError_t launch_expert_ffn_backward(const Shape& sh, const void* x_perm,
                                       const int32_t* offsets, const void* w_gate,
                                       const void* w_up, const void* w_down,
                                       const void* dy_perm, void* dx_perm, void* dw_gate,
                                       void* dw_up, void* dw_down, bool dw_f32, void* ws,
                                       cudaStream_t st) {
  const BackwardWs L = backward_ws(sh);
  const GroupedShape g{sh.T * sh.k, (int)sh.N, sh.bf16};
  int32_t* err = at<int32_t>(ws, L.header);
  float *pre_a = at<float>(ws, L.pre_a), *pre_u = at<float>(ws, L.pre_u);
  void* h = at<void>(ws, L.h);
  void* da = sh.bf16 ? at<void>(ws, L.da) : pre_a;
  void* du = sh.bf16 ? at<void>(ws, L.du) : pre_u;
  const int d = (int)sh.d, F = (int)sh.F;
  cudaError_t e;
  if (sh.bf16) {
    e = launch_swiglu_backward_tc(g, x_perm, w_gate, w_up, dy_perm, w_down, pre_a, pre_u, h, da,
                                  du, d, F, offsets, err, st);
  } else {
    float* dh = at<float>(ws, L.dh);
    const GroupedJob pre[3] = {{Form::kDx, dy_perm, w_down, nullptr, nullptr, dh, F, d, true},
                               {Form::kFwd, x_perm, w_gate, nullptr, nullptr, pre_a, d, F, true},
                               {Form::kFwd, x_perm, w_up, nullptr, nullptr, pre_u, d, F, true}};
    e = launch_grouped_jobs(g, pre, 3, offsets, err, st);
    if (e != cudaSuccess) return e;
    e = swiglu_backward(sh, dh, offsets, h, da, du, st);
  }
  if (e != cudaSuccess) return e;
  const GroupedJob dx{Form::kDx, da, w_gate, du, w_up, dx_perm, d, F, false};
  e = launch_grouped_jobs(g, &dx, 1, offsets, err, st);
  if (e != cudaSuccess) return e;
  const GroupedJob dw[3] = {
      {Form::kDw, da, x_perm, nullptr, nullptr, dw_gate, d, F, dw_f32},
      {Form::kDw, du, x_perm, nullptr, nullptr, dw_up, d, F, dw_f32},
      {Form::kDw, dy_perm, h, nullptr, nullptr, dw_down, F, d, dw_f32}};
  return launch_grouped_jobs(g, dw, 3, offsets, err, st);
}

}  // namespace moe
