// One AdamW step over many tensors at once, run between layer calls on the
// gradients of a backward pass (Loshchilov and Hutter, "Decoupled Weight Decay
// Regularization"). For every element, with t the step count after this step:
//   m = b1 m + (1 - b1) g            v = b2 v + (1 - b2) g g
//   p = (1 - lr wd) p - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// in fp32, whatever the types of the weights and gradients.
//
// States live in flat buffers of 256-element blocks; a tensor starts at a
// block of its own and its last block is padded (the padding stays zero).
//  32 bits: m and v as float.
//  8 bits:  m and r = sqrt(v) as e4m3 codes with one float scale per block,
//           scale = max |value| * (1 / 448) (448 is the largest e4m3 value; the
//           conversion saturates, so a quotient rounded above it is 448). The
//           root spans half the exponent range of v, so it fits a format with
//           4 exponent bits; a code that would round to zero from a positive r
//           takes the smallest step instead, because a second moment of zero
//           under a first moment that is not would blow the next update up.
//           The update itself uses the fp32 values of this step; only what is
//           kept for the next step is rounded to 8 bits.
// m, r and the codes come from explicitly rounded operations (no fused
// multiply-add), so the states are exactly reproducible from the formulas.
//
// The step count lives on the device, so a captured step counts on when it is
// replayed. Each thread block reads it, works out the step's coefficients in
// double precision and takes a ticket; the last one adds one to the count. One
// warp per state block: lane i owns elements 8 i .. 8 i + 7, so all accesses are
// 8- to 16-byte vectors and the block's maxima are warp reductions.
#include <cuda_fp8.h>
#include <float.h>
#include <math.h>

#include "grouped.cuh"

namespace moe {
namespace {

constexpr int kBlock = 256;
constexpr int kAdamThreads = 256;
constexpr int kAdamTable = 1024;  // tensors whose first blocks fit in shared memory

struct AdamState {  // moe_adamw_step's `state`, on the device
  int64_t step;
  uint32_t tickets;  // thread blocks that have read the count; zero between steps
  uint32_t unused;
};

struct AdamArgs {
  const moe_adamw_tensor_t* table;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  AdamState* state;
  int n_tensors;
  int64_t blocks;
  double lr, beta1, beta2;
  float b1, omb1, b2, omb2, eps, keep;
};

// 1 - b^t, kept out of the update kernel's registers.
__device__ __noinline__ double correction(double b, int64_t t) {
  return 1.0 - pow(b, (double)t);
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, float* v);
template <>
__device__ __forceinline__ void load8<float>(const float* p, int n, float* v) {
  if (n == 8) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.f;
  }
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, int n, float* v) {
  if (n == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? __bfloat162float(p[i]) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void save8(T* p, int n, const float* v);
template <>
__device__ __forceinline__ void save8<float>(float* p, int n, const float* v) {
  if (n == 8) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = v[i];
  }
}
template <>
__device__ __forceinline__ void save8<__nv_bfloat16>(__nv_bfloat16* p, int n, const float* v) {
  if (n == 8) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = __float2bfloat16_rn(v[i]);
  }
}

// Eight e4m3 codes times their block's scale (every e4m3 value is exact in
// half precision, which the conversion goes through).
__device__ __forceinline__ void widen8(const uint8_t* p, float scale, float* v) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  const uint32_t w[2] = {u.x, u.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        (__nv_fp8x2_storage_t)((w[i >> 1] >> (16 * (i & 1))) & 0xffffu), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[2 * i] = __fmul_rn(f.x, scale);
    v[2 * i + 1] = __fmul_rn(f.y, scale);
  }
}

// Codes of 8 values of a block and the block's scale. The maximum is taken on
// the magnitudes' bits, so a NaN (larger than infinity there) reaches the
// scale instead of being passed over. The quotients by the block's one scale
// are correctly rounded by Markstein's method (IBM J. Res. Dev. 34, 1990): from
// y = 1 / scale rounded, q = v y, and q + (v - q scale) y with fused
// operations. Scales whose reciprocal or remainders would leave the normal
// range (and NaN) take the divide.
template <bool ROOT>
__device__ __forceinline__ void narrow8(const float* v, uint8_t* p, float* scale_out, int lane) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  top = __reduce_max_sync(0xffffffffu, top);
  const float scale = __fmul_rn(__uint_as_float(top), 1.0f / 448.0f);
  uint32_t w[2] = {0, 0};
  if (scale > 0.f) {
    float q[8];
    if (scale > 1e-18f && scale < 1e18f) {
      const float y = __frcp_rn(scale);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float q0 = __fmul_rn(v[i], y);
        q[i] = __fmaf_rn(__fmaf_rn(-q0, scale, v[i]), y, q0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(v[i], scale);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f = make_float2(q[2 * i], q[2 * i + 1]);
      if (ROOT) {  // 2^-9 is the smallest step
        if (f.x > 0.f) f.x = fmaxf(f.x, 0.001953125f);
        if (f.y > 0.f) f.y = fmaxf(f.y, 0.001953125f);
      }
      w[i >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3)
                   << (16 * (i & 1));
    }
  }
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  if (lane == 0) *scale_out = scale;
}

template <typename PT, typename GT, bool EIGHT>
__global__ void __launch_bounds__(kAdamThreads) adamw_kernel(const AdamArgs a) {
  __shared__ int64_t s_first[kAdamTable];
  __shared__ float s_size, s_inv_root;  // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  griddep_wait();
  griddep_launch_dependents();
  if (threadIdx.x == 0 || threadIdx.x == 32) {  // a warp each
    const int64_t t = a.state->step + 1;
    const bool first = threadIdx.x == 0;
    const double c = correction(first ? a.beta1 : a.beta2, t);
    if (first)
      s_size = (float)(a.lr / c);
    else
      s_inv_root = (float)(1.0 / sqrt(c));
  }
  const int n_t = a.n_tensors;
  const bool in_smem = n_t <= kAdamTable;
  if (in_smem)
    for (int i = threadIdx.x; i < n_t; i += kAdamThreads) s_first[i] = a.table[i].first_block;
  __syncthreads();
  const float size = s_size, inv_root = s_inv_root;
  if (threadIdx.x == 0) {  // both of the block's reads of the count are done
    __threadfence();
    if (atomicAdd(&a.state->tickets, 1u) == gridDim.x - 1) {
      a.state->tickets = 0;
      a.state->step += 1;
    }
  }
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kAdamThreads / 32);
  for (int64_t b = (int64_t)blockIdx.x * (kAdamThreads / 32) + (threadIdx.x >> 5); b < a.blocks;
       b += warps) {
    int lo = 0, hi = n_t - 1;  // last tensor whose first block is <= b
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((in_smem ? s_first[mid] : a.table[mid].first_block) <= b)
        lo = mid;
      else
        hi = mid - 1;
    }
    const moe_adamw_tensor_t tn = a.table[lo];
    const int64_t at = (b - tn.first_block) * kBlock + lane * 8;  // in the tensor
    const int64_t left = at < 0 ? 0 : tn.n - at;  // no tensor has blocks before its own
    const int n = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
    const int64_t sat = b * kBlock + lane * 8;  // in the states
    float g[8], p[8], m[8], v[8], r[8];
    load8<GT>(static_cast<const GT*>(tn.grad) + at, n, g);
    if (tn.master)
      load8<float>(tn.master + at, n, p);
    else
      load8<PT>(static_cast<const PT*>(tn.param) + at, n, p);
    if (EIGHT) {
      widen8(static_cast<const uint8_t*>(a.m) + sat, a.m_scale[b], m);
      widen8(static_cast<const uint8_t*>(a.v) + sat, a.v_scale[b], r);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(r[i], r[i]);
    } else {
      load8<float>(static_cast<const float*>(a.m) + sat, 8, m);
      load8<float>(static_cast<const float*>(a.v) + sat, 8, v);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[i] = __fadd_rn(__fmul_rn(m[i], a.b1), __fmul_rn(g[i], a.omb1));
      v[i] = __fadd_rn(__fmul_rn(v[i], a.b2), __fmul_rn(__fmul_rn(g[i], a.omb2), g[i]));
      r[i] = __fsqrt_rn(v[i]);
      // the weights' quotient takes the fast divide (2 units), like its root
      const float step = __fdividef(m[i], __fmaf_rn(r[i], inv_root, a.eps));
      p[i] = __fsub_rn(__fmul_rn(p[i], a.keep), __fmul_rn(step, size));
    }
    if (tn.master) save8<float>(tn.master + at, n, p);
    save8<PT>(static_cast<PT*>(tn.param) + at, n, p);
    if (EIGHT) {
      narrow8<false>(m, static_cast<uint8_t*>(a.m) + sat, a.m_scale + b, lane);
      narrow8<true>(r, static_cast<uint8_t*>(a.v) + sat, a.v_scale + b, lane);
    } else {
      save8<float>(static_cast<float*>(a.m) + sat, 8, m);
      save8<float>(static_cast<float*>(a.v) + sat, 8, v);
    }
  }
}

template <typename PT, typename GT>
cudaError_t run_adamw(const AdamArgs& a, bool eight, cudaStream_t st) {
  int64_t grid = (a.blocks + kAdamThreads / 32 - 1) / (kAdamThreads / 32);
  const int64_t cap = (int64_t)num_sms() * 16;
  if (grid > cap) grid = cap;
  if (grid < 1) grid = 1;  // no tensors: the step still counts
  return launch_pdl(eight ? adamw_kernel<PT, GT, true> : adamw_kernel<PT, GT, false>,
                    dim3((unsigned)grid), dim3(kAdamThreads), 0, st, a);
}

bool ptr_ok(const void* p, uintptr_t mask) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & mask) == 0;
}

}  // namespace
}  // namespace moe

extern "C" moe_status_t moe_adamw_step(const moe_adamw_t* opt, const moe_adamw_params_t* params,
                                       const moe_adamw_tensor_t* table, void* m, float* m_scale,
                                       void* v, float* v_scale, void* state,
                                       moe_stream_t stream) {
  using namespace moe;
  if (opt == nullptr || params == nullptr) return MOE_ERR_INVALID_ARG;
  const moe_adamw_t& o = *opt;
  const moe_adamw_params_t& h = *params;
  if (o.n_tensors < 0 || o.total_blocks < 0 ||
      (o.param_dtype != MOE_F32 && o.param_dtype != MOE_BF16) ||
      (o.grad_dtype != MOE_F32 && o.grad_dtype != MOE_BF16) ||
      (o.state_bits != 8 && o.state_bits != 32))
    return MOE_ERR_INVALID_ARG;
  // betas in [0, 1), finite rates; eps > 0 (0 / 0 for an element that never
  // had a gradient), and with a quotient that the fast divide is good for: a
  // normal float below 2^126, to which sqrt(v) adds at most 2^91
  if (!(h.beta1 >= 0.0 && h.beta1 < 1.0 && h.beta2 >= 0.0 && h.beta2 < 1.0) ||
      !isfinite(h.lr) || h.lr < 0.0 || !isfinite(h.weight_decay) || h.weight_decay < 0.0 ||
      !(h.eps >= FLT_MIN && h.eps <= 1e30))
    return MOE_ERR_INVALID_ARG;
  if (!ptr_ok(state, 15)) return MOE_ERR_INVALID_ARG;
  const bool eight = o.state_bits == 8, any = o.total_blocks > 0;
  if (any && (o.n_tensors == 0 || !ptr_ok(table, 15) || !ptr_ok(m, 15) || !ptr_ok(v, 15) ||
              (eight && (!ptr_ok(m_scale, 15) || !ptr_ok(v_scale, 15)))))
    return MOE_ERR_INVALID_ARG;
  const size_t blocks = (size_t)o.total_blocks, codes = blocks * kBlock * (eight ? 1 : 4);
  const size_t scales = eight ? blocks * 4 : 0;
  const Span spans[6] = {{table, any ? o.n_tensors * sizeof(moe_adamw_tensor_t) : 0, false},
                         {m, codes, true},
                         {m_scale, scales, true},
                         {v, codes, true},
                         {v_scale, scales, true},
                         {state, sizeof(AdamState), true}};
  if (!disjoint(spans)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  AdamArgs a;
  a.table = table;
  a.m = m;
  a.v = v;
  a.m_scale = m_scale;
  a.v_scale = v_scale;
  a.state = static_cast<AdamState*>(state);
  a.n_tensors = any ? o.n_tensors : 0;
  a.lr = h.lr;
  a.beta1 = h.beta1;
  a.beta2 = h.beta2;
  a.blocks = o.total_blocks;
  a.b1 = (float)h.beta1;
  a.omb1 = (float)(1.0 - h.beta1);
  a.b2 = (float)h.beta2;
  a.omb2 = (float)(1.0 - h.beta2);
  a.eps = (float)h.eps;
  a.keep = (float)(1.0 - h.lr * h.weight_decay);
  const bool pb = o.param_dtype == MOE_BF16, gb = o.grad_dtype == MOE_BF16;
  cudaError_t e;
  if (pb)
    e = gb ? run_adamw<__nv_bfloat16, __nv_bfloat16>(a, eight, st)
           : run_adamw<__nv_bfloat16, float>(a, eight, st);
  else
    e = gb ? run_adamw<float, __nv_bfloat16>(a, eight, st)
           : run_adamw<float, float>(a, eight, st);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
