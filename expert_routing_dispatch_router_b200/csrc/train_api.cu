// C ABI of the training calls: argument checks and launch order. Like the
// forward calls, every check runs on the host before the first launch, and
// nothing here allocates or synchronises.
#include <nvtx3/nvToolsExt.h>

#include "grouped.cuh"

namespace moe {
moe_status_t shape_from_config(const moe_config_t* c, Shape* sh);
}  // namespace moe

using namespace moe;

namespace {

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

bool dev_ok(const void* p) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

constexpr size_t kGroupedWs = 256;  // the error word and unit counters

moe_status_t grouped_check(const moe_grouped_t* c) {
  if (c == nullptr) return MOE_ERR_INVALID_ARG;
  if (c->rows < 0 || c->groups <= 0 || c->n_in <= 0 || c->n_out <= 0) return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_F32 && c->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (c->groups > kMaxExperts || c->n_in % 8 != 0 || c->n_out % 8 != 0 ||
      !grouped_fits(c->rows, c->groups, c->n_in, c->n_out))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status_t ws_check(const void* ws, size_t ws_bytes, size_t need) {
  if (ws == nullptr || ws_bytes < need) return MOE_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status_t grouped_call(const moe_grouped_t* c, Form form, const void* a, const void* b,
                          const int32_t* offsets, void* out, moe_dtype_t out_dtype, void* ws,
                          size_t ws_bytes, moe_stream_t stream) {
  moe_status_t s = grouped_check(c);
  if (s != MOE_OK) return s;
  const bool bf16 = c->dtype == MOE_BF16, out_f32 = out_dtype == MOE_F32;
  if (out_dtype != c->dtype && !(form == Form::kDw && out_f32)) return MOE_ERR_INVALID_ARG;
  if (c->rows == 0 && form != Form::kDw) return MOE_OK;  // no rows: nothing to write
  const size_t es = bf16 ? 2 : 4, os = out_f32 ? 4 : 2;
  const size_t w = (size_t)c->groups * c->n_in * c->n_out;
  const size_t ri = (size_t)c->rows * c->n_in, ro = (size_t)c->rows * c->n_out;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!dev_ok(out)) return MOE_ERR_INVALID_ARG;
  if (c->rows == 0)  // a gradient without rows is zero
    return cuda_status(cudaMemsetAsync(out, 0, w * os, st));
  if (!dev_ok(a) || !dev_ok(b) || !dev_ok(offsets)) return MOE_ERR_INVALID_ARG;
  if ((s = ws_check(ws, ws_bytes, kGroupedWs)) != MOE_OK) return s;
  const Span spans[5] = {
      {a, (form == Form::kFwd ? ri : ro) * es, false},
      {b, (form == Form::kDw ? ri : w) * es, false},
      {offsets, ((size_t)c->groups + 1) * 4, false},
      {ws, kGroupedWs, true},
      {out, form == Form::kDw ? w * os : (form == Form::kFwd ? ro : ri) * es, true}};
  if (!disjoint(spans)) return MOE_ERR_INVALID_ARG;
  const GroupedShape g{c->rows, c->groups, bf16};
  const GroupedJob job{form, a, b, nullptr, nullptr, out, c->n_in, c->n_out, out_f32};
  return cuda_status(launch_grouped_jobs(g, &job, 1, offsets, static_cast<int32_t*>(ws), st));
}

struct Sizes {  // bytes of the layer's buffers
  size_t tok, rows, slots4, w_router, w, off;
};
Sizes sizes_of(const Shape& sh) {
  Sizes z;
  z.tok = (size_t)sh.T * sh.d * sh.es;
  z.rows = (size_t)sh.T * sh.k * sh.d * sh.es;
  z.slots4 = (size_t)sh.T * sh.k * 4;
  z.w_router = (size_t)sh.E * sh.d * 4;
  z.w = (size_t)sh.N * sh.F * sh.d * sh.es;
  z.off = (size_t)(sh.N + 1) * 4;
  return z;
}

// Config checks of the backward calls: those of the forward ones, and unit
// numbers of the products that fit 32 bits.
moe_status_t backward_shape(const moe_config_t* cfg, Shape* sh) {
  const moe_status_t s = shape_from_config(cfg, sh);
  if (s != MOE_OK) return s;
  if (!grouped_fits(sh->T * sh->k, sh->N, sh->d, sh->F)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool dw_dtype_ok(const Shape& sh, moe_dtype_t t) {
  return t == MOE_F32 || (t == MOE_BF16 && sh.bf16);
}

}  // namespace

extern "C" {

size_t moe_grouped_workspace_size(const moe_grouped_t* shape) {
  return grouped_check(shape) == MOE_OK ? kGroupedWs : 0;
}

moe_status_t moe_grouped_matmul(const moe_grouped_t* shape, const void* x, const void* w,
                                const int32_t* offsets, void* y, void* ws, size_t ws_bytes,
                                moe_stream_t stream) {
  NvtxRange range("moe_grouped_matmul");
  return grouped_call(shape, Form::kFwd, x, w, offsets, y,
                      shape ? shape->dtype : MOE_F32, ws, ws_bytes, stream);
}

moe_status_t moe_grouped_matmul_dx(const moe_grouped_t* shape, const void* dy, const void* w,
                                   const int32_t* offsets, void* dx, void* ws, size_t ws_bytes,
                                   moe_stream_t stream) {
  NvtxRange range("moe_grouped_matmul_dx");
  return grouped_call(shape, Form::kDx, dy, w, offsets, dx,
                      shape ? shape->dtype : MOE_F32, ws, ws_bytes, stream);
}

moe_status_t moe_grouped_matmul_dw(const moe_grouped_t* shape, const void* dy, const void* x,
                                   const int32_t* offsets, void* dw, moe_dtype_t dw_dtype,
                                   void* ws, size_t ws_bytes, moe_stream_t stream) {
  NvtxRange range("moe_grouped_matmul_dw");
  return grouped_call(shape, Form::kDw, dy, x, offsets, dw, dw_dtype, ws, ws_bytes, stream);
}

size_t moe_backward_workspace_size(const moe_config_t* cfg) {
  Shape sh;
  if (backward_shape(cfg, &sh) != MOE_OK) return 0;
  return backward_ws(sh).total;
}

moe_status_t moe_expert_ffn_backward(const moe_config_t* cfg, const void* x_perm,
                                     const int32_t* offsets, const void* w_gate,
                                     const void* w_up, const void* w_down, const void* dy_perm,
                                     void* dx_perm, void* dw_gate, void* dw_up, void* dw_down,
                                     moe_dtype_t dw_dtype, void* ws, size_t ws_bytes,
                                     moe_stream_t stream) {
  NvtxRange range("moe_expert_ffn_backward");
  Shape sh;
  moe_status_t s = backward_shape(cfg, &sh);
  if (s != MOE_OK) return s;
  if (!dw_dtype_ok(sh, dw_dtype)) return MOE_ERR_INVALID_ARG;
  if (sh.N == 0) return MOE_OK;  // no routed experts: nothing is read or written
  if (!dev_ok(dw_gate) || !dev_ok(dw_up) || !dev_ok(dw_down)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const Sizes z = sizes_of(sh);
  const size_t dwb = z.w / sh.es * (dw_dtype == MOE_F32 ? 4 : 2);
  if (sh.T == 0) {  // the gradient of no tokens
    for (void* p : {dw_gate, dw_up, dw_down})
      if (cudaMemsetAsync(p, 0, dwb, st) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if (!dev_ok(x_perm) || !dev_ok(offsets) || !dev_ok(w_gate) || !dev_ok(w_up) ||
      !dev_ok(w_down) || !dev_ok(dy_perm) || !dev_ok(dx_perm))
    return MOE_ERR_INVALID_ARG;
  if ((s = ws_check(ws, ws_bytes, backward_ws(sh).total)) != MOE_OK) return s;
  const Span spans[11] = {{x_perm, z.rows, false}, {offsets, z.off, false},
                          {w_gate, z.w, false},    {w_up, z.w, false},
                          {w_down, z.w, false},    {dy_perm, z.rows, false},
                          {dx_perm, z.rows, true}, {dw_gate, dwb, true},
                          {dw_up, dwb, true},      {dw_down, dwb, true},
                          {ws, backward_ws(sh).total, true}};
  if (!disjoint(spans)) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_expert_ffn_backward(sh, x_perm, offsets, w_gate, w_up, w_down,
                                                dy_perm, dx_perm, dw_gate, dw_up, dw_down,
                                                dw_dtype == MOE_F32, ws, st));
}

moe_status_t moe_combine_backward(const moe_config_t* cfg, const void* dout, const void* x,
                                  const void* y_perm, const int32_t* topk_idx,
                                  const float* topk_gate, const int32_t* slot_row,
                                  void* dy_perm, float* dgate, moe_stream_t stream) {
  NvtxRange range("moe_combine_backward");
  Shape sh;
  const moe_status_t s = backward_shape(cfg, &sh);
  if (s != MOE_OK) return s;
  if (sh.T == 0) return MOE_OK;  // empty batch: nothing is read or written
  if (!dev_ok(dout) || !dev_ok(x) || !dev_ok(y_perm) || !dev_ok(topk_idx) ||
      !dev_ok(topk_gate) || !dev_ok(slot_row) || !dev_ok(dy_perm) || !dev_ok(dgate))
    return MOE_ERR_INVALID_ARG;
  const Sizes z = sizes_of(sh);
  const Span spans[8] = {{dout, z.tok, false},         {x, z.tok, false},
                         {y_perm, z.rows, false},      {topk_idx, z.slots4, false},
                         {topk_gate, z.slots4, false}, {slot_row, z.slots4, false},
                         {dy_perm, z.rows, true},      {dgate, z.slots4, true}};
  if (!disjoint(spans)) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_combine_backward(sh, dout, x, y_perm, topk_idx, topk_gate, slot_row,
                                             dy_perm, dgate,
                                             reinterpret_cast<cudaStream_t>(stream)));
}

moe_status_t moe_input_backward(const moe_config_t* cfg, const void* dout, const void* x,
                                const float* w_router, const int32_t* topk_idx,
                                const float* topk_gate, const int32_t* slot_row,
                                const float* dgate, const void* dx_perm, void* dx,
                                float* dw_router, void* ws, size_t ws_bytes,
                                moe_stream_t stream) {
  NvtxRange range("moe_input_backward");
  Shape sh;
  moe_status_t s = backward_shape(cfg, &sh);
  if (s != MOE_OK) return s;
  if (!dev_ok(dw_router)) return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const Sizes z = sizes_of(sh);
  if (sh.T == 0)  // the gradient of no tokens
    return cuda_status(cudaMemsetAsync(dw_router, 0, z.w_router, st));
  if (!dev_ok(dout) || !dev_ok(x) || !dev_ok(w_router) || !dev_ok(topk_idx) ||
      !dev_ok(topk_gate) || !dev_ok(slot_row) || !dev_ok(dgate) || !dev_ok(dx_perm) ||
      !dev_ok(dx))
    return MOE_ERR_INVALID_ARG;
  if ((s = ws_check(ws, ws_bytes, backward_ws(sh).total)) != MOE_OK) return s;
  const Span spans[11] = {{dout, z.tok, false},         {x, z.tok, false},
                          {w_router, z.w_router, false}, {topk_idx, z.slots4, false},
                          {topk_gate, z.slots4, false}, {slot_row, z.slots4, false},
                          {dgate, z.slots4, false},     {dx_perm, z.rows, false},
                          {dx, z.tok, true},            {dw_router, z.w_router, true},
                          {ws, backward_ws(sh).total, true}};
  if (!disjoint(spans)) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_input_backward(sh, dout, x, w_router, topk_idx, topk_gate, slot_row,
                                           dgate, dx_perm, dx, dw_router, ws, st));
}

moe_status_t moe_layer_backward(const moe_config_t* cfg, const void* dout, const void* x,
                                const float* w_router, const void* w_gate, const void* w_up,
                                const void* w_down, const int32_t* topk_idx,
                                const float* topk_gate, const int32_t* offsets,
                                const int32_t* slot_row, const void* x_perm, const void* y_perm,
                                void* dx, float* dw_router, void* dw_gate, void* dw_up,
                                void* dw_down, moe_dtype_t dw_dtype, void* ws, size_t ws_bytes,
                                moe_stream_t stream) {
  NvtxRange range("moe_layer_backward");
  Shape sh;
  moe_status_t s = backward_shape(cfg, &sh);
  if (s != MOE_OK) return s;
  if (!dw_dtype_ok(sh, dw_dtype) || !dev_ok(dw_router)) return MOE_ERR_INVALID_ARG;
  if (sh.N > 0 && (!dev_ok(dw_gate) || !dev_ok(dw_up) || !dev_ok(dw_down)))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const Sizes z = sizes_of(sh);
  const size_t dwb = z.w / sh.es * (dw_dtype == MOE_F32 ? 4 : 2);
  if (sh.T == 0) {
    if (cudaMemsetAsync(dw_router, 0, z.w_router, st) != cudaSuccess) return MOE_ERR_CUDA;
    if (sh.N > 0)
      for (void* p : {dw_gate, dw_up, dw_down})
        if (cudaMemsetAsync(p, 0, dwb, st) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if (!dev_ok(dout) || !dev_ok(x) || !dev_ok(w_router) || !dev_ok(topk_idx) ||
      !dev_ok(topk_gate) || !dev_ok(slot_row) || !dev_ok(dx))
    return MOE_ERR_INVALID_ARG;
  if (sh.N > 0 && (!dev_ok(w_gate) || !dev_ok(w_up) || !dev_ok(w_down) || !dev_ok(offsets) ||
                   !dev_ok(x_perm) || !dev_ok(y_perm)))
    return MOE_ERR_INVALID_ARG;
  const BackwardWs L = backward_ws(sh);
  if ((s = ws_check(ws, ws_bytes, L.total)) != MOE_OK) return s;
  const size_t on = sh.N > 0 ? 1 : 0;
  const Span spans[18] = {{dout, z.tok, false},          {x, z.tok, false},
                          {w_router, z.w_router, false}, {topk_idx, z.slots4, false},
                          {topk_gate, z.slots4, false},  {slot_row, z.slots4, false},
                          {offsets, on * z.off, false},  {x_perm, on * z.rows, false},
                          {y_perm, on * z.rows, false},  {w_gate, z.w, false},
                          {w_up, z.w, false},            {w_down, z.w, false},
                          {dx, z.tok, true},             {dw_router, z.w_router, true},
                          {dw_gate, dwb, true},          {dw_up, dwb, true},
                          {dw_down, dwb, true},          {ws, L.total, true}};
  if (!disjoint(spans)) return MOE_ERR_INVALID_ARG;
  uint8_t* base = static_cast<uint8_t*>(ws);
  void* dy_perm = base + L.dy_perm;
  void* dx_perm = base + L.dx_perm;
  float* dgate = reinterpret_cast<float*>(base + L.dgate);
  cudaError_t e;
  {
    NvtxRange r("moe.combine_backward");
    e = launch_combine_backward(sh, dout, x, y_perm, topk_idx, topk_gate, slot_row, dy_perm,
                                dgate, st);
  }
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  if (sh.N > 0) {
    NvtxRange r("moe.expert_ffn_backward");
    e = launch_expert_ffn_backward(sh, x_perm, offsets, w_gate, w_up, w_down, dy_perm, dx_perm,
                                   dw_gate, dw_up, dw_down, dw_dtype == MOE_F32, ws, st);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
  }
  NvtxRange r("moe.input_backward");
  return cuda_status(launch_input_backward(sh, dout, x, w_router, topk_idx, topk_gate, slot_row,
                                           dgate, dx_perm, dx, dw_router, ws, st));
}

}  // extern "C"
