// Grouped products of float operands, on the CUDA cores: every form, any sizes
// that are multiples of 8.
//
// Each output tile of 64 x 64 is one block's work: 16 steps of the contraction
// at a time go through shared memory (both operands transposed to
// contraction-major, so a thread's 4 + 4 operands are two 16-byte reads) and
// 256 threads hold 4 x 4 sums each, in fp32. Blocks walk a list of tiles made
// on the spot from the offsets; the tiles of up to three independent products
// form one list, so the small products of a layer share a launch.
//   kFwd, kDx  tile = 64 rows of one segment x 64 output columns
//   kDw        tile = 64 x 64 of one group's matrix; a group without rows
//              contracts nothing and writes zeros
#include "grouped.cuh"

namespace moe {
namespace {

constexpr int kTile = 64, kStep = 16, kSimtThreads = 256;

struct SimtArgs {
  GroupedJob job[kMaxJobs];
  int n_jobs;
  int groups;
  int64_t rows;
  const int32_t* offsets;
};

// Stages 4 consecutive elements along the operand's contiguous direction.
// KCONT: the contraction index is contiguous; p points at (line, k0 + 4 q).
template <bool KCONT>
__device__ __forceinline__ void stage(float (*s)[kTile + 4], int line, int kk, float4 v) {
  if (KCONT) {
    s[kk][line] = v.x;
    s[kk + 1][line] = v.y;
    s[kk + 2][line] = v.z;
    s[kk + 3][line] = v.w;
  } else {
    *reinterpret_cast<float4*>(&s[kk][line]) = v;
  }
}

// acc += A B over one source. lines are tile rows (i) or columns (j).
template <Form FORM>
__device__ __forceinline__ void accumulate(const float* __restrict__ a, const float* __restrict__ b,
                                           int row0, int n_rows, int i0, int j0, int n_in,
                                           int n_out, float (*sa)[kTile + 4],
                                           float (*sb)[kTile + 4], float acc[4][4]) {
  const int tid = threadIdx.x, ti = (tid >> 4) * 4, tj = (tid & 15) * 4;
  const int K = FORM == Form::kFwd ? n_in : (FORM == Form::kDx ? n_out : n_rows);
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = 0; k0 < K; k0 += kStep) {
    float4 va = zero, vb = zero;
    // A: contraction-contiguous rows (kFwd, kDx) or output-contiguous (kDw)
    const int line = tid >> 2, kq = (tid & 3) * 4;   // 64 lines x 4 quads of k
    const int kr = tid >> 4, lq = (tid & 15) * 4;    // 16 k x 16 quads of lines
    if (FORM != Form::kDw) {
      if (line < n_rows && k0 + kq < K) va = load4(a + (int64_t)(row0 + line) * K + k0 + kq);
    } else if (k0 + kr < K && i0 + lq < n_out) {
      va = load4(a + (int64_t)(row0 + k0 + kr) * n_out + i0 + lq);
    }
    // B: w[j][k] (kFwd), w[k][j] (kDx), x[row k][j] (kDw)
    if (FORM == Form::kFwd) {
      if (j0 + line < n_out && k0 + kq < K) vb = load4(b + (int64_t)(j0 + line) * n_in + k0 + kq);
    } else if (k0 + kr < K && j0 + lq < n_in) {
      const int64_t at = FORM == Form::kDx ? k0 + kr : row0 + k0 + kr;
      vb = load4(b + at * n_in + j0 + lq);
    }
    __syncthreads();  // the previous step's reads are done
    if (FORM != Form::kDw)
      stage<true>(sa, line, kq, va);
    else
      stage<false>(sa, lq, kr, va);
    if (FORM == Form::kFwd)
      stage<true>(sb, line, kq, vb);
    else
      stage<false>(sb, lq, kr, vb);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kStep; ++k) {
      const float4 x = *reinterpret_cast<const float4*>(&sa[k][ti]);
      const float4 y = *reinterpret_cast<const float4*>(&sb[k][tj]);
      const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[p][q] = fmaf(xs[p], ys[q], acc[p][q]);
    }
  }
}

template <Form FORM>
__device__ __forceinline__ void run_tile(const GroupedJob& job, int64_t unit, int groups,
                                         const int32_t* s_off, const int32_t* s_tile,
                                         float (*sa)[kTile + 4], float (*sb)[kTile + 4]) {
  const int n_in = job.n_in, n_out = job.n_out;
  const int cols = FORM == Form::kFwd ? n_out : n_in;
  const int jt = (cols + kTile - 1) / kTile;
  const int tid = threadIdx.x, ti = (tid >> 4) * 4, tj = (tid & 15) * 4;
  float acc[4][4];
#pragma unroll
  for (int p = 0; p < 4; ++p)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[p][q] = 0.f;
  int e, row0, n_rows, i0 = 0;
  const int j0 = (int)(unit % jt) * kTile;
  if (FORM == Form::kDw) {
    const int it = (n_out + kTile - 1) / kTile;
    const int64_t rest = unit / jt;
    i0 = (int)(rest % it) * kTile;
    e = (int)(rest / it);
    row0 = s_off[e];
    n_rows = s_off[e + 1] - row0;
  } else {
    const int t = (int)(unit / jt);
    e = segment_of(s_tile, groups, t);
    row0 = s_off[e] + (t - s_tile[e]) * kTile;
    n_rows = s_off[e + 1] - row0;
    if (n_rows > kTile) n_rows = kTile;
  }
  const int64_t wn = (int64_t)n_in * n_out;
  const float* b = static_cast<const float*>(job.b) + (FORM == Form::kDw ? 0 : e * wn);
  accumulate<FORM>(static_cast<const float*>(job.a), b, row0, n_rows, i0, j0, n_in, n_out, sa,
                       sb, acc);
  if (FORM == Form::kDx && job.a2 != nullptr)
    accumulate<FORM>(static_cast<const float*>(job.a2),
                         static_cast<const float*>(job.b2) + e * wn, row0, n_rows, i0, j0, n_in,
                         n_out, sa, sb, acc);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const bool in = FORM == Form::kDw ? i0 + ti + p < n_out : ti + p < n_rows;
    if (in && j0 + tj < cols) {
      const int64_t at = FORM == Form::kDw
                             ? e * wn + (int64_t)(i0 + ti + p) * n_in + j0 + tj
                             : (int64_t)(row0 + ti + p) * cols + j0 + tj;
      const float4 v = make_float4(acc[p][0], acc[p][1], acc[p][2], acc[p][3]);
      store4(static_cast<float*>(job.out) + at, v);
    }
  }
}

__global__ void __launch_bounds__(kSimtThreads)
    grouped_simt_kernel(const __grid_constant__ SimtArgs args) {
  __shared__ __align__(16) float sa[kStep][kTile + 4];
  __shared__ __align__(16) float sb[kStep][kTile + 4];
  __shared__ int32_t s_off[kMaxExperts + 1], s_tile[kMaxExperts + 1], s_warp[32];
  griddep_wait();
  griddep_launch_dependents();
  segment_table<kSimtThreads>(args.offsets, args.groups, args.rows, kTile, 0, s_off, s_tile,
                              s_warp);
  int64_t first[kMaxJobs + 1];
  first[0] = 0;
#pragma unroll
  for (int q = 0; q < kMaxJobs; ++q) {
    int64_t n = 0;
    if (q < args.n_jobs) {
      const GroupedJob& j = args.job[q];
      const int it = (j.n_out + kTile - 1) / kTile, jt = (j.n_in + kTile - 1) / kTile;
      n = j.form == Form::kDw ? (int64_t)args.groups * it * jt
                              : (int64_t)s_tile[args.groups] * (j.form == Form::kFwd ? it : jt);
    }
    first[q + 1] = first[q] + n;
  }
  for (int64_t u = blockIdx.x; u < first[kMaxJobs]; u += gridDim.x) {
    const int q = u >= first[2] ? 2 : (u >= first[1] ? 1 : 0);
    const GroupedJob& j = args.job[q];
    const int64_t unit = u - first[q];
    if (j.form == Form::kFwd)
      run_tile<Form::kFwd>(j, unit, args.groups, s_off, s_tile, sa, sb);
    else if (j.form == Form::kDx)
      run_tile<Form::kDx>(j, unit, args.groups, s_off, s_tile, sa, sb);
    else
      run_tile<Form::kDw>(j, unit, args.groups, s_off, s_tile, sa, sb);
  }
}

}  // namespace

cudaError_t launch_grouped_simt(const GroupedShape& g, const GroupedJob* jobs, int n_jobs,
                                const int32_t* offsets, cudaStream_t st) {
  SimtArgs a;
  a.n_jobs = n_jobs;
  a.groups = g.groups;
  a.rows = g.rows;
  a.offsets = offsets;
  int64_t most = 0;  // no more blocks than tiles there can be
  for (int q = 0; q < n_jobs; ++q) {
    a.job[q] = jobs[q];
    const int64_t it = (jobs[q].n_out + kTile - 1) / kTile;
    const int64_t jt = (jobs[q].n_in + kTile - 1) / kTile;
    const int64_t rt = g.rows / kTile + (g.rows < g.groups ? g.rows : g.groups);
    most += jobs[q].form == Form::kDw ? g.groups * it * jt
                                      : rt * (jobs[q].form == Form::kFwd ? it : jt);
  }
  for (int q = n_jobs; q < kMaxJobs; ++q) a.job[q] = GroupedJob{};
  const int64_t cap = (int64_t)num_sms() * 6;
  const unsigned blocks = (unsigned)(most < 1 ? 1 : (most < cap ? most : cap));
  return launch_pdl(grouped_simt_kernel, dim3(blocks), dim3(kSimtThreads), 0, st, a);
}

cudaError_t launch_grouped_jobs(const GroupedShape& g, const GroupedJob* jobs, int n_jobs,
                                const int32_t* offsets, int32_t* err, cudaStream_t st) {
  if (!g.bf16) return launch_grouped_simt(g, jobs, n_jobs, offsets, st);
  if (jobs[0].form == Form::kDw)
    return launch_grouped_dw_tc(g, jobs, n_jobs, offsets, err, st);
  for (int q = 0; q < n_jobs; ++q) {
    const cudaError_t e = launch_grouped_rows_tc(g, jobs[q], offsets, err, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

bool grouped_fits(int64_t rows, int64_t groups, int64_t n_in, int64_t n_out) {
  const int64_t row_units = (rows / 64 + groups) * ((n_in > n_out ? n_in : n_out) / 64 + 1);
  const int64_t dw_units = groups * (n_in / 64 + 1) * (n_out / 64 + 1);
  return row_units < (1ll << 31) && dw_units < (1ll << 31) && rows < (1ll << 31) - 256;
}

}  // namespace moe
