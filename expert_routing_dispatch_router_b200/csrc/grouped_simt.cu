// Grouped products of float operands, on the CUDA cores: every form, any sizes
// that are multiples of 8.
//
// Each output tile is one block's work: 16 steps of the contraction at a time go
// through shared memory (both operands transposed to contraction-major, so a
// thread's 4 + 4 operands are two 16-byte reads; the next step's loads are in
// flight meanwhile) and a thread holds 4 x 4 sums, in fp32. Tiles are 64 x 64,
// one team of 256 threads; or, where those would leave SMs idle, 32 x 32 with
// four teams of 64 threads that take every fourth step and add their sums in a
// fixed order at the end: a small layer has few tiles with long contractions.
// Blocks walk a list of tiles made on the spot from the offsets; the tiles of up
// to three independent products form one list, so the small products of a layer
// share a launch.
//   kFwd, kDx  tile = rows of one segment x output columns
//   kDw        tile of one group's matrix; a group without rows contracts
//              nothing and writes zeros. The rows are summed in chains of kChain
//              and the chains' sums added: in one chain over millions of rows of
//              one sign the terms fall below a step of the sum (1.5e-2 off at
//              2^24 rows)
#include "grouped.cuh"

namespace moe {
namespace {

constexpr int kStep = 16, kSimtThreads = 256, kChain = 1024;

struct SimtArgs {
  GroupedJob job[kMaxJobs];
  int n_jobs;
  int groups;
  int64_t rows;
  const int32_t* offsets;
};

template <int TILE>
struct SimtCfg {
  static constexpr int kTeamThreads = (TILE / 4) * (TILE / 4);
  static constexpr int kTeams = kSimtThreads / kTeamThreads;
  static constexpr int kVecs = TILE * kStep / 4 / kTeamThreads;  // float4 per operand
  static constexpr int kLine = TILE + 4;  // padded line of a staged operand
};
// Staged operands of the teams, then (reused) the teams' sums of a tile.
template <int TILE>
union SimtSmem {
  float stage[SimtCfg<TILE>::kTeams][2][kStep][SimtCfg<TILE>::kLine];
  float sums[SimtCfg<TILE>::kTeams][TILE][TILE];
};

template <int TILE>
__device__ __forceinline__ void team_sync(int team) {
  if (SimtCfg<TILE>::kTeams == 1)
    __syncthreads();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "n"(SimtCfg<TILE>::kTeamThreads) : "memory");
}

// A thread's vectors of one operand for the step at k0. KCONT: the contraction
// index is contiguous, p + line * ld + k; else p + k * ld + line. Vector v of
// the step covers line v / 4, k 4 (v % 4) .. (KCONT), or k v / (TILE / 4) and
// lines 4 (v % (TILE / 4)) ..
template <int TILE, bool KCONT>
__device__ __forceinline__ void fetch(const float* __restrict__ p, int64_t ld, int lines, int K,
                                      int k0, int th, float4* v) {
  using C = SimtCfg<TILE>;
#pragma unroll
  for (int q = 0; q < C::kVecs; ++q) {
    const int i = th + q * C::kTeamThreads;
    const int line = KCONT ? i >> 2 : (i % (TILE / 4)) * 4;
    const int k = k0 + (KCONT ? (i & 3) * 4 : i / (TILE / 4));
    v[q] = line < lines && k < K ? load4(p + (KCONT ? line * ld + k : k * ld + line))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
  }
}
template <int TILE, bool KCONT>
__device__ __forceinline__ void stage(float (*s)[SimtCfg<TILE>::kLine], int th, const float4* v) {
  using C = SimtCfg<TILE>;
#pragma unroll
  for (int q = 0; q < C::kVecs; ++q) {
    const int i = th + q * C::kTeamThreads;
    if (KCONT) {
      const int line = i >> 2, k = (i & 3) * 4;
      s[k][line] = v[q].x;
      s[k + 1][line] = v[q].y;
      s[k + 2][line] = v[q].z;
      s[k + 3][line] = v[q].w;
    } else {
      *reinterpret_cast<float4*>(&s[i / (TILE / 4)][(i % (TILE / 4)) * 4]) = v[q];
    }
  }
}

// acc += this team's steps of A B over one source.
template <int TILE, Form FORM>
__device__ __forceinline__ void accumulate(const float* __restrict__ a,
                                           const float* __restrict__ b, int row0, int n_rows,
                                           int i0, int j0, int n_in, int n_out,
                                           SimtSmem<TILE>& sm, float acc[4][4]) {
  using C = SimtCfg<TILE>;
  constexpr bool AK = FORM != Form::kDw, BK = FORM == Form::kFwd;
  const int team = threadIdx.x / C::kTeamThreads, th = threadIdx.x % C::kTeamThreads;
  const int ti = th / (TILE / 4) * 4, tj = th % (TILE / 4) * 4;
  const int K = FORM == Form::kFwd ? n_in : (FORM == Form::kDx ? n_out : n_rows);
  // A: rows (kFwd, kDx) or dy columns; B: weights, or x columns
  const float* pa = a + (AK ? (int64_t)row0 * K : (int64_t)row0 * n_out + i0);
  const int la = AK ? n_rows : n_out - i0;
  const float* pb = b + (BK ? (int64_t)j0 * n_in
                            : (FORM == Form::kDx ? 0 : (int64_t)row0 * n_in) + j0);
  const int lb = (BK ? n_out : n_in) - j0;
  const int64_t da = AK ? K : n_out, db = n_in;
  float4 va[C::kVecs], vb[C::kVecs];
  int k0 = team * kStep;
  if (k0 < K) {
    fetch<TILE, AK>(pa, da, la, K, k0, th, va);
    fetch<TILE, BK>(pb, db, lb, K, k0, th, vb);
  }
  for (; k0 < K; k0 += C::kTeams * kStep) {
    team_sync<TILE>(team);  // the previous step's reads are done
    stage<TILE, AK>(sm.stage[team][0], th, va);
    stage<TILE, BK>(sm.stage[team][1], th, vb);
    team_sync<TILE>(team);
    const int next = k0 + C::kTeams * kStep;
    if (next < K) {
      fetch<TILE, AK>(pa, da, la, K, next, th, va);
      fetch<TILE, BK>(pb, db, lb, K, next, th, vb);
    }
#pragma unroll
    for (int k = 0; k < kStep; ++k) {
      const float4 x = *reinterpret_cast<const float4*>(&sm.stage[team][0][k][ti]);
      const float4 y = *reinterpret_cast<const float4*>(&sm.stage[team][1][k][tj]);
      const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[p][q] = fmaf(xs[p], ys[q], acc[p][q]);
    }
  }
}

template <int TILE, Form FORM>
__device__ __forceinline__ void run_tile(const GroupedJob& job, int64_t unit, int groups,
                                         const int32_t* s_off, const int32_t* s_tile,
                                         SimtSmem<TILE>& sm) {
  using C = SimtCfg<TILE>;
  const int n_in = job.n_in, n_out = job.n_out;
  const int cols = FORM == Form::kFwd ? n_out : n_in;
  const int jt = (cols + TILE - 1) / TILE;
  float acc[4][4];
#pragma unroll
  for (int p = 0; p < 4; ++p)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[p][q] = 0.f;
  int e, row0, n_rows, i0 = 0;
  const int j0 = (int)(unit % jt) * TILE;
  if (FORM == Form::kDw) {
    const int it = (n_out + TILE - 1) / TILE;
    const int64_t rest = unit / jt;
    i0 = (int)(rest % it) * TILE;
    e = (int)(rest / it);
    row0 = s_off[e];
    n_rows = s_off[e + 1] - row0;
  } else {
    const int t = (int)(unit / jt);
    e = segment_of(s_tile, groups, t);
    row0 = s_off[e] + (t - s_tile[e]) * TILE;
    n_rows = s_off[e + 1] - row0;
    if (n_rows > TILE) n_rows = TILE;
  }
  const int64_t wn = (int64_t)n_in * n_out;
  const float* b = static_cast<const float*>(job.b) + (FORM == Form::kDw ? 0 : e * wn);
  const float* a = static_cast<const float*>(job.a);
  if (FORM == Form::kDw) {
    float chain[4][4];
    for (int c0 = 0; c0 < n_rows; c0 += kChain) {
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q) chain[p][q] = 0.f;
      accumulate<TILE, FORM>(a, b, row0 + c0, n_rows - c0 < kChain ? n_rows - c0 : kChain, i0, j0,
                             n_in, n_out, sm, chain);
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[p][q] += chain[p][q];
    }
  } else {
    accumulate<TILE, FORM>(a, b, row0, n_rows, i0, j0, n_in, n_out, sm, acc);
  }
  if (FORM == Form::kDx && job.a2 != nullptr)
    accumulate<TILE, FORM>(static_cast<const float*>(job.a2),
                           static_cast<const float*>(job.b2) + e * wn, row0, n_rows, i0, j0, n_in,
                           n_out, sm, acc);
  const int team = threadIdx.x / C::kTeamThreads, th = threadIdx.x % C::kTeamThreads;
  const int ti = th / (TILE / 4) * 4, tj = th % (TILE / 4) * 4;
  float* out = static_cast<float*>(job.out);
  const int lines = FORM == Form::kDw ? n_out - i0 : n_rows;  // of this tile
  auto put = [&](int p, int q, float4 v) {
    if (p < lines && j0 + q < cols)
      store4(out + (FORM == Form::kDw ? e * wn + (int64_t)(i0 + p) * n_in
                                      : (int64_t)(row0 + p) * cols) + j0 + q, v);
  };
  if (C::kTeams == 1) {
#pragma unroll
    for (int p = 0; p < 4; ++p)
      put(ti + p, tj, make_float4(acc[p][0], acc[p][1], acc[p][2], acc[p][3]));
    return;
  }
  __syncthreads();  // every team has read its staged operands
#pragma unroll
  for (int p = 0; p < 4; ++p)
    *reinterpret_cast<float4*>(&sm.sums[team][ti + p][tj]) =
        make_float4(acc[p][0], acc[p][1], acc[p][2], acc[p][3]);
  __syncthreads();
  const int p = threadIdx.x / (TILE / 4), q = threadIdx.x % (TILE / 4) * 4;
  if (p < TILE) {
    float4 v = *reinterpret_cast<const float4*>(&sm.sums[0][p][q]);
#pragma unroll
    for (int g = 1; g < C::kTeams; ++g) {
      const float4 w = *reinterpret_cast<const float4*>(&sm.sums[g][p][q]);
      v.x += w.x;
      v.y += w.y;
      v.z += w.z;
      v.w += w.w;
    }
    put(p, q, v);
  }
  __syncthreads();  // the sums are read before the next tile is staged
}

template <int TILE>
__global__ void __launch_bounds__(kSimtThreads)
    grouped_simt_kernel(const __grid_constant__ SimtArgs args) {
  __shared__ __align__(16) SimtSmem<TILE> sm;
  __shared__ int32_t s_off[kMaxExperts + 1], s_tile[kMaxExperts + 1], s_warp[32];
  griddep_wait();
  griddep_launch_dependents();
  segment_table<kSimtThreads>(args.offsets, args.groups, args.rows, TILE, 0, s_off, s_tile,
                              s_warp);
  int64_t first[kMaxJobs + 1];
  first[0] = 0;
#pragma unroll
  for (int q = 0; q < kMaxJobs; ++q) {
    int64_t n = 0;
    if (q < args.n_jobs) {
      const GroupedJob& j = args.job[q];
      const int it = (j.n_out + TILE - 1) / TILE, jt = (j.n_in + TILE - 1) / TILE;
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
      run_tile<TILE, Form::kFwd>(j, unit, args.groups, s_off, s_tile, sm);
    else if (j.form == Form::kDx)
      run_tile<TILE, Form::kDx>(j, unit, args.groups, s_off, s_tile, sm);
    else if constexpr (TILE == 64)  // weight gradients have these tiles only
      run_tile<TILE, Form::kDw>(j, unit, args.groups, s_off, s_tile, sm);
  }
}

// Most tiles the jobs can have.
int64_t simt_tiles(const GroupedShape& g, const GroupedJob* jobs, int n_jobs, int tile) {
  int64_t most = 0;
  for (int q = 0; q < n_jobs; ++q) {
    const int64_t it = (jobs[q].n_out + tile - 1) / tile, jt = (jobs[q].n_in + tile - 1) / tile;
    const int64_t rt = g.rows / tile + (g.rows < g.groups ? g.rows : g.groups);
    most += jobs[q].form == Form::kDw ? g.groups * it * jt
                                      : rt * (jobs[q].form == Form::kFwd ? it : jt);
  }
  return most;
}

}  // namespace

cudaError_t launch_grouped_simt(const GroupedShape& g, const GroupedJob* jobs, int n_jobs,
                                const int32_t* offsets, cudaStream_t st) {
  SimtArgs a;
  a.n_jobs = n_jobs;
  a.groups = g.groups;
  a.rows = g.rows;
  a.offsets = offsets;
  for (int q = 0; q < kMaxJobs; ++q) a.job[q] = q < n_jobs ? jobs[q] : GroupedJob{};
  // 32 x 32 tiles where 64 x 64 ones would not give every SM two blocks (dx of
  // 8 x 26 rows, 256 columns from 512: 26 -> 12 us with the launch) or would be
  // half empty on average; large products are faster with 64 x 64 (34 to 36 TFLOP/s).
  // Weight gradients contract over a segment's rows, often fewer than the four
  // teams' first steps.
  const bool small = jobs[0].form != Form::kDw &&
                     (g.rows / g.groups <= 32 ||
                      simt_tiles(g, jobs, n_jobs, 64) < 2 * num_sms());
  const int64_t most = simt_tiles(g, jobs, n_jobs, small ? 32 : 64);
  const int64_t cap = (int64_t)num_sms() * 6;
  const unsigned blocks = (unsigned)(most < 1 ? 1 : (most < cap ? most : cap));
  return launch_pdl(small ? grouped_simt_kernel<32> : grouped_simt_kernel<64>, dim3(blocks),
                    dim3(kSimtThreads), 0, st, a);
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
  return row_units < (1ll << 31) && dw_units < (1ll << 31) && rows <= kMaxGroupedRows &&
         n_in <= kMaxGroupedDim && n_out <= kMaxGroupedDim;
}

}  // namespace moe
