// C ABI of the layer-norm entry points: host-side validation, the choice of
// the row layout and launches. The contract is in include/ssm_layernorm.h.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "../../include/ssm_layernorm.h"
#include "device_info.cuh"
#include "kernel_layernorm.cuh"

namespace {

using ssm::aligned;
using ssm::NormParams;
using bf16 = __nv_bfloat16;

// Dynamic shared memory that needs no permission beside the kernels' own.
constexpr size_t kSmallSmem = 47 * 1024;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// How a row is spread: G lanes (short rows) or wpr warps, n groups a thread.
struct Shape {
  int g = 32, wpr = 1, n = 1;
  int threads = 256, per = 1;  // of a block; rows of a block
};

// Groups of a thread, for rows of more than 16 of them. Single elements: at
// most 8 (4 where bfloat16 ones are normed): more of them cost residency
// (registers) than they save barriers, fewer the reverse (32768 x 511 float32,
// backward: 158 us for twice the bytes with 8, 182 with 4, 236 with 2; 511
// bfloat16, forward: 532 us with 4, 828 with 8). 16-byte groups: 2 to `most`
// (4; in the backward pass, which keeps two sums for every element, 2, and 3 of
// float32), as many as leave the fewest lanes idle, and of these the most, for
// fewer warps have to meet then (bfloat16 forward, with residual: 131072 x 768 174 us
// with 2, 130 with 3 and no barrier; 16384 x 5120 175 us with 2, 118 with 4;
// 32768 x 2560 127 us with 2, 142 with 4 and idle lanes; 16384 x 4096 98 us
// with 2, 102 with 4; float32 backward: 65536 x 768 153 us with 2, 129 with 3;
// 32768 x 1024 94 us with 2, 132 with 4).
Shape shape_of(int dim, int v, int most) {
  Shape s;
  const int nv = int(ceil_div(dim, v));
  if (nv <= 16) {
    s.g = nv <= 4 ? 4 : nv <= 8 ? 8 : 16;
  } else if (v == 1) {
    // (rows wider than 16 warps' worth of that, the launch bound, take more)
    most = std::max<int>(most, int(ceil_div(nv, 512)));
    s.wpr = int(ceil_div(nv, 32 * most));
    s.n = int(ceil_div(nv, 32 * s.wpr));
  } else {
    int idle = 1 << 30;
    for (int n = nv <= 32 ? 1 : 2; n <= std::max(most, int(ceil_div(nv, 512)));
         ++n) {
      const int wpr = int(ceil_div(nv, 32 * n)), left = 32 * n * wpr - nv;
      if (wpr > 16 || left > idle) continue;
      idle = left;
      s.wpr = wpr;
      s.n = n;
    }
  }
  const int lanes = s.g < 32 ? s.g : 32 * s.wpr;
  s.per = std::max(1, 256 / lanes);
  s.threads = lanes * s.per;
  return s;
}

// Most blocks the backward pass runs on (and partial rows it leaves): what
// may be resident at once, or one for each step of rows if there are fewer.
int parts_of(const Shape &s, int64_t rows, int sms) {
  const int per_sm = std::max(1, 1536 / s.threads);
  return int(std::min<int64_t>(ceil_div(rows, s.per), int64_t(sms) * per_sm));
}

// Blocks of `threads` that an SM holds at once.
int resident(const void *kern, int threads, size_t smem) {
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, smem) !=
          cudaSuccess ||
      n < 1) {
    cudaGetLastError();
    n = 1;
  }
  return n;
}

template <typename T, int V, int N, int G>
int launch_fwd(const NormParams &p, const Shape &s, int sms, cudaStream_t st) {
  const int64_t steps = ceil_div(p.rows, s.per);
  auto kern = ssm::norm::layernorm_fwd_kernel<T, V, N, G>;
  const size_t smem =
      ssm::norm::shared_params(V, N) ? size_t(p.dim) * 2 * sizeof(float) : 0;
  if (smem > kSmallSmem &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           int(smem)) != cudaSuccess) {
    cudaGetLastError();
    return SSM_ERR_CUDA;
  }
  const int64_t grid = std::min<int64_t>(
      steps, int64_t(sms) * resident(reinterpret_cast<const void *>(kern),
                                     s.threads, smem));
  kern<<<unsigned(grid), s.threads, smem, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

template <typename T, int V, int N, int G>
int launch_bwd(NormParams p, const Shape &s, int sms, cudaStream_t st) {
  auto kern = ssm::norm::layernorm_bwd_kernel<T, V, N, G>;
  const size_t smem =
      (size_t(p.part ? (s.per - 1) * 2 : 0) +
       (ssm::norm::shared_weight(V, G) ? 1 : 0)) *
      p.dim * sizeof(float);
  if (smem > kSmallSmem &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           int(smem)) != cudaSuccess) {
    cudaGetLastError();
    return SSM_ERR_CUDA;
  }
  p.parts = std::min(p.parts,
                     sms * resident(reinterpret_cast<const void *>(kern),
                                    s.threads, smem));
  kern<<<unsigned(p.parts), s.threads, smem, st>>>(p);
  if (cudaGetLastError() != cudaSuccess) return SSM_ERR_CUDA;
  if (!p.part) return SSM_OK;
  ssm::norm::layernorm_cols_kernel<<<dim3(unsigned(ceil_div(p.dim, 32)), 2),
                                     256, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

template <typename T, int V, bool BWD, int N, int G>
int launch(const NormParams &p, const Shape &s, int sms, cudaStream_t st) {
  if constexpr (BWD) return launch_bwd<T, V, N, G>(p, s, sms, st);
  else return launch_fwd<T, V, N, G>(p, s, sms, st);
}

template <typename T, int V, bool BWD>
int pick(const NormParams &p, const Shape &s, int sms, cudaStream_t st) {
  if (s.g == 4) return launch<T, V, BWD, 1, 4>(p, s, sms, st);
  if (s.g == 8) return launch<T, V, BWD, 1, 8>(p, s, sms, st);
  if (s.g == 16) return launch<T, V, BWD, 1, 16>(p, s, sms, st);
  if (s.n == 1) return launch<T, V, BWD, 1, 32>(p, s, sms, st);
  if (s.n == 2) return launch<T, V, BWD, 2, 32>(p, s, sms, st);
  if constexpr (V < 8 || !BWD) {
    if (s.n <= 3) return launch<T, V, BWD, 3, 32>(p, s, sms, st);
    if (s.n <= 4) return launch<T, V, BWD, 4, 32>(p, s, sms, st);
  }
  if constexpr (V == 1) {
    if (s.n <= 8) return launch<T, V, BWD, 8, 32>(p, s, sms, st);
    return launch<T, V, BWD, 16, 32>(p, s, sms, st);
  }
  return SSM_ERR_UNSUPPORTED;
}

int run(const NormParams &p, bool wide, bool bwd, int dtype, const Shape &s,
        int sms, cudaStream_t st) {
  if (dtype == SSM_F32) {
    if (wide)
      return bwd ? pick<float, 4, true>(p, s, sms, st)
                 : pick<float, 4, false>(p, s, sms, st);
    return bwd ? pick<float, 1, true>(p, s, sms, st)
               : pick<float, 1, false>(p, s, sms, st);
  }
  if (wide)
    return bwd ? pick<bf16, 8, true>(p, s, sms, st)
               : pick<bf16, 8, false>(p, s, sms, st);
  return bwd ? pick<bf16, 1, true>(p, s, sms, st)
             : pick<bf16, 1, false>(p, s, sms, st);
}

int check(int64_t rows, int64_t dim, int dtype) {
  if (rows <= 0 || dim <= 0) return SSM_ERR_INVALID;
  if (dtype != SSM_F32 && dtype != SSM_BF16) return SSM_ERR_UNSUPPORTED;
  if (dim > SSM_LAYERNORM_MAX_DIM) return SSM_ERR_UNSUPPORTED;
  if (rows > (int64_t(1) << 42)) return SSM_ERR_INVALID;
  return SSM_OK;
}

// Whether rows move in 16-byte groups: every row starts on a 16-byte boundary
// and so do the parameters' groups.
bool wide_rows(int64_t dim, size_t esz,
               std::initializer_list<const void *> list) {
  if (dim * esz % 16 != 0) return false;
  for (const void *q : list)
    if (q && !aligned(q, 16)) return false;
  return true;
}

Shape row_shape(int64_t dim, bool wide, size_t esz, bool bwd) {
  if (!wide) return shape_of(int(dim), 1, bwd || esz == 4 ? 8 : 4);
  return shape_of(int(dim), int(16 / esz), bwd ? (esz == 4 ? 3 : 2) : 4);
}

}  // namespace

extern "C" {

int ssm_layernorm_workspace(int device, int64_t rows, int64_t dim, int dtype,
                            size_t *bytes) {
  if (!bytes) return SSM_ERR_INVALID;
  *bytes = 0;
  int rc = check(rows, dim, dtype);
  if (rc != SSM_OK) return rc;
  int sms = 0;
  rc = ssm::device_sms(device, &sms);
  if (rc != SSM_OK) return rc;
  const size_t esz = dtype == SSM_F32 ? 4 : 2;
  int parts = parts_of(row_shape(dim, false, esz, true), rows, sms);
  if (dim * esz % 16 == 0)
    parts = std::max(parts,
                     parts_of(row_shape(dim, true, esz, true), rows, sms));
  *bytes = size_t(parts) * 2 * dim * sizeof(float);
  return SSM_OK;
}

int ssm_layernorm_fwd(int device, const void *x, const void *residual,
                      const float *weight, const float *bias, float eps,
                      void *y, void *sum, float *mean, float *rstd,
                      int64_t rows, int64_t dim, int dtype,
                      struct CUstream_st *stream) {
  if (!x || !y || (sum && !residual)) return SSM_ERR_INVALID;
  int rc = check(rows, dim, dtype);
  if (rc != SSM_OK) return rc;
  const size_t esz = dtype == SSM_F32 ? 4 : 2;
  for (const void *q : {x, residual, static_cast<const void *>(y),
                        static_cast<const void *>(sum)})
    if (q && !aligned(q, esz)) return SSM_ERR_ALIGN;
  for (const float *q : {weight, bias, static_cast<const float *>(mean),
                         static_cast<const float *>(rstd)})
    if (q && !aligned(q, 4)) return SSM_ERR_ALIGN;
  const size_t all = size_t(rows) * dim * esz, row = dim * sizeof(float),
               stats = size_t(rows) * sizeof(float);
  if (ssm::clash({{y, all}, {sum, all}, {mean, stats}, {rstd, stats}},
                 {{weight, row}, {bias, row}}) ||
      ssm::clash({{mean, stats}, {rstd, stats}}, {{x, all}, {residual, all}}) ||
      ssm::clash({{y, all}, {sum, all}}, {{x, all}, {residual, all}}, true))
    return SSM_ERR_INVALID;
  int sms = 0;
  rc = ssm::device_ready(device, &sms);
  if (rc != SSM_OK) return rc;
  NormParams p{};
  p.x = x; p.residual = residual; p.weight = weight; p.bias = bias;
  p.y = y; p.sum = sum; p.mean = mean; p.rstd = rstd; p.eps = eps;
  p.rows = rows; p.dim = int(dim);
  const bool wide = wide_rows(dim, esz, {x, residual, y, sum, weight, bias});
  const Shape s = row_shape(dim, wide, esz, false);
  p.wpr = s.wpr;
  return run(p, wide, false, dtype, s, sms,
             reinterpret_cast<cudaStream_t>(stream));
}

int ssm_layernorm_bwd(int device, const void *dy, const void *x,
                      const float *mean, const float *rstd,
                      const float *weight, const void *dsum, void *dx,
                      float *dweight, float *dbias, void *workspace,
                      size_t workspace_bytes, int64_t rows, int64_t dim,
                      int dtype, struct CUstream_st *stream) {
  if (!dy || !x || !mean || !rstd || !dx) return SSM_ERR_INVALID;
  int rc = check(rows, dim, dtype);
  if (rc != SSM_OK) return rc;
  const size_t esz = dtype == SSM_F32 ? 4 : 2;
  for (const void *q : {dy, x, dsum, static_cast<const void *>(dx)})
    if (q && !aligned(q, esz)) return SSM_ERR_ALIGN;
  for (const float *q :
       {mean, rstd, weight, static_cast<const float *>(dweight),
        static_cast<const float *>(dbias)})
    if (q && !aligned(q, 4)) return SSM_ERR_ALIGN;
  const size_t all = size_t(rows) * dim * esz, row = dim * sizeof(float),
               stats = size_t(rows) * sizeof(float);
  if (ssm::clash({{dx, all}, {dweight, row}, {dbias, row}},
                 {{mean, stats}, {rstd, stats}, {weight, row}}) ||
      ssm::clash({{dweight, row}, {dbias, row}},
                 {{dy, all}, {x, all}, {dsum, all}}) ||
      ssm::clash({{dx, all}}, {{dy, all}, {x, all}, {dsum, all}}, true))
    return SSM_ERR_INVALID;
  int sms = 0;
  rc = ssm::device_ready(device, &sms);
  if (rc != SSM_OK) return rc;
  NormParams p{};
  p.x = x; p.dy = dy; p.dsum = dsum; p.dx = dx; p.weight = weight;
  p.mean = const_cast<float *>(mean); p.rstd = const_cast<float *>(rstd);
  p.dweight = dweight; p.dbias = dbias;
  p.rows = rows; p.dim = int(dim);
  const bool wide = wide_rows(dim, esz, {dy, x, dsum, dx, weight});
  const Shape s = row_shape(dim, wide, esz, true);
  p.wpr = s.wpr;
  p.parts = parts_of(s, rows, sms);
  if (dweight || dbias) {
    const size_t need = size_t(p.parts) * 2 * dim * sizeof(float);
    if (!workspace || workspace_bytes < need) return SSM_ERR_INVALID;
    if (!aligned(workspace, 4)) return SSM_ERR_ALIGN;
    if (ssm::clash({{workspace, need}},
                   {{dx, all}, {dweight, row}, {dbias, row}, {dy, all},
                    {x, all}, {dsum, all}, {mean, stats}, {rstd, stats},
                    {weight, row}}))
      return SSM_ERR_INVALID;
    p.part = static_cast<float *>(workspace);
  }
  return run(p, wide, true, dtype, s, sms,
             reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
