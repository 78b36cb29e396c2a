// Layer norm over the last dimension, with the residual sum in front, and its
// backward pass. Both are bound by DRAM: the row is read once into registers,
// and everything else happens there.
//
//   s = x (+ residual, rounded to the stream's type: the sum is stored and
//       the norm reads what is stored, so that the backward pass, which reads
//       the stored sum again, differentiates exactly this)
//   mean = sum(s) / D, var = sum((s - mean)^2) / D (two passes over registers:
//       no cancellation however far the mean is from zero)
//   y = (s - mean) rstd w + b,  rstd = 1 / sqrt(var + eps)
//
// Backward, with xhat = (s - mean) rstd and u = dy w:
//   dx = rstd (u - mean(u) - xhat mean(u xhat)) + dsum
//   dw = sum over rows of dy xhat,  db = sum over rows of dy
// dw and db: a thread keeps its columns over all rows its block takes, blocks
// write one partial row each, and a second kernel adds those in a fixed order.
// No atomics: every result is the same on every run.
//
// Layout. A row belongs to G lanes of a warp (G < 32, short rows) or to
// `wpr` whole warps; a thread holds N groups of V consecutive elements (V: 16
// bytes where rows allow it, else 1), group i at column (i * lanes + lane) V.
//
// bfloat16 with residual, 32768 x 2560: 127 us (5.3 TB/s, 0.81 of the copy
// rate), backward with dsum 139 us (0.74: two sums an element hold registers);
// 131072 x 768: 130 us (0.95), backward 170. Single elements (32768 x 511
// float32, backward): 68 us of 31, bound by the number of loads.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace ssm {

struct NormParams {
  const void *x, *residual;      // [rows, dim]
  const float *weight, *bias;    // [dim] or nullptr
  void *y, *sum;                 // [rows, dim]; sum or nullptr
  float *mean, *rstd;            // [rows] (forward: or nullptr)
  float eps;
  int64_t rows;
  int dim;
  int wpr;                       // warps per row (G == 32)
  // backward
  const void *dy, *dsum;         // [rows, dim]; dsum or nullptr
  void *dx;
  float *part;                   // [2, parts, dim]: dw's, db's, or nullptr
  float *dweight, *dbias;
  int parts;                     // partial rows: blocks of the first kernel
};

namespace norm {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }

// V elements as they lie in memory, in registers.
template <typename T, int V>
struct Raw {
  uint32_t w[V == 1 ? 1 : 4];

  // Read once: streamed past the caches' other contents.
  __device__ __forceinline__ void load(const T *p) {
    if constexpr (V == 1) {
      if constexpr (sizeof(T) == 4) w[0] = __float_as_uint(*p);
      else w[0] = uint32_t(*reinterpret_cast<const uint16_t *>(p)) << 16;
    } else {
      const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
      w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < (V == 1 ? 1 : 4); ++j) w[j] = 0u;
  }
  __device__ __forceinline__ float at(int j) const {
    if constexpr (V == 1 || sizeof(T) == 4)
      return __uint_as_float(w[j]);
    else
      return __uint_as_float(j % 2 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
  }
};

template <typename T, int V>
__device__ __forceinline__ void store(T *p, const float (&f)[V]) {
  if constexpr (V == 1) {
    *p = T(f[0]);
  } else if constexpr (sizeof(T) == 4) {
    __stcs(reinterpret_cast<float4 *>(p),
           make_float4(f[0], f[1], f[2], f[3]));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
          : "=r"(w[j])
          : "f"(f[2 * j + 1]), "f"(f[2 * j]));
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
  }
}

// V parameters.
template <int V>
__device__ __forceinline__ void load_param(const float *p, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = __ldg(p);
  } else {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4 *>(p + j));
      f[j] = v.x; f[j + 1] = v.y; f[j + 2] = v.z; f[j + 3] = v.w;
    }
  }
}

// Sums over a row's threads. `red` has room for two values of each warp, for
// two calls in turn (`slot` 0, 1), so that one barrier a call is enough.
template <int G>
__device__ __forceinline__ void row_sum2(float &a, float &b, int wpr,
                                         float2 *red, int slot) {
#pragma unroll
  for (int d = G / 2; d > 0; d >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, d);
    b += __shfl_xor_sync(0xffffffffu, b, d);
  }
  if constexpr (G == 32) {
    if (wpr > 1) {
      const int warp = threadIdx.x / 32;
      float2 *r = red + slot * 32;
      if (threadIdx.x % 32 == 0) r[warp] = make_float2(a, b);
      __syncthreads();
      const int first = warp / wpr * wpr;
      a = b = 0.0f;
      for (int w = 0; w < wpr; ++w) {
        const float2 v = r[first + w];
        a += v.x;
        b += v.y;
      }
    }
  }
}

// Where a thread's parameters wait in shared memory rather than registers, of
// which its elements take too many there: forward weight and bias, backward
// the weight (65536 x 1024 bfloat16, backward: 126 us with it in registers,
// 104 so; 32768 x 2560: 139 either way).
__host__ __device__ constexpr bool shared_params(int v, int n) {
  return v == 8 && n > 2;
}
__host__ __device__ constexpr bool shared_weight(int v, int g) {
  return v == 8 && g == 32;
}

// Blocks stay for many rows: a thread's parameters are read once, and the next
// row is on its way while this one is reduced and written.
template <typename T, int V, int N, int G>
__global__ void __launch_bounds__(512)
    layernorm_fwd_kernel(const __grid_constant__ NormParams p) {
  __shared__ float2 red[64];
  const int lanes = G < 32 ? G : 32 * p.wpr;       // threads of a row
  const int per = blockDim.x / lanes;              // rows of a block
  const int lane = threadIdx.x % lanes, group = threadIdx.x / lanes;
  const float inv = 1.0f / float(p.dim);
  const int64_t steps = (p.rows + per - 1) / per;
  constexpr bool SH = shared_params(V, N);
  extern __shared__ __align__(16) float par[];
  float w[SH ? 1 : N][V], b[SH ? 1 : N][V];
  if constexpr (SH) {
    for (int c = threadIdx.x; c < p.dim; c += blockDim.x) {
      par[c] = p.weight ? p.weight[c] : 1.0f;
      par[p.dim + c] = p.bias ? p.bias[c] : 0.0f;
    }
    __syncthreads();
  } else
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * lanes + lane) * V;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      w[i][j] = 1.0f;
      b[i][j] = 0.0f;
    }
    if (c < p.dim && p.weight) load_param<V>(p.weight + c, w[i]);
    if (c < p.dim && p.bias) load_param<V>(p.bias + c, b[i]);
  }
  Raw<T, V> nx[N], nr[N];
  auto fetch = [&](int64_t st) {
    const int64_t row = st * per + group;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * lanes + lane) * V;
      nx[i].zero();
      nr[i].zero();
      if (row < p.rows && c < p.dim) {
        nx[i].load(static_cast<const T *>(p.x) + row * p.dim + c);
        if (p.residual)
          nr[i].load(static_cast<const T *>(p.residual) + row * p.dim + c);
      }
    }
  };
  fetch(blockIdx.x);
  for (int64_t st = blockIdx.x; st < steps; st += gridDim.x) {
    const int64_t row = st * per + group;
    const bool in = row < p.rows;
    const int64_t base = row * p.dim;
    float f[N][V];
    float s = 0.0f, none = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        f[i][j] = nx[i].at(j);
        if (p.residual) f[i][j] = to_f(T(f[i][j] + nr[i].at(j)));
        s += f[i][j];
      }
    fetch(st + gridDim.x);
    if (p.sum) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (i * lanes + lane) * V;
        if (in && c < p.dim)
          store<T, V>(static_cast<T *>(p.sum) + base + c, f[i]);
      }
    }
    row_sum2<G>(s, none, p.wpr, red, 0);
    const float mean = s * inv;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * lanes + lane) * V;
      if (c < p.dim) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          f[i][j] -= mean;
          q = fmaf(f[i][j], f[i][j], q);
        }
      }
    }
    row_sum2<G>(q, none, p.wpr, red, 1);
    const float rstd = 1.0f / sqrtf(fmaf(q, inv, p.eps));
    if (in && lane == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * lanes + lane) * V;
      if (in && c < p.dim) {
        if constexpr (SH) {
#pragma unroll
          for (int j = 0; j < V; j += 4) {
            const float4 a = *reinterpret_cast<const float4 *>(par + c + j);
            const float4 e =
                *reinterpret_cast<const float4 *>(par + p.dim + c + j);
            f[i][j] = fmaf(f[i][j] * rstd, a.x, e.x);
            f[i][j + 1] = fmaf(f[i][j + 1] * rstd, a.y, e.y);
            f[i][j + 2] = fmaf(f[i][j + 2] * rstd, a.z, e.z);
            f[i][j + 3] = fmaf(f[i][j + 3] * rstd, a.w, e.w);
          }
        } else
#pragma unroll
        for (int j = 0; j < V; ++j)
          f[i][j] = fmaf(f[i][j] * rstd, w[i][j], b[i][j]);
        store<T, V>(static_cast<T *>(p.y) + base + c, f[i]);
      }
    }
  }
}

// Columns sums of short rows go over many rows a thread: every kFold rows the
// running sums are folded into a second pair, so that the rounding of a long
// sum does not grow with its length.
constexpr int kFold = 32;

template <typename T, int V, int N, int G>
__global__ void __launch_bounds__(512, V == 1 && N <= 4 ? 2 : 1)
    layernorm_bwd_kernel(const __grid_constant__ NormParams p) {
  constexpr bool FOLD = N * V <= 8;
  constexpr bool LEAN = shared_weight(V, G);
  __shared__ float2 red[64];
  extern __shared__ __align__(16) float cols[];  // [per - 1, 2, dim] at the end
  const int lanes = G < 32 ? G : 32 * p.wpr;
  const int per = blockDim.x / lanes;
  const int lane = threadIdx.x % lanes, group = threadIdx.x / lanes;
  const float inv = 1.0f / float(p.dim);
  const int64_t steps = (p.rows + per - 1) / per;
  float dw[N][V], db[N][V], dw2[N][V], db2[N][V];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j)
      dw[i][j] = db[i][j] = dw2[i][j] = db2[i][j] = 0.0f;
  float w[LEAN ? 1 : N][V];
  float *ws = cols + (p.part ? (per - 1) * 2 * p.dim : 0);
  if constexpr (LEAN) {
    for (int c = threadIdx.x; c < p.dim; c += blockDim.x)
      ws[c] = p.weight ? p.weight[c] : 1.0f;
    __syncthreads();
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * lanes + lane) * V;
#pragma unroll
      for (int j = 0; j < V; ++j) w[i][j] = 1.0f;
      if (c < p.dim && p.weight) load_param<V>(p.weight + c, w[i]);
    }
  }
  Raw<T, V> nx[N], ng[N];
  float nmean = 0.0f, nrstd = 0.0f;
  auto fetch = [&](int64_t st) {
    const int64_t row = st * per + group;
    const bool in = row < p.rows;
    nmean = in ? p.mean[row] : 0.0f;
    nrstd = in ? p.rstd[row] : 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * lanes + lane) * V;
      nx[i].zero();
      ng[i].zero();
      if (in && c < p.dim) {
        const int64_t at = row * p.dim + c;
        nx[i].load(static_cast<const T *>(p.x) + at);
        ng[i].load(static_cast<const T *>(p.dy) + at);
      }
    }
  };
  fetch(blockIdx.x);
  int fold = 0, slot = 0;
  for (int64_t st = blockIdx.x; st < steps; st += gridDim.x, slot ^= 1) {
    const int64_t row = st * per + group;
    const bool in = row < p.rows;
    const int64_t base = row * p.dim;
    const float mean = nmean, rstd = nrstd;
    float x[N][V], g[N][V];
    // (needed last: on its way while the row is summed)
    Raw<T, V> ds[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * lanes + lane) * V;
      ds[i].zero();
      if (in && c < p.dim && p.dsum)
        ds[i].load(static_cast<const T *>(p.dsum) + base + c);
    }
    float su = 0.0f, sux = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * lanes + lane) * V;
      const bool live = c < p.dim;
      float wi[V];
      if constexpr (LEAN) {
#pragma unroll
        for (int j = 0; j < V; j += 4) {
          const float4 v =
              *reinterpret_cast<const float4 *>(ws + (live ? c + j : 0));
          wi[j] = v.x; wi[j + 1] = v.y; wi[j + 2] = v.z; wi[j + 3] = v.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) wi[j] = w[i][j];
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        x[i][j] = live ? (nx[i].at(j) - mean) * rstd : 0.0f;
        g[i][j] = ng[i].at(j);
        dw[i][j] = fmaf(g[i][j], x[i][j], dw[i][j]);
        db[i][j] += g[i][j];
        g[i][j] *= wi[j];
        su += g[i][j];
        sux = fmaf(g[i][j], x[i][j], sux);
      }
    }
    fetch(st + gridDim.x);
    row_sum2<G>(su, sux, p.wpr, red, slot);
    su *= inv;
    sux *= inv;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * lanes + lane) * V;
      if (in && c < p.dim) {
        float o[V];
#pragma unroll
        for (int j = 0; j < V; ++j)
          o[j] = fmaf(g[i][j] - su - x[i][j] * sux, rstd, ds[i].at(j));
        store<T, V>(static_cast<T *>(p.dx) + base + c, o);
      }
    }
    if (FOLD && ++fold == kFold) {
      fold = 0;
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          dw2[i][j] += dw[i][j];
          db2[i][j] += db[i][j];
          dw[i][j] = db[i][j] = 0.0f;
        }
    }
  }
  if (!p.part) return;
  if (FOLD) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        dw[i][j] += dw2[i][j];
        db[i][j] += db2[i][j];
      }
  }
  // the block's row groups, in order, into the first one's sums
  if (group > 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * lanes + lane) * V;
      if (c < p.dim) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          cols[(int64_t(group - 1) * 2) * p.dim + c + j] = dw[i][j];
          cols[(int64_t(group - 1) * 2 + 1) * p.dim + c + j] = db[i][j];
        }
      }
    }
  }
  __syncthreads();
  if (group == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * lanes + lane) * V;
      if (c < p.dim) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          for (int k = 0; k + 1 < per; ++k) {
            dw[i][j] += cols[(int64_t(k) * 2) * p.dim + c + j];
            db[i][j] += cols[(int64_t(k) * 2 + 1) * p.dim + c + j];
          }
          p.part[int64_t(blockIdx.x) * p.dim + c + j] = dw[i][j];
          p.part[(int64_t(p.parts) + blockIdx.x) * p.dim + c + j] = db[i][j];
        }
      }
    }
  }
}

// dweight and dbias from the blocks' partial rows: 32 columns a block, eight
// warps over the rows, in a fixed order.
__global__ void __launch_bounds__(256)
    layernorm_cols_kernel(const __grid_constant__ NormParams p) {
  __shared__ float red[8][32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + lane;
  const float *src = p.part + int64_t(blockIdx.y) * p.parts * p.dim;
  float *dst = blockIdx.y == 0 ? p.dweight : p.dbias;
  float s = 0.0f;
  if (c < p.dim)
#pragma unroll 4
    for (int r = warp; r < p.parts; r += 8) s += src[int64_t(r) * p.dim + c];
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < p.dim && dst) {
    for (int w = 1; w < 8; ++w) s += red[w][lane];
    dst[c] = s;
  }
}

}  // namespace norm
}  // namespace ssm
