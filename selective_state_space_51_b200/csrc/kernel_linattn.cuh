// Linear attention with a decay for each head, in chunks of 64 steps on the
// tensor cores, for every supported shape and both activation types.
//
// With c_i the sum of the log decays inside the chunk up to step i, S the
// state in front of it:
//   y_i = si e^{c_i} q_i S + sp sum_{j <= i} e^{c_i - c_j} (q_i . k_j) v_j
//   S  <- e^{c_C} S + sw sum_j e^{c_C - c_j} k_j (x) v_j
// A block of eight warps owns one head, one tile of 64 value columns and one
// segment of a sequence: S stays in float32 registers (each warp 16 key rows,
// and half of the columns where there are 64 keys), the chunk's q, k, v and the
// bfloat16 planes of S in shared memory.
//
// The backward pass is three such passes. dq_i reads the same states as y_i,
// transposed: it is linear attention of (query dy, key v, value k). dk and dv
// run backwards in time: dk is that of (query v, key dy, value q), dv that of
// (query k, key q, value dy). Counted from the end, step i sits at token
// t = T - 1 - i, and the decay between two steps is shifted by one: step i
// carries the log decay of token t + 1.
//
// Types. The tensor cores multiply bfloat16 and add float32, so every operand
// is a sum of bfloat16 planes: x = x0 + x1 + x2, each the rounding of what
// the ones before leave (8 significant bits each, 24 in all: float32 exactly).
// bfloat16 inputs are one plane, float32 inputs three. A product of two
// operands takes the plane pairs (a, b) with a + b < 3; what is left out is
// below 2^-24 of the product. The state's write takes three planes of the
// weighted key for both types, so the float32 state has float32 accuracy.
// Reading the state and the decayed scores takes PS planes: two where only
// bfloat16 results come of them (2^-17 of a term is lost, nothing beside the
// results' rounding; one plane would add as much as that rounding is), three
// for float32 results and for the decay's gradient, which sums differences of
// them.
//
// Bound by the tensor pipe's mma.sync rate and by what feeds it: six products
// for float32 operands, at 40% of the pipe's cycles. 64 steps a chunk and 64
// value columns a block leave room for two blocks an SM (one with three planes
// of 128-wide keys). float32, 64 x up to 512 steps, 8 heads of 64: 195 us, the
// bytes alone 42; backward, 3 x 1000 steps, 6 heads of 48 x 77: 192 us with
// its ten short launches.
#pragma once

#include <cuda_bf16.h>
#include <math_constants.h>
#include <stdint.h>

#include "device_math.cuh"
#include "linattn_params.cuh"

namespace ssm {
namespace la {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const bf16 *p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p)));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], const bf16 *p) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(smem_u32(p)));
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4],
                                    uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float lo2(uint32_t v) {
  return __uint_as_float(v << 16);
}
__device__ __forceinline__ float hi2(uint32_t v) {
  return __uint_as_float(v & 0xffff0000u);
}

// The first N bfloat16 planes of a pair of floats.
template <int N>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&p)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    p[n] = pack2(x, y);
    x -= lo2(p[n]);
    y -= hi2(p[n]);
  }
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }

// The log decay of one token and head.
template <typename T>
__device__ __forceinline__ double gate_at(const LaParams &p, int64_t b,
                                          int64_t t, int h) {
  double g = 0.0;
  if (p.log_decay)
    g = double(to_f(static_cast<const T *>(
        p.log_decay)[(b * p.seqlen + t) * p.heads + h]));
  if (p.head_log_decay) g += double(p.head_log_decay[h]);
  return g;
}

// Where the rows of a chunk come from: row r is step `first + r`.
struct Rows {
  int64_t first;  // token of row 0
  int dir;        // +1, or -1 in reverse
  int64_t len;    // tokens of this sequence
  __device__ __forceinline__ int64_t token(int r) const {
    return first + int64_t(dir) * r;
  }
  __device__ __forceinline__ bool live(int r) const { return token(r) < len; }
};

constexpr int kThreads = 256;

// A thread's part of one [64][COLS] tile as it lies in memory: COLS / 32
// groups of 8 elements. All of a chunk's loads are issued before the first is
// used. Rows past the sequence's length and columns past `cols` are zero
// whatever the memory holds.
template <typename T, int COLS>
struct RawTile {
  static constexpr int IT = COLS / 32;
  static constexpr int W = sizeof(T) == 2 ? 1 : 2;  // 16-byte words a group
  uint4 w[IT][W];

  __device__ __forceinline__ static int row(int i) {
    return (int(threadIdx.x) + i * kThreads) / (COLS / 8);
  }
  __device__ __forceinline__ static int col(int i) {
    return (int(threadIdx.x) + i * kThreads) % (COLS / 8) * 8;
  }

  __device__ __forceinline__ void load(const T *src, int64_t stride, int cols,
                                       const Rows &rows, bool vec) {
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int r = row(i), c = col(i);
#pragma unroll
      for (int k = 0; k < W; ++k) w[i][k] = make_uint4(0u, 0u, 0u, 0u);
      if (rows.live(r) && c < cols) {
        const T *s = src + rows.token(r) * stride + c;
        if (vec && c + 8 <= cols) {
#pragma unroll
          for (int k = 0; k < W; ++k)
            w[i][k] = __ldg(reinterpret_cast<const uint4 *>(s) + k);
        } else if constexpr (sizeof(T) == 4) {
          uint32_t x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            x[j] = c + j < cols ? __float_as_uint(s[j]) : 0u;
          w[i][0] = make_uint4(x[0], x[1], x[2], x[3]);
          w[i][1] = make_uint4(x[4], x[5], x[6], x[7]);
        } else {
          const uint16_t *h = reinterpret_cast<const uint16_t *>(s);
          uint32_t x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = c + j < cols ? h[j] : 0u;
          w[i][0] = make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16,
                               x[4] | x[5] << 16, x[6] | x[7] << 16);
        }
      }
    }
  }

  // The NP planes of the tile, in shared memory with rows of COLS + 8.
  template <int NP>
  __device__ __forceinline__ void store(bf16 *dst) const {
    constexpr int LD = COLS + 8;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      bf16 *d = dst + row(i) * LD + col(i);
      if constexpr (NP == 1) {
        *reinterpret_cast<uint4 *>(d) = w[i][0];
      } else {
        const float x[8] = {
            __uint_as_float(w[i][0].x), __uint_as_float(w[i][0].y),
            __uint_as_float(w[i][0].z), __uint_as_float(w[i][0].w),
            __uint_as_float(w[i][1].x), __uint_as_float(w[i][1].y),
            __uint_as_float(w[i][1].z), __uint_as_float(w[i][1].w)};
        uint32_t pl[4][NP];
#pragma unroll
        for (int j = 0; j < 4; ++j) split2<NP>(x[2 * j], x[2 * j + 1], pl[j]);
#pragma unroll
        for (int n = 0; n < NP; ++n)
          *reinterpret_cast<uint4 *>(d + n * kLaChunk * LD) =
              make_uint4(pl[0][n], pl[1][n], pl[2][n], pl[3][n]);
      }
    }
  }
};

// Brings the rows of a tile to the L2 cache, one chunk ahead of their loads.
template <typename T>
__device__ __forceinline__ void prefetch_tile(const T *src, int64_t stride,
                                              int cols, const Rows &rows) {
  const int lines = (cols * int(sizeof(T)) + 127) / 128;
  for (int i = threadIdx.x; i < kLaChunk * lines; i += kThreads) {
    const int r = i / lines, l = i % lines;
    if (rows.live(r))
      asm volatile("prefetch.global.L2 [%0];" ::"l"(
          src + rows.token(r) * stride + l * (128 / int(sizeof(T)))));
  }
}

// A step whose log decay is below this starts the state anew (e^g is about to
// leave float32's normal numbers, which end at e^-87.3).
constexpr double kRestart = -87.0;

// The chunk's decays, in units of log2. At a step that starts the state anew
// the sums restart (so that they stay finite and small), and nothing before it
// is read.
// The sums are formed in 64 bits and kept as a pair of floats: a difference of
// two of them is then exact to float32 however much the chunk decays.
struct alignas(16) Gates {
  float hi[kLaChunk], lo[kLaChunk];  // c_i since the last restart
  int from[kLaChunk];                // the last restart at or before step i
  float read[kLaChunk];              // e^{c_i}, 0 behind a restart
  float write[kLaChunk];             // e^{c_C - c_i}, 0 before a restart
  float2 keep;                       // of e^{c_C} (see keep_of), 0 with a restart
  double end;                        // c_C, -infinity with a restart
};

// 2^x for a 64-bit x: the float32 rounding of x is put back to first order.
// What leaves float32's normal numbers is 0, as ex2 has it.
__device__ __forceinline__ float ex2_d(double x) {
  if (x < -126.0) return 0.0f;
  const float hi = float(x);
  return ex2(hi) * fmaf(float(x - double(hi)), kLn2, 1.0f);
}

// What is kept of a state over a chunk, 2^x, as {m, b}: S <- b S + (m S + ...).
// A kept part near 1 is {2^x - 1, 1}: rounded as one number it would be off by
// up to 2^-24, always to the same side where a head's decay is the same for
// every step, which over the 1600 chunks that a decay of e^-0.00001 a step lets
// through made 1e-5 of the state.
__device__ __forceinline__ float2 keep_of(double x) {
  return x > -1.0 ? make_float2(expm1f(float(x * 0.6931471805599453)), 1.0f)
                  : make_float2(ex2_d(x), 0.0f);
}
__device__ __forceinline__ bool none_kept(float2 keep) {
  return keep.x == 0.0f && keep.y == 0.0f;
}

// The decay of one step, from its log decay.
__device__ __forceinline__ float decay_of(double g) {
  return g < kRestart ? 0.0f : ex2_d(g * 1.4426950408889634);
}

template <typename T>
__device__ __forceinline__ void load_gates(Gates &g, const LaParams &p,
                                           const Rows &rows, int64_t b,
                                           int h, int reverse) {
  const int lane = threadIdx.x;  // one warp's work
  double c[2];
  int from[2];
  double sum = 0.0;
  int last = 0;
  bool any = false;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int r = 2 * lane + j;
    const int64_t t = rows.token(r) + (reverse ? 1 : 0);
    double x = 0.0;
    if (t < rows.len) x = gate_at<T>(p, b, t, h);
    if (x < kRestart) {
      sum = 0.0;
      last = r;
      any = true;
    } else {
      sum += x * 1.4426950408889634;
    }
    c[j] = sum;
    from[j] = any ? last : -1;
  }
  // prefix over the lanes: (sum since the restart, restart or -1)
  double ps = sum;
  int pr = any ? last : -1;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const double os = __shfl_up_sync(0xffffffffu, ps, d);
    const int orr = __shfl_up_sync(0xffffffffu, pr, d);
    if (lane >= d) {
      if (pr < 0) {
        ps += os;
        pr = orr;
      }
    }
  }
  double es = __shfl_up_sync(0xffffffffu, ps, 1);
  int er = __shfl_up_sync(0xffffffffu, pr, 1);
  if (lane == 0) {
    es = 0.0;
    er = -1;
  }
  const double end = __shfl_sync(0xffffffffu, ps, 31);
  const int end_r = __shfl_sync(0xffffffffu, pr, 31);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int r = 2 * lane + j;
    if (from[j] < 0) {
      c[j] += es;
      from[j] = er;
    }
    const float hi = float(c[j]);
    g.hi[r] = hi;
    g.lo[r] = float(c[j] - double(hi));
    g.from[r] = from[j] < 0 ? 0 : from[j];
    g.read[r] = from[j] < 0 ? ex2_d(c[j]) : 0.0f;
    g.write[r] = r >= end_r ? ex2_d(end - c[j]) : 0.0f;
  }
  if (lane == 0) {
    g.keep = end_r < 0 ? keep_of(end) : make_float2(0.0f, 0.0f);
    g.end = end_r < 0 ? end : -CUDART_INF;
  }
}

template <typename T, int NP, int PS, int QD, bool STATE_ONLY>
struct Layout {
  static constexpr int LDQ = QD + 8, LDV = kLaTile + 8;
  static constexpr int TQ = kLaChunk * LDQ, TV = kLaChunk * LDV;
  static constexpr int TS = QD * LDV;
  static constexpr int K = 0;                       // bf16 offsets
  static constexpr int V = K + NP * TQ;
  static constexpr int Q = V + NP * TV;
  static constexpr int S = Q + (STATE_ONLY ? 0 : NP * TQ);
  static constexpr int END = S + (STATE_ONLY ? 0 : PS * TS);
  static constexpr int BYTES = END * 2 + 2 * int(sizeof(Gates));
};

// The state in the warps' accumulators, in the usual m16n8 layout. With 128
// key rows a warp owns 16 of them and all 64 columns; with 64, 16 rows and one
// half of the columns.
template <int QD>
struct StateMap {
  static constexpr int NT = QD == 128 ? 8 : 4;  // n-tiles of a warp
  __device__ __forceinline__ static int row0() {
    const int warp = threadIdx.x / 32;
    return (QD == 128 ? warp : warp % 4) * 16;
  }
  __device__ __forceinline__ static int col0() {
    return QD == 128 ? 0 : int(threadIdx.x) / 128 * 32;
  }
  template <class F>
  __device__ __forceinline__ static void each(F f) {
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int hr = 0; hr < 2; ++hr)
        f(n, hr, row0() + lane / 4 + hr * 8, col0() + n * 8 + (lane % 4) * 2);
  }
};

// MINB: resident blocks the registers are held to.
//
// Warp w computes rows 16 (w % 4).. of y, columns 32 (w / 4)... The tensor
// cores may truncate where they add to an accumulator, so products of the
// leading planes go to an accumulator of their own (`hi`), all smaller ones to
// a second (`lo`): the result then takes a few truncations, not six times as
// many.
template <typename T, int NP, int PS, int QD, bool STATE_ONLY, int MINB>
__global__ void __launch_bounds__(kThreads, MINB)
    linattn_kernel(const __grid_constant__ LaParams p) {
  using Lay = Layout<T, NP, PS, QD, STATE_ONLY>;
  using Map = StateMap<QD>;
  constexpr int NT = Map::NT;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  bf16 *sm = reinterpret_cast<bf16 *>(smem_raw);
  bf16 *Ks = sm + Lay::K, *Vs = sm + Lay::V;
  bf16 *Qs = sm + Lay::Q, *Ss = sm + Lay::S;
  Gates *gates = reinterpret_cast<Gates *>(sm + Lay::END);

  const LaJob &job = p.job[blockIdx.y];
  // tiles of one head, then heads, are neighbours: they read the same q and k
  unsigned x = blockIdx.x;
  const int tile = int(x % unsigned(job.tiles));
  x /= unsigned(job.tiles);
  const unsigned local = x % unsigned(p.bhs);
  const int seg = int(x / unsigned(p.bhs));
  const int h = int((p.bh0 + local) % unsigned(p.heads));
  const int64_t b = (p.bh0 + local) / unsigned(p.heads);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int wm = warp % 4, wn = warp / 4;
  const int64_t L = p.seqlen;
  int64_t len = L;
  if (p.lengths) {
    const int64_t n = p.lengths[b];
    len = n < 0 ? 0 : n > L ? L : n;
  }
  const int64_t total = p.nseg * p.seg_len;
  const int kh = h / (p.heads / job.k_heads);
  const int qh = h / (p.heads / job.q_heads);
  const int vh = h / (p.heads / job.v_heads);
  const int c0 = tile * kLaTile;
  const int vcols = min(job.vd - c0, kLaTile);
  const T *kb = static_cast<const T *>(job.k) + b * L * job.k_stride +
                int64_t(kh) * job.qd;
  const T *qb = static_cast<const T *>(job.q) + b * L * job.q_stride +
                int64_t(qh) * job.qd;
  const T *vb = static_cast<const T *>(job.v) + b * L * job.v_stride +
                int64_t(vh) * job.vd + c0;
  constexpr int VE = 16 / sizeof(T);
  auto vec_ok = [&](const T *s, int64_t stride) {
    return (reinterpret_cast<uintptr_t>(s) % 16) == 0 && stride % VE == 0;
  };
  const bool kvec = vec_ok(kb, job.k_stride), qvec = vec_ok(qb, job.q_stride),
             vvec = vec_ok(vb, job.v_stride);

  const int64_t bh = b * p.heads + h;
  constexpr int64_t SF = int64_t(QD) * kLaTile;
  float *seg_state =
      p.nseg > 1
          ? job.seg_state +
                ((int64_t(local) * p.nseg + seg) * job.tiles + tile) * SF
          : nullptr;

  float S[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) S[n][j] = 0.0f;
  if (!STATE_ONLY) {
    if (p.nseg > 1) {
      Map::each([&](int n, int hr, int row, int col) {
        const float2 v = *reinterpret_cast<const float2 *>(
            seg_state + row * kLaTile + col);
        S[n][2 * hr] = v.x;
        S[n][2 * hr + 1] = v.y;
      });
    } else if (job.init) {
      const float *src = job.init + bh * job.qd * job.vd;
      Map::each([&](int n, int hr, int row, int col) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (row < job.qd && c0 + col + j < job.vd)
            S[n][2 * hr + j] = src[int64_t(row) * job.state_rs +
                                   int64_t(c0 + col + j) * job.state_cs];
      });
    }
  }

  double seg_sum = 0.0;  // of the chunks' log decays
  const int chunks = int(p.seg_len / kLaChunk);
  auto rows_of = [&](int ch) {
    Rows rows;
    const int64_t i0 = int64_t(seg) * p.seg_len + int64_t(ch) * kLaChunk;
    rows.first = job.reverse ? total - 1 - i0 : i0;
    rows.dir = job.reverse ? -1 : 1;
    rows.len = len;
    return rows;
  };
  bool ready = false;  // this chunk's decays are summed
  for (int ch = 0; ch < chunks; ++ch) {
    Gates &gt = gates[ch & 1];
    const Rows rows = rows_of(ch);
    const int64_t lowest =
        job.reverse ? rows.first - (kLaChunk - 1) : rows.first;
    const bool idle = lowest >= len;
    if (idle) {
      // no live step: the state stays, the rows of y behind the sequence are 0
      if (!STATE_ONLY && lowest < L) {
        const int64_t n = L - lowest < kLaChunk ? L - lowest : kLaChunk;
        for (int64_t i = threadIdx.x; i < n * vcols; i += kThreads) {
          const int64_t t = lowest + i / vcols;
          const int64_t at =
              ((b * L + t) * p.heads + h) * job.vd + c0 + i % vcols;
          if (job.y_f32)
            static_cast<float *>(job.y)[at] = 0.0f;
          else
            static_cast<T *>(job.y)[at] = T(0.0f);
        }
      }
      continue;
    }
    if constexpr (!STATE_ONLY) {
      // between tokens `edge` - 1 and `edge`: what the decay's gradient needs
      const int64_t edge = job.reverse ? rows.first + 1 : rows.first;
      if (job.anchor && (edge & (p.anchor_len - 1)) == 0 && edge > 0 &&
          edge < len) {
        const int64_t at = edge / p.anchor_len;
        float *dst =
            job.anchor +
            ((bh * p.anchors + (job.reverse ? p.anchors - at : at)) *
                 job.tiles +
             tile) *
                SF;
        Map::each([&](int n, int hr, int row, int col) {
          *reinterpret_cast<float2 *>(dst + row * kLaTile + col) =
              make_float2(S[n][2 * hr], S[n][2 * hr + 1]);
        });
      }
    }

    {
      RawTile<T, QD> rk, rq;
      RawTile<T, kLaTile> rv;
      rk.load(kb, job.k_stride, job.qd, rows, kvec);
      rv.load(vb, job.v_stride, vcols, rows, vvec);
      if constexpr (!STATE_ONLY)
        rq.load(qb, job.q_stride, job.qd, rows, qvec);
      if (ch + 1 < chunks) {
        const Rows next = rows_of(ch + 1);
        prefetch_tile(kb, job.k_stride, job.qd, next);
        prefetch_tile(vb, job.v_stride, vcols, next);
        if constexpr (!STATE_ONLY)
          prefetch_tile(qb, job.q_stride, job.qd, next);
      }
      __syncthreads();  // the last chunk's reads are done
      if (warp == 0 && !ready) load_gates<T>(gt, p, rows, b, h, job.reverse);
      rk.template store<NP>(Ks);
      rv.template store<NP>(Vs);
      if constexpr (!STATE_ONLY) {
        rq.template store<NP>(Qs);
        Map::each([&](int n, int hr, int row, int col) {
          uint32_t pl[PS];
          split2<PS>(S[n][2 * hr], S[n][2 * hr + 1], pl);
#pragma unroll
          for (int s = 0; s < PS; ++s)
            *reinterpret_cast<uint32_t *>(Ss + s * Lay::TS + row * Lay::LDV +
                                          col) = pl[s];
        });
      }
    }
    __syncthreads();

    if constexpr (!STATE_ONLY) {
      const int r0 = wm * 16 + lane / 4;  // rows r0 and r0 + 8 of this lane
      // ---- scores: 16 rows, all columns up to the diagonal
      float P[8][4];
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) P[n][j] = 0.0f;
      {
        float lo[NP > 1 ? 8 : 1][4];
        if constexpr (NP > 1) {
#pragma unroll
          for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) lo[n][j] = 0.0f;
        }
#pragma unroll
        for (int ks = 0; ks < QD / 16; ++ks) {
          uint32_t a[NP][4];
#pragma unroll
          for (int s = 0; s < NP; ++s)
            ldsm4(a[s], Qs + s * Lay::TQ + (wm * 16 + lane % 16) * Lay::LDQ +
                            ks * 16 + (lane / 16) * 8);
#pragma unroll
          for (int n2 = 0; n2 < 4; ++n2) {
            if (n2 <= wm) {
              uint32_t bk[NP][4];
#pragma unroll
              for (int s = 0; s < NP; ++s)
                ldsm4(bk[s], Ks + s * Lay::TQ +
                                 (n2 * 16 + lane % 8 + (lane / 16) * 8) *
                                     Lay::LDQ +
                                 ks * 16 + ((lane / 8) % 2) * 8);
#pragma unroll
              for (int s = 0; s < NP; ++s)
#pragma unroll
                for (int u = 0; u < NP; ++u) {
                  if constexpr (NP > 1) {
                    if (s + u > 0 && s + u < 3) {
                      mma(lo[2 * n2], a[s], bk[u][0], bk[u][1]);
                      mma(lo[2 * n2 + 1], a[s], bk[u][2], bk[u][3]);
                    }
                  }
                  if (s + u == 0) {
                    mma(P[2 * n2], a[0], bk[0][0], bk[0][1]);
                    mma(P[2 * n2 + 1], a[0], bk[0][2], bk[0][3]);
                  }
                }
            }
          }
        }
        if constexpr (NP > 1) {
#pragma unroll
          for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) P[n][j] += lo[n][j];
        }
      }
      // ---- decay
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        const int r = r0 + 8 * hr;
        const float chi = gt.hi[r], clo = gt.lo[r];
        const int from = gt.from[r];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          if (n < 2 * wm + 2) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int c = n * 8 + (lane % 4) * 2 + j;
              const float d =
                  ex2((chi - gt.hi[c]) + (clo - gt.lo[c])) * job.sp;
              P[n][2 * hr + j] =
                  (c <= r && c >= from) ? P[n][2 * hr + j] * d : 0.0f;
            }
          }
        }
      }
      // ---- the state's part, columns 32 wn .. 32 wn + 31
      constexpr bool OLO = NP > 1 || PS > 1;
      float O[4][4], lo[OLO ? 4 : 1][4];
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          O[n][j] = 0.0f;
          if (OLO) lo[OLO ? n : 0][j] = 0.0f;
        }
#pragma unroll
      for (int ks = 0; ks < QD / 16; ++ks) {
        uint32_t a[NP][4];
#pragma unroll
        for (int s = 0; s < NP; ++s)
          ldsm4(a[s], Qs + s * Lay::TQ + (wm * 16 + lane % 16) * Lay::LDQ +
                          ks * 16 + (lane / 16) * 8);
#pragma unroll
        for (int n2 = 0; n2 < 2; ++n2) {
          uint32_t bs[PS][4];
#pragma unroll
          for (int s = 0; s < PS; ++s)
            ldsm4t(bs[s], Ss + s * Lay::TS +
                              (ks * 16 + lane % 16) * Lay::LDV + wn * 32 +
                              n2 * 16 + (lane / 16) * 8);
#pragma unroll
          for (int s = 0; s < NP; ++s)
#pragma unroll
            for (int u = 0; u < PS; ++u) {
              if constexpr (OLO) {
                if (s + u > 0 && s + u < 3) {
                  mma(lo[2 * n2], a[s], bs[u][0], bs[u][1]);
                  mma(lo[2 * n2 + 1], a[s], bs[u][2], bs[u][3]);
                }
              }
              if (s + u == 0) {
                mma(O[2 * n2], a[0], bs[0][0], bs[0][1]);
                mma(O[2 * n2 + 1], a[0], bs[0][2], bs[0][3]);
              }
            }
        }
      }
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        const float rd = gt.read[r0 + 8 * hr] * job.si;
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int j = 2 * hr; j < 2 * hr + 2; ++j) {
            // a restart forgets the state whatever it held
            O[n][j] = rd == 0.0f ? 0.0f : O[n][j] * rd;
            if constexpr (OLO)
              lo[n][j] = rd == 0.0f ? 0.0f : lo[n][j] * rd;
          }
      }
      // ---- scores times values
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if (kk <= wm) {
          uint32_t a[PS][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t pl[PS];
            split2<PS>(P[2 * kk + i / 2][2 * (i % 2)],
                       P[2 * kk + i / 2][2 * (i % 2) + 1], pl);
#pragma unroll
            for (int s = 0; s < PS; ++s) a[s][i] = pl[s];
          }
#pragma unroll
          for (int n2 = 0; n2 < 2; ++n2) {
            uint32_t bv[NP][4];
#pragma unroll
            for (int s = 0; s < NP; ++s)
              ldsm4t(bv[s], Vs + s * Lay::TV +
                                (kk * 16 + lane % 16) * Lay::LDV + wn * 32 +
                                n2 * 16 + (lane / 16) * 8);
#pragma unroll
            for (int s = 0; s < PS; ++s)
#pragma unroll
              for (int u = 0; u < NP; ++u) {
                if constexpr (OLO) {
                  if (s + u > 0 && s + u < 3) {
                    mma(lo[2 * n2], a[s], bv[u][0], bv[u][1]);
                    mma(lo[2 * n2 + 1], a[s], bv[u][2], bv[u][3]);
                  }
                }
                if (s + u == 0) {
                  mma(O[2 * n2], a[0], bv[0][0], bv[0][1]);
                  mma(O[2 * n2 + 1], a[0], bv[0][2], bv[0][3]);
                }
              }
          }
        }
      }
      if constexpr (OLO) {
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) O[n][j] += lo[n][j];
      }
      // ---- y, and the row dots the decay's gradient is made of
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        const int r = r0 + 8 * hr;
        const int64_t t = rows.token(r);
        const bool in = t < L, live = t < len;
        float dot = 0.0f;
        if (in) {
          const int64_t at = ((b * L + t) * p.heads + h) * job.vd + c0;
          const T *ds =
              job.dot ? static_cast<const T *>(job.dot) +
                            (b * L + t) * job.dot_stride +
                            int64_t(h / (p.heads / job.dot_heads)) * job.vd +
                            c0
                      : nullptr;
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const int c = wn * 32 + n * 8 + (lane % 4) * 2;
            const float v0 = live ? O[n][2 * hr] : 0.0f;
            const float v1 = live ? O[n][2 * hr + 1] : 0.0f;
            if (job.y_f32) {
              float *y = static_cast<float *>(job.y) + at + c;
              if (c + 1 < vcols && job.vd % 2 == 0) {
                *reinterpret_cast<float2 *>(y) = make_float2(v0, v1);
              } else {
                if (c < vcols) y[0] = v0;
                if (c + 1 < vcols) y[1] = v1;
              }
            } else {
              T *y = static_cast<T *>(job.y) + at + c;
              if (c + 1 < vcols && job.vd % 2 == 0) {
                if constexpr (sizeof(T) == 2)
                  *reinterpret_cast<uint32_t *>(y) = pack2(v0, v1);
                else
                  *reinterpret_cast<float2 *>(y) = make_float2(v0, v1);
              } else {
                if (c < vcols) y[0] = T(v0);
                if (c + 1 < vcols) y[1] = T(v1);
              }
            }
            if (ds && live) {
              if (c < vcols) dot += v0 * to_f(ds[c]);
              if (c + 1 < vcols) dot += v1 * to_f(ds[c + 1]);
            }
          }
        }
        if (job.rows) {
          dot += __shfl_xor_sync(0xffffffffu, dot, 1);
          dot += __shfl_xor_sync(0xffffffffu, dot, 2);
          if (in && lane % 4 == 0)
            job.rows[((int64_t(2 * tile + wn) * p.batch + b) * p.heads + h) *
                         L + t] = dot;
        }
      }
    }

    // the next chunk's decays, by a warp whose rows have the fewest scores;
    // where an SM holds one block only, for another would fill the wait (2 x
    // 4096 steps, 16 heads of 128, float32: 641 us without, 620 so; 64 x 512
    // steps, 8 heads of 64, two blocks an SM: 199 without, 204 so)
    ready = MINB == 1 && ch + 1 < chunks;
    if (warp == 0 && ready)
      load_gates<T>(gates[(ch + 1) & 1], p, rows_of(ch + 1), b, h,
                    job.reverse);

    // ---- the state: S <- keep S + (weighted k)^T v
    const float2 keep = gt.keep;
    if constexpr (STATE_ONLY) seg_sum += gt.end;
    float U[NT][4], lo[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) U[n][j] = lo[n][j] = 0.0f;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      uint32_t kr[NP][4], a[3][4];
#pragma unroll
      for (int s = 0; s < NP; ++s)
        ldsm4t(kr[s], Ks + s * Lay::TQ +
                          (kk * 16 + lane % 8 + (lane / 16) * 8) * Lay::LDQ +
                          Map::row0() + ((lane / 8) % 2) * 8);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float f0 = 0.0f, f1 = 0.0f;
#pragma unroll
        for (int s = NP - 1; s >= 0; --s) {
          f0 += lo2(kr[s][i]);
          f1 += hi2(kr[s][i]);
        }
        const float2 w = *reinterpret_cast<const float2 *>(
            gt.write + kk * 16 + (lane % 4) * 2 + (i / 2) * 8);
        uint32_t pl[3];
        split2<3>(f0 * (w.x * job.sw), f1 * (w.y * job.sw), pl);
#pragma unroll
        for (int s = 0; s < 3; ++s) a[s][i] = pl[s];
      }
#pragma unroll
      for (int n2 = 0; n2 < NT / 2; ++n2) {
        uint32_t bv[NP][4];
#pragma unroll
        for (int s = 0; s < NP; ++s)
          ldsm4t(bv[s], Vs + s * Lay::TV +
                            (kk * 16 + lane % 16) * Lay::LDV + Map::col0() +
                            n2 * 16 + (lane / 16) * 8);
#pragma unroll
        for (int s = 0; s < 3; ++s)
#pragma unroll
          for (int u = 0; u < NP; ++u) {
            if (s + u > 0 && s + u < 3) {
              mma(lo[2 * n2], a[s], bv[u][0], bv[u][1]);
              mma(lo[2 * n2 + 1], a[s], bv[u][2], bv[u][3]);
            }
            if (s + u == 0) {
              mma(U[2 * n2], a[0], bv[0][0], bv[0][1]);
              mma(U[2 * n2 + 1], a[0], bv[0][2], bv[0][3]);
            }
          }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float u = U[n][j] + lo[n][j];
        S[n][j] = none_kept(keep)
                      ? u
                      : fmaf(keep.y, S[n][j], fmaf(keep.x, S[n][j], u));
      }
  }

  if constexpr (STATE_ONLY) {
    Map::each([&](int n, int hr, int row, int col) {
      *reinterpret_cast<float2 *>(seg_state + row * kLaTile + col) =
          make_float2(S[n][2 * hr], S[n][2 * hr + 1]);
    });
    if (tile == 0 && threadIdx.x == 0)
      job.seg_decay[int64_t(local) * p.nseg + seg] = exp2(seg_sum);
  } else if (job.last && seg == p.nseg - 1) {
    // running backwards, the first token's own decay is still to come
    float f = 1.0f;
    if (job.reverse && len > 0)
      f = decay_of(gate_at<T>(p, b, 0, h));
    float *dst = job.last + bh * job.qd * job.vd;
    Map::each([&](int n, int hr, int row, int col) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (row < job.qd && c0 + col + j < job.vd)
          dst[int64_t(row) * job.state_rs +
              int64_t(c0 + col + j) * job.state_cs] =
              f == 0.0f ? 0.0f : S[n][2 * hr + j] * f;
    });
  }
}

// The states in front of the segments, from what each segment adds on its own:
// S_{m+1} = decay_m S_m + U_m, in place (entry m takes S_m; the last segment's
// own part is not formed here), in 64 bits. One thread per state element.
template <int QD>
__global__ void __launch_bounds__(256)
    linattn_join_kernel(const __grid_constant__ LaParams p) {
  const LaJob &job = p.job[blockIdx.z];
  constexpr int SF = QD * kLaTile;
  const int per = SF * job.tiles;
  const int el = int(blockIdx.x) * 256 + int(threadIdx.x);
  if (el >= per) return;
  const int tile = el / SF, row = el % SF / kLaTile,
            col = el % kLaTile + tile * kLaTile;
  for (int64_t local = blockIdx.y; local < p.bhs; local += gridDim.y) {
    const int64_t bh = p.bh0 + local;
    double S = 0.0;
    if (job.init && row < job.qd && col < job.vd)
      S = job.init[bh * job.qd * job.vd + int64_t(row) * job.state_rs +
                   int64_t(col) * job.state_cs];
    float *u = job.seg_state + local * p.nseg * per + el;  // (a segment: per)
    const double *d = job.seg_decay + local * p.nseg;
    // sixteen segments' parts are on their way at a time
    const int n = p.nseg - 1;
    for (int m = 0; m < n; m += 16) {
      float a[16];
      double k[16];
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (m + j < n) {
          a[j] = u[int64_t(m + j) * per];
          k[j] = d[m + j];
        }
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (m + j < n) {
          u[int64_t(m + j) * per] = float(S);
          S = k[j] == 0.0 ? double(a[j]) : fma(k[j], S, double(a[j]));
        }
    }
    u[int64_t(n) * per] = float(S);
  }
}

__device__ __forceinline__ double block_sum(double v, double *red) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < int(blockDim.x) / 32; ++w) s += red[w];
  __syncthreads();
  return s;
}

// The log decay's gradient. With G the gradient of the state,
//   dg_t = <a_t S_{t-1}, G_t> = dg_{t+1} + q_t . dq_t - k_t . dk_t,
// summed backwards inside each group of steps from its end, where the product
// of the state and its gradient is formed from the states the two passes left
// there: what the differences are off by then adds up over one group only,
// and the products' own errors over groups that know nothing of each other.
// Where a float32 result comes of them, groups are 128 steps and the sums
// 64-bit: of 2048 steps and in float32, the sum of a head's gradients
// over 2 x 16384 steps was 2.7e-5 off (the plain form: 9e-7). Alone beside
// bfloat16, segments of 2048 steps are as good as the output. A step that
// starts the state anew has no gradient, and the sum starts from 0 there: the
// differences behind it cancel in exact arithmetic only, and what rounding
// leaves of them is not the business of the steps in front. One block per
// (sequence, head, group).
template <typename T>
__global__ void __launch_bounds__(256)
    linattn_gate_kernel(const __grid_constant__ LaGateParams p) {
  __shared__ double red[8];
  __shared__ double warp_tot[8];
  __shared__ bool warp_anew[8];
  const int64_t x = blockIdx.x;
  const int seg = int(x % p.nseg);
  const int64_t bh = x / p.nseg;
  const int64_t b = bh / p.heads;
  const int h = int(bh % p.heads);
  const int64_t L = p.seqlen;
  int64_t len = L;
  if (p.lengths) {
    const int64_t n = p.lengths[b];
    len = n < 0 ? 0 : n > L ? L : n;
  }
  const int64_t t0 = int64_t(seg) * p.seg_len;
  const int64_t t1 = t0 + p.seg_len;
  const double head = p.head_log_decay ? double(p.head_log_decay[h]) : 0.0;
  auto log_of = [&](float g) { return double(g) + head; };
  // the product of the state behind the group and its gradient
  const float *S = nullptr, *G = nullptr;
  int64_t n = 0;
  double end = 0.0;
  if (t1 < len) {
    S = p.fwd_state + (bh * p.nseg + seg + 1) * p.state_floats;
    G = p.rev_state + (bh * p.nseg + p.nseg - 1 - seg) * p.state_floats;
    n = p.state_floats;
  } else if (p.dh_last && t0 < len) {
    S = p.last_state + bh * p.last_floats;
    G = p.dh_last + bh * p.last_floats;
    n = p.last_floats;
  }
  if (n) {
    float s = 0.0f;
#pragma unroll 16
    for (int64_t i = threadIdx.x; i < n; i += 256) s = fmaf(S[i], G[i], s);
    end = block_sum(double(s), red);
    if (t1 < len) {  // the decay of the next group's first token
      const float a = decay_of(log_of(
          p.log_decay ? to_f(static_cast<const T *>(
                            p.log_decay)[(b * L + t1) * p.heads + h])
                      : 0.0f));
      end = a == 0.0f ? 0.0 : end * double(a);
    }
  }
  // backwards, a whole segment at a time where it is one of 2048: thread i has
  // the i-th kRun tokens from the end, all on their way at once (8 x 24 heads
  // of 2048 tokens: 18 us with a token a thread in eight rounds, 13 so)
  constexpr int kRun = 8;
  double carry = end, part = 0.0;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int64_t hi = t1; hi > t0; hi -= 256 * kRun) {
    const int64_t last = hi - 1 - int64_t(threadIdx.x) * kRun;
    double v[kRun];
    float u[kRun], w[kRun];
    T g[kRun];
    auto in = [&](int j) { return last - j >= t0 && last - j < len; };
    const int64_t at = (b * p.heads + h) * L + last;
    const int64_t step = p.batch * p.heads * L;
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      w[j] = in(j) ? p.rows_q[at - j] : 0.0f;
      u[j] = in(j) ? p.rows_k[at - j] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < kRun; ++j)
      g[j] = p.log_decay && in(j)
                 ? static_cast<const T *>(
                       p.log_decay)[(b * L + last - j) * p.heads + h]
                 : T(0.0f);
#pragma unroll
    for (int j = 0; j < kRun; ++j) v[j] = double(w[j]) - double(u[j]);
    for (int k = 1; k < p.parts; ++k) {
      const float *q = p.rows_q + k * step, *r = p.rows_k + k * step;
#pragma unroll
      for (int j = 0; j < kRun; ++j)
        if (in(j)) v[j] += double(q[at - j]) - double(r[at - j]);
    }
    // sums since the last restart behind each token; `anew`: there is one in
    // this thread's tokens so far (bits), its warp's, the block's
    uint32_t anew = 0u;
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      const bool starts = in(j) && log_of(to_f(g[j])) < kRestart;
      anew |= uint32_t(starts) << j;
      v[j] = starts ? 0.0 : j ? v[j] + v[j - 1] : v[j];
    }
    double sum = v[kRun - 1];
    int any = anew != 0u;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const double o = __shfl_up_sync(0xffffffffu, sum, d);
      const int oa = __shfl_up_sync(0xffffffffu, any, d);
      if (lane >= d && !any) {
        sum += o;
        any = oa;
      }
    }
    if (lane == 31) {
      warp_tot[warp] = sum;
      warp_anew[warp] = any;
    }
    // what lies behind this thread's tokens in its warp
    double before = __shfl_up_sync(0xffffffffu, sum, 1);
    int cut = __shfl_up_sync(0xffffffffu, any, 1);
    if (lane == 0) {
      before = 0.0;
      cut = 0;
    }
    __syncthreads();
    double behind = carry;
    for (int i = 0; i < 8; ++i) {
      if (i == warp && !cut) before += behind;
      behind = warp_anew[i] ? warp_tot[i] : behind + warp_tot[i];
    }
    carry = behind;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      const int64_t t = last - j;
      if (t >= t0 && t < L) {
        // (a step that starts the state anew does not depend on its decay)
        const bool live = t < len && !(anew >> j & 1u);
        const bool whole = (anew & ((2u << j) - 1u)) == 0u;
        const double out = live ? (whole ? before + v[j] : v[j]) : 0.0;
        if (p.dlog_decay)
          static_cast<T *>(p.dlog_decay)[(b * L + t) * p.heads + h] =
              T(float(out));
        part += out;
      }
    }
  }
  if (p.part) {
    part = block_sum(part, red);
    if (threadIdx.x == 0) p.part[(b * p.nseg + seg) * p.heads + h] = part;
  }
}

// out[h] = sum over n rows of part[n][heads], in a fixed order.
__global__ void __launch_bounds__(128)
    linattn_head_sum_kernel(const double *part, int64_t n, int heads,
                            float *out) {
  __shared__ double red[4];
  const int h = blockIdx.x;
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 128)
    s += part[i * heads + h];
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = s;
  __syncthreads();
  if (threadIdx.x == 0) out[h] = float(red[0] + red[1] + red[2] + red[3]);
}

// The gradient of a shared head: out[r][g][d] = sum of the group's heads, in
// order, of part[r][h][d].
template <typename T>
__global__ void __launch_bounds__(256)
    linattn_group_sum_kernel(const float *part, int64_t rows, int groups,
                             int per, int d, T *out) {
  const int64_t n = rows * groups * d;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n;
       i += int64_t(gridDim.x) * 256) {
    const int64_t rg = i / d;
    const int c = int(i % d);
    float s = 0.0f;
    for (int k = 0; k < per; ++k) s += part[(rg * per + k) * d + c];
    out[i] = T(s);
  }
}

// ---- one token: S <- a S + k (x) v in place, y = scale q S.
// Bound by the state's bytes (read and written once). A block of 8 warps owns
// one head and LPR W value columns: LPR lanes (16 where 64 columns are all
// there are) share a key row, W columns each, so that a warp takes 32 / LPR
// rows at a time and a block 256 / LPR; eight of them a thread are on their
// way at once, the first before anything else is read. The rows' parts of y
// are added through shared memory in a fixed order.
// 256 x 40 heads of 128 x 128 float32: 201 us, 6.7 TB/s.
template <typename T, int W, int LPR>
__global__ void __launch_bounds__(256)
    linattn_step_kernel(const __grid_constant__ LaStepParams p) {
  constexpr int COLS = LPR * W, STEP = 256 / LPR, ROWS = 8;
  __shared__ float ks[kLaMaxKey], qs[kLaMaxKey];
  __shared__ float part[8][COLS];
  const int tiles = (p.dv + COLS - 1) / COLS;
  const int tile = int(blockIdx.x % unsigned(tiles));
  const int64_t bh = blockIdx.x / unsigned(tiles);
  const int64_t b = bh / p.heads;
  const int h = int(bh % p.heads), g = h / (p.heads / p.groups);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int first = threadIdx.x / LPR, at = lane % LPR * W;
  const int c0 = tile * COLS + at;
  float *S = p.state + bh * p.dk * p.dv + c0;
  float x[ROWS][W];
  auto fetch = [&](int r0) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int r = r0 + STEP * i;
      if (r >= p.dk || c0 >= p.dv) break;
      const float *s = S + int64_t(r) * p.dv;
      if constexpr (W == 4) {
        const float4 u = __ldcs(reinterpret_cast<const float4 *>(s));
        x[i][0] = u.x; x[i][1] = u.y; x[i][2] = u.z; x[i][3] = u.w;
      } else {
        x[i][0] = s[0];
      }
    }
  };
  fetch(first);
  const T *kp = static_cast<const T *>(p.k) + b * p.k_stride + g * p.dk;
  const T *qp = static_cast<const T *>(p.q) + b * p.q_stride + g * p.dk;
  const T *vp = static_cast<const T *>(p.v) + b * p.v_stride + h * p.dv + c0;
  for (int i = threadIdx.x; i < p.dk; i += 256) {
    ks[i] = to_f(kp[i]);
    qs[i] = to_f(qp[i]);
  }
  double gd = 0.0;
  if (p.log_decay)
    gd = double(to_f(static_cast<const T *>(p.log_decay)[bh]));
  if (p.head_log_decay) gd += double(p.head_log_decay[h]);
  const float2 a = gd < kRestart ? make_float2(0.0f, 0.0f)
                                 : keep_of(gd * 1.4426950408889634);
  float v[W], y[W];
#pragma unroll
  for (int j = 0; j < W; ++j) {
    v[j] = c0 + j < p.dv ? to_f(vp[j]) : 0.0f;
    y[j] = 0.0f;
  }
  __syncthreads();
#pragma unroll 1
  for (int r0 = first; r0 < p.dk; r0 += STEP * ROWS) {
    if (r0 != first) fetch(r0);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int r = r0 + STEP * i;
      if (r >= p.dk || c0 >= p.dv) break;
#pragma unroll
      for (int j = 0; j < W; ++j) {
        // a = 0 starts anew, whatever the state held
        const float kv = ks[r] * v[j];
        x[i][j] = none_kept(a)
                      ? kv
                      : fmaf(a.y, x[i][j], fmaf(a.x, x[i][j], kv));
        y[j] = fmaf(qs[r], x[i][j], y[j]);
      }
      float *s = S + int64_t(r) * p.dv;
      if constexpr (W == 4)
        __stcs(reinterpret_cast<float4 *>(s),
               make_float4(x[i][0], x[i][1], x[i][2], x[i][3]));
      else
        s[0] = x[i][0];
    }
  }
#pragma unroll
  for (int j = 0; j < W; ++j) {
    if (LPR == 16) y[j] += __shfl_xor_sync(0xffffffffu, y[j], 16);
    if (lane < LPR) part[warp][at + j] = y[j];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < COLS; i += 256) {
    const int c = tile * COLS + i;
    if (c < p.dv) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < 8; ++w) s += part[w][i];
      static_cast<T *>(p.y)[bh * p.dv + c] = T(s * p.scale);
    }
  }
}

}  // namespace la
}  // namespace ssm
