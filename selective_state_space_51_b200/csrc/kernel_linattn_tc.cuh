// Linear attention with a decay for each head on the fifth-generation tensor
// cores: the pass of kernel_linattn.cuh (same mathematics, same jobs), for
// bfloat16 rows on 16-byte boundaries, key and value sizes up to 128, in
// chunks of 128 steps, one block for a whole head.
//
// Four products a chunk, each D[128][n] in TMEM:
//   P  [step i][step j]  = Q K^T            both from shared memory
//   O1 [step i][value]   = Q S              S: its bfloat16 copy in shared memory
//   U^T[value][key]      = (w V)^T K        (w V)^T from TMEM
//   O2 [step i][value]   = P' V             P' (decayed scores) from TMEM
//   y = read_i O1 + O2,  S^T <- keep S^T + U^T (float32, registers)
// The weighted values need three bfloat16 planes for a float32 state; as the A
// operand in TMEM they cost no shared memory and no bank traffic, and the
// state's transpose lies in the same lanes (one value column a lane) as the
// product that is added to it. They go through two buffers of 32 steps.
//
// Warps 0-7 compute: warp w has lanes 32 (w % 4).. of every TMEM tile and half
// w / 4 of its columns. Warp 8 loads q, k and v by TMA, two chunks deep; warp
// 9 issues the products; warp 10 sums the decays, one chunk ahead. Everything
// between them goes through mbarriers with bounded waits.
//
// The decay e^{c_i - c_j}: outside the 32 x 32 blocks on the diagonal it is
// e^{c_i - c_r} e^{c_r - c_j}, r the last step of j's block: both factors are
// at most 1 for decays (no overflow), so a block costs one exponential a row
// and two products an element. On the diagonal it is formed directly.
#pragma once

#include "kernel_linattn.cuh"
#include "tcgen05.cuh"

namespace ssm {
namespace lat {

constexpr int kChunk = 128;
constexpr int kWarps = 11, kThreads = 32 * kWarps;
constexpr int kCompute = 256;

struct Params {
  CUtensorMap map[3][3];  // [job][q, k, v]
  LaParams p;             // seg_len: a multiple of kChunk
  int *status;
};

// The decays of a chunk; arrays by row (token order). Steps are counted in
// the order of time, which in reverse is from the last row.
struct Gates {
  float hi[kChunk], lo[kChunk];  // c since the last restart
  float read[kChunk];            // si e^{c_i}, 0 behind a restart
  float write[kChunk];           // sw e^{c_C - c_i}, 0 before a restart
  float near[kChunk];            // e^{c_r - c_j}, r: the last step of j's 32
  unsigned char from[kChunk];    // the last restart at or before the step
  float keep;
  int dead;
  uint32_t tmem;
  uint64_t bars[20];
};

enum Bar {
  kFull0, kFull1,      // q, k, v of a stage have arrived
  kEmpty0, kEmpty1,    // the stage's products are done
  kScores,             // P
  kRead,               // O1
  kWFull0, kWFull1, kWEmpty0, kWEmpty1,
  kUpdate,             // U
  kGo,                 // P' stored, O1 read
  kOut,                // O2
  kState,              // S stored, U read
  kOutRead,            // O2 read
  kGates, kGatesFree,
  kClean,              // rows behind the sequence's end zeroed
  kFin,
};

template <int QD, int TV, int PS, bool STATE_ONLY>
struct Lay {
  static constexpr int Q = kChunk * QD * 2, V = kChunk * TV * 2;
  static constexpr int STAGE = (STATE_ONLY ? Q : 2 * Q) + V;  // k, v(, q)
  static constexpr int S = STATE_ONLY ? 0 : PS * TV * QD * 2;
  static constexpr int GATES = 2 * STAGE + S;
  static constexpr int BYTES = GATES + int(sizeof(Gates));
  // TMEM columns
  static constexpr uint32_t P = 0, O = 128, U = 256, W = 384;
};

template <int QD, int TV, int PS, bool STATE_ONLY>
__global__ void __launch_bounds__(kThreads, 1)
    linattn_tc_kernel(const __grid_constant__ Params pp) {
  using L_ = Lay<QD, TV, PS, STATE_ONLY>;
  using la::bf16;
  using la::ex2_d;
  using la::pack2;
  extern __shared__ __align__(1024) unsigned char smem[];
  Gates &gt = *reinterpret_cast<Gates *>(smem + L_::GATES);
  const uint32_t base = tc::smem_addr(smem);
  const LaParams &p = pp.p;
  const LaJob &job = p.job[blockIdx.y];
  const CUtensorMap *maps = pp.map[blockIdx.y];

  int64_t x = blockIdx.x;
  const int h = int(x % p.heads);
  x /= p.heads;
  const int64_t b = x % p.batch;
  const int seg = int(x / p.batch);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t L = p.seqlen;
  int64_t len = L;
  if (p.lengths) {
    const int64_t n = p.lengths[b];
    len = n < 0 ? 0 : n > L ? L : n;
  }
  const bool rev = job.reverse;
  const int64_t total = p.nseg * p.seg_len;
  const int chunks = int(p.seg_len / kChunk);
  // first token of chunk c, in the order of time
  auto low = [&](int c) {
    const int64_t i0 = int64_t(seg) * p.seg_len + int64_t(c) * kChunk;
    return rev ? total - i0 - kChunk : i0;
  };
  // chunks [first, last) hold live steps
  int first = 0, last = chunks;
  if (rev) {
    const int64_t over = low(0) - len;  // chunk c is live: low(c) < len
    if (over >= 0)
      first = int(over / kChunk + 1 < chunks ? over / kChunk + 1 : chunks);
  } else {
    const int64_t left = len - low(0);
    const int64_t n = left <= 0 ? 0 : (left + kChunk - 1) / kChunk;
    if (n < chunks) last = int(n);
  }
  const int n_live = last - first;

  auto bar = [&](int i) {
    return base + uint32_t(L_::GATES) +
           uint32_t(reinterpret_cast<const char *>(&gt.bars[i]) -
                    reinterpret_cast<const char *>(&gt));
  };
  volatile int *dead = &gt.dead;
  auto wait = [&](int i, uint32_t parity) {
    return tc::bar_wait(bar(i), parity & 1u, dead, pp.status);
  };
  if (warp == 9) {
    tc::tmem_alloc(base + uint32_t(L_::GATES) +
                       uint32_t(reinterpret_cast<const char *>(&gt.tmem) -
                                reinterpret_cast<const char *>(&gt)),
                   512);
  }
  if (threadIdx.x == 0) {
    gt.dead = 0;
    for (int i = 0; i <= kFin; ++i) {
      const bool all = i == kWFull0 || i == kWFull1 || i == kGo ||
                       i == kState || i == kOutRead || i == kGatesFree ||
                       i == kClean;
      tc::bar_init(bar(i), all ? kCompute : 1);
    }
    tc::fence_init();
  }
  tc::before_sync();
  __syncthreads();
  tc::after_sync();
  const uint32_t tmem = gt.tmem;
  // the chunk in which the sequence ends before its rows do
  const int64_t end_low = len / kChunk * kChunk;
  auto ragged = [&](int c) { return len < L && low(c) == end_low; };
  const int64_t bh = b * p.heads + h;

  if (warp == 8) {
    // ---- loads: stage it % 2, two chunks deep
    const int kh = h / (p.heads / job.k_heads);
    const int qh = h / (p.heads / job.q_heads);
    const int vh = h / (p.heads / job.v_heads);
    for (int it = 0; it < n_live; ++it) {
      const int st = it & 1;
      if (it >= 2 && !wait(kEmpty0 + st, uint32_t(it / 2 - 1))) break;
      if (lane == 0) {
        const int tok = int(low(first + it));
        const uint32_t s = base + st * L_::STAGE;
        tc::bar_expect(bar(kFull0 + st), L_::STAGE);
        for (int c = 0; c < QD / 64; ++c) {
          tc::load_box(s + c * 16384, &maps[1], bar(kFull0 + st), c * 64, kh,
                       tok, int(b));
          if (!STATE_ONLY)
            tc::load_box(s + L_::Q + L_::V + c * 16384, &maps[0],
                         bar(kFull0 + st), c * 64, qh, tok, int(b));
        }
        for (int c = 0; c < TV / 64; ++c)
          tc::load_box(s + L_::Q + c * 16384, &maps[2], bar(kFull0 + st),
                       c * 64, vh, tok, int(b));
      }
      __syncwarp();
    }
    if (*dead) {  // nothing may still be on its way into this block's memory
      for (int it = n_live > 2 ? n_live - 2 : 0; it < n_live; ++it)
        for (int i = 0; i < 1 << 16; ++i)
          if (tc::bar_try(bar(kFull0 + (it & 1)), uint32_t(it / 2) & 1u)) break;
    }
  } else if (warp == 9) {
    // ---- products
    constexpr uint32_t kScoreShape = tc::shape(128, false);
    constexpr uint32_t kReadShape = tc::shape(TV, false);
    constexpr uint32_t kUpdateShape = tc::shape(QD, true);
    constexpr uint32_t kOutShape = tc::shape(TV, true);
    bool alive = true;
    for (int it = 0; it < n_live && alive; ++it) {
      const int st = it & 1;
      const uint32_t K = base + st * L_::STAGE, V = K + L_::Q,
                     Q = V + L_::V, S = base + 2 * L_::STAGE;
      alive = wait(kFull0 + st, it / 2);
      if (alive && ragged(first + it)) alive = wait(kClean, 0);
      if (!alive) break;
      tc::after_sync();
      if constexpr (!STATE_ONLY) {
        if (lane == 0) {
#pragma unroll
          for (int ks = 0; ks < QD / 16; ++ks) {
            const uint32_t off = (ks / 4) * 16384 + (ks % 4) * 32;
            tc::mma_ss(tmem + L_::P, tc::operand(Q + off, 0),
                       tc::operand(K + off, 0), kScoreShape, ks > 0);
          }
          tc::commit(bar(kScores));
        }
        __syncwarp();
      }
      alive = wait(kState, it);
      if (!alive) break;
      if constexpr (!STATE_ONLY) {
        if (it > 0) alive = wait(kOutRead, it - 1);
        if (!alive) break;
        tc::after_sync();
        if (lane == 0) {
#pragma unroll
          for (int s = PS - 1; s >= 0; --s)
#pragma unroll
            for (int ks = 0; ks < QD / 16; ++ks)
              tc::mma_ss(
                  tmem + L_::O,
                  tc::operand(Q + (ks / 4) * 16384 + (ks % 4) * 32, 0),
                  tc::operand(S + s * TV * QD * 2 + (ks / 4) * TV * 128 +
                                  (ks % 4) * 32,
                              0),
                  kReadShape, ks > 0 || s < PS - 1);
          tc::commit(bar(kRead));
        }
        __syncwarp();
      }
      for (int qr = 0; qr < 4 && alive; ++qr) {
        if constexpr (!STATE_ONLY) {
          if (qr == 2) {
            alive = wait(kGo, it);
            if (!alive) break;
            tc::after_sync();
            if (lane == 0) {
#pragma unroll
              for (int s = PS - 1; s >= 0; --s)
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                  tc::mma_ts(tmem + L_::O,
                             tmem + L_::P + (ks / 4) * 64 + s * 32 +
                                 (ks % 4) * 8,
                             tc::operand(V + ks * 2048, 16384), kOutShape,
                             ks > 0 || s < PS - 1);
              tc::commit(bar(kOut));
            }
            __syncwarp();
          }
        }
        const int buf = qr & 1;
        alive = wait(kWFull0 + buf, it * 2 + qr / 2);
        if (!alive) break;
        tc::after_sync();
        if (lane == 0) {
#pragma unroll
          for (int s = 2; s >= 0; --s)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
              tc::mma_ts(tmem + L_::U,
                         tmem + L_::W + buf * 48 + s * 16 + ks * 8,
                         tc::operand(K + (qr * 2 + ks) * 2048, 16384),
                         kUpdateShape, qr > 0 || s < 2 || ks > 0);
          tc::commit(bar(kWEmpty0 + buf));
          if (qr == 3) {
            tc::commit(bar(kUpdate));
            tc::commit(bar(kEmpty0 + st));
          }
        }
        __syncwarp();
      }
    }
    // every product is done before the block goes
    if (lane == 0) tc::commit(bar(kFin));
    __syncwarp();
    for (int i = 0; i < 1 << 16; ++i)
      if (tc::bar_try(bar(kFin), 0)) break;
  } else if (warp == 10) {
    // ---- decays: four steps a lane, in the order of time
    auto fetch = [&](int it, double (&g)[4]) {
      const int64_t lo = low(first + it);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int s = 4 * lane + j;
        const int64_t t = rev ? lo + kChunk - s : lo + s;
        g[j] = t < len ? la::gate_at<bf16>(p, b, t, h) * 1.4426950408889634
                       : 0.0;
      }
    };
    double g[4];
    if (n_live > 0) fetch(0, g);
    for (int it = 0; it < n_live; ++it) {
      double c[4], sum = 0.0;
      int from[4], lastr = -1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (g[j] < -126.0) {
          sum = 0.0;
          lastr = 4 * lane + j;
        } else {
          sum += g[j];
        }
        c[j] = sum;
        from[j] = lastr;
      }
      if (it + 1 < n_live) fetch(it + 1, g);
      double ps = sum;
      int pr = lastr;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const double os = __shfl_up_sync(0xffffffffu, ps, d);
        const int orr = __shfl_up_sync(0xffffffffu, pr, d);
        if (lane >= d && pr < 0) {
          ps += os;
          pr = orr;
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
      const double blk = __shfl_sync(0xffffffffu, ps, lane | 7);
      const int blk_r = __shfl_sync(0xffffffffu, pr, lane | 7);
      if (it > 0 && !wait(kGatesFree, it - 1)) break;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int s = 4 * lane + j;
        if (from[j] < 0) {
          c[j] += es;
          from[j] = er;
        }
        const int r = rev ? kChunk - 1 - s : s;
        const float hi = float(c[j]);
        gt.hi[r] = hi;
        gt.lo[r] = float(c[j] - double(hi));
        gt.from[r] = (unsigned char)(from[j] < 0 ? 0 : from[j]);
        gt.read[r] = from[j] < 0 ? ex2_d(c[j]) * job.si : 0.0f;
        gt.write[r] = s >= end_r ? ex2_d(end - c[j]) * job.sw : 0.0f;
        gt.near[r] = s >= blk_r ? ex2_d(blk - c[j]) : 0.0f;
      }
      if (lane == 0) gt.keep = end_r < 0 ? ex2_d(end) : 0.0f;
      __syncwarp();
      if (lane == 0) tc::bar_arrive(bar(kGates));
    }
  } else {
    // ---- warps 0-7
    const int q4 = warp % 4, half = warp / 4;
    const int r = q4 * 32 + lane;  // this thread's TMEM lane
    const uint32_t mine = tmem + (uint32_t(q4 * 32) << 16);
    const bool has_v = q4 * 32 < TV;  // lanes of value columns
    constexpr int NS = QD / 2;        // state columns (keys) of a thread
    constexpr int NO = TV / 2;        // value columns of a thread
    const int k0 = half * NS;
    constexpr int64_t SF = int64_t(QD) * kLaTile;
    const int tiles = (job.vd + kLaTile - 1) / kLaTile;
    // element (key, value r) of a segment's state
    float *seg_state =
        p.nseg > 1 ? job.seg_state +
                         ((bh * p.nseg + seg) * tiles + r / kLaTile) * SF +
                         r % kLaTile
                   : nullptr;
    const bool seg_row = r / kLaTile < tiles;
    float S[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) S[i] = 0.0f;
    if (!STATE_ONLY && r < TV) {
      if (p.nseg > 1) {
        if (seg_row) {
#pragma unroll
          for (int i = 0; i < NS; ++i)
            S[i] = seg_state[int64_t(k0 + i) * kLaTile];
        }
      } else if (job.init && r < job.vd) {
        const float *src =
            job.init + bh * job.qd * job.vd + int64_t(r) * job.state_cs;
#pragma unroll
        for (int i = 0; i < NS; ++i)
          if (k0 + i < job.qd) S[i] = src[int64_t(k0 + i) * job.state_rs];
      }
    }
    // rows of y behind the sequence's last live chunk
    auto zeros = [&](int from_chunk, int to_chunk) {
      for (int c = from_chunk; c < to_chunk; ++c) {
        const int64_t lo = low(c);
        const int64_t n = L - lo < kChunk ? L - lo : kChunk;
        for (int64_t i = threadIdx.x; i < n * job.vd; i += kCompute) {
          const int64_t at =
              ((b * L + lo + i / job.vd) * p.heads + h) * job.vd + i % job.vd;
          if (job.y_f32)
            static_cast<float *>(job.y)[at] = 0.0f;
          else
            static_cast<bf16 *>(job.y)[at] = bf16(0.0f);
        }
      }
    };
    if (!STATE_ONLY) {
      zeros(0, first);
      zeros(last, chunks);
    }
    // the bfloat16 planes of this thread's part of the state
    auto put_state = [&]() {
      if constexpr (!STATE_ONLY) {
        if (r < TV) {
#pragma unroll
          for (int i = 0; i < NS; i += 8) {
            uint32_t w[4][PS];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              la::split2<PS>(S[i + 2 * j], S[i + 2 * j + 1], w[j]);
            const int k = k0 + i;
            unsigned char *dst = smem + 2 * L_::STAGE + (k / 64) * TV * 128 +
                                 r * 128 + ((k % 64 / 8) ^ (r % 8)) * 16;
#pragma unroll
            for (int s = 0; s < PS; ++s)
              *reinterpret_cast<uint4 *>(dst + s * TV * QD * 2) =
                  make_uint4(w[0][s], w[1][s], w[2][s], w[3][s]);
          }
        }
        tc::fence_async();
      }
      tc::before_sync();
      tc::bar_arrive(bar(kState));
    };
    put_state();
    float seg_keep = 1.0f;
    bool alive = true;
    for (int it = 0; it < n_live && alive; ++it) {
      const int st = it & 1;
      unsigned char *Ks = smem + st * L_::STAGE, *Vs = Ks + L_::Q;
      const int64_t lo = low(first + it);
      alive = wait(kFull0 + st, it / 2) && wait(kGates, it);
      if (!alive) break;
      if (ragged(first + it)) {
        // rows behind the sequence's end: zeros, whatever was loaded
        const int dead_from = int(len - lo);
        for (int i = threadIdx.x + dead_from * 8; i < kChunk * 8;
             i += kCompute) {
#pragma unroll
          for (int c = 0; c < QD / 64; ++c)
            *reinterpret_cast<uint4 *>(Ks + c * 16384 + i * 16) =
                make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int c = 0; c < TV / 64; ++c)
            *reinterpret_cast<uint4 *>(Vs + c * 16384 + i * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        }
        tc::fence_async();
        tc::bar_arrive(bar(kClean));
        alive = wait(kClean, 0);
        if (!alive) break;
      }
      const float keep = gt.keep;
      seg_keep *= keep;

      // weighted values of steps 32 qr + 16 half .. + 15, this lane's column
      auto weigh = [&](int qr) {
        const int buf = qr & 1, use = it * 2 + qr / 2;
        if (use > 0 && !wait(kWEmpty0 + buf, use - 1)) return false;
        tc::after_sync();
        if (has_v) {
          const int t0 = qr * 32 + half * 16;
          const unsigned char *col =
              Vs + (r / 64) * 16384 + (r % 8) * 2;
          const int ch = r % 64 / 8;
          uint32_t pl[3][8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int t = t0 + 2 * i;
            const float2 w =
                *reinterpret_cast<const float2 *>(gt.write + t);
            const float v0 = __uint_as_float(
                uint32_t(*reinterpret_cast<const uint16_t *>(
                    col + t * 128 + ((ch ^ ((2 * i) % 8)) * 16)))
                << 16);
            const float v1 = __uint_as_float(
                uint32_t(*reinterpret_cast<const uint16_t *>(
                    col + (t + 1) * 128 + ((ch ^ ((2 * i + 1) % 8)) * 16)))
                << 16);
            uint32_t s3[3];
            la::split2<3>(v0 * w.x, v1 * w.y, s3);
#pragma unroll
            for (int s = 0; s < 3; ++s) pl[s][i] = s3[s];
          }
#pragma unroll
          for (int s = 0; s < 3; ++s)
            tc::tmem_st8(mine + L_::W + buf * 48 + s * 16 + half * 8, pl[s]);
          tc::tmem_wait_st();
        }
        tc::before_sync();
        tc::bar_arrive(bar(kWFull0 + buf));
        return true;
      };
      alive = weigh(0) && weigh(1);
      if (!alive) break;

      float O[STATE_ONLY ? 1 : NO];
      if constexpr (!STATE_ONLY) {
        // ---- P -> P'
        alive = wait(kScores, it);
        if (!alive) break;
        tc::after_sync();
        uint32_t pv[64];
        // step of this row, and of the rows of a 32-block, in time
        const int si = rev ? kChunk - 1 - r : r;
        const int tb = rev ? 3 - q4 : q4;  // this warp's block in time
        const int from = gt.from[r];
        const float chi = gt.hi[r], clo = gt.lo[r];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int jb = rev ? 3 - (2 * half + u) : 2 * half + u;  // in time
          if (jb <= tb)
            tc::tmem_ld32(mine + L_::P + half * 64 + u * 32, pv + 32 * u);
        }
        tc::tmem_wait_ld();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int nb = 2 * half + u;          // block of rows j
          const int jb = rev ? 3 - nb : nb;     // in time
          uint32_t *v = pv + 32 * u;
          if (jb > tb) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0u;
          } else if (jb < tb) {
            const int ref = rev ? nb * 32 : nb * 32 + 31;  // row of r
            float e = 0.0f;
            if (from <= jb * 32 + 31)
              e = ex2((chi - gt.hi[ref]) + (clo - gt.lo[ref])) * job.sp;
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 f =
                  *reinterpret_cast<const float4 *>(gt.near + nb * 32 + i);
              const float d[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
              for (int j = 0; j < 4; ++j)
                v[i + j] =
                    __float_as_uint(__uint_as_float(v[i + j]) * (e * d[j]));
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int j = nb * 32 + i;
              const int sj = rev ? kChunk - 1 - j : j;
              const float d =
                  ex2((chi - gt.hi[j]) + (clo - gt.lo[j])) * job.sp;
              v[i] = (sj <= si && sj >= from)
                         ? __float_as_uint(__uint_as_float(v[i]) * d)
                         : 0u;
            }
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t w[PS][16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            uint32_t pl[PS];
            la::split2<PS>(__uint_as_float(pv[32 * u + 2 * i]),
                           __uint_as_float(pv[32 * u + 2 * i + 1]), pl);
#pragma unroll
            for (int s = 0; s < PS; ++s) w[s][i] = pl[s];
          }
#pragma unroll
          for (int s = 0; s < PS; ++s)
            tc::tmem_st16(mine + L_::P + half * 64 + s * 32 + u * 16, w[s]);
        }
        tc::tmem_wait_st();
        // ---- O1, before its columns take O2
        alive = wait(kRead, it);
        if (!alive) break;
        tc::after_sync();
        const float rd = gt.read[r];
#pragma unroll
        for (int u = 0; u < NO; u += 32) {
          uint32_t t[32];
          tc::tmem_ld32(mine + L_::O + half * NO + u, t);
          tc::tmem_wait_ld();
          // a restart forgets the state whatever it held
#pragma unroll
          for (int i = 0; i < 32; ++i)
            O[u + i] = rd == 0.0f ? 0.0f : __uint_as_float(t[i]) * rd;
        }
        tc::before_sync();
        tc::bar_arrive(bar(kGo));
      }
      alive = weigh(2) && weigh(3);
      if (!alive) break;
      tc::bar_arrive(bar(kGatesFree));

      if constexpr (!STATE_ONLY) {
        // ---- y
        alive = wait(kOut, it);
        if (!alive) break;
        tc::after_sync();
#pragma unroll
        for (int u = 0; u < NO; u += 32) {
          uint32_t t[32];
          tc::tmem_ld32(mine + L_::O + half * NO + u, t);
          tc::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) O[u + i] += __uint_as_float(t[i]);
        }
        tc::before_sync();
        tc::bar_arrive(bar(kOutRead));
        const int64_t t = lo + r;
        if (t < L) {
          const bool live = t < len;
          const int64_t row = (b * L + t) * p.heads + h;
          const int c0 = half * NO;
          if (job.y_f32) {
            float *y = static_cast<float *>(job.y) + row * job.vd + c0;
#pragma unroll
            for (int i = 0; i < NO; i += 4)
              if (c0 + i < job.vd)
                *reinterpret_cast<float4 *>(y + i) =
                    live ? make_float4(O[i], O[i + 1], O[i + 2], O[i + 3])
                         : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          } else {
            bf16 *y = static_cast<bf16 *>(job.y) + row * job.vd + c0;
#pragma unroll
            for (int i = 0; i < NO; i += 8)
              if (c0 + i < job.vd)
                *reinterpret_cast<uint4 *>(y + i) =
                    live ? make_uint4(pack2(O[i], O[i + 1]),
                                      pack2(O[i + 2], O[i + 3]),
                                      pack2(O[i + 4], O[i + 5]),
                                      pack2(O[i + 6], O[i + 7]))
                         : make_uint4(0u, 0u, 0u, 0u);
          }
          if (job.rows) {
            // the row dots the decay's gradient is made of
            float dot = 0.0f;
            if (live) {
              const bf16 *ds =
                  static_cast<const bf16 *>(job.dot) +
                  (b * L + t) * job.dot_stride +
                  int64_t(h / (p.heads / job.dot_heads)) * job.vd + c0;
#pragma unroll
              for (int i = 0; i < NO; i += 8)
                if (c0 + i < job.vd) {
                  const uint4 v = __ldg(reinterpret_cast<const uint4 *>(ds + i));
                  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    dot = fmaf(O[i + 2 * j], la::lo2(w[j]), dot);
                    dot = fmaf(O[i + 2 * j + 1], la::hi2(w[j]), dot);
                  }
                }
            }
            job.rows[((int64_t(half) * p.batch + b) * p.heads + h) * L + t] =
                dot;
          }
        }
      }

      // ---- the state
      alive = wait(kUpdate, it);
      if (!alive) break;
      tc::after_sync();
#pragma unroll
      for (int u = 0; u < NS; u += 32) {
        uint32_t t[32];
        tc::tmem_ld32(mine + L_::U + k0 + u, t);
        tc::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i)
          S[u + i] = keep == 0.0f
                         ? __uint_as_float(t[i])
                         : fmaf(keep, S[u + i], __uint_as_float(t[i]));
      }
      put_state();
    }
    if (alive && r < TV) {
      if constexpr (STATE_ONLY) {
        if (seg_row) {
#pragma unroll
          for (int i = 0; i < NS; ++i)
            seg_state[int64_t(k0 + i) * kLaTile] = S[i];
        }
        if (threadIdx.x == 0) job.seg_decay[bh * p.nseg + seg] = seg_keep;
      } else if (job.last && seg == p.nseg - 1 && r < job.vd) {
        // running backwards, the first token's own decay is still to come
        float f = 1.0f;
        if (rev && len > 0)
          f = ex2_d(la::gate_at<bf16>(p, b, 0, h) * 1.4426950408889634);
        float *dst =
            job.last + bh * job.qd * job.vd + int64_t(r) * job.state_cs;
#pragma unroll
        for (int i = 0; i < NS; ++i)
          if (k0 + i < job.qd)
            dst[int64_t(k0 + i) * job.state_rs] = f == 0.0f ? 0.0f : S[i] * f;
      }
    }
  }
  tc::before_sync();
  __syncthreads();
  tc::after_sync();
  if (warp == 9) tc::tmem_free(tmem, 512);
}

}  // namespace lat
}  // namespace ssm
