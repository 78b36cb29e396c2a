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
// One warpgroup each (a thread has one TMEM lane): 0 turns P into P', 1 weighs
// the values and holds the state, 2 scales O1 in its place (O2 is added to it
// there) and hands y to a TMA store.
// Of the fourth, warp 12 moves q, k, v (two chunks deep) and y, 13 issues the
// products, 14 and 15 sum the decays ahead of their chunks. Everything between them goes
// through mbarriers with bounded waits; the registers are divided by need.
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
constexpr int kThreads = 512;

struct Params {
  CUtensorMap map[3][4];  // [job][q, k, v, y]
  LaParams p;             // seg_len: a multiple of kChunk
  int *status;
};

// The decays of a chunk; arrays by row (token order). Steps are counted in
// the order of time, which in reverse is from the last row.
struct Gates {
  float hi[kChunk], lo[kChunk];  // c since the last restart
  float near[kChunk];            // e^{c_r - c_j}, r: the last step of j's 32
  float read[kChunk];            // si e^{c_i}, 0 behind a restart
  float write[kChunk];           // sw e^{c_C - c_i}, 0 before a restart
  unsigned char from[kChunk];    // the last restart at or before the step
  float keep;
  int dead;
  uint32_t tmem;
  uint64_t bars[26];
};

enum Bar {
  kFull0, kFull1,      // q, k, v of a stage have arrived
  kEmpty0, kEmpty1,    // the stage's products are done
  kScores,             // P
  kRead,               // O1
  kOut,                // O2
  kUpdate,             // U
  kWEmpty0, kWEmpty1,  // a buffer of weighted values has been used
  kGatesA, kGatesB, kGatesC,  // hi, lo, near, from; write, keep; read
  kStored,             // y has been read by its store
  kSingle,             // (barriers above: one arrival; below: a warpgroup's)
  kWFull0 = kSingle, kWFull1,
  kScored,             // P'
  kReadDone,           // O1 read
  kOutRead,            // O2 read
  kState,              // S stored, U read
  kFreeA, kFreeB, kFreeC,
  kStaged,             // y in shared memory
  kClean,              // rows behind the sequence's end zeroed
  kFin,                // (one arrival)
};

template <int QD, int TV, int PS, bool STATE_ONLY>
struct Lay {
  static constexpr int Q = kChunk * QD * 2, V = kChunk * TV * 2;
  static constexpr int STAGE = (STATE_ONLY ? Q : 2 * Q) + V;  // k, v(, q)
  static constexpr int S = 2 * STAGE;
  // y: in the place of the chunk's q where there is no room of its own
  static constexpr bool OVER_Q = QD == 128 && TV == 128;
  static constexpr int Y = S + (STATE_ONLY ? 0 : PS * TV * QD * 2);
  static constexpr int GATES = Y + (STATE_ONLY || OVER_Q ? 0 : V);
  static constexpr int BYTES = GATES + int(sizeof(Gates));
  // TMEM columns
  static constexpr uint32_t P = 0, O = 128, U = 256, W = 384;
};

// A 16-byte group of a 128-byte row in the 128-byte swizzle.
__device__ __forceinline__ int swizzled(int row, int group) {
  return row * 128 + ((group ^ (row % 8)) * 16);
}

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

  unsigned x = blockIdx.x;
  const int h = int(x % unsigned(p.heads));
  x /= unsigned(p.heads);
  const int64_t b = x % unsigned(p.batch);
  const int seg = int(x / unsigned(p.batch));
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t L = p.seqlen;
  int64_t len = L;
  if (p.lengths) {
    const int64_t n = p.lengths[b];
    len = n < 0 ? 0 : n > L ? L : n;
  }
  const bool rev = job.reverse;
  const int chunks = int(p.seg_len / kChunk);
  // live chunks of this segment, in the order of time: `n_live` of them from
  // the one whose first token is `low0`; the rest lie behind the sequence's
  // end (`idle_low`: the first token of all of these)
  const int64_t seg_low = rev ? (p.nseg - 1 - seg) * p.seg_len
                              : seg * p.seg_len;
  int64_t n_left = (len - seg_low + kChunk - 1) / kChunk;
  n_left = n_left < 0 ? 0 : n_left < chunks ? n_left : chunks;
  const int n_live = int(n_left);
  const int64_t idle_low = seg_low + int64_t(n_live) * kChunk;
  const int low0 = int(rev ? idle_low - kChunk : seg_low);
  auto low = [&](int it) { return rev ? low0 - it * kChunk : low0 + it * kChunk; };
  // the chunk in which the sequence ends before its rows do, or -1
  const int ragged =
      len < L && len % kChunk != 0 && n_live > 0
          ? (len / kChunk * kChunk == low(rev ? 0 : n_live - 1)
                 ? (rev ? 0 : n_live - 1)
                 : -1)
          : -1;

  auto in_gates = [&](const void *q) {
    return base + uint32_t(L_::GATES) +
           uint32_t(static_cast<const char *>(q) -
                    reinterpret_cast<const char *>(&gt));
  };
  auto bar = [&](int i) { return in_gates(&gt.bars[i]); };
  volatile int *dead = &gt.dead;
  auto wait = [&](int i, int use) {
    return tc::bar_wait(bar(i), uint32_t(use) & 1u, dead, pp.status);
  };
  if (warp == 13) tc::tmem_alloc(in_gates(&gt.tmem), 512);
  if (threadIdx.x == 0) {
    gt.dead = 0;
    for (int i = 0; i <= kFin; ++i)
      tc::bar_init(bar(i), i >= kSingle && i < kFin ? 128 : 1);
    tc::fence_init();
  }
  tc::before_sync();
  __syncthreads();
  tc::after_sync();
  const uint32_t tmem = gt.tmem;
  const int64_t bh = b * p.heads + h;
  const int r = threadIdx.x % 128;  // a warpgroup's thread: its TMEM lane
  const uint32_t mine = tmem + (uint32_t(r / 32 * 32) << 16);

  if (warp >= 12) {
    if (warp == 12) {
      // ---- q, k, v in (stage it % 2), y out
      const int kh = h / (p.heads / job.k_heads);
      const int qh = h / (p.heads / job.q_heads);
      const int vh = h / (p.heads / job.v_heads);
      auto load = [&](int it) {
        if (lane == 0) {
          const int st = it & 1, tok = low(it);
          const uint32_t s = base + st * L_::STAGE, f = bar(kFull0 + st);
          tc::bar_expect(f, L_::STAGE);
          for (int c = 0; c < QD / 64; ++c) {
            tc::load_box(s + c * 16384, &maps[1], f, c * 64, kh, tok, int(b));
            if (!STATE_ONLY)
              tc::load_box(s + L_::Q + L_::V + c * 16384, &maps[0], f, c * 64,
                           qh, tok, int(b));
          }
          for (int c = 0; c < TV / 64; ++c)
            tc::load_box(s + L_::Q + c * 16384, &maps[2], f, c * 64, vh, tok,
                         int(b));
        }
        __syncwarp();
      };
      int loaded = 0;
#pragma unroll 1
      for (; loaded < n_live && loaded < 2; ++loaded) load(loaded);
#pragma unroll 1
      for (int it = 0; it < n_live; ++it) {
        const int st = it & 1;
        if (!STATE_ONLY && !job.y_f32) {
          if (!wait(kStaged, it)) break;
          if (lane == 0) {
            const uint32_t y =
                base + (L_::OVER_Q ? st * L_::STAGE + L_::Q + L_::V : L_::Y);
#pragma unroll
            for (int c = 0; c < TV / 64; ++c)
              if (c * 64 < job.vd)
              tc::store_box(&maps[3], y + c * 16384, c * 64, h,
                            low(it), int(b));
            tc::store_read();
            tc::bar_arrive(bar(kStored));
          }
          __syncwarp();
        }
        if (it + 2 < n_live) {
          if (!wait(kEmpty0 + st, it / 2)) break;
          load(it + 2);
          ++loaded;
        }
      }
      if (*dead)  // nothing may still be on its way into this block's memory
#pragma unroll 1
        for (int it = loaded > 2 ? loaded - 2 : 0; it < loaded; ++it)
#pragma unroll 1
          for (int i = 0; i < 1 << 16; ++i)
            if (tc::bar_try(bar(kFull0 + (it & 1)), uint32_t(it / 2) & 1u))
              break;
    } else if (warp == 13) {
      // ---- products, issued by one thread
      if (lane == 0) {
        constexpr uint32_t kScoreShape = tc::shape(128, false);
        constexpr uint32_t kReadShape = tc::shape(TV, false);
        constexpr uint32_t kUpdateShape = tc::shape(QD, true);
        constexpr uint32_t kOutShape = tc::shape(TV, true);
        // an operand's description for each step of 16 is the first one's
        // plus the bytes between them (in units of 16)
        const uint64_t stage0 = tc::operand(base, 16384);
        const uint64_t state0 = tc::operand(base + L_::S, 0);
        constexpr uint64_t kStage = L_::STAGE / 16, kV = L_::Q / 16,
                           kQ = (L_::Q + L_::V) / 16;
        auto one = [&](int i, int use) {
          return tc::bar_wait_one(bar(i), uint32_t(use) & 1u, dead, pp.status);
        };
        // K-major: 64 steps to a 128-byte row, then `far` on
        auto along = [](int ks, int far) {
          return uint64_t((ks >> 2) * far + (ks & 3) * 2);
        };
        auto scores = [&](int it) {
          const int st = it & 1;
          const uint64_t K = stage0 + st * kStage, Q = K + kQ;
          if (!one(kFull0 + st, it / 2)) return false;
          if (it == ragged && !one(kClean, 0)) return false;
          tc::after_sync();
          if (!STATE_ONLY) {
#pragma unroll
            for (int ks = 0; ks < QD / 16; ++ks)
              tc::mma_ss(tmem + L_::P, Q + along(ks, 1024),
                         K + along(ks, 1024), kScoreShape, ks > 0);
            tc::commit(bar(kScores));
          }
          return true;
        };
        bool alive = n_live > 0 && scores(0);
#pragma unroll 1
        for (int it = 0; it < n_live && alive; ++it) {
          const int st = it & 1;
          const uint64_t K = stage0 + st * kStage, V = K + kV, Q = K + kQ;
          alive = one(kState, it);
          // the state's update first: the next chunk waits for it; what reads
          // the state, and the scores' product, fill in behind
#pragma unroll 1
          for (int qr = 0; qr < 4 && alive; ++qr) {
            const int buf = qr & 1;
            alive = one(kWFull0 + buf, it * 2 + qr / 2);
            if (!alive) break;
            tc::after_sync();
            // planes from the smallest to the leading one, two steps of 16
            const uint32_t w = tmem + L_::W + buf * 48;
            const uint64_t k0 = K + uint64_t(qr * 256);
#pragma unroll
            for (int s = 2; s >= 0; --s) {
              tc::mma_ts(tmem + L_::U, w + s * 16, k0, kUpdateShape,
                         qr > 0 || s < 2);
              tc::mma_ts(tmem + L_::U, w + s * 16 + 8, k0 + 128, kUpdateShape,
                         true);
            }
            tc::commit(bar(kWEmpty0 + buf));
            if (qr == 3) tc::commit(bar(kUpdate));
            if constexpr (!STATE_ONLY) {
              if (qr == 0) {
                alive = it == 0 || one(kOutRead, it - 1);
                if (!alive) break;
                tc::after_sync();
#pragma unroll
                for (int i = 0; i < PS * QD / 16; ++i) {
                  const int s = PS - 1 - i / (QD / 16), ks = i % (QD / 16);
                  tc::mma_ss(tmem + L_::O, Q + along(ks, 1024),
                             state0 + uint64_t(s * TV * QD / 8) +
                                 along(ks, TV * 8),
                             kReadShape, i > 0);
                }
                tc::commit(bar(kRead));
              }
            }
          }
          if (!alive) break;
          if constexpr (!STATE_ONLY) {
            // O2 is added to the scaled O1
            alive = one(kScored, it) && one(kReadDone, it);
            if (!alive) break;
            tc::after_sync();
#pragma unroll
            for (int i = 0; i < PS * 8; ++i) {
              const int s = PS - 1 - i / 8, ks = i % 8;
              tc::mma_ts(tmem + L_::O,
                         tmem + L_::P + (ks / 2) * 32 + s * 16 + (ks % 2) * 8,
                         V + uint64_t(ks * 128), kOutShape, true);
            }
            tc::commit(bar(kOut));
          }
          tc::commit(bar(kEmpty0 + st));
          if (it + 1 < n_live) alive = scores(it + 1);
        }
      }
      __syncwarp();
      // every product is done before the block goes
      if (lane == 0) tc::commit(bar(kFin));
      __syncwarp();
#pragma unroll 1
      for (int i = 0; i < 1 << 16; ++i)
        if (tc::bar_try(bar(kFin), 0)) break;
    } else {
      // ---- decays: every second chunk each, four steps a lane in the order
      // of time; the next values are on their way while these are summed
      const bf16 *gate = static_cast<const bf16 *>(p.log_decay);
      const double head = p.head_log_decay ? p.head_log_decay[h] : 0.0;
      unsigned short raw[4];
      auto fetch = [&](int it) {
        const int lo = low(it);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int s = 4 * lane + j;
          const int64_t t = rev ? lo + kChunk - s : lo + s;
          raw[j] = 0;
          if (gate && t < len)
            raw[j] = __ldg(reinterpret_cast<const unsigned short *>(gate) +
                           (b * L + t) * p.heads + h);
        }
      };
      // The last chunk's values have been written (by the other warp) and
      // used. Without the first wait the second could run a phase ahead of
      // its barrier and pass on the parity of an old one.
      auto turn = [&](int written, int used, int it) {
        return it == 0 || (wait(written, it - 1) && wait(used, it - 1));
      };
      if (warp - 14 < n_live) fetch(warp - 14);
#pragma unroll 1
      for (int it = warp - 14; it < n_live; it += 2) {
        double c[4], sum = 0.0;
        int from[4], lastr = -1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int lo = low(it);
          const int s = 4 * lane + j;
          const int64_t t = rev ? lo + kChunk - s : lo + s;
          const double g =
              t < len ? (double(__uint_as_float(uint32_t(raw[j]) << 16)) +
                         head) *
                            1.4426950408889634
                      : 0.0;
          if (g < -126.0) {
            sum = 0.0;
            lastr = s;
          } else {
            sum += g;
          }
          c[j] = sum;
          from[j] = lastr;
        }
        if (it + 2 < n_live) fetch(it + 2);
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
        float hi[4], lo4[4], near[4], read[4], write[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int s = 4 * lane + j;
          if (from[j] < 0) {
            c[j] += es;
            from[j] = er;
          }
          hi[j] = float(c[j]);
          lo4[j] = float(c[j] - double(hi[j]));
          near[j] = s >= blk_r ? ex2_d(blk - c[j]) : 0.0f;
          read[j] = from[j] < 0 ? ex2_d(c[j]) * job.si : 0.0f;
          write[j] = s >= end_r ? ex2_d(end - c[j]) * job.sw : 0.0f;
          from[j] = from[j] < 0 ? 0 : from[j];
        }
        const float keep = end_r < 0 ? ex2_d(end) : 0.0f;
        // in reverse, a lane's four steps are its four rows backwards
        const int row = rev ? kChunk - 4 - 4 * lane : 4 * lane;
        auto put = [&](float *dst, const float (&v)[4]) {
          *reinterpret_cast<float4 *>(dst + row) =
              rev ? make_float4(v[3], v[2], v[1], v[0])
                  : make_float4(v[0], v[1], v[2], v[3]);
        };
        if (!STATE_ONLY) {
          if (!turn(kGatesA, kFreeA, it)) break;
          put(gt.hi, hi);
          put(gt.lo, lo4);
          put(gt.near, near);
          *reinterpret_cast<uchar4 *>(gt.from + row) =
              rev ? make_uchar4(from[3], from[2], from[1], from[0])
                  : make_uchar4(from[0], from[1], from[2], from[3]);
          __syncwarp();
          if (lane == 0) tc::bar_arrive(bar(kGatesA));
          if (!turn(kGatesC, kFreeC, it)) break;
          put(gt.read, read);
          __syncwarp();
          if (lane == 0) tc::bar_arrive(bar(kGatesC));
        }
        if (!turn(kGatesB, kFreeB, it)) break;
        put(gt.write, write);
        if (lane == 0) gt.keep = keep;
        __syncwarp();
        if (lane == 0) tc::bar_arrive(bar(kGatesB));
      }
    }
  } else if (warp < 4) {
    // ---- scores: P -> P'
    tc::fewer_registers<88>();
    // the step of this row in time, and its warp's block of 32
    const int step = rev ? kChunk - 1 - r : r;
    const int tb = rev ? 3 - warp : warp;
#pragma unroll 1
    for (int it = 0; !STATE_ONLY && it < n_live; ++it) {
      if (!wait(kGatesA, it) || !wait(kScores, it)) break;
      tc::after_sync();
      const int from = gt.from[r];
      const float chi = gt.hi[r], clo = gt.lo[r];
#pragma unroll 1
      for (int nb = 0; nb < 4; ++nb) {     // blocks of 32 rows j
        const int jb = rev ? 3 - nb : nb;  // in time
        uint32_t v[32], late[PS == 2 ? 16 : 1];
        if (jb > tb) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0u;
        } else {
          tc::tmem_ld32(mine + L_::P + nb * 32, v);
          tc::tmem_wait_ld();
          if (jb < tb) {
            const int ref = rev ? nb * 32 : nb * 32 + 31;  // row of step r
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
            // rows of steps in [from, step] of this block, as bits
            const int lo_s = max(from - jb * 32, 0), hi_s = step - jb * 32;
            uint32_t keep_bits = (0xffffffffu >> (31 - hi_s)) &
                                 (0xffffffffu << lo_s);
            if (rev) keep_bits = __brev(keep_bits);
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 fh =
                  *reinterpret_cast<const float4 *>(gt.hi + nb * 32 + i);
              const float4 fl =
                  *reinterpret_cast<const float4 *>(gt.lo + nb * 32 + i);
              const float dh[4] = {fh.x, fh.y, fh.z, fh.w};
              const float dl[4] = {fl.x, fl.y, fl.z, fl.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float d = ex2((chi - dh[j]) + (clo - dl[j])) * job.sp;
                v[i + j] =
                    keep_bits >> (i + j) & 1u
                        ? __float_as_uint(__uint_as_float(v[i + j]) * d)
                        : 0u;
              }
            }
          }
        }
        // P' takes the place of its block of P: 16 columns a plane
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          uint32_t pl[PS];
          la::split2<PS>(__uint_as_float(v[2 * i]),
                         __uint_as_float(v[2 * i + 1]), pl);
          v[i] = pl[0];
          if constexpr (PS == 2) late[i] = pl[1];
        }
        tc::tmem_st16(mine + L_::P + nb * 32, v);
        if constexpr (PS == 2) tc::tmem_st16(mine + L_::P + nb * 32 + 16, late);
      }
      tc::tmem_wait_st();
      tc::bar_arrive(bar(kFreeA));
      tc::before_sync();
      tc::bar_arrive(bar(kScored));
    }
  } else if (warp < 8) {
    // ---- the weighted values and the state; lane: a value column
    tc::more_registers<208>();
    const bool has_v = r / 32 * 32 < TV;
    constexpr int64_t SF = int64_t(QD) * kLaTile;
    const int tiles = (job.vd + kLaTile - 1) / kLaTile;
    // element (key, value r) of a segment's state
    float *seg_state =
        p.nseg > 1 && r / kLaTile < tiles
            ? job.seg_state +
                  ((bh * p.nseg + seg) * tiles + r / kLaTile) * SF +
                  r % kLaTile
            : nullptr;
    float S[QD];
#pragma unroll
    for (int i = 0; i < QD; ++i) S[i] = 0.0f;
    if (!STATE_ONLY && r < TV) {
      if (p.nseg > 1) {
        if (seg_state) {
#pragma unroll
          for (int i = 0; i < QD; ++i) S[i] = seg_state[i * kLaTile];
        }
      } else if (job.init && r < job.vd) {
        const float *src =
            job.init + bh * job.qd * job.vd + int64_t(r) * job.state_cs;
#pragma unroll
        for (int i = 0; i < QD; ++i)
          if (i < job.qd) S[i] = src[int64_t(i) * job.state_rs];
      }
    }
    // the bfloat16 planes of the state
    auto put_state = [&]() {
      if constexpr (!STATE_ONLY) {
        if (r < TV) {
#pragma unroll
          for (int i = 0; i < QD; i += 8) {
            uint32_t w[4][PS];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              la::split2<PS>(S[i + 2 * j], S[i + 2 * j + 1], w[j]);
            unsigned char *dst = smem + L_::S + (i / 64) * TV * 128 +
                                 swizzled(r, i % 64 / 8);
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
    float keep = 0.0f, next_keep = 0.0f, seg_keep = 1.0f;
    // a chunk's values are there, zeros behind the sequence's end
    auto begin = [&](int it) {
      const int st = it & 1;
      if (!wait(kFull0 + st, it / 2) || !wait(kGatesB, it)) return false;
      if (it == ragged) {
        // whatever was loaded
        unsigned char *Ks = smem + st * L_::STAGE, *Vs = Ks + L_::Q;
        const int dead_from = int(len - low(it));
#pragma unroll 1
        for (int i = r + dead_from * 8; i < kChunk * 8; i += 128) {
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
        if (!wait(kClean, 0)) return false;
      }
      next_keep = gt.keep;
      return true;
    };
    // weighted values of 32 steps, this lane's column
    auto weigh = [&](int it, int qr) {
      const int buf = qr & 1, use = it * 2 + qr / 2;
      if (use > 0 && !wait(kWEmpty0 + buf, use - 1)) return false;
      tc::after_sync();
      if (has_v) {
        const unsigned char *col = smem + (it & 1) * L_::STAGE + L_::Q +
                                   (r / 64) * 16384 + qr * 4096 + (r % 8) * 2;
        const float *wt = gt.write + qr * 32;
        const int group = r % 64 / 8;
        uint32_t pl[3][16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 w = *reinterpret_cast<const float2 *>(wt + 2 * i);
          const float v0 = __uint_as_float(
              uint32_t(*reinterpret_cast<const uint16_t *>(
                  col + 2 * i * 128 + ((group ^ ((2 * i) % 8)) * 16)))
              << 16);
          const float v1 = __uint_as_float(
              uint32_t(*reinterpret_cast<const uint16_t *>(
                  col + (2 * i + 1) * 128 +
                  ((group ^ ((2 * i + 1) % 8)) * 16)))
              << 16);
          uint32_t s3[3];
          la::split2<3>(v0 * w.x, v1 * w.y, s3);
#pragma unroll
          for (int s = 0; s < 3; ++s) pl[s][i] = s3[s];
        }
#pragma unroll
        for (int s = 0; s < 3; ++s)
          tc::tmem_st16(mine + L_::W + buf * 48 + s * 16, pl[s]);
        tc::tmem_wait_st();
      }
      tc::before_sync();
      tc::bar_arrive(bar(kWFull0 + buf));
      return true;
    };
    put_state();
    // The first quarter of a chunk's values is weighed before the last
    // chunk's update is waited for: there is a buffer free for it, and the
    // products of the last quarter are still under way.
    bool alive = n_live == 0 || begin(0);
#pragma unroll 1
    for (int i = 0; i < 4 * n_live && alive; ++i) {
      const int it = i / 4;
      alive = weigh(it, i % 4);
      if (!alive) break;
      if (i % 4 == 0) {
        if (it == 0) {
          keep = next_keep;
          seg_keep *= keep;
          continue;
        }
      } else if (i % 4 < 3) {
        continue;
      } else {
        tc::bar_arrive(bar(kFreeB));
        if (it + 1 < n_live) {
          alive = begin(it + 1);
          continue;
        }
      }
      // here after the first quarter of every chunk but the first, and at the
      // very end: the update of the chunk before
      const int done = i % 4 == 0 ? it - 1 : it;
      alive = wait(kUpdate, done);
      if (!alive) break;
      tc::after_sync();
      if (keep == 0.0f) {  // a restart forgets the state whatever it held
#pragma unroll
        for (int i = 0; i < QD; ++i) S[i] = 0.0f;
      }
#pragma unroll
      for (int u = 0; u < QD; u += 32) {
        uint32_t t[32];
        tc::tmem_ld32(mine + L_::U + u, t);
        tc::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i)
          S[u + i] = fmaf(keep, S[u + i], __uint_as_float(t[i]));
      }
      put_state();
      keep = next_keep;
      if (done + 1 < n_live) seg_keep *= keep;
    }
    if (alive && r < TV) {
      if constexpr (STATE_ONLY) {
        if (seg_state) {
#pragma unroll
          for (int i = 0; i < QD; ++i) seg_state[i * kLaTile] = S[i];
        }
        if (r == 0) job.seg_decay[bh * p.nseg + seg] = seg_keep;
      } else if (job.last && seg == p.nseg - 1 && r < job.vd) {
        // running backwards, the first token's own decay is still to come
        float f = 1.0f;
        if (rev && len > 0)
          f = ex2_d(la::gate_at<bf16>(p, b, 0, h) * 1.4426950408889634);
        float *dst =
            job.last + bh * job.qd * job.vd + int64_t(r) * job.state_cs;
#pragma unroll
        for (int i = 0; i < QD; ++i)
          if (i < job.qd)
            dst[int64_t(i) * job.state_rs] = f == 0.0f ? 0.0f : S[i] * f;
      }
    }
  } else {
    // ---- y; lane: a step
    tc::fewer_registers<88>();
    if constexpr (!STATE_ONLY) {
      // rows of y behind the sequence's last live chunk
#pragma unroll 1
      for (int64_t t = idle_low + r; t < seg_low + p.seg_len && t < L;
           t += 128) {
        const int64_t at = ((b * L + t) * p.heads + h) * job.vd;
        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
        for (int i = 0; i < job.vd; i += 8) {  // 8 elements: 16 or 32 bytes
          if (job.y_f32) {
            uint4 *y =
                reinterpret_cast<uint4 *>(static_cast<float *>(job.y) + at + i);
            y[0] = z;
            y[1] = z;
          } else {
            *reinterpret_cast<uint4 *>(static_cast<bf16 *>(job.y) + at + i) = z;
          }
        }
      }
#pragma unroll 1
      for (int it = 0; it < n_live; ++it) {
        const int st = it & 1;
        // O1, scaled in its place: O2 is added to it there
        if (!wait(kGatesC, it) || !wait(kRead, it)) break;
        tc::after_sync();
        const float rd = gt.read[r];
#pragma unroll 1
        for (int u = 0; u < TV; u += 32) {
          uint32_t v[32];
          tc::tmem_ld32(mine + L_::O + u, v);
          tc::tmem_wait_ld();
          // a restart forgets the state whatever it held
#pragma unroll
          for (int i = 0; i < 32; ++i)
            v[i] = rd == 0.0f ? 0u
                              : __float_as_uint(__uint_as_float(v[i]) * rd);
          tc::tmem_st16(mine + L_::O + u, v);
          tc::tmem_st16(mine + L_::O + u + 16, v + 16);
        }
        tc::tmem_wait_st();
        tc::bar_arrive(bar(kFreeC));
        tc::before_sync();
        tc::bar_arrive(bar(kReadDone));
        const int64_t t = low(it) + r;
        const bool live = t < len;
        const bool staged = !job.y_f32;
        if (staged && !L_::OVER_Q && it > 0 && !wait(kStored, it - 1)) break;
        if (!wait(kOut, it)) break;
        tc::after_sync();
        unsigned char *ys =
            smem + (L_::OVER_Q ? st * L_::STAGE + L_::Q + L_::V : L_::Y);
        const int64_t row = (b * L + t) * p.heads + h;
        const bf16 *ds =
            job.rows ? static_cast<const bf16 *>(job.dot) +
                           (b * L + t) * job.dot_stride +
                           int64_t(h / (p.heads / job.dot_heads)) * job.vd
                     : nullptr;
        float dot = 0.0f;
#pragma unroll 1
        for (int u = 0; u < TV; u += 32) {
          uint32_t v[32];
          tc::tmem_ld32(mine + L_::O + u, v);
          tc::tmem_wait_ld();
          if (!live) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0u;
          }
          if (staged) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                w[j] = pack2(__uint_as_float(v[i + 2 * j]),
                             __uint_as_float(v[i + 2 * j + 1]));
              *reinterpret_cast<uint4 *>(
                  ys + (u / 64) * 16384 +
                  swizzled(r, u % 64 / 8 + i / 8)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else if (t < L) {
            float *y = static_cast<float *>(job.y) + row * job.vd + u;
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              if (u + i < job.vd)
                *reinterpret_cast<uint4 *>(y + i) =
                    make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          }
          if (ds && live) {
            // the row dots the decay's gradient is made of
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              if (u + i < job.vd) {
                const uint4 q =
                    __ldg(reinterpret_cast<const uint4 *>(ds + u + i));
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  dot = fmaf(__uint_as_float(v[i + 2 * j]), la::lo2(w[j]),
                             dot);
                  dot = fmaf(__uint_as_float(v[i + 2 * j + 1]),
                             la::hi2(w[j]), dot);
                }
              }
          }
        }
        tc::before_sync();
        tc::bar_arrive(bar(kOutRead));
        if (staged) {
          tc::fence_async();
          tc::bar_arrive(bar(kStaged));
        }
        if (job.rows && t < L) job.rows[(b * p.heads + h) * L + t] = dot;
      }
    }
  }
  tc::before_sync();
  __syncthreads();
  tc::after_sync();
  if (warp == 13) tc::tmem_free(tmem, 512);
}

}  // namespace lat
}  // namespace ssm
