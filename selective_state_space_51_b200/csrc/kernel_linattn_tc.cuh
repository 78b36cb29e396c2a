// Linear attention with a decay for each head on the fifth-generation tensor
// cores: the pass of kernel_linattn.cuh (same mathematics, same jobs), for
// bfloat16 rows on 16-byte boundaries, key and value sizes up to 128, in
// chunks of 128 steps, one block for a whole head.
//
// Four products a chunk, each D[128][n] in TMEM:
//   P  [step i][step j]  = Q K^T            both from shared memory
//   O1 [step i][value]   = Q S              S: a bfloat16 copy in shared memory
//   U^T[value][key]      = (w V)^T K        (w V)^T from TMEM
//   O2 [step i][value]   = P' V             P' (decayed scores) from TMEM
//   y = read_i O1 + O2,  S^T <- keep S^T + U^T (float32, registers)
// The weighted values need three bfloat16 planes for a float32 state; as the A
// operand in TMEM they cost no shared memory and no bank traffic, and the
// state's transpose lies in the same lanes (one value column a lane) as the
// product that is added to it. The decayed scores and the copy of the state have
// two planes each, beside which only the result's own rounding is seen.
//
// Three warpgroups (a thread has one TMEM lane) share the chunk's 128 weighted
// steps, which all need the same arithmetic, and have a task of their own
// each: the first turns P into P', the second holds the state, the third
// scales O1 in its place (O2 is added to it there) and hands y to a TMA store.
// The weighted values pass through three buffers of 32, 32 and 16 steps: the
// first and the third group have theirs ready while the last chunk's state is
// still being added up, the second follows once it is. Of the fourth
// warpgroup, warp 12 moves q, k, v (two chunks deep, but for the q of 128-wide
// keys and values) and y, 13 issues the products, 14 and 15 sum the decays ahead
// of their chunks. Everything between them goes through mbarriers with bounded
// waits; the registers are divided by need.
//
// A wait by parity has to come within one phase of its barrier: every wait
// here is for a phase that cannot be followed by the next before it returns.
// Whichever role gives a wait up says so itself (`dead`): the last chunk's are
// waited for by nobody else.
//
// The decay e^{c_i - c_j}: outside the 32 x 32 blocks on the diagonal it is
// e^{c_i - c_r} e^{c_r - c_j}, r the last step of j's block: both factors are
// at most 1 for decays (no overflow), so a block costs one exponential a row
// and two products an element. On the diagonal it is formed directly.
//
// 148 heads x 8192 steps of (128, 128): 365 us, 3.4 TB/s (0.52 of the copy
// rate); bound by a chunk's chain (state, its copy, products, weighted values,
// update: 5.7 us), with 45% of the issue slots and 43% of the tensor pipe busy.
// With one plane, loops unrolled past the instruction cache took 370 us and
// short ones 288; eight warps doing all of it in turn, 160 heads, 1.1 ms.
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

enum Bar {
  kFull0, kFull1,      // k, v (ONE_Q: v) of a stage have arrived
  kFullQ0, kFullQ1,    // its q (ONE_Q: the first of them alone)
  kFullK0, kFullK1,    // ONE_Q: its k
  kEmpty0, kEmpty1,    // the stage's products are done
  kScores,             // P
  kRead,               // O1
  kOut,                // O2
  kUpdate,             // U
  kUsed,               // (3) slots 0, 1, 2 of weighted values have been used
  kGates = kUsed + 3,  // hi, lo, near, from
  kWeights0, kWeights1,  // write, keep of every second chunk
  kStored,             // y has been read by its store
  // the barriers above take one arrival, these a warpgroup's ...
  kWeighed,            // (5) a slot of weighted values is there
  kScored = kWeighed + 5,  // P'
  kReadDone,           // O1 scaled
  kOutRead,            // O2 read
  kState,              // S stored, U read
  kStaged,             // y in shared memory
  kClean,              // rows behind the sequence's end zeroed
  kGatesFree,          // ... two warpgroups' ...
  kWeightsFree0, kWeightsFree1,  // ... and three
  kFin,                // one
  kBars
};

// The decays of a chunk; arrays by row (token order). Steps are counted in
// the order of time, which in reverse is from the last row.
constexpr int kNoRestart = 255;
struct Gates {
  float hi[kChunk];              // c since the last restart: hi + lo
  float near[kChunk];            // e^{c_r - c_j}, r: the last step of j's 32
  float write[2][kChunk];        // sw e^{c_C - c_i}, 0 before a restart
  unsigned short lo[kChunk];     // (bfloat16)
  unsigned char from[kChunk];    // the last restart at or before the step
  float2 keep[2];                // of e^{c_C} (la::keep_of), 0 with a restart
  double end[2];                 // c_C, -infinity with a restart
  int staged, dotted;            // what becomes of y (see the third group)
  int dead;
  uint32_t tmem;
  uint64_t bars[kBars];
};

// The slots a chunk's weighted values come in: the first step, 8-step groups,
// the buffer. Slot 0 is the first warpgroup's, 1 the third's (which both fill
// them ahead), the others the second's.
__host__ __device__ constexpr int slot_step(int s) {
  return s < 3 ? s * 32 : s == 3 ? 80 : 112;
}
__host__ __device__ constexpr int slot_groups(int s) {
  return s == 2 || s == 4 ? 2 : 4;
}
__host__ __device__ constexpr int slot_buffer(int s) {
  return s < 3 ? s : s == 3 ? 0 : 2;
}

// Planes of the decayed scores and of the state that is read. One of each adds
// a rounding as large as the result's own (prompts: 2.34e-3 off, where the last
// rounding alone makes 1.66e-3); with two the rest is not seen beside it. They
// cost 148 heads x 8192 steps of (128, 128) 281 -> 365 us: the state's second
// copy is on the chunk's chain, and there is more code than the instruction
// cache holds (4 times the misses).
constexpr int PS = 2;

template <int QD, int TV, bool STATE_ONLY>
struct Lay {
  static constexpr int Q = kChunk * QD * 2, V = kChunk * TV * 2;
  // Two stages of q, k, v and two planes of the state are more than there is
  // where both sizes are 128: one q then, which is loaded once its forerunner
  // has been multiplied with the state, and y in the place of the chunk's k.
  static constexpr bool ONE_Q = QD == 128 && TV == 128 && !STATE_ONLY;
  static constexpr int STAGE = (STATE_ONLY || ONE_Q ? Q : 2 * Q) + V;
  static constexpr int Q0 = ONE_Q ? 2 * STAGE : Q + V;  // (of a stage: k, v, q)
  static constexpr int S = 2 * STAGE + (ONE_Q ? Q : 0);
  static constexpr int Y = S + (STATE_ONLY ? 0 : PS * TV * QD * 2);
  static constexpr int GATES = Y + (STATE_ONLY || ONE_Q ? 0 : V);
  static constexpr int BYTES = GATES + int(sizeof(Gates));
  // TMEM columns
  static constexpr uint32_t P = 0, O = 128, U = 256, W = 384;
};

// Two planes of a pair of floats, the first cut off (exact to subtract, and no
// conversion), the second rounded: 2^-16 of the value at most is lost.
__device__ __forceinline__ void planes(float2 x, uint32_t (&p)[PS]) {
  static_assert(PS == 2, "");
  const uint32_t a = __float_as_uint(x.x), b = __float_as_uint(x.y);
  p[0] = __byte_perm(a, b, 0x7632);
  const float2 r = fma2(make_float2(__uint_as_float(a & 0xffff0000u),
                                    __uint_as_float(b & 0xffff0000u)),
                        make_float2(-1.0f, -1.0f), x);
  p[1] = la::pack2(r.x, r.y);
}

// A 16-byte group of a 128-byte row in the 128-byte swizzle.
__device__ __forceinline__ int swizzled(int row, int group) {
  return row * 128 + ((group ^ (row % 8)) * 16);
}

template <int QD, int TV, bool STATE_ONLY>
__global__ void __launch_bounds__(kThreads, 1)
    linattn_tc_kernel(const __grid_constant__ Params pp) {
  using L_ = Lay<QD, TV, STATE_ONLY>;
  constexpr bool ONE_Q = L_::ONE_Q;
  using la::bf16;
  using la::pack2;
  extern __shared__ __align__(1024) unsigned char smem[];
  Gates &gt = *reinterpret_cast<Gates *>(smem + L_::GATES);
  const uint32_t base = tc::smem_addr(smem);
  const LaParams &p = pp.p;
  const LaJob &job = p.job[blockIdx.y];
  const CUtensorMap *maps = pp.map[blockIdx.y];

  const unsigned local = blockIdx.x % unsigned(p.bhs);
  const int seg = int(blockIdx.x / unsigned(p.bhs));
  const int h = int((p.bh0 + local) % unsigned(p.heads));
  const int64_t b = (p.bh0 + local) / unsigned(p.heads);
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
  auto low = [&](int it) {
    return rev ? low0 - it * kChunk : low0 + it * kChunk;
  };
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
  auto wait = [&](int i, int use) {
    return tc::bar_wait(bar(i), uint32_t(use) & 1u);
  };
  if (warp == 13) tc::tmem_alloc(in_gates(&gt.tmem), 512);
  if (threadIdx.x == 0) {
    gt.dead = 0;
    gt.staged = !job.y_f32;
    gt.dotted = job.rows != nullptr;
#pragma unroll 1
    for (int i = 0; i < kBars; ++i)
      tc::bar_init(bar(i), i < kWeighed || i == kFin ? 1
                           : i < kGatesFree          ? 128
                           : i == kGatesFree         ? 256
                                                     : 384);
    tc::fence_init();
  }
  tc::before_sync();
  __syncthreads();
  tc::after_sync();
  // all of TMEM is this block's: it starts at column 0
  constexpr uint32_t tmem = 0;
  const bool fit = gt.tmem == tmem;
  const int64_t bh = b * p.heads + h;
  const int r = threadIdx.x % 128;  // a warpgroup's thread: its TMEM lane
  const uint32_t mine = tmem + (uint32_t(r / 32 * 32) << 16);

  // The weighted values of one slot, this lane's value column, as three
  // planes in the slot's buffer.
  auto weigh = [&](int it, int slot) {
    // the buffer is free: slots 0 and 2 follow the whole last chunk (which the
    // second warpgroup has waited for), 1 its last use, 3 and 4 the slots
    // before them in their buffers
    const int buf = slot_buffer(slot);
    if (slot == 0 && it > 0 && !wait(kUpdate, it - 1)) return false;
    if (slot == 1 && it > 0 && !wait(kUsed + 1, it - 1)) return false;
    if (slot >= 3 && !wait(kUsed + buf, it)) return false;
    if (r / 32 * 32 < TV) {
      tc::after_sync();
      const int t0 = slot_step(slot), groups = slot_groups(slot);
      const unsigned char *col = smem + (it & 1) * L_::STAGE + L_::Q +
                                 (r / 64) * 16384 + t0 * 128 + (r % 8) * 2;
      const float *wt = gt.write[it & 1] + t0;
      const int group = r % 64 / 8;
      uint32_t dst = mine + L_::W + buf * 48;
#pragma unroll 1
      for (int g = 0; g < groups; ++g, col += 1024, wt += 8, dst += 4) {
        uint32_t pl[3][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 w = *reinterpret_cast<const float2 *>(wt + 2 * i);
          const uint32_t v0 = *reinterpret_cast<const uint16_t *>(
              col + 2 * i * 128 + ((group ^ (2 * i % 8)) * 16));
          const uint32_t v1 = *reinterpret_cast<const uint16_t *>(
              col + (2 * i + 1) * 128 + ((group ^ ((2 * i + 1) % 8)) * 16));
          float2 x = mul2(make_float2(__uint_as_float(v0 << 16),
                                      __uint_as_float(v1 << 16)),
                          w);
#pragma unroll
          for (int s = 0; s < 3; ++s) {
            pl[s][i] = pack2(x.x, x.y);
            if (s < 2)
              x = fma2(make_float2(la::lo2(pl[s][i]), la::hi2(pl[s][i])),
                       make_float2(-1.0f, -1.0f), x);
          }
        }
#pragma unroll
        for (int s = 0; s < 3; ++s)
          tc::tmem_st4(dst + s * groups * 4, pl[s]);
      }
      tc::tmem_wait_st();
      tc::before_sync();
    }
    tc::bar_arrive(bar(kWeighed + slot));
    return true;
  };
  // The barrier of chunk `it`'s q, and how often it has been used.
  auto q_full = [&](int it) {
    return ONE_Q ? int(kFullQ0) : kFullQ0 + (it & 1);
  };
  auto q_use = [&](int it) { return ONE_Q ? it : it / 2; };
  // Whether chunk `it`'s values and weights are there.
  auto chunk_in = [&](int it) {
    return wait(kFull0 + (it & 1), it / 2) &&
           wait(kWeights0 + (it & 1), it / 2);
  };

  if (warp >= 12) {
    // The code of a chunk's round, over all roles, has to stay within the SM's
    // instruction cache (about 32 KB of it is hot here): warps that run alone
    // wait for little else, so loops are rolled and nothing is inlined twice.
    if (warp == 12) {
      // ---- q, k, v in (stage it % 2), y out
      const int kh = h / (p.heads / job.k_heads);
      const int qh = h / (p.heads / job.q_heads);
      const int vh = h / (p.heads / job.v_heads);
      const bool staged = !STATE_ONLY && !job.y_f32;
      // k and v come as soon as their stage's products are done. With one q, k
      // comes once the y in its place has been read, and q after its
      // forerunner's last product; both are brought to L2 before.
      int it = 0;
#pragma unroll 1
      for (; fit && it < n_live + 2; ++it) {
        const int st = it & 1;
        const uint32_t s = base + st * L_::STAGE, f = bar(kFull0 + st);
        if (it < n_live) {
          if (it >= 2 && !wait(kEmpty0 + st, it / 2 - 1)) break;
          if (lane == 0) {
            tc::bar_expect(f, ONE_Q ? L_::V : L_::Q + L_::V);
#pragma unroll 1
            for (int c = 0; c < QD / 64; ++c)
              if constexpr (ONE_Q) {
                tc::prefetch_box(&maps[1], c * 64, kh, low(it), int(b));
                tc::prefetch_box(&maps[0], c * 64, qh, low(it), int(b));
              } else {
                tc::load_box(s + c * 16384, &maps[1], f, c * 64, kh, low(it),
                             int(b));
              }
#pragma unroll 1
            for (int c = 0; c < TV / 64; ++c)
              tc::load_box(s + L_::Q + c * 16384, &maps[2], f, c * 64, vh,
                           low(it), int(b));
          }
          __syncwarp();
        }
        if (STATE_ONLY) continue;
        if (it >= 2 && staged) {
          if (!wait(kStaged, it - 2)) break;
          if (lane == 0) {
            const uint32_t y = ONE_Q ? s : base + L_::Y;
#pragma unroll 1
            for (int c = 0; c * 64 < job.vd; ++c)
              tc::store_box(&maps[3], y + c * 16384, c * 64, h, low(it - 2),
                            int(b));
            tc::store_read();
            tc::bar_arrive(bar(kStored));
          }
          __syncwarp();
        }
        if (it >= n_live) continue;
        if constexpr (ONE_Q) {
          if (lane == 0) {
            tc::bar_expect(bar(kFullK0 + st), L_::Q);
#pragma unroll 1
            for (int c = 0; c < QD / 64; ++c)
              tc::load_box(s + c * 16384, &maps[1], bar(kFullK0 + st), c * 64,
                           kh, low(it), int(b));
          }
          __syncwarp();
          if (it > 0 && !wait(kRead, it - 1)) break;
        }
        if (lane == 0) {
          const uint32_t q = ONE_Q ? base : s, fq = bar(q_full(it));
          tc::bar_expect(fq, L_::Q);
#pragma unroll 1
          for (int c = 0; c < QD / 64; ++c)
            tc::load_box(q + L_::Q0 + c * 16384, &maps[0], fq, c * 64, qh,
                         low(it), int(b));
        }
        __syncwarp();
      }
      if (it < n_live + 2) {
        // given up: nothing may still be on its way into this block's memory
        gt.dead = 1;
        const int loaded = it < n_live ? it + 1 : n_live;
#pragma unroll 1
        for (it = loaded > 3 ? loaded - 3 : 0; it < loaded; ++it)
#pragma unroll 1
          for (int i = 0; i < 1 << 12; ++i)
            if (tc::bar_try(bar(kFull0 + (it & 1)), uint32_t(it / 2) & 1u) &&
                (STATE_ONLY ||
                 tc::bar_try(bar(q_full(it)), uint32_t(q_use(it)) & 1u)) &&
                (!ONE_Q || tc::bar_try(bar(kFullK0 + (it & 1)),
                                       uint32_t(it / 2) & 1u)))
              break;
      }
    } else if (warp == 13) {
      // ---- products, in a converged warp with uniform operands
      constexpr uint32_t kScoreShape = tc::shape(128, false);
      constexpr uint32_t kReadShape = tc::shape(TV, false);
      constexpr uint32_t kUpdateShape = tc::shape(QD, true);
      constexpr uint32_t kOutShape = tc::shape(TV, true);
      const uint32_t e = tc::elected();
      // an operand's description for each step of 16 is the first one's plus
      // the bytes between them (in units of 16)
      const uint64_t stage0 = tc::operand(base, 16384);
      const uint64_t state0 = tc::operand(base + L_::S, 0);
      constexpr uint64_t kStage = L_::STAGE / 16, kV = L_::Q / 16,
                         kQ = L_::Q0 / 16;
      bool alive = fit;
      // round i: chunk i - 1's update, reading and output, then chunk i's
      // scores, which are decayed while the state is brought up to date
#pragma unroll 1
      for (int i = 0; i <= n_live && alive; ++i) {
        if (i > 0) {
          const int it = i - 1, st = it & 1;
          const uint64_t K = stage0 + st * kStage, V = K + kV,
                         Q = (ONE_Q ? stage0 : K) + kQ;
          alive = wait(kState, it);
          // the state's update first: the next chunk waits for it
#pragma unroll 1
          for (int slot = 0; slot < 5 && alive; ++slot) {
            alive = wait(kWeighed + slot, it);
            if (!alive) break;
            tc::after_sync();
            const int n = slot_groups(slot) / 2, buf = slot_buffer(slot);
            uint32_t w = tmem + L_::W + buf * 48;
            uint64_t k = K + uint64_t(slot_step(slot) * 8);
#pragma unroll 1
            for (int j = 0; j < n; ++j, w += 8, k += 128) {  // 16 steps
              // planes from the smallest to the leading one
              tc::mma_ts(e, tmem + L_::U, w + 16 * n, k, kUpdateShape,
                         (slot | j) != 0);
              tc::mma_ts(e, tmem + L_::U, w + 8 * n, k, kUpdateShape, true);
              tc::mma_ts(e, tmem + L_::U, w, k, kUpdateShape, true);
            }
            if (slot < 3) tc::commit(e, bar(kUsed + slot));
            if constexpr (!STATE_ONLY) {
              if (slot == 1) {
                if (it > 0) alive = wait(kOutRead, it - 1);
                if (!alive) break;
                tc::after_sync();
#pragma unroll 1
                for (int s = PS - 1; s >= 0; --s)
#pragma unroll
                  for (int c = 0; c < QD / 64; ++c)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                      tc::mma_ss(e, tmem + L_::O, Q + c * 1024 + ks * 2,
                                 state0 + uint64_t(s * TV * QD / 8 +
                                                   c * TV * 8 + ks * 2),
                                 kReadShape, s < PS - 1 || c + ks > 0);
                tc::commit(e, bar(kRead));
              }
            }
          }
          if (!alive) break;
          tc::commit(e, bar(kUpdate));
          if constexpr (!STATE_ONLY) {
            // O2 is added to the scaled O1
            alive = wait(kScored, it) && wait(kReadDone, it);
            if (!alive) break;
            tc::after_sync();
#pragma unroll 1
            for (int s = PS - 1; s >= 0; --s)
#pragma unroll
              for (int ks = 0; ks < 8; ++ks)
                tc::mma_ts(e, tmem + L_::O, tmem + L_::P + ks * 16 + s * 8,
                           V + uint64_t(ks * 128), kOutShape, true);
            tc::commit(e, bar(kOut));
          }
          tc::commit(e, bar(kEmpty0 + st));
        }
        if (i < n_live) {
          const int st = i & 1;
          const uint64_t K = stage0 + st * kStage,
                         Q = (ONE_Q ? stage0 : K) + kQ;
          alive = wait(kFull0 + st, i / 2) &&
                  (!ONE_Q || wait(kFullK0 + st, i / 2)) &&
                  (STATE_ONLY || wait(q_full(i), q_use(i))) &&
                  (i != ragged || wait(kClean, 0));
          if (!alive) break;
          tc::after_sync();
          if constexpr (!STATE_ONLY) {
            // K-major: 64 steps to a 128-byte row
#pragma unroll
            for (int c = 0; c < QD / 64; ++c)
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                tc::mma_ss(e, tmem + L_::P, Q + c * 1024 + ks * 2,
                           K + c * 1024 + ks * 2, kScoreShape, c + ks > 0);
            tc::commit(e, bar(kScores));
          }
        }
      }
      if (!alive) gt.dead = 1;
      // every product is done before the block goes
      tc::commit(e, bar(kFin));
      int left = 1 << 16;
#pragma unroll 1
      while (left > 0 && !tc::bar_try(bar(kFin), 0)) --left;
      if (left == 0) gt.dead = 1;
      __syncwarp();
    } else {
      // ---- decays: every second chunk each, four steps a lane in the order
      // of time; the next values are on their way while these are summed
      const unsigned short *gate =
          p.log_decay ? static_cast<const unsigned short *>(p.log_decay) +
                            b * L * p.heads + h
                      : nullptr;
      const double head = p.head_log_decay ? p.head_log_decay[h] : 0.0;
      unsigned short raw[4] = {0, 0, 0, 0};
      auto token = [&](int it, int j) {
        const int s = 4 * lane + j;
        return rev ? low(it) + kChunk - s : low(it) + s;
      };
      auto fetch = [&](int it) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = token(it, j);
          if (gate && t < len) raw[j] = __ldg(gate + int64_t(t) * p.heads);
        }
      };
      // round -1 only reads
      bool alive = true;
#pragma unroll 1
      for (int it = warp - 16; it < n_live && alive; it += 2) {
        double c[4], sum = 0.0;
        int from[4], lastr = -1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const double g =
              it >= 0 && token(it, j) < len
                  ? double(__uint_as_float(uint32_t(raw[j]) << 16)) + head
                  : 0.0;
          sum += g * 1.4426950408889634;
          if (g < la::kRestart) {
            sum = 0.0;
            lastr = 4 * lane + j;
          }
          c[j] = sum;
          from[j] = lastr;
        }
        if (it + 2 < n_live) fetch(it + 2);
        if (it < 0) continue;
        double ps = sum;
        int pr = lastr;
#pragma unroll 1
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
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (from[j] < 0) {
            c[j] += es;
            from[j] = er;
          }
        auto pick = [](int j, const auto (&v)[4]) {
          return j & 2 ? (j & 1 ? v[3] : v[2]) : (j & 1 ? v[1] : v[0]);
        };
        // (a weight e^-x is off by x e^-x 2^-24 at most for the rounding of
        // x); this warp's own last weights have been used
        const int par = it & 1;
        if (it >= 2) alive = wait(kWeightsFree0 + par, it / 2 - 1);
        if (!alive) break;
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
          const int s = 4 * lane + j, row = rev ? kChunk - 1 - s : s;
          gt.write[par][row] =
              s >= end_r ? ex2(float(end - pick(j, c))) * job.sw : 0.0f;
        }
        if (lane == 0) {
          gt.keep[par] =
              end_r < 0 ? la::keep_of(end) : make_float2(0.0f, 0.0f);
          if (STATE_ONLY) gt.end[par] = end_r < 0 ? end : -CUDART_INF;
        }
        __syncwarp();
        if (lane == 0) tc::bar_arrive(bar(kWeights0 + par));
        if constexpr (!STATE_ONLY) {
          // the last chunk's values have been written (by the other warp) and
          // used; without the first wait this one could run a phase ahead of
          // its barrier and pass on the parity of an old one
          if (it > 0) alive = wait(kGates, it - 1) && wait(kGatesFree, it - 1);
          if (!alive) break;
#pragma unroll 1
          for (int j = 0; j < 4; ++j) {
            const int s = 4 * lane + j, row = rev ? kChunk - 1 - s : s;
            const double cj = pick(j, c);
            const int fj = pick(j, from);
            const float hi = float(cj);
            gt.hi[row] = hi;
            gt.lo[row] =
                (unsigned short)pack2(float(cj - double(hi)), 0.0f);
            gt.near[row] = s >= blk_r ? ex2(float(blk - cj)) : 0.0f;
            gt.from[row] = (unsigned char)(fj < 0 ? kNoRestart : fj);
          }
          __syncwarp();
          if (lane == 0) tc::bar_arrive(bar(kGates));
        }
      }
      if (!alive) gt.dead = 1;
    }
  } else if (warp < 4) {
    // ---- scores: P -> P'
    tc::fewer_registers<88>();
    // the step of this row in time, and its warp's block of 32
    const int step = rev ? kChunk - 1 - r : r;
    const int tb = rev ? 3 - warp : warp;
    int it = 0;
#pragma unroll 1
    for (; it < n_live; ++it) {
      if (!chunk_in(it) || (it == ragged && !wait(kClean, 0)) || !weigh(it, 0))
        break;
      tc::bar_arrive(bar(kWeightsFree0 + (it & 1)));
      if constexpr (STATE_ONLY) continue;
      if (!wait(kGates, it) || !wait(kScores, it)) break;
      tc::after_sync();
      const int rs = gt.from[r], from = rs == kNoRestart ? 0 : rs;
      const float chi = gt.hi[r],
                  clo = __uint_as_float(uint32_t(gt.lo[r]) << 16);
      // P' takes the place of its 16 columns of P: 8 a plane
      auto put = [&](int col, const uint32_t *v) {
        uint32_t w[PS][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t pl[PS];
          planes(make_float2(__uint_as_float(v[2 * i]),
                             __uint_as_float(v[2 * i + 1])),
                 pl);
#pragma unroll
          for (int s = 0; s < PS; ++s) w[s][i] = pl[s];
        }
#pragma unroll
        for (int s = 0; s < PS; ++s)
          tc::tmem_st8(mine + L_::P + col + s * 8, w[s]);
      };
#pragma unroll 1
      for (int nb = 0; nb < 4; ++nb) {     // 32 rows j
        const int jb = rev ? 3 - nb : nb;  // in time
        uint32_t v[32];
        if (jb < tb) {
          tc::tmem_ld32(mine + L_::P + nb * 32, v);
          const int ref = rev ? nb * 32 : nb * 32 + 31;  // row of step r
          const float e =
              from <= jb * 32 + 31
                  ? ex2((chi - gt.hi[ref]) +
                        (clo - __uint_as_float(uint32_t(gt.lo[ref]) << 16))) *
                        job.sp
                  : 0.0f;
          tc::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 f =
                *reinterpret_cast<const float4 *>(gt.near + nb * 32 + i);
            const float2 d[2] = {make_float2(f.x, f.y),
                                 make_float2(f.z, f.w)};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float2 x =
                  mul2(make_float2(__uint_as_float(v[i + 2 * j]),
                                   __uint_as_float(v[i + 2 * j + 1])),
                       mul2(make_float2(e, e), d[j]));
              v[i + 2 * j] = __float_as_uint(x.x);
              v[i + 2 * j + 1] = __float_as_uint(x.y);
            }
          }
          put(nb * 32, v);
          put(nb * 32 + 16, v + 16);
        } else if (jb == tb) {
          // rows of steps in [from, step] of this block of 32, as bits
          const int lo_s = max(from - jb * 32, 0), hi_s = step - jb * 32;
          uint32_t bits =
              (0xffffffffu >> (31 - hi_s)) & (0xffffffffu << lo_s);
          if (rev) bits = __brev(bits);
#pragma unroll 1
          for (int c = nb * 32; c < nb * 32 + 32; c += 16, bits >>= 16) {
            tc::tmem_ld16(mine + L_::P + c, v);
            tc::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const float4 fh =
                  *reinterpret_cast<const float4 *>(gt.hi + c + i);
              const uint2 fl = *reinterpret_cast<const uint2 *>(gt.lo + c + i);
              const float dh[4] = {fh.x, fh.y, fh.z, fh.w};
              const float dl[4] = {la::lo2(fl.x), la::hi2(fl.x),
                                   la::lo2(fl.y), la::hi2(fl.y)};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float d = ex2((chi - dh[j]) + (clo - dl[j])) * job.sp;
                v[i + j] = bits >> (i + j) & 1u
                               ? __float_as_uint(__uint_as_float(v[i + j]) * d)
                               : 0u;
              }
            }
            put(c, v);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = 0u;
#pragma unroll
          for (int c = 0; c < 32; c += 8)
            if (PS == 2 || c % 16 == 0)
              tc::tmem_st8(mine + L_::P + nb * 32 + c, v);
        }
      }
      tc::tmem_wait_st();
      tc::bar_arrive(bar(kGatesFree));
      tc::before_sync();
      tc::bar_arrive(bar(kScored));
    }
    if (it < n_live) gt.dead = 1;
  } else if (warp < 8) {
    // ---- the weighted values and the state; lane: a value column
    tc::more_registers<208>();
    constexpr int64_t SF = int64_t(QD) * kLaTile;
    const int tiles = (job.vd + kLaTile - 1) / kLaTile;
    // element (key, value r) of a segment's state
    float *seg_state =
        p.nseg > 1 && r / kLaTile < tiles
            ? job.seg_state +
                  ((int64_t(local) * p.nseg + seg) * tiles + r / kLaTile) *
                      SF +
                  r % kLaTile
            : nullptr;
    float2 S[QD / 2];
    {
      const float *src = nullptr;
      int keys = 0;
      int64_t stride = kLaTile;
      if (!STATE_ONLY && p.nseg > 1) {
        src = seg_state;
        keys = QD;
      } else if (!STATE_ONLY && job.init && r < job.vd) {
        src = job.init + bh * job.qd * job.vd + int64_t(r) * job.state_cs;
        keys = job.qd;
        stride = job.state_rs;
      }
      if (!src) keys = 0;
#pragma unroll
      for (int i = 0; i < QD; ++i) {
        const float x = i < keys ? *src : 0.0f;
        (i % 2 ? S[i / 2].y : S[i / 2].x) = x;
        src += stride;
      }
    }
    // the bfloat16 planes of the state
    auto put_state = [&]() {
      if constexpr (!STATE_ONLY) {
        if (r < TV) {
          // (the swizzle of a row's first group; the others are 16 bytes times
          // their number away, without carries)
          const uint32_t at = base + L_::S + swizzled(r, 0);
#pragma unroll
          for (int i = 0; i < QD; i += 8) {
            uint32_t w[4][PS];
#pragma unroll
            for (int j = 0; j < 4; ++j) planes(S[i / 2 + j], w[j]);
            const uint32_t dst = at ^ uint32_t(i % 64 / 8 * 16);
#pragma unroll
            for (int s = 0; s < PS; ++s)
              tc::smem_st4(dst + (i / 64) * TV * 128 + s * TV * QD * 2,
                           w[0][s], w[1][s], w[2][s], w[3][s]);
          }
        }
        tc::fence_async();
      }
      tc::before_sync();
      tc::bar_arrive(bar(kState));
    };
    double seg_sum = 0.0;  // of the chunks' log decays
    put_state();
    bool alive = fit;
    // In turn: the slots of chunk it, the arrival of chunk it + 1, the update.
#pragma unroll 1
    for (int it = -1; alive && it < n_live; ++it) {
#pragma unroll 1
      for (int slot = 2; slot < 5 && alive && it >= 0; ++slot)
        alive = weigh(it, slot);
      if (alive && it + 1 < n_live) {
        alive = chunk_in(it + 1);
        if (ONE_Q && alive && it + 1 == ragged)
          alive = wait(kFullK0 + ((it + 1) & 1), (it + 1) / 2);
        if (alive && it + 1 == ragged) {
          // rows behind the sequence's end: zeros, whatever was loaded
          unsigned char *Ks = smem + ((it + 1) & 1) * L_::STAGE,
                        *Vs = Ks + L_::Q;
          const int dead_from = int(len - low(it + 1));
#pragma unroll 1
          for (int z = r + dead_from * 8; z < kChunk * 8; z += 128) {
#pragma unroll
            for (int c = 0; c < QD / 64; ++c)
              *reinterpret_cast<uint4 *>(Ks + c * 16384 + z * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int c = 0; c < TV / 64; ++c)
              *reinterpret_cast<uint4 *>(Vs + c * 16384 + z * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
          }
          tc::fence_async();
          tc::bar_arrive(bar(kClean));
          alive = wait(kClean, 0);
        }
      }
      if (!alive) break;
      if (it < 0) continue;
      const float2 keep = gt.keep[it & 1];
      if (STATE_ONLY) seg_sum += gt.end[it & 1];
      tc::bar_arrive(bar(kWeightsFree0 + (it & 1)));
      alive = wait(kUpdate, it);
      if (!alive) break;
      tc::after_sync();
      if (la::none_kept(keep)) {  // a restart forgets whatever it held
#pragma unroll
        for (int i = 0; i < QD / 2; ++i) S[i] = make_float2(0.0f, 0.0f);
      }
#pragma unroll
      for (int u = 0; u < QD; u += 32) {
        uint32_t t[32];
        tc::tmem_ld32(mine + L_::U + u, t);
        tc::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          S[u / 2 + i] =
              fma2(make_float2(keep.y, keep.y), S[u / 2 + i],
                   fma2(make_float2(keep.x, keep.x), S[u / 2 + i],
                        make_float2(__uint_as_float(t[2 * i]),
                                    __uint_as_float(t[2 * i + 1]))));
      }
      put_state();
    }
    if (!alive) gt.dead = 1;
    float *dst = nullptr;
    int keys = 0;
    int64_t stride = kLaTile;
    if (STATE_ONLY) {
      dst = seg_state;
      keys = QD;
      if (r == 0)
        job.seg_decay[int64_t(local) * p.nseg + seg] = exp2(seg_sum);
    } else if (job.last && seg == p.nseg - 1 && r < job.vd) {
      dst = job.last + bh * job.qd * job.vd + int64_t(r) * job.state_cs;
      keys = job.qd;
      stride = job.state_rs;
      // running backwards, the first token's own decay is still to come
      if (rev && len > 0) {
        const float f = la::decay_of(la::gate_at<bf16>(p, b, 0, h));
#pragma unroll
        for (int i = 0; i < QD / 2; ++i)
          S[i] = f == 0.0f ? make_float2(0.0f, 0.0f)
                           : mul2(S[i], make_float2(f, f));
      }
    }
    if (!alive || !dst) keys = 0;
#pragma unroll
    for (int i = 0; i < QD; ++i) {
      if (i < keys) *dst = i % 2 ? S[i / 2].y : S[i / 2].x;
      dst += stride;
    }
  } else {
    // ---- y; lane: a step
    tc::fewer_registers<88>();
    {
      // rows of y behind the sequence's last live chunk
#pragma unroll 1
      for (int64_t t = STATE_ONLY ? L : idle_low + r;
           t < seg_low + p.seg_len && t < L; t += 128) {
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
      // In turn: O1 of chunk it is scaled, slot 1 of chunk it + 1 weighed
      // (while the output's products run), chunk it put out.
      int it = -1;
#pragma unroll 1
      for (; it < n_live; ++it) {
        const int st = it & 1;
        if (!STATE_ONLY && it >= 0) {
          // O1, scaled in its place: O2 is added to it there
          if (!wait(kGates, it) || !wait(kRead, it)) break;
          tc::after_sync();
          const float rd =
              gt.from[r] == kNoRestart ? ex2(gt.hi[r]) * job.si : 0.0f;
#pragma unroll 1
          for (int u = 0; u < TV; u += 32) {
            uint32_t v[32];
            tc::tmem_ld32(mine + L_::O + u, v);
            tc::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 x =
                  mul2(make_float2(__uint_as_float(v[i]),
                                   __uint_as_float(v[i + 1])),
                       make_float2(rd, rd));
              v[i] = __float_as_uint(x.x);
              v[i + 1] = __float_as_uint(x.y);
            }
            if (rd == 0.0f) {  // a restart forgets the state whatever it held
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = 0u;
            }
            tc::tmem_st16(mine + L_::O + u, v);
            tc::tmem_st16(mine + L_::O + u + 16, v + 16);
          }
          tc::tmem_wait_st();
          tc::bar_arrive(bar(kGatesFree));
          tc::before_sync();
          tc::bar_arrive(bar(kReadDone));
        }
        if (it + 1 < n_live) {
          if (!chunk_in(it + 1) || (it + 1 == ragged && !wait(kClean, 0)) ||
              !weigh(it + 1, 1))
            break;
          tc::bar_arrive(bar(kWeightsFree0 + ((it + 1) & 1)));
        }
        if (STATE_ONLY || it < 0) continue;
        const int64_t t = low(it) + r;
        const bool live = t < len;
        const bool staged = !job.y_f32;
        if (staged && it > 0 && !wait(kStored, it - 1)) break;
        if (!wait(kOut, it)) break;
        tc::after_sync();
        unsigned char *ys = smem + (ONE_Q ? st * L_::STAGE : L_::Y);
        const int64_t row = (b * L + t) * p.heads + h;
        float dot = 0.0f;
        // (the flags are read in the loop, so that it stays one loop)
        volatile const int *is_staged = &gt.staged, *is_dotted = &gt.dotted;
#pragma unroll 1
        for (int u = 0; u < TV; u += 32) {
          uint32_t v[32];
          tc::tmem_ld32(mine + L_::O + u, v);
          tc::tmem_wait_ld();
          if (!live) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0u;
          }
          if (*is_staged) {
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
          if (*is_dotted && live) {
            // the row dots the decay's gradient is made of
            const bf16 *ds = static_cast<const bf16 *>(job.dot) +
                             (b * L + t) * job.dot_stride +
                             int64_t(h / (p.heads / job.dot_heads)) * job.vd;
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
      if (it < n_live) gt.dead = 1;
    }
  }
  tc::before_sync();
  __syncthreads();
  tc::after_sync();
  if (warp == 13) tc::tmem_free(gt.tmem, 512);
  if (threadIdx.x == 0 && gt.dead) *pp.status = 1;
}

}  // namespace lat
}  // namespace ssm
