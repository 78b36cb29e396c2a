// C ABI of the linear-attention entry points: host-side validation, the split
// of long sequences, workspaces and launches. The contract is in
// include/ssm_linattn.h.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "../../include/ssm_linattn.h"
#include "device_info.cuh"
#include "kernel_linattn_tc.cuh"
#include "tensor_map.cuh"

namespace {

using ssm::aligned;
using ssm::LaGateParams;
using ssm::LaJob;
using ssm::LaParams;
using ssm::LaStepParams;
using bf16 = __nv_bfloat16;

// Beyond what a device holds: sizes up to these overflow no index.
constexpr int64_t kMaxElements = int64_t(1) << 42;
constexpr int64_t kMaxSteps = int64_t(1) << 36;
// The tensor-memory kernel counts tokens in 32 bits, up to two chunks past the
// end.
constexpr int64_t kMaxTcSteps = int64_t(1) << 30;
// The decay's gradient sums differences inside a group of steps: at most 2048
// where it is bfloat16 (rounded by 2^-9), 128 where it is float32. The
// tensor-memory kernel's passes, which are for the former only, leave states at
// the ends of segments, and the segment is the group; the other kernel's leave
// them wherever they are wanted.
constexpr int64_t kGateSegment = 2048;
constexpr int64_t kGateExact = 128;

// Shared memory that lets one block of the tensor-memory kernel (which takes
// all of TMEM) onto an SM at a time.
constexpr int kOnePerSm = 120 * 1024;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int key_pad(int64_t d) { return d <= 64 ? 64 : 128; }

// Checks shared by every entry; fills dense strides in.
int check_dims(ssm_linattn_dims *d, int dtype, int64_t max_value) {
  if (d->batch <= 0 || d->seqlen <= 0 || d->heads <= 0 || d->groups <= 0 ||
      d->dk <= 0 || d->dv <= 0 || d->heads % d->groups != 0)
    return SSM_ERR_INVALID;
  if (dtype != SSM_F32 && dtype != SSM_BF16) return SSM_ERR_UNSUPPORTED;
  if (d->dk > ssm::kLaMaxKey || d->dv > max_value || d->heads > (1 << 20))
    return SSM_ERR_UNSUPPORTED;
  if (d->q_stride == 0) d->q_stride = d->groups * d->dk;
  if (d->k_stride == 0) d->k_stride = d->groups * d->dk;
  if (d->v_stride == 0) d->v_stride = d->heads * d->dv;
  if (d->q_stride < d->groups * d->dk || d->k_stride < d->groups * d->dk ||
      d->v_stride < d->heads * d->dv)
    return SSM_ERR_INVALID;
  int64_t rows = 0, n = 0, st = 0;
  if (__builtin_mul_overflow(d->batch, d->seqlen, &rows) ||
      rows > kMaxElements || d->seqlen > kMaxSteps)
    return SSM_ERR_INVALID;
  for (int64_t s : {d->q_stride, d->k_stride, d->v_stride, d->heads * d->dk})
    if (__builtin_mul_overflow(rows, s, &n) || n > kMaxElements)
      return SSM_ERR_INVALID;
  if (__builtin_mul_overflow(d->batch * d->heads, d->dk * d->dv, &st) ||
      st > kMaxElements)
    return SSM_ERR_INVALID;
  if (d->batch * d->heads > 0x7fffffff) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}

// Which kernel runs a call's passes: the tensor-memory kernel takes bfloat16
// rows on 16-byte boundaries, the other one everything.
enum class Path { kAny, kTc };

struct Plan {
  int nseg = 1;
  int64_t seg_len = 0;
  // heads that run uncut before the others, which are cut (forward)
  int64_t whole = 0;
  int64_t whole_len = 0;
  // byte offsets into the workspace; jobs: y or dq, dk, dv
  size_t state[3] = {0, 0, 0}, decay[3] = {0, 0, 0};
  size_t part_dq = 0, part_dk = 0, rows_q = 0, rows_k = 0, part_head = 0,
         last = 0, anchor[2] = {0, 0};
  // groups of steps that the decay's gradient is summed in (backward)
  int groups = 0;
  int64_t group_len = 0;
  size_t bytes = 0;
};

size_t take(size_t *at, size_t floats) {
  const size_t here = *at;
  *at += (floats * sizeof(float) + 255) / 256 * 256;
  return here;
}

// Segments: where one block for each sequence, head and tile leaves over half
// of the GPU idle, a sequence is cut so that about two blocks (one of the
// tensor-memory kernel) are there for each SM, of at least 128 (512) steps: 1 x
// 65536 steps of 8 heads of 128 take 290 us in 18 segments a head; uncut,
// eight SMs would go through 512 chunks of 5.7 us each. The states in front of
// the segments cost one more reading of k and v, so a grid that fills the GPU
// by itself is not cut. (Two are counted for float32 with 128-wide keys too, of
// which an SM holds one: its blocks then come in two rounds.)
void cut(Plan *pl, int64_t blocks, int64_t L, int sms, Path path,
         int64_t most) {
  const int chunk = path == Path::kTc ? ssm::lat::kChunk : ssm::kLaChunk;
  const int64_t slots = int64_t(sms) * (path == Path::kTc ? 1 : 2);
  int64_t n = 1;
  if (blocks * 2 <= slots)
    n = std::min(slots / blocks,
                 std::max<int64_t>(1, L / (path == Path::kTc ? 512 : 128)));
  n = std::max(n, ceil_div(L, most));
  const int64_t chunks = ceil_div(L, chunk);
  const int64_t per = ceil_div(chunks, n);
  pl->seg_len = per * chunk;
  pl->nseg = int(ceil_div(chunks, per));
}

Plan plan_fwd(const ssm_linattn_dims &d, Path path, int sms) {
  Plan pl;
  const int64_t tiles = ceil_div(d.dv, ssm::kLaTile);
  const int64_t all = d.batch * d.heads;
  // One block an SM: where the last round of blocks would leave over half of
  // the SMs idle, its heads are cut (4 x 8192 x 40 heads of 128, one plane of
  // the state: 550 us with 12 heads in a round of their own, 359 to 406 us with
  // these cut).
  auto cut_for = [&](int64_t heads) {
    cut(&pl, heads * (path == Path::kTc ? 1 : tiles), d.seqlen, sms, path,
        int64_t(1) << 40);
  };
  cut_for(all);
  if (path == Path::kTc && all > sms && all % sms != 0) {
    cut_for(all % sms);
    if (pl.nseg > 1) pl.whole = all / sms * sms;
    else cut_for(all);
  }
  pl.whole_len =
      ceil_div(d.seqlen, ssm::lat::kChunk) * ssm::lat::kChunk;
  if (pl.nseg > 1) {
    const size_t bh = size_t(all - pl.whole);
    pl.state[0] = take(&pl.bytes, bh * pl.nseg * tiles * key_pad(d.dk) *
                                      ssm::kLaTile);
    pl.decay[0] = take(&pl.bytes, bh * pl.nseg * 2);  // 64-bit
  }
  return pl;
}

// gate: with the decays' gradients; exact: one of which is float32.
Plan plan_bwd(const ssm_linattn_dims &d, Path path, bool gate, bool exact,
              int sms) {
  Plan pl;
  const int64_t tk = ceil_div(d.dk, ssm::kLaTile),
                tv = ceil_div(d.dv, ssm::kLaTile);
  const size_t bh = size_t(d.batch) * d.heads;
  cut(&pl, d.batch * d.heads * (path == Path::kTc ? 3 : 2 * tk + tv),
      d.seqlen, sms, path,
      gate && path == Path::kTc ? kGateSegment : int64_t(1) << 40);
  if (pl.nseg > 1)
    for (int j = 0; j < 3; ++j) {
      pl.state[j] = take(&pl.bytes, bh * pl.nseg * (j < 2 ? tk : tv) *
                                        key_pad(j < 2 ? d.dv : d.dk) *
                                        ssm::kLaTile);
      pl.decay[j] = take(&pl.bytes, bh * pl.nseg * 2);  // 64-bit
    }
  if (d.groups != d.heads) {
    pl.part_dq = take(&pl.bytes, bh * d.seqlen * d.dk);
    pl.part_dk = take(&pl.bytes, bh * d.seqlen * d.dk);
  }
  if (gate) {
    pl.rows_q = take(&pl.bytes, bh * d.seqlen * 2 * tk);
    pl.rows_k = take(&pl.bytes, bh * d.seqlen * 2 * tk);
    pl.groups = pl.nseg;
    pl.group_len = pl.seg_len;
    if (path == Path::kAny) {
      pl.group_len = exact ? kGateExact : kGateSegment;
      pl.groups = int(ceil_div(d.seqlen, pl.group_len));
      if (pl.groups > 1)
        for (size_t &a : pl.anchor)
          a = take(&pl.bytes, bh * pl.groups * tk * key_pad(d.dv) *
                                  ssm::kLaTile);
    }
    pl.part_head = take(&pl.bytes, bh * pl.groups * 2);  // 64-bit
    pl.last = take(&pl.bytes, bh * d.dk * d.dv);
  }
  return pl;
}

// The states in front of the segments, from what each of them adds.
template <int QD>
void join(const LaParams &p, int n, int tiles, cudaStream_t s) {
  const int blocks = QD * ssm::kLaTile * tiles / 256;
  ssm::la::linattn_join_kernel<QD>
      <<<dim3(unsigned(blocks), unsigned(std::min(p.bhs, 65535)), unsigned(n)),
         256, 0, s>>>(p);
}

// Every job of `p` (n of them), which share QD and PS.
template <typename T, int NP, int PS, int QD>
int launch_jobs(const LaParams &p, int n, cudaStream_t s) {
  constexpr int MINB = NP == 3 && QD == 128 ? 1 : 2;
  int tiles = 0;
  for (int j = 0; j < n; ++j) tiles = std::max(tiles, p.job[j].tiles);
  // jobs of one launch have the same tile count (the caller groups them)
  const int64_t one = int64_t(tiles) * p.bhs;
  if (one > 0x7fffffff / p.nseg) return SSM_ERR_UNSUPPORTED;
  if (p.nseg > 1) {
    auto kern = ssm::la::linattn_kernel<T, NP, PS, QD, true, MINB>;
    constexpr int smem = ssm::la::Layout<T, NP, PS, QD, true>::BYTES;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem) != cudaSuccess) {
      cudaGetLastError();
      return SSM_ERR_CUDA;
    }
    kern<<<dim3(unsigned(one * (p.nseg - 1)), n),
           ssm::la::kThreads, smem, s>>>(p);
    if (cudaGetLastError() != cudaSuccess) return SSM_ERR_CUDA;
    join<QD>(p, n, tiles, s);
    if (cudaGetLastError() != cudaSuccess) return SSM_ERR_CUDA;
  }
  auto kern = ssm::la::linattn_kernel<T, NP, PS, QD, false, MINB>;
  constexpr int smem = ssm::la::Layout<T, NP, PS, QD, false>::BYTES;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           smem) != cudaSuccess) {
    cudaGetLastError();
    return SSM_ERR_CUDA;
  }
  kern<<<dim3(unsigned(one * p.nseg), n),
           ssm::la::kThreads, smem, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

int run_jobs(const LaParams &p, int n, int dtype, bool exact, cudaStream_t s) {
  const int qd = key_pad(p.job[0].qd);
  if (dtype == SSM_F32)
    return qd == 64 ? launch_jobs<float, 3, 3, 64>(p, n, s)
                    : launch_jobs<float, 3, 3, 128>(p, n, s);
  if (exact)
    return qd == 64 ? launch_jobs<bf16, 1, 3, 64>(p, n, s)
                    : launch_jobs<bf16, 1, 3, 128>(p, n, s);
  return qd == 64 ? launch_jobs<bf16, 1, 2, 64>(p, n, s)
                  : launch_jobs<bf16, 1, 2, 128>(p, n, s);
}

// ---- the tensor-memory kernel
__device__ int g_linattn_status;

int *status_word(int device) {
  static std::atomic<int *> known[64];
  int *w = known[device].load(std::memory_order_relaxed);
  if (!w) {
    void *q = nullptr;
    if (cudaGetSymbolAddress(&q, g_linattn_status) != cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    w = static_cast<int *>(q);
    known[device].store(w, std::memory_order_relaxed);
  }
  return w;
}

bool tc_rows(const void *q, int64_t stride, int64_t d) {
  return aligned(q, 16) && stride % 8 == 0 && d % 8 == 0 &&
         stride < (int64_t(1) << 36);
}

// Whether every pass of a call can run there.
bool tc_takes(const ssm_linattn_dims &d, int dtype, const void *q,
              const void *k, const void *v,
              std::initializer_list<const void *> dense) {
  if (dtype != SSM_BF16 || d.dv > 128 || d.seqlen > kMaxTcSteps ||
      d.batch >= (int64_t(1) << 31) || !tc_rows(q, d.q_stride, d.dk) ||
      !tc_rows(k, d.k_stride, d.dk) || !tc_rows(v, d.v_stride, d.dv) ||
      d.seqlen * d.q_stride >= (int64_t(1) << 38) ||
      d.seqlen * d.k_stride >= (int64_t(1) << 38) ||
      d.seqlen * d.v_stride >= (int64_t(1) << 38) ||
      d.seqlen * d.heads * d.dv >= (int64_t(1) << 38))
    return false;
  for (const void *a : dense)
    if (a && !aligned(a, 16)) return false;
  return true;
}

template <int QD, int TV>
int launch_tc(const ssm::lat::Params &pp, int n, cudaStream_t s) {
  const LaParams &p = pp.p;
  const int64_t one = p.bhs;
  if (one > 0x7fffffff / p.nseg) return SSM_ERR_UNSUPPORTED;
  if (p.nseg > 1) {
    auto kern = ssm::lat::linattn_tc_kernel<QD, TV, true>;
    constexpr int smem = ssm::lat::Lay<QD, TV, true>::BYTES;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem < kOnePerSm ? kOnePerSm : smem) !=
        cudaSuccess) {
      cudaGetLastError();
      return SSM_ERR_CUDA;
    }
    kern<<<dim3(unsigned(one * (p.nseg - 1)), n), ssm::lat::kThreads,
           smem < kOnePerSm ? kOnePerSm : smem, s>>>(pp);
    if (cudaGetLastError() != cudaSuccess) return SSM_ERR_CUDA;
    int tiles = 0;
    for (int j = 0; j < n; ++j) tiles = std::max(tiles, p.job[j].tiles);
    join<QD>(p, n, tiles, s);
    if (cudaGetLastError() != cudaSuccess) return SSM_ERR_CUDA;
  }
  auto kern = ssm::lat::linattn_tc_kernel<QD, TV, false>;
  constexpr int need = ssm::lat::Lay<QD, TV, false>::BYTES;
  constexpr int smem = need < kOnePerSm ? kOnePerSm : need;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           smem) != cudaSuccess) {
    cudaGetLastError();
    return SSM_ERR_CUDA;
  }
  kern<<<dim3(unsigned(one * p.nseg), n), ssm::lat::kThreads, smem, s>>>(pp);
  return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

// The jobs of `p` (n of them), which share their sizes.
int run_tc(const LaParams &p, int n, int device, cudaStream_t s) {
  ssm::lat::Params pp{};
  pp.p = p;
  pp.status = status_word(device);
  if (!pp.status) return SSM_ERR_CUDA;
  for (int i = 0; i < n; ++i) {
    const LaJob &j = p.job[i];
    if (!ssm::row_map(&pp.map[i][0], j.q, p.batch, p.seqlen, j.q_heads, j.qd,
                      j.q_stride, ssm::lat::kChunk) ||
        !ssm::row_map(&pp.map[i][1], j.k, p.batch, p.seqlen, j.k_heads, j.qd,
                      j.k_stride, ssm::lat::kChunk) ||
        !ssm::row_map(&pp.map[i][2], j.v, p.batch, p.seqlen, j.v_heads, j.vd,
                      j.v_stride, ssm::lat::kChunk) ||
        (!j.y_f32 &&
         !ssm::row_map(&pp.map[i][3], j.y, p.batch, p.seqlen, p.heads, j.vd,
                       int64_t(p.heads) * j.vd, ssm::lat::kChunk)))
      return SSM_ERR_CUDA;
  }
  const bool q64 = p.job[0].qd <= 64, v64 = p.job[0].vd <= 64;
  return q64 ? (v64 ? launch_tc<64, 64>(pp, n, s)
                    : launch_tc<64, 128>(pp, n, s))
             : (v64 ? launch_tc<128, 64>(pp, n, s)
                    : launch_tc<128, 128>(pp, n, s));
}

// Every token's rows of a tensor, from the first element to the last.
ssm::Span rows_span(const void *at, const ssm_linattn_dims &d, int64_t stride,
                    int64_t row, size_t esz) {
  return {at, size_t((d.batch * d.seqlen - 1) * stride + row) * esz};
}

ssm::Span state_span(const float *at, const ssm_linattn_dims &d) {
  return {at, size_t(d.batch * d.heads * d.dk * d.dv) * sizeof(float)};
}

bool check_floats(std::initializer_list<const float *> list) {
  for (const float *q : list)
    if (q && !aligned(q, 4)) return false;
  return true;
}

LaParams common(const ssm_linattn_dims &d, const Plan &pl,
                const void *log_decay, const float *head_log_decay,
                const int *lengths) {
  LaParams p{};
  p.log_decay = log_decay;
  p.head_log_decay = head_log_decay;
  p.lengths = lengths;
  p.batch = d.batch;
  p.seqlen = d.seqlen;
  p.heads = int(d.heads);
  p.nseg = pl.nseg;
  p.seg_len = pl.seg_len;
  p.anchors = pl.groups;
  p.anchor_len = int(pl.group_len);
  p.bhs = int(d.batch * d.heads);
  return p;
}

template <typename T>
void group_sum(const float *part, const ssm_linattn_dims &d, void *out,
               int sms, cudaStream_t s) {
  const int64_t n = d.batch * d.seqlen * d.groups * d.dk;
  const int64_t grid = std::min<int64_t>(ceil_div(n, 256), int64_t(sms) * 16);
  ssm::la::linattn_group_sum_kernel<T><<<unsigned(grid), 256, 0, s>>>(
      part, d.batch * d.seqlen, int(d.groups), int(d.heads / d.groups),
      int(d.dk), static_cast<T *>(out));
}

}  // namespace

extern "C" {

int ssm_linattn_workspace(int device, ssm_linattn_dims dims, int dtype,
                          int backward, size_t *bytes) {
  if (!bytes) return SSM_ERR_INVALID;
  *bytes = 0;
  int rc = check_dims(&dims, dtype,
                      backward ? ssm::kLaMaxKey : SSM_LINATTN_MAX_VALUE);
  if (rc != SSM_OK) return rc;
  int sms = 0;
  rc = ssm::device_sms(device, &sms);
  if (rc != SSM_OK) return rc;
  for (Path path : {Path::kAny, Path::kTc}) {
    if (path == Path::kTc && (dtype != SSM_BF16 || dims.dv > 128)) continue;
    if (!backward) {
      *bytes = std::max(*bytes, plan_fwd(dims, path, sms).bytes);
      continue;
    }
    // every kind of call that is not ruled out
    const bool gate = !(backward & SSM_LINATTN_NO_DECAY_GRADIENT),
               head = gate && !(backward & SSM_LINATTN_NO_HEAD_GRADIENT) &&
                      path == Path::kAny;
    *bytes = std::max(*bytes, plan_bwd(dims, path, false, false, sms).bytes);
    if (gate)
      *bytes = std::max(*bytes, plan_bwd(dims, path, true, dtype == SSM_F32,
                                         sms).bytes);
    if (head)
      *bytes = std::max(*bytes, plan_bwd(dims, path, true, true, sms).bytes);
  }
  return SSM_OK;
}

int ssm_linattn_fwd(int device, const void *q, const void *k, const void *v,
                    const void *log_decay, const float *head_log_decay,
                    float scale, const int32_t *lengths, const float *h0,
                    void *y, float *h_last, void *workspace,
                    size_t workspace_bytes, ssm_linattn_dims dims, int dtype,
                    struct CUstream_st *stream) {
  // ---- host-side validation: nothing touches the GPU before it passes
  if (!q || !k || !v || !y) return SSM_ERR_INVALID;
  int rc = check_dims(&dims, dtype, SSM_LINATTN_MAX_VALUE);
  if (rc != SSM_OK) return rc;
  const size_t esz = dtype == SSM_F32 ? 4 : 2;
  for (const void *a : {q, k, v, log_decay, static_cast<const void *>(y)})
    if (a && !aligned(a, esz)) return SSM_ERR_ALIGN;
  // y is written in pairs of values
  if (dims.dv % 2 == 0 && !aligned(y, 2 * esz)) return SSM_ERR_ALIGN;
  if (!check_floats({head_log_decay, h0, h_last,
                     reinterpret_cast<const float *>(lengths)}))
    return SSM_ERR_ALIGN;
  const int64_t G = dims.groups * dims.dk, H = dims.heads * dims.dv;
  const ssm::Span out_y = rows_span(y, dims, H, H, esz),
                  in_h = state_span(h0 == h_last ? nullptr : h0, dims),
                  out_h = state_span(h_last, dims);
  const auto reads = {
      rows_span(q, dims, dims.q_stride, G, esz),
      rows_span(k, dims, dims.k_stride, G, esz),
      rows_span(v, dims, dims.v_stride, H, esz),
      rows_span(log_decay, dims, dims.heads, dims.heads, esz),
      ssm::Span{head_log_decay, size_t(dims.heads) * sizeof(float)},
      ssm::Span{lengths, size_t(dims.batch) * sizeof(int32_t)}, in_h};
  if (ssm::clash({out_y, out_h}, reads)) return SSM_ERR_INVALID;
  int sms = 0;
  rc = ssm::device_ready(device, &sms);
  if (rc != SSM_OK) return rc;
  const Path path =
      tc_takes(dims, dtype, q, k, v, {y}) ? Path::kTc : Path::kAny;
  const Plan pl = plan_fwd(dims, path, sms);
  if (pl.bytes > workspace_bytes || (pl.bytes && !workspace))
    return SSM_ERR_INVALID;
  if (workspace && !aligned(workspace, 16)) return SSM_ERR_ALIGN;
  if (pl.bytes && ssm::clash({{workspace, pl.bytes}, out_y, out_h}, reads))
    return SSM_ERR_INVALID;
  unsigned char *ws = static_cast<unsigned char *>(workspace);

  LaParams p = common(dims, pl, log_decay, head_log_decay, lengths);
  LaJob &j = p.job[0];
  j.q = q; j.k = k; j.v = v; j.y = y;
  j.q_stride = dims.q_stride; j.k_stride = dims.k_stride;
  j.v_stride = dims.v_stride;
  j.q_heads = j.k_heads = int(dims.groups);
  j.v_heads = int(dims.heads);
  j.qd = int(dims.dk); j.vd = int(dims.dv);
  j.tiles = int(ceil_div(dims.dv, ssm::kLaTile));
  j.init = h0; j.last = h_last;
  j.state_rs = j.vd; j.state_cs = 1;
  j.sp = j.si = scale; j.sw = 1.0f;
  if (pl.nseg > 1) {
    j.seg_state = reinterpret_cast<float *>(ws + pl.state[0]);
    j.seg_decay = reinterpret_cast<double *>(ws + pl.decay[0]);
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (path == Path::kAny) return run_jobs(p, 1, dtype, false, s);
  if (pl.whole > 0) {
    LaParams first = p;
    first.nseg = 1;
    first.seg_len = pl.whole_len;
    first.bhs = int(pl.whole);
    rc = run_tc(first, 1, device, s);
    if (rc != SSM_OK) return rc;
    p.bh0 = int(pl.whole);
    p.bhs -= int(pl.whole);
  }
  return run_tc(p, 1, device, s);
}

int ssm_linattn_step(int device, const void *q, const void *k, const void *v,
                     const void *log_decay, const float *head_log_decay,
                     float scale, float *state, void *y, ssm_linattn_dims dims,
                     int dtype, struct CUstream_st *stream) {
  if (!q || !k || !v || !state || !y) return SSM_ERR_INVALID;
  if (dims.seqlen != 1) return SSM_ERR_INVALID;
  int rc = check_dims(&dims, dtype, SSM_LINATTN_MAX_VALUE);
  if (rc != SSM_OK) return rc;
  const size_t esz = dtype == SSM_F32 ? 4 : 2;
  for (const void *a : {q, k, v, log_decay, static_cast<const void *>(y)})
    if (a && !aligned(a, esz)) return SSM_ERR_ALIGN;
  if (!check_floats({head_log_decay, state})) return SSM_ERR_ALIGN;
  const int64_t G = dims.groups * dims.dk, H = dims.heads * dims.dv;
  if (ssm::clash({state_span(state, dims), rows_span(y, dims, H, H, esz)},
                 {rows_span(q, dims, dims.q_stride, G, esz),
                  rows_span(k, dims, dims.k_stride, G, esz),
                  rows_span(v, dims, dims.v_stride, H, esz),
                  rows_span(log_decay, dims, dims.heads, dims.heads, esz),
                  {head_log_decay, size_t(dims.heads) * sizeof(float)}}))
    return SSM_ERR_INVALID;
  int sms = 0;
  rc = ssm::device_ready(device, &sms);
  if (rc != SSM_OK) return rc;
  LaStepParams p{};
  p.q = q; p.k = k; p.v = v;
  p.q_stride = dims.q_stride; p.k_stride = dims.k_stride;
  p.v_stride = dims.v_stride;
  p.log_decay = log_decay; p.head_log_decay = head_log_decay;
  p.scale = scale; p.state = state; p.y = y;
  p.batch = dims.batch; p.heads = int(dims.heads);
  p.groups = int(dims.groups); p.dk = int(dims.dk); p.dv = int(dims.dv);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool wide = p.dv % 4 == 0 && aligned(state, 16);
  const bool half = wide ? p.dv <= 64 : p.dv <= 16;
  const int64_t grid =
      p.batch * p.heads * ceil_div(p.dv, (wide ? 4 : 1) * (half ? 16 : 32));
  if (grid > 0x7fffffff) return SSM_ERR_UNSUPPORTED;
  auto pick = [&](auto type) {
    using T = decltype(type);
    return wide ? (half ? ssm::la::linattn_step_kernel<T, 4, 16>
                        : ssm::la::linattn_step_kernel<T, 4, 32>)
                : (half ? ssm::la::linattn_step_kernel<T, 1, 16>
                        : ssm::la::linattn_step_kernel<T, 1, 32>);
  };
  auto kern = dtype == SSM_F32 ? pick(float()) : pick(bf16());
  kern<<<unsigned(grid), 256, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

int ssm_linattn_bwd(int device, const void *q, const void *k, const void *v,
                    const void *log_decay, const float *head_log_decay,
                    float scale, const int32_t *lengths, const float *h0,
                    const void *dy, const float *dh_last, void *dq, void *dk,
                    void *dv, void *dlog_decay, float *dhead_log_decay,
                    float *dh0, void *workspace, size_t workspace_bytes,
                    ssm_linattn_dims dims, int dtype,
                    struct CUstream_st *stream) {
  // ---- host-side validation: nothing touches the GPU before it passes
  if (!q || !k || !v || !dy || !dq || !dk || !dv) return SSM_ERR_INVALID;
  if ((dlog_decay && !log_decay) || (dhead_log_decay && !head_log_decay))
    return SSM_ERR_INVALID;
  int rc = check_dims(&dims, dtype, ssm::kLaMaxKey);
  if (rc != SSM_OK) return rc;
  const size_t esz = dtype == SSM_F32 ? 4 : 2;
  for (const void *a : {q, k, v, log_decay, dy, static_cast<const void *>(dq),
                        static_cast<const void *>(dk),
                        static_cast<const void *>(dv),
                        static_cast<const void *>(dlog_decay)})
    if (a && !aligned(a, esz)) return SSM_ERR_ALIGN;
  // gradients are written in pairs of values
  if (dims.dk % 2 == 0 && (!aligned(dq, 2 * esz) || !aligned(dk, 2 * esz)))
    return SSM_ERR_ALIGN;
  if (dims.dv % 2 == 0 && !aligned(dv, 2 * esz)) return SSM_ERR_ALIGN;
  if (!check_floats({head_log_decay, h0, dh_last, dhead_log_decay, dh0,
                     reinterpret_cast<const float *>(lengths)}))
    return SSM_ERR_ALIGN;
  const int H = int(dims.heads), G = int(dims.groups), K = int(dims.dk),
            V = int(dims.dv);
  const int64_t dy_stride = int64_t(H) * V;
  const size_t heads_bytes = size_t(H) * sizeof(float);
  const int64_t qk = int64_t(G) * K;
  const ssm::Span writes[] = {
      rows_span(dq, dims, qk, qk, esz), rows_span(dk, dims, qk, qk, esz),
      rows_span(dv, dims, dy_stride, dy_stride, esz),
      rows_span(dlog_decay, dims, H, H, esz),
      ssm::Span{dhead_log_decay, heads_bytes}, state_span(dh0, dims)};
  const auto reads = {
      rows_span(q, dims, dims.q_stride, qk, esz),
      rows_span(k, dims, dims.k_stride, qk, esz),
      rows_span(v, dims, dims.v_stride, dy_stride, esz),
      rows_span(log_decay, dims, H, H, esz),
      ssm::Span{head_log_decay, heads_bytes},
      ssm::Span{lengths, size_t(dims.batch) * sizeof(int32_t)},
      state_span(h0, dims), rows_span(dy, dims, dy_stride, dy_stride, esz),
      state_span(dh_last, dims)};
  if (ssm::clash({writes[0], writes[1], writes[2], writes[3], writes[4],
                  writes[5]},
                 reads))
    return SSM_ERR_INVALID;
  int sms = 0;
  rc = ssm::device_ready(device, &sms);
  if (rc != SSM_OK) return rc;
  const bool gate = dlog_decay || dhead_log_decay;
  // The heads' own gradient is float32 and sums differences over all steps:
  // the two planes that fit beside the stages there leave it 5.6e-5 off (8192
  // steps of long memory), the other kernel's three planes 3e-7.
  const Path path = tc_takes(dims, dtype, q, k, v, {dy, dq, dk, dv}) &&
                            !dhead_log_decay
                        ? Path::kTc
                        : Path::kAny;
  const Plan pl =
      plan_bwd(dims, path, gate, dtype == SSM_F32 || dhead_log_decay, sms);
  if (pl.bytes > workspace_bytes || (pl.bytes && !workspace))
    return SSM_ERR_INVALID;
  if (workspace && !aligned(workspace, 16)) return SSM_ERR_ALIGN;
  if (pl.bytes &&
      ssm::clash({{workspace, pl.bytes}, writes[0], writes[1], writes[2],
                  writes[3], writes[4], writes[5]},
                 reads))
    return SSM_ERR_INVALID;
  if (gate && dims.batch * dims.heads > 0x7fffffff / pl.groups)
    return SSM_ERR_UNSUPPORTED;
  unsigned char *ws = static_cast<unsigned char *>(workspace);
  auto at = [&](size_t off) { return reinterpret_cast<float *>(ws + off); };
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);

  const bool shared = G != H;
  LaJob jq{}, jk{}, jv{};
  // dq: query dy, key v, value k
  jq.q = dy; jq.q_stride = dy_stride; jq.q_heads = H;
  jq.k = v; jq.k_stride = dims.v_stride; jq.k_heads = H;
  jq.v = k; jq.v_stride = dims.k_stride; jq.v_heads = G;
  jq.qd = V; jq.vd = K;
  jq.y = shared ? static_cast<void *>(at(pl.part_dq)) : dq;
  jq.init = h0; jq.state_rs = 1; jq.state_cs = V;
  jq.sp = jq.si = scale; jq.sw = 1.0f;
  // dk: query v, key dy, value q, backwards
  jk.q = v; jk.q_stride = dims.v_stride; jk.q_heads = H;
  jk.k = dy; jk.k_stride = dy_stride; jk.k_heads = H;
  jk.v = q; jk.v_stride = dims.q_stride; jk.v_heads = G;
  jk.qd = V; jk.vd = K;
  jk.y = shared ? static_cast<void *>(at(pl.part_dk)) : dk;
  jk.init = dh_last; jk.state_rs = 1; jk.state_cs = V;
  jk.sp = jk.sw = scale; jk.si = 1.0f;
  jk.reverse = 1;
  jq.y_f32 = jk.y_f32 = shared;
  jq.tiles = jk.tiles = int(ceil_div(K, ssm::kLaTile));
  // dv: query k, key q, value dy, backwards
  jv.q = k; jv.q_stride = dims.k_stride; jv.q_heads = G;
  jv.k = q; jv.k_stride = dims.q_stride; jv.k_heads = G;
  jv.v = dy; jv.v_stride = dy_stride; jv.v_heads = H;
  jv.qd = K; jv.vd = V;
  jv.y = dv;
  jv.init = dh_last; jv.last = dh0; jv.state_rs = V; jv.state_cs = 1;
  jv.sp = jv.sw = scale; jv.si = 1.0f;
  jv.reverse = 1;
  jv.tiles = int(ceil_div(V, ssm::kLaTile));
  if (pl.nseg > 1) {
    LaJob *all[3] = {&jq, &jk, &jv};
    for (int i = 0; i < 3; ++i) {
      all[i]->seg_state = at(pl.state[i]);
      all[i]->seg_decay = reinterpret_cast<double *>(ws + pl.decay[i]);
    }
  }
  if (gate) {
    jq.dot = q; jq.dot_stride = dims.q_stride; jq.dot_heads = G;
    jk.dot = k; jk.dot_stride = dims.k_stride; jk.dot_heads = G;
    jq.rows = at(pl.rows_q);
    jk.rows = at(pl.rows_k);
    if (dh_last) jq.last = at(pl.last);  // [dk, dv] through the strides
    if (path == Path::kAny && pl.groups > 1) {
      jq.anchor = at(pl.anchor[0]);
      jk.anchor = at(pl.anchor[1]);
    }
  }

  LaParams p = common(dims, pl, log_decay, head_log_decay, lengths);
  p.job[0] = jq;
  p.job[1] = jk;
  // one launch for all three where they are of one kind
  const bool one = (K <= ssm::kLaTile) == (V <= ssm::kLaTile);
  p.job[2] = jv;
  auto run = [&](int n, bool exact) {
    return path == Path::kTc ? run_tc(p, n, device, s)
                             : run_jobs(p, n, dtype, exact, s);
  };
  rc = run(one ? 3 : 2, gate);
  if (rc == SSM_OK && !one) {
    p.job[0] = jv;
    rc = run(1, false);
  }
  if (rc != SSM_OK) return rc;

  if (shared) {
    if (dtype == SSM_F32) {
      group_sum<float>(at(pl.part_dq), dims, dq, sms, s);
      group_sum<float>(at(pl.part_dk), dims, dk, sms, s);
    } else {
      group_sum<bf16>(at(pl.part_dq), dims, dq, sms, s);
      group_sum<bf16>(at(pl.part_dk), dims, dk, sms, s);
    }
    if (cudaGetLastError() != cudaSuccess) return SSM_ERR_CUDA;
  }
  if (gate) {
    LaGateParams g{};
    g.rows_q = at(pl.rows_q);
    g.rows_k = at(pl.rows_k);
    // the other kernel's passes leave row dots for each 32 columns
    g.parts = path == Path::kTc ? 1 : 2 * jq.tiles;
    if (pl.groups > 1) {
      g.fwd_state = path == Path::kAny ? jq.anchor : jq.seg_state;
      g.rev_state = path == Path::kAny ? jk.anchor : jk.seg_state;
    }
    g.state_floats = int64_t(jq.tiles) * key_pad(V) * ssm::kLaTile;
    g.last_state = at(pl.last);
    g.dh_last = dh_last;
    g.last_floats = int64_t(K) * V;
    g.dlog_decay = dlog_decay;
    g.part = dhead_log_decay
                 ? reinterpret_cast<double *>(ws + pl.part_head)
                 : nullptr;
    g.log_decay = log_decay;
    g.head_log_decay = head_log_decay;
    g.lengths = lengths;
    g.batch = dims.batch; g.seqlen = dims.seqlen; g.heads = H;
    g.nseg = pl.groups; g.seg_len = pl.group_len;
    const int64_t grid = dims.batch * H * pl.groups;
    if (dtype == SSM_F32)
      ssm::la::linattn_gate_kernel<float><<<unsigned(grid), 256, 0, s>>>(g);
    else
      ssm::la::linattn_gate_kernel<bf16><<<unsigned(grid), 256, 0, s>>>(g);
    if (dhead_log_decay)
      ssm::la::linattn_head_sum_kernel<<<H, 128, 0, s>>>(
          g.part, dims.batch * pl.groups, H, dhead_log_decay);
    if (cudaGetLastError() != cudaSuccess) return SSM_ERR_CUDA;
  }
  return SSM_OK;
}

int ssm_linattn_sync_status(int device, struct CUstream_st *stream) {
  int sms = 0;
  int rc = ssm::device_ready(device, &sms);
  if (rc != SSM_OK) return rc;
  int *word = status_word(device);
  if (!word || cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) !=
                   cudaSuccess) {
    cudaGetLastError();
    return SSM_ERR_CUDA;
  }
  int value = 0;
  if (cudaMemcpy(&value, word, sizeof(int), cudaMemcpyDeviceToHost) !=
      cudaSuccess)
    return SSM_ERR_CUDA;
  if (value == 0) return SSM_OK;
  value = 0;
  if (cudaMemcpy(word, &value, sizeof(int), cudaMemcpyHostToDevice) !=
      cudaSuccess)
    return SSM_ERR_CUDA;
  return SSM_ERR_TIMEOUT;
}

}  // extern "C"
