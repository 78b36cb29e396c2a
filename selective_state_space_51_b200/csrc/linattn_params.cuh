// Launch parameters shared by the linear-attention kernels (plain pointers
// and sizes).
#pragma once

#include <stdint.h>

namespace ssm {

constexpr int kLaChunk = 64;   // steps per chunk of the chunked form
constexpr int kLaTile = 64;    // value columns per block
constexpr int kLaMaxKey = 128; // widest key (and, backward, value)

// One pass of linear attention with decay over every sequence and head:
//   y_i = sp * sum_{j <= i} decay(j, i) (q_i . k_j) v_j + si * (...) of the
// incoming state, S <- decay S + sw * k v. The backward pass is three of them
// (see kernel_linattn.cuh), so q, k and v here are whatever the pass reads as
// query, key and value.
struct LaJob {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // elements from a token to the next
  int q_heads, k_heads, v_heads;         // heads in each (H, or G shared)
  int qd, vd;                            // key size, value size
  int tiles;                             // value tiles of kLaTile columns
  void *y;                               // [b, L, heads, vd]: T or float
  int y_f32;
  const float *init;                     // state in front or nullptr
  float *last;                           // state behind or nullptr
  int state_rs, state_cs;                // strides of init/last: key, value
  int reverse;                           // time runs from the end
  float sp, sw, si;                      // factors of P, the write, the read
  const void *dot;                       // row-dot operand [.., vd] or nullptr
  int64_t dot_stride;
  int dot_heads;
  float *rows;                           // [2 tiles, b, heads, L] row dots,
                                         // of 32 columns each
  float *seg_state;                      // [bhs, nseg, tiles, QD, 64]
  double *seg_decay;                     // [bhs, nseg]
  float *anchor;                         // [b, heads, anchors, tiles, QD, 64]
                                         // or nullptr: the state in front of
                                         // every anchor_len-th token
};

struct LaParams {
  LaJob job[3];
  const void *log_decay;        // [b, L, H] activation type or nullptr
  const float *head_log_decay;  // [H] or nullptr
  const int *lengths;           // [b] or nullptr
  int64_t batch, seqlen;
  int heads;
  int nseg;                     // segments per sequence
  int64_t seg_len;              // steps per segment, a multiple of the chunk
  int anchors;                  // groups of anchor_len tokens in a sequence
  int anchor_len;               // a power of 2, and of chunks
  int bh0, bhs;                 // the sequences' heads of this launch, counted
                                // through all: bhs of them from bh0 on
};

// The log decay's gradient from the row dots and the states at the ends of
// groups of steps (nseg of seg_len steps: anchor_len of them, or a segment).
struct LaGateParams {
  const float *rows_q, *rows_k;  // row dots of dq with q, of dk with k
  int parts;                           // of 32 columns each
  const float *fwd_state, *rev_state;  // anchor (seg_state) of the dq and dk
                                       // passes
  int64_t state_floats;                // floats of one state, all tiles
  const float *last_state, *dh_last;   // [b, H, dk, dv], dh_last or nullptr
  int64_t last_floats;                 // dk dv
  void *dlog_decay;                    // [b, L, H] activation type or nullptr
  double *part;                        // [b, nseg, H] sums or nullptr
  const void *log_decay;
  const float *head_log_decay;
  const int *lengths;
  int64_t batch, seqlen;
  int heads, nseg;
  int64_t seg_len;
};

struct LaStepParams {
  const void *q, *k, *v;        // [b, G, dk], [b, G, dk], [b, H, dv]
  int64_t q_stride, k_stride, v_stride;
  const void *log_decay;        // [b, H] or nullptr
  const float *head_log_decay;  // [H] or nullptr
  float scale;
  float *state;                 // [b, H, dk, dv]
  void *y;                      // [b, H, dv]
  int64_t batch;
  int heads, groups, dk, dv;
};

}  // namespace ssm
