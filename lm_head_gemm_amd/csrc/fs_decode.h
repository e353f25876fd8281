// Internal header of the 8-bit and beam search kernels: their argument blocks,
// launchers and what they share with the host code of the first ABI part.
#pragma once

#include "../../include/flashsample_decode.h"
#include "fs_common.h"

namespace fs {

// Records a launch status for fs_last_hip_error() and returns FS_ERR_HIP.
fs_status_t fail_hip(hipError_t e);

struct RowsI8Args {
  const void* x;
  int64_t ldx;
  const void* residual;   // or null
  int64_t ldr;
  const void* gain;       // null: codes of x itself, no norm
  void* sum;              // where h = x + residual goes (with a residual)
  int64_t lds;
  int8_t* codes;
  int64_t ldc;
  float* scales;
  int32_t M, D;
  float eps;
};

struct ProductI8Args {
  const int8_t* q;
  int64_t ldq;
  const float* q_scales;
  const int8_t* w;
  int64_t ldw;
  const float* w_scales;
  int32_t M, N, K;
  void* out;
  int64_t ldo;
  int32_t out_bf16;
};

struct BeamSelectArgs {
  const void* logits;
  int64_t ld;
  int32_t bf16;
  const float* scores;
  const uint8_t* finished;   // or null
  int32_t pad;
  int32_t B, beams, V, n;
  int32_t chunk, n_chunks;   // vocabulary entries per chunk, chunks per row
  uint64_t* cand;            // [B * beams, n_chunks, n] candidate keys, best first (0: none)
  double* sums;              // [B * beams, n_chunks] sum of e^(l - max) per chunk
  float* maxima;             // [B * beams, n_chunks] largest logit per chunk
  float* out_scores;
  int32_t* out_parents;
  int32_t* out_tokens;
};

struct BeamReorderArgs {
  fs_beam_layout_t from, to;
  const int32_t* parents;
  int32_t n_states, B, beams;
  int32_t in_place;
};

hipError_t launch_rows_i8(const RowsI8Args& a, bool bf16, bool gain_bf16, hipStream_t stream);
hipError_t launch_product_i8(const ProductI8Args& a, hipStream_t stream);
// Vocabulary entries per chunk of the selection's first kernel.
int32_t beam_chunk(int64_t rows, int64_t V, bool bf16);
hipError_t launch_beam_select(const BeamSelectArgs& a, hipStream_t stream);
// states, out: host arrays of a.n_states device addresses (in place: the same one twice).
hipError_t launch_beam_reorder(const BeamReorderArgs& a, const void* const* states, void* const* out,
                               hipStream_t stream);

}  // namespace fs
