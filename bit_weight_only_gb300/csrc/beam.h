// beam.h -- beam selection: parameters, limits and the launch call.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "qgemv.h"

namespace qgemv {

constexpr int kMaxBeams = 64;      // of a sequence
constexpr int kMaxWidth = 64;      // candidates kept of a sequence
constexpr int kMaxBeamSeqs = 4096;
constexpr int kBeamChunk = 512;    // values of a row that are summed up together

// Workspace: a count of arrivals for each of kMaxBeamSeqs sequences, 0 between
// calls (in one place whatever the sizes of a call); for each chunk of each row
// its largest logit and the sum of exp(x - that).
struct BeamParams {
  const void* logits;
  int64_t row_stride, vocab;
  const float* scores;
  int64_t n_seqs;
  int beams, width;
  float* out_scores;
  int32_t* out_beams;
  int32_t* out_tokens;
  unsigned* arrived;  // [kMaxBeamSeqs]
  float2* chunks;     // [rows][n_chunks]
  int n_chunks;       // of a row
};

inline int64_t beam_chunks(int64_t vocab) { return (vocab + kBeamChunk - 1) / kBeamChunk; }
cudaError_t launch_beam(const BeamParams& p, int dtype, cudaStream_t s);

}  // namespace qgemv
