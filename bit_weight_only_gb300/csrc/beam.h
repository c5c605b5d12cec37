// beam.h -- beam selection: parameters, limits and the launch call.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "qgemv.h"

namespace qgemv {

constexpr int kMaxBeams = 64;   // of a sequence
constexpr int kMaxWidth = 64;   // candidates kept of a sequence
constexpr int kMaxParts = 32;   // parts of a row, each a block's
constexpr int kMaxBeamSeqs = 4096;

// Workspace: a count of arrivals for each of kMaxBeamSeqs sequences, 0 between
// calls (in one place whatever the sizes of a call); for each row and part the candidates' keys (uint64 [width],
// descending, 0: none), then the largest logit and the sum of exponentials.
struct BeamParams {
  const void* logits;
  int64_t row_stride, vocab;
  const float* scores;
  int64_t n_seqs;
  int beams, width;
  float* out_scores;
  int32_t* out_beams;
  int32_t* out_tokens;
  unsigned* arrived;           // [kMaxBeamSeqs]
  unsigned long long* keys;    // [rows][parts][width]
  float2* sums;                // [rows][parts]
  int parts;
  int tiles;        // of a part, at most
};

int beam_parts(int64_t rows, int64_t vocab, int sms);
cudaError_t launch_beam(const BeamParams& p, int dtype, cudaStream_t s);

}  // namespace qgemv
