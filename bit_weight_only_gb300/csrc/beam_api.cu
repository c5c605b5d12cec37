// beam_api.cu -- the C ABI of beam search's selection (include/qgemv.h):
// argument checks on the host, then the launches.
#include "api_checks.h"
#include "beam.h"

namespace {

using namespace qgemv;

bool beam_sizes_ok(int64_t n_seqs, int beams, int64_t vocab, int width) {
  return n_seqs >= 0 && n_seqs <= kMaxBeamSeqs && beams >= 1 && beams <= kMaxBeams && vocab >= 1 &&
         vocab <= (int64_t(1) << 30) && width >= 1 && width <= kMaxWidth;
}

}  // namespace

extern "C" {

int64_t qgemv_beam_ws_bytes(int64_t n_seqs, int beams, int64_t vocab, int width) {
  if (!beam_sizes_ok(n_seqs, beams, vocab, width)) return 0;
  const int64_t rows = (n_seqs > 0 ? n_seqs : 1) * beams;
  return 4 * kMaxBeamSeqs + rows * beam_chunks(vocab) * static_cast<int64_t>(sizeof(float2));
}

int qgemv_beam_select(int dtype, const void* logits, int64_t row_stride, int64_t vocab, const float* scores, int64_t n_seqs,
                      int beams, int width, float* out_scores, int32_t* out_beams, int32_t* out_tokens, void* ws,
                      int64_t ws_bytes, void* stream) {
  const int size = dtype_size(dtype);
  if (size == 0) return fail(QGEMV_ERR_ARG, "unknown dtype %d", dtype);
  if (!beam_sizes_ok(n_seqs, beams, vocab, width))
    return fail(QGEMV_ERR_ARG, "%lld sequences of %d beams, %lld tokens, %d kept: at most %d of %d, 2^30 and %d",
                (long long)n_seqs, beams, (long long)vocab, width, kMaxBeamSeqs, kMaxBeams, kMaxWidth);
  if (n_seqs == 0) return report_error(QGEMV_OK, "");
  if (row_stride < 0 || row_stride > (int64_t(1) << 38)) return fail(QGEMV_ERR_ARG, "row_stride outside [0, 2^38]");
  if (!logits || !scores || !out_scores || !out_beams || !out_tokens || !ws) return fail(QGEMV_ERR_ARG, "an argument is NULL");
  if (reinterpret_cast<uintptr_t>(logits) & (size - 1)) return fail(QGEMV_ERR_ALIGN, "logits must be aligned to their elements");
  if ((reinterpret_cast<uintptr_t>(scores) | reinterpret_cast<uintptr_t>(out_scores) | reinterpret_cast<uintptr_t>(out_beams) |
       reinterpret_cast<uintptr_t>(out_tokens)) & 3)
    return fail(QGEMV_ERR_ALIGN, "scores and outputs must be 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(ws) & 15) return fail(QGEMV_ERR_ALIGN, "the workspace must be 16-byte aligned");
  const int64_t need = qgemv_beam_ws_bytes(n_seqs, beams, vocab, width);
  if (ws_bytes < need)
    return fail(QGEMV_ERR_ARG, "the workspace has %lld bytes, %lld are needed", (long long)ws_bytes, (long long)need);
  BeamParams p = {};
  p.logits = logits;
  p.row_stride = row_stride;
  p.vocab = vocab;
  p.scores = scores;
  p.n_seqs = n_seqs;
  p.beams = beams;
  p.width = width;
  p.out_scores = out_scores;
  p.out_beams = out_beams;
  p.out_tokens = out_tokens;
  p.arrived = static_cast<unsigned*>(ws);
  p.chunks = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + 4 * kMaxBeamSeqs);
  p.n_chunks = static_cast<int>(beam_chunks(vocab));
  return done(launch_beam(p, dtype, static_cast<cudaStream_t>(stream)), "launching the selection");
}

}  // extern "C"
