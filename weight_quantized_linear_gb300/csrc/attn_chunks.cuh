// attn_chunks.cuh -- what the two kernels of attention over chunks share.
#pragma once

#include "kv_i4.cuh"

namespace wql {

// What CTAs leave unfinished, [CTA]; (m, l) and O of up to `rows` rows, [CTA][0: of the unit found begun, 1: of the one begun].
struct ChunkParts {
  int4* begun;   // {row of q, tokens, tokens that the first row sees, K/V head} of the unit that it began; no tokens: none
  int* went_on;  // of the unit that it found begun: 0: none, 1: it goes on, 2: it ends here
  float2* ml;
  float* part;
  int rows;
};

// Sequences of a few rows: attn_steps_i4.cu.
struct StepArgs {
  const __half* q;
  long long q_stride;
  const int *cu, *kv_lens;
  int B, T, Hq, Hkv, G, few;  // few: tokens of a chunk at most that are taken here, few * G <= kFewRows; up to 8 of these rows are cheaper
  const uint8_t* cache;
  int pages;
  FastDiv bpp;  // blocks of a page
  const int* table;
  int width, cap;
  float scale_log2;  // of any sign
  __half* out;
  float* lse;
  ChunkParts parts;
  unsigned* err;
};
constexpr int kFewRows = 16;
cudaError_t launch_attn_steps_i4(const StepArgs& a, int D, int ctas, cudaStream_t s);

}  // namespace wql
