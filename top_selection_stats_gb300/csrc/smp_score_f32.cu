// smp_score_f32.cu -- smp_token_logprobs for binary32 logits.
#include "smp_score_kernel.cuh"

namespace smp {
int score_f32(const ScoreArgs& a, cudaStream_t st) { return score_rows<SMP_F32>(a, st); }
}  // namespace smp
