// smp_score_f16.cu -- smp_token_logprobs for binary16 logits.
#include "smp_score_kernel.cuh"

namespace smp {
int score_f16(const ScoreArgs& a, cudaStream_t st) { return score_rows<SMP_F16>(a, st); }
}  // namespace smp
