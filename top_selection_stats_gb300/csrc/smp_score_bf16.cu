// smp_score_bf16.cu -- smp_token_logprobs for bfloat16 logits.
#include "smp_score_kernel.cuh"

namespace smp {
int score_bf16(const ScoreArgs& a, cudaStream_t st) { return score_rows<SMP_BF16>(a, st); }
}  // namespace smp
