// smp_distill_bf16.cu -- smp_distill_loss' kernel for bf16 logits.
#include "smp_distill_kernel.cuh"

namespace smp {
int distill_bf16(const DistillArgs& a, cudaStream_t st) { return distill_rows<SMP_BF16>(a, st); }
}  // namespace smp
