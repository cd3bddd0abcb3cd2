// smp_distill_f16.cu -- smp_distill_loss' kernel for f16 logits.
#include "smp_distill_kernel.cuh"

namespace smp {
int distill_f16(const DistillArgs& a, cudaStream_t st) { return distill_rows<SMP_F16>(a, st); }
}  // namespace smp
