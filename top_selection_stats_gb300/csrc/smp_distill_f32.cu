// smp_distill_f32.cu -- smp_distill_loss' kernel for f32 logits.
#include "smp_distill_kernel.cuh"

namespace smp {
int distill_f32(const DistillArgs& a, cudaStream_t st) { return distill_rows<SMP_F32>(a, st); }
}  // namespace smp
