// smp_score_grad.cu -- the gradient of log probabilities and entropy with
// respect to the logits (smp_token_logprobs_grad).  One CTA per row.  With
// d_j = (x_j - m) s, s = log2(e) / T and p_j = 2^(d_j - log2 of the mass),
//     grad_j = p_j (a + b d_j) + [j = target] g / T,
//     a = -(g + g_H (H - L)) / T,   b = -g_H ln 2 / T.
// 2^d flushes results below 2^-126 to zero, which a small T would make
// visible: p is taken times 2^24 and a, b times 2^-24.
#include "smp_score.cuh"

namespace smp {
namespace {

constexpr int GT = 256;

template <int DT>
__global__ void __launch_bounds__(GT) grad_kernel(const GradArgs a) {
  using TY = ScType<DT>;
  const int r = blockIdx.x;
  const typename TY::raw* row = static_cast<const typename TY::raw*>(a.logits) + (size_t)r * a.ld;
  typename TY::raw* out = static_cast<typename TY::raw*>(a.grad) + (size_t)r * a.gld;
  const uint32_t* bm = a.bitmask ? a.bitmask + (size_t)r * a.W : nullptr;
  const float T = a.temperature ? a.temperature[r] : 1.f;
  const int t = a.targets ? a.targets[r] : -1;
  const float m = a.stats[2 * (size_t)r], L = a.stats[2 * (size_t)r + 1];
  const bool live = sc_temperature_ok(T) && t >= -1 && t < a.V && fabsf(m) < INFINITY &&
                    fabsf(L) < INFINITY;
  auto logit = [&](int j) {
    return (!bm || ((bm[j >> 5] >> (j & 31)) & 1u)) ? TY::value(row[j]) : -INFINITY;
  };
  const float s = sc_scale(live ? T : 1.f);
  const bool hit = live && t >= 0 && a.g_lp && logit(t) > -INFINITY;
  __syncthreads();  // the target's logit is read before it may be overwritten
  const float g = hit ? a.g_lp[r] : 0.f;
  const float gh = live && a.g_ent ? a.g_ent[r] : 0.f;
  const float c0 = live ? -(g + (a.g_ent ? gh * (a.entropy[r] - L) : 0.f)) / T * 0x1p-24f : 0.f;
  const float c1 = live ? -gh * SC_LN2 / T * 0x1p-24f : 0.f;
  const float at = live ? g / T : 0.f;
  const float l2 = L / SC_LN2 - 24.f;
  for (int j = threadIdx.x; j < a.V; j += GT) {
    float y = 0.f;
    const float x = live ? logit(j) : -INFINITY;
    if (x > -INFINITY) {
      const float d = fmaxf((x - m) * s, SC_DMIN);
      y = sc_ex2(d - l2) * fmaf(c1, d, c0);
    }
    if (hit && j == t) y += at;
    out[j] = TY::store(y);
  }
}

}  // namespace

int grad_enqueue(const GradArgs& a, int dtype, cudaStream_t st) {
  switch (dtype) {
    case SMP_F32: grad_kernel<SMP_F32><<<a.B, GT, 0, st>>>(a); break;
    case SMP_BF16: grad_kernel<SMP_BF16><<<a.B, GT, 0, st>>>(a); break;
    default: grad_kernel<SMP_F16><<<a.B, GT, 0, st>>>(a); break;
  }
  return cudaGetLastError() == cudaSuccess ? SMP_OK : SMP_ERR_CUDA;
}

}  // namespace smp
