// smp_distill_grad.cu -- the gradient of smp_distill_loss' loss and log
// probabilities with respect to the logits (smp_distill_loss_grad).
//
// Outside the slots grad_j = rho_j D, rho_j = 2^((x_j - m) s - L log2 e) the token's
// share of the mass there and D = (g A - g_lp s) / T one factor for the row; a slot's
// value is (g G_k - g_lp p_k) / T, and the target adds g_lp / T.  The kind of
// divergence is in A and G_k alone.  A CTA writes rho_j D over its segment, slots
// included, and after a barrier the slots' values over those.
//
// D is handled as a mantissa and a power of two, so that neither a small T nor
// gradients near the ends of binary32 make it 0 or infinite: usually 2^24 goes to
// rho (2^x flushes results below 2^-126, which a small T would make visible), and the
// whole power where it is beyond 2^60.
#include "smp_train.cuh"

namespace smp {
namespace {

constexpr int DGT = 256;  // threads
constexpr int DGSEG = 8192;

template <int DT>
__global__ void __launch_bounds__(DGT) distill_grad_kernel(const DistillGradArgs a, const int nc) {
  using TY = ScType<DT>;
  const int r = blockIdx.x / nc, c = blockIdx.x % nc, tid = threadIdx.x, K = a.K;
  const int j0 = c * DGSEG, j1 = min(a.V, j0 + DGSEG);
  const typename TY::raw* row = static_cast<const typename TY::raw*>(a.logits) + (size_t)r * a.ld;
  typename TY::raw* out = static_cast<typename TY::raw*>(a.grad) + (size_t)r * a.gld;
  const uint32_t* bm = a.bitmask ? a.bitmask + (size_t)r * a.W : nullptr;
  const float T = a.temperature ? a.temperature[r] : 1.f;
  float m = a.stats[4 * (size_t)r];
  const float Lr = a.stats[4 * (size_t)r + 1], A = a.stats[4 * (size_t)r + 2], mass = a.stats[4 * (size_t)r + 3];
  int t = a.targets ? a.targets[r] : -1;
  const bool live = sc_temperature_ok(T) && t >= -1 && t < a.V && fabsf(A) < INFINITY && mass >= 0.f;
  float g = live && a.g_loss ? a.g_loss[r] : 0.f, gl = live && t >= 0 && a.g_lp ? a.g_lp[r] : 0.f;
  if (gl != 0.f && !(a.logprobs[r] > -INFINITY)) gl = 0.f;
  // g, gl = (gm, glm) 2^ge;  T = Tm 2^Te;  D = Dm 2^De
  int ge, le, Te, De;
  frexpf(g, &ge);
  frexpf(gl, &le);
  ge = g == 0.f ? le : gl == 0.f ? ge : max(ge, le);
  const float gm = ldexpf(g, -ge), glm = ldexpf(gl, -ge), Tm = frexpf(live ? T : 1.f, &Te);
  float Dm = frexpf(gm * A - glm * mass, &De) / Tm;
  De += ge - Te;
  const int shift = De > -60 && De < 60 ? 24 : max(-250, min(250, De));
  Dm = ldexpf(Dm, De - shift);
  float l2 = Lr / SC_LN2 - (float)shift;
  const float s = sc_scale(live ? T : 1.f);
  if (m == -INFINITY) m = l2 = Dm = 0.f;  // every legal token has a slot
  const float at_target = ldexpf(glm / Tm, ge - Te);
  const bool none = !live || (g == 0.f && gl == 0.f);
  for (int j = j0 + tid; j < j1; j += DGT) {
    float y = 0.f;
    if (!none && (!bm || ((bm[j >> 5] >> (j & 31)) & 1u))) {
      const float x = TY::value(row[j]);
      if (x > -INFINITY) y = sc_ex2(fmaf(x - m, s, -l2)) * Dm;
      if (j == t) y += at_target;
    }
    out[j] = TY::store(y);
  }
  if (none) return;
  __syncthreads();
  for (int k = tid; k < K; k += DGT) {
    const int id = a.ids[(size_t)r * K + k];
    if (id < j0 || id >= j1) continue;
    float y = gm * a.slot_g[(size_t)r * K + k];
    if (gl != 0.f) y += (id == t ? glm : 0.f) - glm * expf(a.slot_lp[(size_t)r * K + k]);
    out[id] = TY::store(ldexpf(y / Tm, ge - Te));
  }
}

template <int DT>
int launch_distill_grad(const DistillGradArgs& a, cudaStream_t st) {
  const int nc = (a.V + DGSEG - 1) / DGSEG;
  if ((long long)a.B * nc > 0x7fffffffLL) return SMP_ERR_CAPACITY;
  distill_grad_kernel<DT><<<(unsigned)(a.B * nc), DGT, 0, st>>>(a, nc);
  return sc_ok(cudaGetLastError()) ? SMP_OK : SMP_ERR_CUDA;
}

}  // namespace

int distill_grad_enqueue(const DistillGradArgs& a, int dtype, cudaStream_t st) {
  switch (dtype) {
    case SMP_F32: return launch_distill_grad<SMP_F32>(a, st);
    case SMP_BF16: return launch_distill_grad<SMP_BF16>(a, st);
    default: return launch_distill_grad<SMP_F16>(a, st);
  }
}

}  // namespace smp
