// smp_distill.cu -- divergence of a student's distribution from a teacher's top
// tokens (smp_distill_loss).  One CTA per row.
#include "smp_distill.cuh"

namespace smp {
namespace {

constexpr int DT_THREADS = 256;

template <int DT>
__global__ void __launch_bounds__(DT_THREADS) distill_kernel(const DistillArgs a) {
  using TY = ScType<DT>;
  __shared__ int ids[DI_MAX_K];
  __shared__ float xk[DI_MAX_K], sm[DT_THREADS / 32], sS[DT_THREADS / 32];
  const int r = blockIdx.x, tid = threadIdx.x, K = a.K;
  const typename TY::raw* row = static_cast<const typename TY::raw*>(a.logits) + (size_t)r * a.ld;
  const uint32_t* bm = a.bitmask ? a.bitmask + (size_t)r * a.W : nullptr;
  auto legal = [&](int j) { return !bm || ((bm[j >> 5] >> (j & 31)) & 1u); };
  const float T = a.temperature ? a.temperature[r] : 1.f;
  const int t = a.targets ? a.targets[r] : -1;
  int wrong = sc_temperature_ok(T) && t >= -1 && t < a.V ? 0 : DI_INVALID;
  const float s = sc_scale(wrong ? 1.f : T);
  for (int k = tid; k < K; k += DT_THREADS) {
    const int id = a.ids[(size_t)r * K + k];
    const bool in = id >= 0 && id < a.V;
    if (!in && id != -1) wrong |= DI_INVALID;
    ids[k] = in ? id : -1;
    xk[k] = in && legal(id) ? TY::value(row[id]) : -INFINITY;
  }
  const float xt = !wrong && t >= 0 && legal(t) ? TY::value(row[t]) : -INFINITY;
  __syncthreads();
  for (int k = tid; k < K; k += DT_THREADS)
    for (int i = 0; i < k; ++i)
      if (ids[k] >= 0 && ids[i] == ids[k]) wrong |= DI_INVALID;
  Soft st{-INFINITY, 0.f, 0.f};
  for (int j = tid; j < a.V; j += DT_THREADS) {
    if (!legal(j)) continue;
    bool member = false;
    for (int k = 0; k < K; ++k) member |= ids[k] == j;
    if (member) continue;
    const float x = TY::value(row[j]);
    if (!(x < INFINITY)) wrong |= DI_NONFINITE;
    sc_add(st, x, s);
  }
  st = sc_warp_merge(st, s);
  if ((tid & 31) == 0) {
    sm[tid / 32] = st.m;
    sS[tid / 32] = st.S;
  }
  int all = 0;
  if (__syncthreads_or(wrong & DI_INVALID)) all |= DI_INVALID;
  if (__syncthreads_or(wrong & DI_NONFINITE)) all |= DI_NONFINITE;
  if (tid >= 32) return;
  st = tid < DT_THREADS / 32 ? Soft{sm[tid], sS[tid], 0.f} : Soft{-INFINITY, 0.f, 0.f};
  st = sc_warp_merge(st, s);
  distill_finish(a, r, T, t, xt, all, st.m, st.S, ids, xk);
}

}  // namespace

int distill_enqueue(const DistillArgs& a, int dtype, cudaStream_t st) {
  switch (dtype) {
    case SMP_F32: distill_kernel<SMP_F32><<<a.B, DT_THREADS, 0, st>>>(a); break;
    case SMP_BF16: distill_kernel<SMP_BF16><<<a.B, DT_THREADS, 0, st>>>(a); break;
    default: distill_kernel<SMP_F16><<<a.B, DT_THREADS, 0, st>>>(a); break;
  }
  return sc_ok(cudaGetLastError()) ? SMP_OK : SMP_ERR_CUDA;
}

}  // namespace smp
