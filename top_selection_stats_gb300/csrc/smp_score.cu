// smp_score.cu -- log probabilities of given tokens, entropy, rank and the n
// most likely alternatives (smp_token_logprobs).  One CTA per row: one pass
// for the softmax state and the rank, then one pass per alternative for the
// best token after the one before.
#include "smp_score.cuh"

namespace smp {
namespace {

constexpr int TT = 256;

// Order key: larger = earlier (larger logit, then smaller id); 0 = none.
__device__ __forceinline__ uint64_t order_key(float x, int id) {
  uint32_t b = __float_as_uint(x + 0.f);  // -0 folds onto +0
  b = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return ((uint64_t)b << 32) | (uint64_t)(0xffffffffu - (uint32_t)id);
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t b = (uint32_t)(k >> 32);
  return __uint_as_float((b & 0x80000000u) ? (b & 0x7fffffffu) : ~b);
}
__device__ __forceinline__ int key_id(uint64_t k) { return (int)(0xffffffffu - (uint32_t)k); }

template <int DT>
__global__ void __launch_bounds__(TT) score_kernel(const ScoreArgs a) {
  using TY = ScType<DT>;
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const typename TY::raw* row = static_cast<const typename TY::raw*>(a.logits) + (size_t)r * a.ld;
  const uint32_t* bm = a.bitmask ? a.bitmask + (size_t)r * a.W : nullptr;
  const float T = a.temperature ? a.temperature[r] : 1.f;
  const int t = a.targets ? a.targets[r] : -1;
  const bool valid = sc_temperature_ok(T) && t >= -1 && t < a.V;
  const float s = sc_scale(valid ? T : 1.f);
  auto logit = [&](int j) {
    return (!bm || ((bm[j >> 5] >> (j & 31)) & 1u)) ? TY::value(row[j]) : -INFINITY;
  };
  __shared__ Soft sw[TT / 32];
  __shared__ uint64_t kw[TT / 32];
  __shared__ int rw[TT / 32], bw[TT / 32];
  const float xt = valid && t >= 0 ? logit(t) : -INFINITY;
  Soft a0{-INFINITY, 0.f, 0.f};
  int ahead = 0, bad = 0;
  for (int j = tid; j < a.V; j += TT) {
    const float x = logit(j);
    if (!(x < INFINITY)) bad = 1;
    else if (x > -INFINITY) {
      sc_add(a0, x, s);
      ahead += (x > xt || (x == xt && j < t));
    }
  }
  for (int o = 16; o > 0; o >>= 1) {
    a0 = sc_merge(a0, sc_shfl_xor(a0, o), s);
    ahead += __shfl_xor_sync(0xffffffffu, ahead, o);
    bad |= __shfl_xor_sync(0xffffffffu, bad, o);
  }
  if (lane == 0) {
    sw[warp] = a0;
    rw[warp] = ahead;
    bw[warp] = bad;
  }
  __syncthreads();
  a0 = sw[0];
  ahead = rw[0];
  bad = bw[0];
  for (int w = 1; w < TT / 32; ++w) {
    a0 = sc_merge(a0, sw[w], s);
    ahead += rw[w];
    bad |= bw[w];
  }
  const int status = !valid ? SMP_ERR_INVALID_PARAM : bad ? SMP_ERR_NONFINITE
                     : a0.m == -INFINITY ? SMP_ERR_EMPTY : SMP_OK;
  if (tid == 0) {
    const bool ok = status == SMP_OK;
    a.status[r] = status;
    if (a.logprobs) a.logprobs[r] = !ok ? sc_nan() : t < 0 ? 0.f : sc_logprob(xt, a0, T);
    if (a.entropy) a.entropy[r] = ok ? sc_entropy(a0) : sc_nan();
    if (a.rank) a.rank[r] = ok && t >= 0 ? ahead : -1;
    if (a.stats) {
      a.stats[2 * (size_t)r] = ok ? a0.m : sc_nan();
      a.stats[2 * (size_t)r + 1] = ok ? SC_LN2 * sc_log2_mass(a0) : sc_nan();
    }
  }
  uint64_t last = ~0ull;
  for (int i = 0; i < a.n; ++i) {
    uint64_t best = 0ull;
    if (status == SMP_OK && last) {
      for (int j = tid; j < a.V; j += TT) {
        const float x = logit(j);
        const uint64_t k = x > -INFINITY ? order_key(x, j) : 0ull;
        if (k < last && k > best) best = k;
      }
    }
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t k = __shfl_xor_sync(0xffffffffu, best, o);
      best = k > best ? k : best;
    }
    __syncthreads();
    if (lane == 0) kw[warp] = best;
    __syncthreads();
    for (int w = 0; w < TT / 32; ++w) best = kw[w] > best ? kw[w] : best;
    last = best;
    if (tid == 0) {
      a.top_ids[(size_t)r * a.n + i] = best ? key_id(best) : -1;
      a.top_lp[(size_t)r * a.n + i] = status != SMP_OK ? sc_nan()
                                      : best ? sc_logprob(key_value(best), a0, T) : -INFINITY;
    }
  }
}

}  // namespace

int score_enqueue(const ScoreArgs& a, int dtype, cudaStream_t st) {
  switch (dtype) {
    case SMP_F32: score_kernel<SMP_F32><<<a.B, TT, 0, st>>>(a); break;
    case SMP_BF16: score_kernel<SMP_BF16><<<a.B, TT, 0, st>>>(a); break;
    default: score_kernel<SMP_F16><<<a.B, TT, 0, st>>>(a); break;
  }
  return cudaGetLastError() == cudaSuccess ? SMP_OK : SMP_ERR_CUDA;
}

}  // namespace smp
