// smp_head.cu -- log probabilities and entropy straight from hidden states and
// the output head's weights (smp_head_logprobs).  Phase 1: a CTA takes 64 rows
// and a chunk of the vocabulary, forms 64 x 64 tiles of logits from shared
// memory and folds them into the rows' softmax states; the state and the
// target's logit, if the chunk holds it, go to the workspace.  Phase 2 joins
// the chunks of a row.
#include "smp_score.cuh"

namespace smp {
namespace {

constexpr int HM = 64, HN = 64, HK = 32;
constexpr int HCHUNK = 1024;  // tokens a workspace entry stands for

int chunks_of(int V) { return (V + HCHUNK - 1) / HCHUNK; }

template <int DT>
__global__ void __launch_bounds__(256) head_kernel(const HeadArgs a) {
  using TY = ScType<DT>;
  __shared__ float sa[HK][HM + 1], sb[HK][HN + 1], sx[HM][HN + 1];
  const int r0 = blockIdx.x * HM, chunk = blockIdx.y, tid = threadIdx.x;
  const int ty = tid / 16, tx = tid % 16;
  const unsigned short* hid = static_cast<const unsigned short*>(a.hidden);
  const unsigned short* wei = static_cast<const unsigned short*>(a.weight);
  const int v1 = min(a.V, (chunk + 1) * HCHUNK);
  const int row = r0 + tid;
  const bool mine = tid < HM && row < a.N;
  const float T = mine && a.temperature ? a.temperature[row] : 1.f;
  const float s = sc_scale(sc_temperature_ok(T) ? T : 1.f);
  const int t = mine && a.targets ? a.targets[row] : -1;
  Soft st{-INFINITY, 0.f, 0.f};
  float xt = -INFINITY;
  bool bad = false;
  for (int v0 = chunk * HCHUNK; v0 < v1; v0 += HN) {
    float acc[4][4] = {};
    for (int k0 = 0; k0 < a.D; k0 += HK) {
      __syncthreads();
      for (int i = tid; i < HM * HK; i += 256) {
        const int k = i % HK, m = i / HK;
        const bool in = k0 + k < a.D;
        sa[k][m] = in && r0 + m < a.N ? TY::value(hid[(size_t)(r0 + m) * a.ldh + k0 + k]) : 0.f;
        sb[k][m] = in && v0 + m < a.V ? TY::value(wei[(size_t)(v0 + m) * a.ldw + k0 + k]) : 0.f;
      }
      __syncthreads();
      for (int k = 0; k < HK; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ty * 4 + i], sb[k][tx * 4 + j], acc[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sx[ty * 4 + i][tx * 4 + j] = acc[i][j];
    __syncthreads();
    if (mine) {
      for (int j = 0; j < HN && v0 + j < v1; ++j) {
        const float x = sx[tid][j];
        if (!(x < INFINITY)) bad = true;
        else if (x > -INFINITY) sc_add(st, x, s);
        if (v0 + j == t) xt = x;
      }
    }
  }
  if (mine) {
    if (bad) st.m = INFINITY;
    a.part[(size_t)chunk * a.N + row] = make_float4(st.m, st.S, st.U, xt);
  }
}

__global__ void __launch_bounds__(128) head_join(const HeadArgs a, int chunks) {
  const int row = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= a.N) return;
  const float T = a.temperature ? a.temperature[row] : 1.f;
  const int t = a.targets ? a.targets[row] : -1;
  const bool valid = sc_temperature_ok(T) && t >= -1 && t < a.V;
  const float s = sc_scale(valid ? T : 1.f);
  Soft st{-INFINITY, 0.f, 0.f};
  float xt = -INFINITY;
  bool bad = false;
  for (int c = lane; c < chunks; c += 32) {
    const float4 p = a.part[(size_t)c * a.N + row];
    if (p.x == INFINITY) bad = true;
    else st = sc_merge(st, Soft{p.x, p.y, p.z}, s);
    xt = fmaxf(xt, p.w);
  }
  for (int o = 16; o > 0; o >>= 1) {
    st = sc_merge(st, sc_shfl_xor(st, o), s);
    xt = fmaxf(xt, __shfl_xor_sync(0xffffffffu, xt, o));
  }
  bad = __any_sync(0xffffffffu, bad);
  if (lane) return;
  const int status = !valid ? SMP_ERR_INVALID_PARAM : bad ? SMP_ERR_NONFINITE
                     : st.m == -INFINITY ? SMP_ERR_EMPTY : SMP_OK;
  const bool ok = status == SMP_OK;
  a.status[row] = status;
  if (a.logprobs) a.logprobs[row] = !ok ? sc_nan() : t < 0 ? 0.f : sc_logprob(xt, st, T);
  if (a.entropy) a.entropy[row] = ok ? sc_entropy(st) : sc_nan();
  if (a.stats) {
    a.stats[2 * (size_t)row] = ok ? st.m : sc_nan();
    a.stats[2 * (size_t)row + 1] = ok ? SC_LN2 * sc_log2_mass(st) : sc_nan();
  }
}

}  // namespace

int64_t head_workspace(int N, int V) { return (int64_t)chunks_of(V) * N * (int64_t)sizeof(float4); }

int head_enqueue(const HeadArgs& a, int dtype, cudaStream_t st) {
  const int chunks = chunks_of(a.V);
  const dim3 grid((a.N + HM - 1) / HM, chunks);
  if (dtype == SMP_BF16) head_kernel<SMP_BF16><<<grid, 256, 0, st>>>(a);
  else head_kernel<SMP_F16><<<grid, 256, 0, st>>>(a);
  head_join<<<(a.N + 3) / 4, 128, 0, st>>>(a, chunks);
  return cudaGetLastError() == cudaSuccess ? SMP_OK : SMP_ERR_CUDA;
}

}  // namespace smp
