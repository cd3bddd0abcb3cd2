// smp_process.cu -- penalties for repeated tokens, biases and grammar masks on
// logits (smp_process_logits).
//
// A CTA takes a segment of a row.  It counts the history's tokens that fall into
// its segment in shared memory (one word a token: copies among the generated
// tokens, and whether the token was seen or has a bias), copies the segment with
// its mask, and then rewrites the tokens that were counted from their raw logits.
// In place the copy is left out: only masked and counted tokens are touched.
#include "smp_train.cuh"

namespace smp {
namespace {

constexpr int PT = 256;        // threads
constexpr int PSEG = 8192;     // tokens of a segment
constexpr uint32_t PSEEN = 0x80000000u, PBIAS = 0x40000000u, PCOUNT = 0x3fffffffu;

template <int DT, int OT>
__global__ void __launch_bounds__(PT) process_kernel(const ProcessArgs a, const int nc, const bool in_place) {
  using TI = ScType<DT>;
  using TO = ScType<OT>;
  __shared__ uint32_t count[PSEG];
  const int r = blockIdx.x / nc, c = blockIdx.x % nc, tid = threadIdx.x;
  const int j0 = c * PSEG, j1 = min(a.V, j0 + PSEG);
  const typename TI::raw* row = static_cast<const typename TI::raw*>(a.logits) + (size_t)r * a.ld;
  typename TO::raw* out = static_cast<typename TO::raw*>(a.out) + (size_t)r * a.old;
  const uint32_t* bm = a.bitmask ? a.bitmask + (size_t)r * a.W : nullptr;
  const int32_t* history = a.history + (size_t)r * a.hld;
  const int32_t* bias_ids = a.bias_ids + (size_t)r * a.NB;
  const float* bias = a.bias + (size_t)r * a.NB;
  const float theta = a.repetition ? a.repetition[r] : 1.f;
  const float presence = a.presence ? a.presence[r] : 0.f, frequency = a.frequency ? a.frequency[r] : 0.f;
  const int length = a.lengths ? a.lengths[r] : a.H, prompt = a.prompts ? a.prompts[r] : 0;
  bool bad = !(theta > 0.f && theta < INFINITY && fabsf(presence) < INFINITY && fabsf(frequency) < INFINITY &&
               length >= 0 && length <= a.H && prompt >= 0 && prompt <= length);
  for (int i = tid; i < PSEG; i += PT) count[i] = 0u;
  for (int i = tid; i < a.NB; i += PT)
    if ((unsigned)bias_ids[i] < (unsigned)a.V && !(bias[i] < INFINITY)) bad = true;
  bad = __syncthreads_or(bad);
  if (c == 0 && tid == 0) a.status[r] = bad ? SMP_ERR_INVALID_PARAM : SMP_OK;
  if (!bad) {
    for (int i = tid; i < length; i += PT) {
      const int t = history[i];
      if (t < j0 || t >= j1) continue;
      if (i < prompt) atomicOr(&count[t - j0], PSEEN);
      else atomicAdd(&count[t - j0], 1u);
    }
    for (int i = tid; i < a.NB; i += PT)
      if (bias_ids[i] >= j0 && bias_ids[i] < j1) atomicOr(&count[bias_ids[i] - j0], PBIAS);
  }
  __syncthreads();
  for (int j = j0 + tid; j < j1; j += PT) {
    const uint32_t n = count[j - j0];
    const bool masked = !bad && bm && !((bm[j >> 5] >> (j & 31)) & 1u);
    if (in_place && !n && !masked) continue;
    float v = TI::value(row[j]);
    if (v > -INFINITY || v != v) {
      if (n & ~PBIAS) {
        v = v > 0.f ? __fdiv_rn(v, theta) : __fmul_rn(v, theta);
        const float copies = (float)(n & PCOUNT);
        v = __fsub_rn(v, __fadd_rn(__fmul_rn(frequency, copies), copies > 0.f ? presence : 0.f));
      }
      if (n & PBIAS) {
        for (int i = 0; i < a.NB; ++i)
          if (bias_ids[i] == j) v = bias[i] == -INFINITY || v == -INFINITY ? -INFINITY : __fadd_rn(v, bias[i]);
      }
    }
    out[j] = TO::store(masked ? -INFINITY : v);
  }
}

template <int DT, int OT>
int launch_process(const ProcessArgs& a, cudaStream_t st) {
  const int nc = (a.V + PSEG - 1) / PSEG;
  if ((long long)a.B * nc > 0x7fffffffLL) return SMP_ERR_CAPACITY;
  process_kernel<DT, OT><<<(unsigned)(a.B * nc), PT, 0, st>>>(a, nc, a.out == a.logits);
  return sc_ok(cudaGetLastError()) ? SMP_OK : SMP_ERR_CUDA;
}

}  // namespace

int process_enqueue(const ProcessArgs& a, int dtype, int out_dtype, cudaStream_t st) {
  if (dtype == SMP_F32) return launch_process<SMP_F32, SMP_F32>(a, st);
  if (dtype == SMP_BF16)
    return out_dtype == SMP_F32 ? launch_process<SMP_BF16, SMP_F32>(a, st) : launch_process<SMP_BF16, SMP_BF16>(a, st);
  return out_dtype == SMP_F32 ? launch_process<SMP_F16, SMP_F32>(a, st) : launch_process<SMP_F16, SMP_F16>(a, st);
}

}  // namespace smp
