// smp_score_api.cu -- argument checks of the scoring calls declared in
// include/smp.h, and the bound on their waits.  Nothing here allocates,
// synchronises or throws.
#include <atomic>
#include <cstdint>

#include "smp_score.cuh"

using namespace smp;

namespace {
bool dtype_ok(int dt) { return dt == SMP_F32 || dt == SMP_BF16 || dt == SMP_F16; }
bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
constexpr int HEAD_MAX = 1 << 20;
std::atomic<long long> g_wait_limit{SC_WAIT};
}  // namespace

extern "C" {

int smp_token_logprobs(const void* logits, smp_dtype dtype, int B, int V, int64_t ld,
                       const uint32_t* bitmask, const float* temperature, const int32_t* targets,
                       float* logprobs, float* entropy, int32_t* rank, float* stats,
                       int32_t* row_status, int n, int32_t* top_ids, float* top_logprobs,
                       smp_stream stream) {
  if (!dtype_ok((int)dtype) || B < 0 || V < 1 || ld < V || n < 0) return SMP_ERR_INVALID_PARAM;
  if (n > SC_MAX_TOP || V > SC_MAX_V) return SMP_ERR_CAPACITY;
  if (B == 0) return SMP_OK;
  if (!logits || !row_status || (targets && !logprobs) || (n > 0 && (!top_ids || !top_logprobs)))
    return SMP_ERR_INVALID_PARAM;
  ScoreArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.bitmask = bitmask;
  a.temperature = temperature;
  a.targets = targets;
  a.logprobs = logprobs;
  a.entropy = entropy;
  a.stats = stats;
  a.rank = rank;
  a.status = row_status;
  a.top_ids = top_ids;
  a.top_lp = top_logprobs;
  a.B = B;
  a.V = V;
  a.W = (V + 31) / 32;
  a.n = n;
  a.wait_limit = g_wait_limit.load(std::memory_order_relaxed);
  cudaStream_t st = (cudaStream_t)stream;
  return dtype == SMP_F32 ? score_f32(a, st) : dtype == SMP_BF16 ? score_bf16(a, st) : score_f16(a, st);
}

int smp_token_logprobs_grad(const void* logits, smp_dtype dtype, int B, int V, int64_t ld,
                            const uint32_t* bitmask, const float* temperature,
                            const int32_t* targets, const float* stats, const float* entropy,
                            const float* grad_logprobs, const float* grad_entropy, void* grad,
                            int64_t grad_ld, smp_stream stream) {
  if (!dtype_ok((int)dtype) || B < 0 || V < 1 || ld < V || grad_ld < V)
    return SMP_ERR_INVALID_PARAM;
  if (V > SC_MAX_V) return SMP_ERR_CAPACITY;
  if (B == 0) return SMP_OK;
  if (!logits || !stats || !grad || (grad_entropy && !entropy) || (grad_logprobs && !targets))
    return SMP_ERR_INVALID_PARAM;
  if (grad == logits && grad_ld != ld) return SMP_ERR_INVALID_PARAM;
  GradArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.gld = grad_ld;
  a.bitmask = bitmask;
  a.temperature = temperature;
  a.targets = targets;
  a.stats = stats;
  a.entropy = entropy;
  a.g_lp = grad_logprobs;
  a.g_ent = grad_entropy;
  a.grad = grad;
  a.B = B;
  a.V = V;
  a.W = (V + 31) / 32;
  return grad_enqueue(a, (int)dtype, (cudaStream_t)stream);
}

int smp_head_logprobs(const void* hidden, int64_t ld_hidden, const void* weight,
                      int64_t ld_weight, smp_dtype dtype, int N, int V, int D,
                      const float* temperature, const int32_t* targets, float* logprobs,
                      float* entropy, float* stats, int32_t* row_status, void* workspace,
                      int64_t workspace_bytes, smp_stream stream) {
  if ((int)dtype != SMP_BF16 && (int)dtype != SMP_F16) return SMP_ERR_INVALID_PARAM;
  if (N < 0 || V < 1 || D < 1 || ld_hidden < D || ld_weight < D || (ld_hidden & 7) ||
      (ld_weight & 7))
    return SMP_ERR_INVALID_PARAM;
  if (V > SC_MAX_V || N > HEAD_MAX || D > HEAD_MAX) return SMP_ERR_CAPACITY;
  if (N == 0) return SMP_OK;
  if (!hidden || !weight || !row_status || !workspace || (targets && !logprobs))
    return SMP_ERR_INVALID_PARAM;
  if (misaligned(hidden) || misaligned(weight) || misaligned(workspace) ||
      workspace_bytes < head_workspace(N, V))
    return SMP_ERR_INVALID_PARAM;
  HeadArgs a{};
  a.hidden = hidden;
  a.weight = weight;
  a.ldh = ld_hidden;
  a.ldw = ld_weight;
  a.temperature = temperature;
  a.targets = targets;
  a.logprobs = logprobs;
  a.entropy = entropy;
  a.stats = stats;
  a.status = row_status;
  a.part = static_cast<float4*>(workspace);
  a.N = N;
  a.V = V;
  a.D = D;
  a.wait_limit = g_wait_limit.load(std::memory_order_relaxed);
  return head_enqueue(a, (int)dtype, (cudaStream_t)stream);
}

int smp_set_scoring_wait_limit(long long cycles) {
  g_wait_limit.store(cycles > 0 ? cycles : SC_WAIT, std::memory_order_relaxed);
  return SMP_OK;
}

int64_t smp_head_workspace(int N, int V) { return N < 1 || V < 1 ? 0 : head_workspace(N, V); }

}  // extern "C"
