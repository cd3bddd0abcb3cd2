// smp_train_api.cu -- argument checks of the processing and distillation calls
// declared in include/smp.h.  Nothing here allocates, synchronises or throws.
#include "smp_train.cuh"

using namespace smp;

namespace {
bool dtype_ok(int dt) { return dt == SMP_F32 || dt == SMP_BF16 || dt == SMP_F16; }
}  // namespace

extern "C" {

int smp_process_logits(const void* logits, smp_dtype dtype, int B, int V, int64_t ld,
                       const int32_t* history, int H, int64_t history_ld, const int32_t* lengths,
                       const int32_t* prompt_lengths, const float* repetition,
                       const float* presence, const float* frequency, const int32_t* bias_ids,
                       const float* bias, int NB, const uint32_t* bitmask, void* out,
                       smp_dtype out_dtype, int64_t out_ld, int32_t* row_status,
                       smp_stream stream) {
  if (!dtype_ok((int)dtype) || (out_dtype != dtype && (int)out_dtype != SMP_F32) || B < 0 || V < 1 || ld < V ||
      out_ld < V || H < 0 || history_ld < H || NB < 0)
    return SMP_ERR_INVALID_PARAM;
  if (V > SC_MAX_V || H > PR_MAX_H || NB > PR_MAX_NB) return SMP_ERR_CAPACITY;
  if (B == 0) return SMP_OK;
  if (!logits || !out || !row_status || (H > 0 && !history) || (NB > 0 && (!bias_ids || !bias)))
    return SMP_ERR_INVALID_PARAM;
  if (out == logits && (out_dtype != dtype || out_ld != ld)) return SMP_ERR_INVALID_PARAM;
  ProcessArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.history = history;
  a.hld = history_ld;
  a.lengths = lengths;
  a.prompts = prompt_lengths;
  a.repetition = repetition;
  a.presence = presence;
  a.frequency = frequency;
  a.bias_ids = bias_ids;
  a.bias = bias;
  a.bitmask = bitmask;
  a.out = out;
  a.old = out_ld;
  a.status = row_status;
  a.B = B;
  a.V = V;
  a.W = (V + 31) / 32;
  a.H = H;
  a.NB = NB;
  return process_enqueue(a, (int)dtype, (int)out_dtype, (cudaStream_t)stream);
}

int smp_distill_loss(const void* logits, smp_dtype dtype, int B, int V, int64_t ld,
                     const uint32_t* bitmask, const float* temperature, const int32_t* teacher_ids,
                     const float* teacher, int K, int kind, const int32_t* targets, float* loss,
                     float* logprobs, float* slot_logprobs, float* slot_grads, float* stats,
                     int32_t* row_status, smp_stream stream) {
  if (!dtype_ok((int)dtype) || B < 0 || V < 1 || ld < V || K < 1 || kind < SMP_DISTILL_FORWARD ||
      kind > SMP_DISTILL_TRUNCATED)
    return SMP_ERR_INVALID_PARAM;
  if (K > DI_MAX_K || V > SC_MAX_V) return SMP_ERR_CAPACITY;
  if (B == 0) return SMP_OK;
  if (!logits || !teacher_ids || !teacher || !loss || !row_status || (targets && !logprobs))
    return SMP_ERR_INVALID_PARAM;
  DistillArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.bitmask = bitmask;
  a.temperature = temperature;
  a.ids = teacher_ids;
  a.teacher = teacher;
  a.targets = targets;
  a.loss = loss;
  a.logprobs = logprobs;
  a.slot_lp = slot_logprobs;
  a.slot_g = slot_grads;
  a.stats = stats;
  a.status = row_status;
  a.B = B;
  a.V = V;
  a.W = (V + 31) / 32;
  a.K = K;
  a.kind = kind;
  a.wait_limit = scoring_wait_limit();
  cudaStream_t st = (cudaStream_t)stream;
  return dtype == SMP_F32 ? distill_f32(a, st) : dtype == SMP_BF16 ? distill_bf16(a, st) : distill_f16(a, st);
}

int smp_distill_loss_grad(const void* logits, smp_dtype dtype, int B, int V, int64_t ld,
                          const uint32_t* bitmask, const float* temperature,
                          const int32_t* teacher_ids, int K, const float* slot_logprobs,
                          const float* slot_grads, const float* stats, const float* grad_loss,
                          const int32_t* targets, const float* logprobs,
                          const float* grad_logprobs, void* grad, int64_t grad_ld,
                          smp_stream stream) {
  if (!dtype_ok((int)dtype) || B < 0 || V < 1 || ld < V || grad_ld < V || K < 1)
    return SMP_ERR_INVALID_PARAM;
  if (K > DI_MAX_K || V > SC_MAX_V) return SMP_ERR_CAPACITY;
  if (B == 0) return SMP_OK;
  if (!logits || !teacher_ids || !slot_grads || !stats || !grad ||
      (grad_logprobs && (!targets || !logprobs || !slot_logprobs)))
    return SMP_ERR_INVALID_PARAM;
  if (grad == logits && grad_ld != ld) return SMP_ERR_INVALID_PARAM;
  DistillGradArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.gld = grad_ld;
  a.bitmask = bitmask;
  a.temperature = temperature;
  a.ids = teacher_ids;
  a.slot_lp = slot_logprobs;
  a.slot_g = slot_grads;
  a.stats = stats;
  a.g_loss = grad_loss;
  a.targets = targets;
  a.logprobs = logprobs;
  a.g_lp = grad_logprobs;
  a.grad = grad;
  a.B = B;
  a.V = V;
  a.W = (V + 31) / 32;
  a.K = K;
  return distill_grad_enqueue(a, (int)dtype, (cudaStream_t)stream);
}

}  // extern "C"
