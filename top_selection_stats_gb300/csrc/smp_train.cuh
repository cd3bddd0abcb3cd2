// smp_train.cuh -- arguments and entry points of the processing and distillation
// calls (smp_process.cu, smp_distill_kernel.cuh, smp_distill_grad.cu,
// smp_train_api.cu).
#pragma once

#include "smp_score.cuh"

namespace smp {

constexpr int DI_MAX_K = 256;         // slots of a teacher
constexpr int PR_MAX_H = 1 << 24;     // history entries: counts are exact in binary32
constexpr int PR_MAX_NB = 4096;       // biases of a row
constexpr float DI_LEAST = 0x1p-24f;  // the teacher's mass outside its slots, at least
constexpr double DI_MOST = 1.0 + 0x1p-10;  // the sum of a teacher's probabilities, at most

struct ProcessArgs {
  const void* logits;
  long long ld;
  const int32_t* history;
  long long hld;
  const int32_t *lengths, *prompts;
  const float *repetition, *presence, *frequency;
  const int32_t* bias_ids;
  const float* bias;
  const uint32_t* bitmask;
  void* out;
  long long old;
  int32_t* status;
  int B, V, W, H, NB;
};
struct DistillArgs {
  const void* logits;
  long long ld;
  const uint32_t* bitmask;
  const float* temperature;
  const int32_t* ids;
  const float* teacher;
  const int32_t* targets;
  float *loss, *logprobs, *slot_lp, *slot_g, *stats;
  int32_t* status;
  int B, V, W, K, kind;
  long long wait_limit;
};
struct DistillGradArgs {
  const void* logits;
  long long ld, gld;
  const uint32_t* bitmask;
  const float* temperature;
  const int32_t* ids;
  const float *slot_lp, *slot_g, *stats, *g_loss;
  const int32_t* targets;
  const float *logprobs, *g_lp;
  void* grad;
  int B, V, W, K;
};

// 16 bytes that start `off` bytes into p[0] (0: p[0] itself, and p[1] is not read).
__device__ __forceinline__ uint4 vector_across(const uint4* p, int off) {
  const uint4 a = p[0], b = off ? p[1] : a;
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t y[5];
  const int k = off >> 2, bits = (off & 3) * 8;
#pragma unroll
  for (int i = 0; i < 5; ++i) y[i] = k == 0 ? w[i] : k == 1 ? w[i + 1] : k == 2 ? w[i + 2] : w[min(i + 3, 7)];
  return make_uint4(__funnelshift_r(y[0], y[1], bits), __funnelshift_r(y[1], y[2], bits),
                    __funnelshift_r(y[2], y[3], bits), __funnelshift_r(y[3], y[4], bits));
}

int process_enqueue(const ProcessArgs& a, int dtype, int out_dtype, cudaStream_t st);
int distill_f32(const DistillArgs& a, cudaStream_t st);
int distill_bf16(const DistillArgs& a, cudaStream_t st);
int distill_f16(const DistillArgs& a, cudaStream_t st);
int distill_grad_enqueue(const DistillGradArgs& a, int dtype, cudaStream_t st);

// The bound that smp_set_scoring_wait_limit holds (smp_score_api.cu).
long long scoring_wait_limit();

}  // namespace smp
