// smp_distill.cuh -- the mathematics of a row of smp_distill_loss, from the softmax
// state of the tokens outside the slots and the slots' own logits.
//
// The mass outside the slots, s, is summed apart from theirs, never as 1 minus
// their sum: a student that puts all but 1e-6 on the teacher's tokens loses no bits
// of it.  With z = x / T, logarithms taken relative to the largest logit m:
//   L = log(mass), log p_k = (x_k - m) / T - L, log s = (m_r - m) / T + L_r - L.
// The loss's derivatives by z, for a slot and for a token j outside, rho_j its
// share of the mass there (bounded, whatever r / s is):
//   forward    p_k (Q + r) - q_k              rho_j (s (Q + r) - r)       Q = sum q
//   reverse    p_k (u_k - loss)               rho_j s (u_r - loss)
//              u_k = log p_k - log q_k, u_r = log s - log r
//   truncated  p_k Q - q_k                    rho_j s Q                   Q = 1 (0 without slots)
// r is 1 minus a sum that is often near 1: the q_k and their sum are taken in
// binary64 (one exponential a slot, off the path of the stream), since reverse
// losses take r's logarithm.
#pragma once

#include "smp_train.cuh"

namespace smp {
namespace {

__device__ __forceinline__ float di_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float di_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

enum { DI_INVALID = 1, DI_NONFINITE = 2, DI_LATE = 4 };

// A row's slots in shared memory.
struct Slots {
  int ids[DI_MAX_K];       // negative: unused
  float x[DI_MAX_K];       // the student's logit, -inf: not legal
  float teacher[DI_MAX_K];  // -inf in unused slots
};

// One warp: the row's results.  rest: the state of the legal tokens outside the
// slots; total: the sum of the teacher's probabilities (not truncated); xt: the target's
// logit (-inf: not legal); wrong: what was found so far.
__device__ __forceinline__ void distill_finish(const DistillArgs& a, int r, float T, int t, float xt, int wrong,
                                               float rest_m, float rest_S, const Slots& slots, double total) {
  const int* ids = slots.ids;
  const float *xk = slots.x, *teacher = slots.teacher;
  const int lane = threadIdx.x & 31, K = a.K;
  const size_t at = (size_t)r * K;
  const float s_scale = sc_scale(wrong & DI_INVALID ? 1.f : T);
  // the student
  float m = rest_m;
  for (int k = lane; k < K; k += 32) {
    if (!(xk[k] < INFINITY)) wrong |= DI_NONFINITE;
    m = fmaxf(m, xk[k]);
  }
  m = di_max(m);
  float S = 0.f;
  for (int k = lane; k < K; k += 32) S += xk[k] == -INFINITY ? 0.f : sc_ex2((xk[k] - m) * s_scale);
  S = di_sum(S);
  const bool bare = rest_m == -INFINITY;  // no legal token outside the slots
  if (!bare) S += rest_S * sc_ex2((rest_m - m) * s_scale);
  const float L = SC_LN2 * log2f(S), Lr = SC_LN2 * log2f(rest_S);
  const float log_s = bare ? -INFINITY : fminf(__fdiv_rn(rest_m - m, T) + (Lr - L), 0.f);
  const float mass = bare ? 0.f : expf(log_s);
  // the teacher
  float top = -INFINITY, size = 0.f;
  float Q, rest = 0.f, log_size = 0.f;
  if (a.kind == SMP_DISTILL_TRUNCATED) {
    for (int k = lane; k < K; k += 32) top = fmaxf(top, teacher[k]);
    top = di_max(top);
    for (int k = lane; k < K; k += 32)
      if (teacher[k] > -INFINITY) size += expf(__fdiv_rn(teacher[k] - top, T));
    size = di_sum(size);
    log_size = logf(size);
    Q = top > -INFINITY ? 1.f : 0.f;
  } else {
    if (total > DI_MOST) wrong |= DI_INVALID;
    Q = (float)total;
    if (!bare) rest = fmaxf((float)(1.0 - total), DI_LEAST);
  }
  const float log_r = logf(rest);
  wrong = __reduce_or_sync(0xffffffffu, wrong);
  const int status = wrong & DI_LATE        ? SMP_ERR_TIMEOUT
                     : wrong & DI_INVALID   ? SMP_ERR_INVALID_PARAM
                     : wrong & DI_NONFINITE ? SMP_ERR_NONFINITE
                     : m == -INFINITY       ? SMP_ERR_EMPTY
                                            : SMP_OK;
  const bool ok = status == SMP_OK;
  auto slot = [&](int k, float& lp, float& p, float& lq, float& q) {
    lp = xk[k] == -INFINITY ? -INFINITY : fminf(__fdiv_rn(xk[k] - m, T) - L, 0.f);
    p = expf(lp);
    lq = teacher[k];
    if (a.kind == SMP_DISTILL_TRUNCATED && lq > -INFINITY) lq = __fdiv_rn(lq - top, T) - log_size;
    q = expf(lq);
  };
  float loss = 0.f;
  for (int k = lane; ok && k < K; k += 32) {
    float lp, p, lq, q;
    slot(k, lp, p, lq, q);
    const float w = a.kind == SMP_DISTILL_REVERSE ? p : q;
    if (w > 0.f) loss += a.kind == SMP_DISTILL_REVERSE ? p * (lp - lq) : q * (lq - lp);
  }
  loss = di_sum(loss);
  if (rest > 0.f) {
    if (a.kind == SMP_DISTILL_REVERSE) loss += mass > 0.f ? mass * (log_s - log_r) : 0.f;
    else loss += rest * (log_r - log_s);
  }
  const bool finite = fabsf(loss) < INFINITY;
  float A = 0.f;
  if (finite) {
    if (a.kind == SMP_DISTILL_REVERSE) A = mass > 0.f ? mass * (log_s - log_r - loss) : 0.f;
    else A = mass * (Q + rest) - rest;
  }
  if (a.slot_lp || a.slot_g) {
    for (int k = lane; k < K; k += 32) {
      float lp, p, lq, q, g = 0.f;
      slot(k, lp, p, lq, q);
      if (ids[k] >= 0 && finite) {
        if (a.kind == SMP_DISTILL_REVERSE) g = p > 0.f ? p * (lp - lq - loss) : 0.f;
        else g = p * (Q + rest) - q;
      }
      if (a.slot_lp) a.slot_lp[at + k] = ok ? lp : sc_nan();
      if (a.slot_g) a.slot_g[at + k] = ok ? g : sc_nan();
    }
  }
  if (lane) return;
  a.status[r] = status;
  a.loss[r] = ok ? loss : sc_nan();
  if (a.targets) a.logprobs[r] = !ok ? sc_nan() : t < 0 ? 0.f : sc_logprob(xt, m, L, T);
  if (a.stats) {
    float* o = a.stats + 4 * (size_t)r;
    o[0] = ok ? rest_m : sc_nan();
    o[1] = ok ? Lr : sc_nan();
    o[2] = ok ? A : sc_nan();
    o[3] = ok ? mass : sc_nan();
  }
}

}  // namespace
}  // namespace smp
