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
// binary64, since reverse losses take r's logarithm.  That is an exponential a slot and
// five additions of lanes for each 32 slots on few binary64 units: under the stream where
// rows are long and slots few, on the row's path otherwise (912 x 128256 takes 43 us with 64
// slots, 63 with 256).
//
// What binary32 costs elsewhere: s = log2(e) / T is rounded once, so that all masses are those
// of a temperature within half a unit of T, which moves L by up to 2^-24 times the mean of |z|;
// a mass is a sum of powers good to 2 units; and a slot's log p is a quotient relative to its
// part's largest logit plus the part's own, two more roundings.  Against 64-bit definitions the
// outputs are off by 2e-7 to 6e-7 (root of the mean square, relative), those of elementary
// binary32 operations with a quotient for each logit by 3e-7 to 4e-7.
#pragma once

#include "smp_train.cuh"

namespace smp {
namespace {

enum { DI_INVALID = 1, DI_NONFINITE = 2, DI_LATE = 4, DI_APART = 8 };  // the last: a slot with lost or over
// A slot's weight is 0 when its logarithm is below this, the least that binary64 has.
constexpr float DI_LEAST_LOG = -745.1332f;

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

// What 32 slots come to, relative to their own largest logit m and teacher value top (0
// where the teacher's values are log probabilities): with d = (x - m) / T, w = 2^((x - m) s),
// y = (teacher - top) (/ T if truncated), e = exp(y),
//   mass = sum w, teach = sum e, and cross, the mean of (y - d) / 2 under e (forward, truncated)
//   or of (d - y) / 2 under w (reverse): halves, as a mean of values at the end of binary32
//   may round past it.
// Terms that are infinite unless their weight in the row is 0 are kept apart, as that is not
// known here: lost is the largest logarithm, relative to m or top, of the weight of a slot that
// the other side does not have, over the largest weight of one whose d has passed binary32.
struct SlotPart {
  float m, mass, top, teach, cross, lost, over;
  int wrong;
  double total;  // sum e in binary64 (not truncated)
};
// A row's slots in shared memory.
struct Slots {
  int ids[DI_MAX_K];     // negative: unused
  float x[DI_MAX_K], d[DI_MAX_K], y[DI_MAX_K], e[DI_MAX_K];
  SlotPart part[DI_MAX_K / 32];
};

// One warp, its lane's slot k0 + lane: fills slots, but for the ids.  id: -1 unused; x:
// -inf not legal; v: the teacher's value.
__device__ __forceinline__ void distill_slots(const DistillArgs& a, Slots& slots, int k0, int id, float x, float v,
                                              float T, float s) {
  const int lane = threadIdx.x & 31;
  const bool truncated = a.kind == SMP_DISTILL_TRUNCATED, reverse = a.kind == SMP_DISTILL_REVERSE;
  SlotPart p;
  p.wrong = 0;
  if (id < 0) v = -INFINITY;
  if (!(x < INFINITY) || !(v < INFINITY)) {
    p.wrong = DI_NONFINITE;
    x = v = -INFINITY;
  }
  p.m = di_max(x);
  p.top = truncated ? di_max(v) : 0.f;
  const bool legal = x > -INFINITY, taught = v > -INFINITY;
  float w = legal ? sc_ex2((x - p.m) * s) : 0.f;
  // 2^x flushes results below 2^-126, which a teacher's lowest finite values weigh up
  if (reverse && legal && w == 0.f) w = __fmul_rn(sc_ex2((x - p.m) * s + 64.f), 0x1p-64f);
  const float d = legal ? __fdiv_rn(x - p.m, T) : -INFINITY;
  const float y = !taught ? -INFINITY : truncated ? __fdiv_rn(v - p.top, T) : v;
  float e = 0.f;
  p.total = 0.0;
  if (truncated) {
    e = taught ? expf(y) : 0.f;
  } else {
    p.total = taught ? exp((double)v) : 0.0;
    e = (float)p.total;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) p.total += __shfl_xor_sync(0xffffffffu, p.total, o);
  }
  p.mass = di_sum(w);
  p.teach = di_sum(e);
  const float weight = reverse ? w : e;
  float cross = 0.f;
  p.lost = -INFINITY;
  p.over = 0.f;
  if (reverse ? legal && !taught : taught && !legal) {
    p.wrong |= DI_APART;
    p.lost = reverse ? d : y;
  } else if (weight > 0.f) {
    cross = __fdiv_rn(weight, reverse ? p.mass : p.teach) * (reverse ? 0.5f * d - 0.5f * y : 0.5f * y - 0.5f * d);
    if (!(cross < INFINITY)) {
      p.wrong |= DI_APART;
      p.over = weight;
      cross = 0.f;
    }
  }
  p.cross = di_sum(cross);
  p.wrong = __reduce_or_sync(0xffffffffu, p.wrong);
  if (p.wrong & DI_APART) {
    p.lost = di_max(p.lost);
    p.over = di_max(p.over);
  }
  slots.x[k0 + lane] = x;
  slots.d[k0 + lane] = d;
  slots.y[k0 + lane] = y;
  slots.e[k0 + lane] = e;
  if (lane == 0) slots.part[k0 / 32] = p;
}

// What the slots of each part need of the row: log p = d + shift, q = scale e.
struct RowResult {
  float shift[DI_MAX_K / 32], scale[DI_MAX_K / 32];
  float loss, weight;  // weight: Q + r
  int ok, finite;
};

// One warp: the row's results, and in `o` what its slots' need.  rest: the state of the legal
// tokens outside the slots; xt: the target's logit (-inf: not legal); wrong: what was found
// so far.
__device__ __forceinline__ void distill_finish(const DistillArgs& a, int r, float T, float s, int t, float xt, int wrong,
                                               float rest_m, float rest_S, const Slots& slots, RowResult& o) {
  const int lane = threadIdx.x & 31, parts = (a.K + 31) / 32;
  const bool reverse = a.kind == SMP_DISTILL_REVERSE, truncated = a.kind == SMP_DISTILL_TRUNCATED;
  SlotPart p{-INFINITY, 0.f, truncated ? -INFINITY : 0.f, 0.f, 0.f, -INFINITY, 0.f, 0, 0.0};
  if (lane < parts) p = slots.part[lane];
  wrong |= p.wrong;
  // the student: lane `parts` has what is outside the slots
  const bool bare = rest_m == -INFINITY;  // no legal token there
  const float own_m = lane == parts ? rest_m : p.m, own_S = lane == parts ? rest_S : p.mass;
  const float m = di_max(own_m);
  const float S = di_sum(own_m == -INFINITY ? 0.f : own_S * sc_ex2((own_m - m) * s));
  const float L = SC_LN2 * log2f(S), Lr = SC_LN2 * log2f(rest_S);
  const float shift = own_m == -INFINITY ? -INFINITY : __fdiv_rn(own_m - m, T) - L;
  const float log_s = bare ? -INFINITY : fminf(__shfl_sync(0xffffffffu, shift, parts) + Lr, 0.f);
  const float mass = bare ? 0.f : expf(log_s);
  // the teacher
  float Q, rest = 0.f, taught = 0.f, scale = 1.f;
  if (truncated) {
    const float top = di_max(p.top);
    const float c = p.top > -INFINITY ? expf(__fdiv_rn(p.top - top, T)) : 0.f, size = di_sum(p.teach * c);
    Q = top > -INFINITY ? 1.f : 0.f;
    scale = Q > 0.f ? __fdiv_rn(c, size) : 0.f;
    taught = p.top > -INFINITY ? __fdiv_rn(p.top - top, T) - logf(size) : 0.f;
  } else {
    double total = 0.0;
    for (int k = 0; k < parts; ++k) total += slots.part[k].total;
    if (total > DI_MOST) wrong |= DI_INVALID;
    Q = (float)total;
    if (!bare) rest = fmaxf((float)(1.0 - total), DI_LEAST);
  }
  wrong = __reduce_or_sync(0xffffffffu, wrong);
  const int status = wrong & DI_LATE        ? SMP_ERR_TIMEOUT
                     : wrong & DI_INVALID   ? SMP_ERR_INVALID_PARAM
                     : wrong & DI_NONFINITE ? SMP_ERR_NONFINITE
                     : m == -INFINITY       ? SMP_ERR_EMPTY
                                            : SMP_OK;
  const bool ok = status == SMP_OK;
  // the slots' part of the loss
  float loss = 0.f;
  const float by = reverse ? expf(shift) : scale;
  if (lane < parts) {
    const float q = by * (reverse ? p.mass : p.teach);  // the part's weight
    if (q > 0.f) loss = q * (p.cross + 0.5f * (reverse ? shift : p.m > -INFINITY ? taught - shift : 0.f));
  }
  loss = di_sum(loss);
  loss = loss > 0x1p127f && loss < 0x1.00001p127f ? 0x1.fffffep127f : 2.f * loss;
  const float log_r = logf(rest);
  if (rest > 0.f) {
    if (reverse) loss += mass > 0.f ? mass * (log_s - log_r) : 0.f;
    else loss += rest * (log_r - log_s);
  }
  if (wrong & DI_APART) {  // of some part; infinite with a weight above 0
    const bool counts = lane < parts && (p.lost + (reverse ? shift : taught) >= DI_LEAST_LOG || by * p.over > 0.f);
    if (__any_sync(0xffffffffu, counts)) loss = INFINITY;
  }
  const bool finite = fabsf(loss) < INFINITY;
  float A = 0.f;
  if (finite) {
    if (reverse) A = mass > 0.f ? mass * (log_s - log_r - loss) : 0.f;
    else A = mass * (Q + rest) - rest;
  }
  if (lane < parts) {
    o.shift[lane] = shift;
    o.scale[lane] = scale;
  }
  if (lane) return;
  o.loss = loss;
  o.weight = Q + rest;
  o.ok = ok;
  o.finite = finite;
  a.status[r] = status;
  a.loss[r] = ok ? loss : sc_nan();
  if (a.targets) a.logprobs[r] = !ok ? sc_nan() : t < 0 ? 0.f : sc_logprob(xt, m, L, T);
  if (a.stats) {
    float* to = a.stats + 4 * (size_t)r;
    to[0] = ok ? rest_m : sc_nan();
    to[1] = ok ? Lr : sc_nan();
    to[2] = ok ? A : sc_nan();
    to[3] = ok ? mass : sc_nan();
  }
}

// A slot's outputs.
__device__ __forceinline__ void distill_slot(const DistillArgs& a, int r, int k, const Slots& slots, const RowResult& o) {
  const float lp = slots.x[k] > -INFINITY ? fminf(slots.d[k] + o.shift[k / 32], 0.f) : -INFINITY, p = expf(lp);
  float g = 0.f;
  if (slots.ids[k] >= 0 && o.finite) {
    if (a.kind == SMP_DISTILL_REVERSE) g = p > 0.f ? p * (lp - slots.y[k] - o.loss) : 0.f;
    else g = p * o.weight - slots.e[k] * o.scale[k / 32];
  }
  const size_t at = (size_t)r * a.K + k;
  if (a.slot_lp) a.slot_lp[at] = o.ok ? lp : sc_nan();
  if (a.slot_g) a.slot_g[at] = o.ok ? g : sc_nan();
}

}  // namespace
}  // namespace smp
