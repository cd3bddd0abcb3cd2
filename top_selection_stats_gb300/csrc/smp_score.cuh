// smp_score.cuh -- what the scoring kernels (smp_score_kernel.cuh,
// smp_score_grad.cu, smp_head.cu) share: the softmax state of a set of values,
// its merge, the results computed from it, and bounded waits.
//
// A set A of values x with largest m, scaled by s = log2(e) / T, is held as
//     m,  S = sum 2^d,  U = sum 2^d d,   d = (x - m) s <= 0,
// in binary32.  From it L = ln 2 log2 S and the entropy, ln 2 (log2 S - U/S),
// a sum of two terms that are both >= 0, so nothing cancels.  x - m is formed
// before the scaling: near the top, where the mass is, it is exact, so the
// results do not lose bits when all logits are far from 0.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/smp.h"

namespace smp {

constexpr float SC_LN2 = 0.6931471805599453f;
// d is clamped here before it is multiplied by 2^d: 2^d is 0 long before, and
// 0 times the d of an illegal token (-inf) would be NaN.
constexpr float SC_DMIN = -1.0e4f;
constexpr int SC_MAX_V = 1 << 24;
constexpr int SC_MAX_TOP = 32;
// SM cycles that a wait may take, unless a call is given fewer (about two seconds); what is
// in flight when one runs out is always given as long as this to land.
constexpr long long SC_WAIT = 4000000000ll;

__device__ __forceinline__ float sc_nan() { return __int_as_float(0x7fffffff); }

// A valid temperature is finite and > 0; its scale log2(e) / T is kept finite.
__device__ __forceinline__ bool sc_temperature_ok(float T) { return T > 0.f && T < INFINITY; }
__device__ __forceinline__ float sc_scale(float T) {
  return fminf(__fdiv_rn(1.4426950408889634f, T), 3.0e38f);
}

__device__ __forceinline__ float sc_ex2(float d) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(d));
  return y;
}

// Two binary32 values handled by one instruction.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(f32x2 r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

struct Soft {
  float m, S, U;
};

// One more value (x = -inf: none).
__device__ __forceinline__ void sc_add(Soft& a, float x, float s) {
  if (x > a.m) {
    const float d = a.m == -INFINITY ? SC_DMIN : fmaxf((a.m - x) * s, SC_DMIN);
    const float c = sc_ex2(d);
    a.U = (a.U + a.S * d) * c;
    a.S *= c;
    a.m = x;
  }
  const float d = x == -INFINITY ? SC_DMIN : fmaxf((x - a.m) * s, SC_DMIN);
  const float e = sc_ex2(d);
  a.S += e;
  a.U = fmaf(e, d, a.U);
}

// The state of the union of two sets.  An empty set has m = -inf, S = U = 0.
__device__ __forceinline__ Soft sc_merge(const Soft& a, const Soft& b, float s) {
  Soft r;
  r.m = fmaxf(a.m, b.m);
  if (r.m == -INFINITY) {
    r.S = 0.f;
    r.U = 0.f;
    return r;
  }
  const float da = fmaxf((a.m - r.m) * s, SC_DMIN), db = fmaxf((b.m - r.m) * s, SC_DMIN);
  const float ca = sc_ex2(da), cb = sc_ex2(db);
  r.S = a.S * ca + b.S * cb;
  r.U = (a.U + a.S * da) * ca + (b.U + b.S * db) * cb;
  return r;
}

__device__ __forceinline__ Soft sc_shfl_xor(const Soft& a, int o) {
  Soft b;
  b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
  b.S = __shfl_xor_sync(0xffffffffu, a.S, o);
  b.U = __shfl_xor_sync(0xffffffffu, a.U, o);
  return b;
}

// The warp's union, in every lane: one rescaling to the common largest, then sums.
__device__ __forceinline__ Soft sc_warp_merge(Soft a, float s) {
  float m = a.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float d = a.m == -INFINITY ? SC_DMIN : fmaxf((a.m - m) * s, SC_DMIN);
  const float c = sc_ex2(d);
  a.U = (a.U + a.S * d) * c;
  a.S *= c;
  a.m = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a.S += __shfl_xor_sync(0xffffffffu, a.S, o);
    a.U += __shfl_xor_sync(0xffffffffu, a.U, o);
  }
  return a;
}

// What a complete row's state gives: L = log of the mass relative to m, the
// entropy, and the log probability of a value.
__device__ __forceinline__ float sc_log_mass(const Soft& a) { return SC_LN2 * log2f(a.S); }
__device__ __forceinline__ float sc_entropy(const Soft& a, float L) {
  return fmaxf(L - SC_LN2 * (a.U / a.S), 0.f);
}
__device__ __forceinline__ float sc_logprob(float x, float m, float L, float T) {
  return x == -INFINITY ? -INFINITY : fminf(__fdiv_rn(x - m, T) - L, 0.f);
}

template <int DT>
struct ScType;
template <>
struct ScType<SMP_F32> {
  using raw = float;
  static __device__ __forceinline__ float value(float v) { return v; }
  static __device__ __forceinline__ float store(float v) { return v; }
};
template <>
struct ScType<SMP_BF16> {
  using raw = unsigned short;
  static __device__ __forceinline__ float value(unsigned short v) {
    return __uint_as_float((uint32_t)v << 16);
  }
  static __device__ __forceinline__ unsigned short store(float v) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
};
template <>
struct ScType<SMP_F16> {
  using raw = unsigned short;
  static __device__ __forceinline__ float value(unsigned short v) {
    return __half2float(__ushort_as_half(v));
  }
  static __device__ __forceinline__ unsigned short store(float v) {
    return __half_as_ushort(__float2half_rn(v));
  }
};

// The values of a 16-byte vector of logits, and back (round to nearest even).
template <int DT>
__device__ __forceinline__ void sc_unpack(const uint4& q, float (&f)[DT == SMP_F32 ? 4 : 8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == SMP_F32) {
      f[i] = __uint_as_float(w[i]);
    } else if constexpr (DT == SMP_BF16) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      f[2 * i] = __half2float(__ushort_as_half((unsigned short)(w[i] & 0xffffu)));
      f[2 * i + 1] = __half2float(__ushort_as_half((unsigned short)(w[i] >> 16)));
    }
  }
}
template <int DT>
__device__ __forceinline__ uint4 sc_pack(const float (&f)[DT == SMP_F32 ? 4 : 8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == SMP_F32)
      w[i] = __float_as_uint(f[i]);
    else if constexpr (DT == SMP_BF16)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    else
      asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The two halves of a cluster-wide barrier (a launch without clusters: its CTA).
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Whether a barrier's phase is complete (shared memory address `bar`).
__device__ __forceinline__ bool sc_done(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0u;
}
// The same after a while: the thread is parked for up to a microsecond.
__device__ __forceinline__ bool sc_park(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(1000u)
      : "memory");
  return ok != 0u;
}
// A wait for a phase, `limit` SM cycles at most from a first look that does not park: with a
// limit of 1 every wait that would wait fails.
__device__ __forceinline__ bool sc_wait(uint32_t bar, uint32_t parity, long long limit) {
  if (sc_done(bar, parity)) return true;
  const long long t0 = clock64();
  do {
    if (clock64() - t0 > limit) return false;
  } while (!sc_park(bar, parity));
  return true;
}

struct ScoreArgs {
  const void* logits;
  long long ld;
  const uint32_t* bitmask;
  const float* temperature;
  const int32_t* targets;
  float *logprobs, *entropy, *stats;
  int32_t *rank, *status, *top_ids;
  float* top_lp;
  int B, V, W, n;
  long long wait_limit;
};
struct GradArgs {
  const void* logits;
  long long ld, gld;
  const uint32_t* bitmask;
  const float* temperature;
  const int32_t* targets;
  const float *stats, *entropy, *g_lp, *g_ent;
  void* grad;
  int B, V, W;
};
struct HeadArgs {
  const void *hidden, *weight;
  long long ldh, ldw;
  const float* temperature;
  const int32_t* targets;
  float *logprobs, *entropy, *stats;
  int32_t* status;
  float4* part;  // workspace
  int N, V, D;
  long long wait_limit;
};

// Whether a runtime call succeeded.  An error is taken off the thread's last error: it is
// reported by this call's status, and a later launch's check must not find it.
inline bool sc_ok(cudaError_t e) {
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess;
}

// SMs of the current device; 0 when it cannot be asked.
inline int sc_sm_count() {
  int dev = 0, sms = 0;
  if (!sc_ok(cudaGetDevice(&dev)) || !sc_ok(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)))
    return 0;
  return sms;
}

int score_f32(const ScoreArgs& a, cudaStream_t st);
int score_bf16(const ScoreArgs& a, cudaStream_t st);
int score_f16(const ScoreArgs& a, cudaStream_t st);
int grad_enqueue(const GradArgs& a, int dtype, cudaStream_t st);
int head_enqueue(const HeadArgs& a, int dtype, cudaStream_t st);
int64_t head_workspace(int N, int V);

}  // namespace smp
