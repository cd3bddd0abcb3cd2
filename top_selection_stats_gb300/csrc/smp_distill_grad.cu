// smp_distill_grad.cu -- the gradient of smp_distill_loss' loss and log
// probabilities with respect to the logits (smp_distill_loss_grad).
//
// Outside the slots grad_j = rho_j D, rho_j = 2^((x_j - m) s - L log2 e) the token's
// share of the mass there and D = (g A - g_lp s) / T one factor for the row; a slot's
// value is (g G_k - g_lp p_k) / T, and the target adds g_lp / T.  The kind of
// divergence is in A and G_k alone.  A warp writes rho_j D to its vectors, slots
// included, and then the slots' values over those.
//
// D is handled as a mantissa and a power of two, so that neither a small T nor
// gradients near the ends of binary32 make it 0 or infinite: usually 2^24 goes to
// rho (2^x flushes results below 2^-126, which a small T would make visible), and the
// whole power where it is beyond 2^60.  In such rows the slots' values are taken at a scale
// where the larger of g and g_lp is near 1, and D in binary64, where neither of its terms
// hides the other; the rest of the kernel is the same for them, as anything more in it costs
// all rows (values of the slots in binary64: 348 to 356 us for the case below).
//
// One read and one write of the row: bound by HBM.  A row is cut into segments, one per
// CTA; a thread has DGU 16-byte vectors in flight and the next ones requested while it
// computes them, the first before the row's parameters are there.  Vectors are aligned in
// the result; where the logits lie otherwise in theirs, a vector is put together from two.
// Two values share an instruction (add, fused multiply-add, multiply).  The slots are
// written over a step's vectors by the same warp right after them, while their lines are
// in L2, and are looked up by each warp for itself, so that no warp waits for another.
// 4096 x 128256 bf16 with 64 slots: 316 us, 6.7 TB/s (a copy of as many bytes: 311); slots
// written at the end of each CTA 393, kept in a table of the CTA with two barriers 320,
// logits through rings of bulk copies 341 to 351.
#include "smp_train.cuh"

namespace smp {
namespace {

constexpr int DGT = 256;     // threads
constexpr int DGCTAS = 8;    // CTAs on an SM
constexpr int DGU = 2;       // vectors a thread has in flight
constexpr int DGSTEPS = 4;   // steps a CTA takes, at most; twice as many with more slots than DGFEW
constexpr int DGFEW = 128;

// rho_j D of two logits (-inf: 0).
struct DistillGradRow {
  float m, s, l2, D;
};
__device__ __forceinline__ void distill_grad_pair(const DistillGradRow& q, float& x0, float& x1) {
  const f32x2 z = add2(pair(x0, x1), pair(-q.m, -q.m));
  float e0, e1;
  unpair(fma2(z, pair(q.s, q.s), pair(-q.l2, -q.l2)), e0, e1);
  unpair(mul2(pair(sc_ex2(e0), sc_ex2(e1)), pair(q.D, q.D)), x0, x1);
}

// What the row's parameters come to: D = q.D 2^-shift with 2^shift in q.l2, and the
// slots' scale, (g, g_lp) / T = (gm, glm) / Tm 2^e.
struct DistillGradScale {
  DistillGradRow q;
  float gm, glm, Tm;
  int e;
};
struct DistillGradIn {
  float m, L, A, mass, T, g, gl;
};
// Any values: mantissas and powers apart.
__device__ __noinline__ DistillGradScale distill_grad_far(const DistillGradIn i) {
  DistillGradScale o;
  o.q.m = i.m;
  if (!(fabsf(i.g) < INFINITY && fabsf(i.gl) < INFINITY)) {
    // An incoming gradient that is not finite: results that are not, at legal tokens alone.
    // Outside the slots 2^x is infinite for a finite logit and 0 for -inf, and D is 1, -1 or (NaN)
    // 0; a slot's value is 2^300 times what a sign comes to, 0 at a token without probability.
    const float D = i.g * i.A - i.gl * i.mass;
    auto sign = [](float v) { return fabsf(v) < INFINITY ? 0.f : v < 0.f ? -1.f : 1.f; };
    o.gm = sign(i.g);
    o.glm = sign(i.gl);
    o.Tm = 1.f;
    o.e = 300;
    o.q.D = D == INFINITY ? 1.f : D == -INFINITY ? -1.f : 0.f;
    o.q.s = 0x1p-100f;
    o.q.l2 = -0x1p100f;
    return o;
  }
  o.q.s = sc_scale(i.T);
  int ge, le, Te, De;
  frexpf(i.g, &ge);
  frexpf(i.gl, &le);
  ge = i.g == 0.f ? le : i.gl == 0.f ? ge : max(ge, le);
  o.gm = ldexpf(i.g, -ge);
  o.glm = ldexpf(i.gl, -ge);
  o.Tm = frexpf(i.T, &Te);
  o.e = ge - Te;
  // in binary64, where neither product hides the other's bits
  const double D = frexp(((double)i.g * i.A - (double)i.gl * i.mass) / i.T, &De);
  // 2^(De - 1) at most goes to rho, so that rho 2^shift is in range where the result is
  const int shift = D == 0.0 || (De > -60 && De <= 24) ? 24 : max(-250, min(250, De - 1));
  o.q.D = (float)ldexp(D, De - shift);
  o.q.l2 = i.L / SC_LN2 - (float)shift;
  return o;
}
// Values of ordinary size: every product and quotient is in range by itself.
__device__ __forceinline__ DistillGradScale distill_grad_scale(const DistillGradIn& i) {
  const float size = fabsf(i.g) + fabsf(i.gl);  // NaN is far too
  DistillGradScale o;
  o.gm = i.g;
  o.glm = i.gl;
  o.Tm = i.T;
  o.e = 0;
  o.q.D = (i.g * i.A - i.gl * i.mass) / i.T * 0x1p-24f;
  o.q.l2 = i.L / SC_LN2 - 24.f;
  o.q.m = i.m;
  o.q.s = sc_scale(i.T);
  if (!(i.T > 0x1p-20f && i.T < 0x1p20f && size > 0x1p-60f && size < 0x1p40f && fabsf(i.A) < 0x1p40f)) o = distill_grad_far(i);
  if (i.m == -INFINITY) o.q.m = o.q.l2 = o.q.D = 0.f;  // every legal token has a slot
  return o;
}

// ALIKE: logits and result start at the same place in their vectors.
template <int DT, bool ALIKE, bool MASK>
__global__ void __launch_bounds__(DGT, DGCTAS) distill_grad_kernel(const DistillGradArgs a, const int nc, const int seg) {
  using TY = ScType<DT>;
  using raw = typename TY::raw;
  constexpr int VE = 16 / (int)sizeof(raw), STEP = DGT * DGU;
  extern __shared__ int2 slot_lists[];
  const int r = blockIdx.x / nc, c = blockIdx.x % nc, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const raw* row = static_cast<const raw*>(a.logits) + (size_t)r * a.ld;
  raw* out = static_cast<raw*>(a.grad) + (size_t)r * a.gld;
  const uint32_t* bm = MASK ? a.bitmask + (size_t)r * a.W : nullptr;
  // Vector v has elements v VE - lead + [0, VE) of the row; [f0, f1) lie inside it.
  const int lead = (int)((reinterpret_cast<uintptr_t>(out) & 15) / sizeof(raw));
  const int f0 = lead ? 1 : 0, f1 = max(f0, (a.V + lead) / VE);
  const int v0 = min(f1, f0 + c * seg), v1 = min(f1, v0 + seg);
  const char* first = reinterpret_cast<const char*>(row - lead);  // of vector 0
  const int off = (int)(reinterpret_cast<uintptr_t>(first) & 15);
  const uint4* src = reinterpret_cast<const uint4*>(first - off);
  uint4* dst = reinterpret_cast<uint4*>(out - lead);
  // The launch gets ready under the end of the work before it on the stream: nothing of
  // a caller's is read or written before that is complete.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  uint4 x[DGU];
  uint32_t bits[MASK ? DGU : 1];
  auto load = [&](int vb) {
#pragma unroll
    for (int u = 0; u < DGU; ++u) {
      const int v = vb + u * DGT;
      if (v < v1) {
        x[u] = ALIKE ? __ldcs(src + v) : vector_across(src + v, off);
        if constexpr (MASK) {
          const int j = v * VE - lead;
          bits[u] = __funnelshift_r(bm[j >> 5], bm[(j + VE - 1) >> 5], j & 31);
        }
      }
    }
  };
  load(v0 + tid);
  DistillGradIn in;
  in.m = a.stats[4 * (size_t)r];
  in.L = a.stats[4 * (size_t)r + 1];
  in.A = a.stats[4 * (size_t)r + 2];
  in.mass = a.stats[4 * (size_t)r + 3];
  in.T = a.temperature ? a.temperature[r] : 1.f;
  in.g = a.g_loss ? a.g_loss[r] : 0.f;
  in.gl = a.g_lp ? a.g_lp[r] : 0.f;
  int target = a.targets ? a.targets[r] : -1;
  const float lp = a.g_lp ? a.logprobs[r] : 0.f;
  const bool live = sc_temperature_ok(in.T) && target >= -1 && target < a.V && fabsf(in.A) < INFINITY && in.mass >= 0.f;
  if (target < 0 || !(lp > -INFINITY)) in.gl = 0.f;  // a target that is not legal has no gradient
  const bool none = !live || (in.g == 0.f && in.gl == 0.f);
  if (!live) in.T = 1.f;
  if (none || in.gl == 0.f) target = -1;
  const DistillGradScale sc = distill_grad_scale(in);

  // The slots among this warp's vectors (and the row's ends): id and value.
  int2* list = slot_lists + warp * a.K;
  int slots = 0;
  if (!none) {
    bool taken = false;
    for (int k0 = 0; k0 < a.K; k0 += 32) {
      const int k = k0 + lane, given = k < a.K ? a.ids[(size_t)r * a.K + k] : -1;
      const bool in_row = given >= 0 && given < a.V;
      const int id = in_row ? given : 0, v = (id + lead) / VE;
      taken |= in_row && id == target;
      const bool end = v < f0 || v >= f1;
      const bool mine = in_row && (end ? c == 0 && warp == 0 : v >= v0 && v < v1 && (v - v0) % DGT / 32 == warp);
      const uint32_t which = __ballot_sync(0xffffffffu, mine);
      if (mine) {
        float y = sc.gm * a.slot_g[(size_t)r * a.K + k];
        if (sc.glm != 0.f) y += (id == target ? sc.glm : 0.f) - sc.glm * expf(a.slot_lp[(size_t)r * a.K + k]);
        list[slots + __popc(which & ((1u << lane) - 1))] = make_int2(id, __float_as_int(ldexpf(y / sc.Tm, sc.e)));
      }
      slots += __popc(which);
    }
    if (__any_sync(0xffffffffu, taken)) target = -1;  // part of a slot's value
    __syncwarp();
  }
  for (int vb = v0; vb < v1; vb += STEP) {
    uint4 now[DGU];
    uint32_t legal[MASK ? DGU : 1];
#pragma unroll
    for (int u = 0; u < DGU; ++u) {
      now[u] = x[u];
      if constexpr (MASK) legal[u] = bits[u];
    }
    if (!none) load(vb + STEP + tid);
#pragma unroll
    for (int u = 0; u < DGU; ++u) {
      const int v = vb + tid + u * DGT;
      if (v >= v1) break;
      if (none) {
        __stcs(dst + v, make_uint4(0, 0, 0, 0));
        continue;
      }
      float f[VE];
      sc_unpack<DT>(now[u], f);
      if constexpr (MASK) {
#pragma unroll
        for (int i = 0; i < VE; ++i) f[i] = ((legal[u] >> i) & 1u) ? f[i] : -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < VE; i += 2) distill_grad_pair(sc.q, f[i], f[i + 1]);
      {
        const int i0 = target - (v * VE - lead);
        if ((unsigned)i0 < (unsigned)VE) {
          const float add = ldexpf(sc.glm / sc.Tm, sc.e);
#pragma unroll
          for (int i = 0; i < VE; ++i)
            if (i0 == i) f[i] += add;
        }
      }
      __stcs(dst + v, sc_pack<DT>(f));
    }
    if (slots) {
      __syncwarp();  // the step's vectors are written
      for (int k = lane; k < slots; k += 32) {
        const int2 s = list[k];
        const int v = (s.x + lead) / VE;
        if (v >= vb && v < min(v1, vb + STEP)) out[s.x] = TY::store(__int_as_float(s.y));
      }
    }
  }
  if (c == 0 && warp == 0) {  // the row's ends, fewer than 2 VE values
    const int head = lead ? min(a.V, VE - lead) : 0;
    const int j = lane < head ? lane : max(head, f1 * VE - lead) + lane - head;
    if (j < a.V) {
      float y = -INFINITY, other = -INFINITY;
      if (!none && (!MASK || ((bm[j >> 5] >> (j & 31)) & 1u))) y = TY::value(row[j]);
      distill_grad_pair(sc.q, y, other);
      if (j == target) y += ldexpf(sc.glm / sc.Tm, sc.e);
      for (int k = 0; k < slots; ++k) y = list[k].x == j ? __int_as_float(list[k].y) : y;
      out[j] = TY::store(none ? 0.f : y);
    }
  }
  // A target outside the slots whose two parts were infinite and opposite: (g A rho + gl (1 - p)) / T,
  // by the warp that wrote it.
  if (sc.e > 60 && target >= 0) {
    const int v = (target + lead) / VE;
    __syncwarp();
    if (lane == 0 && (v < f0 || v >= f1 ? c == 0 && warp == 0 : v >= v0 && v < v1 && (v - v0) % DGT / 32 == warp) &&
        isnan(TY::value(out[target])) && fabsf(a.g_lp[r]) < INFINITY && (!a.g_loss || fabsf(a.g_loss[r]) < INFINITY)) {
      const float A = a.stats[4 * (size_t)r + 2], mass = a.stats[4 * (size_t)r + 3], p = expf(a.logprobs[r]);
      const float rho = mass > 0.f ? __fdiv_rn(p, mass) : 0.f;
      out[target] = TY::store(ldexpf((sc.gm * A * rho + sc.glm * (1.f - p)) / sc.Tm, sc.e));
    }
  }
}

// A CTA takes up to DGSTEPS steps of DGT * DGU vectors of its row, fewer while one round
// of CTAs does not fill the SMs: 256 x 151936 masked 32.7 us with at most 4 steps, 35.5
// with 8; 150 x 128256 with 100 slots 16.9 us with 3, 24.6 with 1; 4096 x 128256 with 64
// slots 316 and 318.  Each warp looks through all slots, so many of them want longer
// segments: 2000 x 128256 with 256 slots 181 us with 8 steps, 205 with 4.
template <int DT>
int launch_distill_grad(const DistillGradArgs& a, int sms, cudaStream_t st) {
  constexpr int VE = DT == SMP_F32 ? 4 : 8;
  const int vectors = a.V / VE > 0 ? a.V / VE : 1;
  const int steps = (vectors + DGT * DGU - 1) / (DGT * DGU);
  const long long share = (long long)a.B * steps / ((long long)DGCTAS * sms);
  const int most = a.K > DGFEW ? 2 * DGSTEPS : DGSTEPS;
  const int per = share < 1 ? 1 : share > most ? most : (int)share;
  const int seg = per * DGT * DGU, nc = (steps + per - 1) / per;
  if ((long long)a.B * nc > 0x7fffffffLL) return SMP_ERR_CAPACITY;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * nc));
  cfg.blockDim = dim3(DGT);
  cfg.stream = st;
  cfg.dynamicSmemBytes = (size_t)(DGT / 32) * a.K * sizeof(int2);
  // whether all rows of the logits and the result start alike
  const size_t size = DT == SMP_F32 ? 4 : 2;
  const bool alike = ((reinterpret_cast<uintptr_t>(a.logits) - reinterpret_cast<uintptr_t>(a.grad)) & 15) == 0 &&
                     ((size_t)(a.ld - a.gld) * size & 15) == 0;
  const auto kernel = a.bitmask ? (alike ? distill_grad_kernel<DT, true, true> : distill_grad_kernel<DT, false, true>)
                                : (alike ? distill_grad_kernel<DT, true, false> : distill_grad_kernel<DT, false, false>);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return sc_ok(cudaLaunchKernelEx(&cfg, kernel, a, nc, seg)) ? SMP_OK : SMP_ERR_CUDA;
}

}  // namespace

int distill_grad_enqueue(const DistillGradArgs& a, int dtype, cudaStream_t st) {
  const int sms = sc_sm_count();
  if (sms < 1) return SMP_ERR_CUDA;
  switch (dtype) {
    case SMP_F32: return launch_distill_grad<SMP_F32>(a, sms, st);
    case SMP_BF16: return launch_distill_grad<SMP_BF16>(a, sms, st);
    default: return launch_distill_grad<SMP_F16>(a, sms, st);
  }
}

}  // namespace smp
