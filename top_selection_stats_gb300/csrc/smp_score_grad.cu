// smp_score_grad.cu -- the gradient of log probabilities and entropy with
// respect to the logits (smp_token_logprobs_grad).  With d_j = (x_j - m) s,
// s = log2(e) / T and p_j = 2^(d_j - log2 of the mass),
//     grad_j = p_j (a + b d_j) + [j = target] g / T,
//     a = -(g + g_H (H - L)) / T,   b = -g_H ln 2 / T.
// 2^d flushes results below 2^-126 to zero, which a small T would make
// visible: p is taken times 2^24 and a, b times 2^-24.  A row whose a, b or g / T leave
// binary32's normal range all the same (T = 1e-40, gradients of 1e-32 or 1e38) takes
// another power than 2^24, with which a and b stay inside it, and has its target's
// value from the formula: only results that pass the range themselves become infinite,
// and 0 probability gives 0, not 0 times infinity.
//
// One read and one write of the row: bound by HBM.  A row is cut into segments,
// one per CTA; a thread has GU 16-byte vectors in flight.  A CTA reads the
// row's parameters first: a row without any gradient (padding, a failed row)
// is then written as zeros without being read.  Two values share an
// instruction (add, multiply, fused multiply-add on pairs), about 5
// instructions a value; one value an instruction, with a comparison for the
// target in each, took 418 us where this takes 297 (4096 x 128256 bf16, 7.1
// TB/s; a copy of as many bytes: 309).
#include "smp_score.cuh"

namespace smp {
namespace {

constexpr int GT = 256;     // threads
constexpr int GU = 2;       // vectors a thread has in flight
constexpr int GSTEPS = 4;   // steps a CTA takes, at most
constexpr int GMAXC = 8;    // in place: CTAs of a row, one cluster

struct GradRow {
  float m, s, c0, c1, l2, at;
  int t;
};

// p_j (a + b d_j) of two logits (-inf: 0).
template <bool ENT>
__device__ __forceinline__ void grad_pair(const GradRow& g, float& x0, float& x1) {
  const f32x2 z = add2(pair(x0, x1), pair(-g.m, -g.m));
  float e0, e1;
  if (ENT) {
    float d0, d1;
    unpair(mul2(z, pair(g.s, g.s)), d0, d1);
    d0 = fmaxf(d0, SC_DMIN);
    d1 = fmaxf(d1, SC_DMIN);
    const f32x2 d = pair(d0, d1);
    unpair(add2(d, pair(-g.l2, -g.l2)), e0, e1);
    const f32x2 w = fma2(d, pair(g.c1, g.c1), pair(g.c0, g.c0));
    unpair(mul2(pair(sc_ex2(e0), sc_ex2(e1)), w), x0, x1);
  } else {
    unpair(fma2(z, pair(g.s, g.s), pair(-g.l2, -g.l2)), e0, e1);
    unpair(mul2(pair(sc_ex2(e0), sc_ex2(e1)), pair(g.c0, g.c0)), x0, x1);
  }
}

template <int DT, bool ENT>
__global__ void __launch_bounds__(GT) grad_kernel(const GradArgs a, const int nc, const int seg,
                                                  const bool in_place) {
  using TY = ScType<DT>;
  using raw = typename TY::raw;
  constexpr int VE = 16 / (int)sizeof(raw);
  const int r = blockIdx.x / nc, tid = threadIdx.x;
  const raw* row = static_cast<const raw*>(a.logits) + (size_t)r * a.ld;
  raw* out = static_cast<raw*>(a.grad) + (size_t)r * a.gld;
  const uint32_t* bm = a.bitmask ? a.bitmask + (size_t)r * a.W : nullptr;
  // The launch gets ready under the end of the work before it on the stream (1 x 128256:
  // 2.3 to 1.9 us): nothing of a caller's is read or written before that is complete.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float T = a.temperature ? a.temperature[r] : 1.f;
  const float m = a.stats[2 * (size_t)r], L = a.stats[2 * (size_t)r + 1];
  const int t = a.targets ? a.targets[r] : -1;
  float g = a.g_lp ? a.g_lp[r] : 0.f;
  const float gh = a.g_ent ? a.g_ent[r] : 0.f;
  const float H = a.g_ent ? a.entropy[r] : 0.f;
  const bool live = sc_temperature_ok(T) && t >= -1 && t < a.V && fabsf(m) < INFINITY && fabsf(L) < INFINITY;
  auto legal = [&](int j) { return !bm || ((bm[j >> 5] >> (j & 31)) & 1u); };
  // a target that is not legal has no gradient
  const float xt = live && t >= 0 && legal(t) ? TY::value(row[t]) : -INFINITY;
  if (!(xt > -INFINITY)) g = 0.f;
  if (in_place) {  // every CTA of the row has read the target's logit before one writes
    cluster_arrive();
    cluster_wait();
  }
  GradRow q;
  q.m = m;
  q.s = sc_scale(live ? T : 1.f);
  q.c0 = -(g + (a.g_ent ? gh * (H - L) : 0.f)) / T * 0x1p-24f;
  q.c1 = -gh * SC_LN2 / T * 0x1p-24f;
  q.l2 = L / SC_LN2 - 24.f;
  q.at = g / T;
  q.t = g != 0.f ? t : -1;
  const bool zero = !live || (g == 0.f && gh == 0.f);
  // with these the factors are in range (H - L is at most 17): no wait for the quotients
  const float size = fmaxf(fabsf(g), fabsf(gh));
  bool far = !zero && !(T > 0x1p-60f && T < 0x1p20f && size > 0x1p-70f && size < 0x1p60f);
  float most;
  if (far) {
    most = fmaxf(fabsf(q.c0), fabsf(q.c1));
    far = !(most >= 0x1p-126f && most < INFINITY && fabsf(q.at) < INFINITY);
  }
  if (far) {
    // Small: p times 2^-24, factors that keep their bits.  Large (T < 1): p times 2^63,
    // a and b up to 2^110, so that b d, with d down to SC_DMIN, stays finite; past 2^173
    // they count as that.
    const bool small = most < 0x1p-126f;
    const float sg = small ? 0x1p24f : 0x1p-32f, st = small ? T : T * 0x1p31f;
    const float gs = g * sg, hs = gh * sg;
    auto factor = [&](float c) { return fabsf(c) > 0x1p110f ? copysignf(0x1p110f, c) : c; };
    q.c0 = factor(-(gs + (a.g_ent ? hs * (H - L) : 0.f)) / st);
    q.c1 = factor(-hs * SC_LN2 / st);
    q.l2 = L / SC_LN2 + (small ? 24.f : -63.f);
    const float lp = (xt - m) / T - L, p = expf(lp);
    q.at = (gs - (p > 0.f ? p * (gs + (a.g_ent ? hs * (lp + H) : 0.f)) : 0.f)) / st * (small ? 0x1p-24f : 0x1p63f);
  }

  // Vectors are aligned in memory: vector v has elements v VE - lead + [0, VE).
  const int lead = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(raw));
  const bool same = (int)((reinterpret_cast<uintptr_t>(out) & 15) / sizeof(raw)) == lead;
  const int vectors = (a.V + lead + VE - 1) / VE;
  const int v0 = (blockIdx.x % nc) * seg, v1 = min(vectors, v0 + seg);
  const uint4* src = reinterpret_cast<const uint4*>(row - lead);
  uint4* dst = reinterpret_cast<uint4*>(out - lead);
  for (int vb = v0 + tid; vb < v1; vb += GT * GU) {
    uint4 x[GU];
    uint32_t bits[GU];
    if (!zero) {
#pragma unroll
      for (int u = 0; u < GU; ++u) {
        const int v = vb + u * GT, j0 = v * VE - lead;
        x[u] = make_uint4(0, 0, 0, 0);
        bits[u] = 0u;
        if (v < v1 && j0 >= 0 && j0 + VE <= a.V) {
          x[u] = __ldcs(src + v);
          if (bm) bits[u] = __funnelshift_r(bm[j0 >> 5], bm[(j0 + VE - 1) >> 5], j0 & 31);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < GU; ++u) {
      const int v = vb + u * GT, j0 = v * VE - lead;
      if (v >= v1) break;
      if (same && j0 >= 0 && j0 + VE <= a.V) {
        if (zero) {
          __stcs(dst + v, make_uint4(0, 0, 0, 0));
          continue;
        }
        float f[VE];
        sc_unpack<DT>(x[u], f);
        if (bm) {
#pragma unroll
          for (int i = 0; i < VE; ++i) f[i] = ((bits[u] >> i) & 1u) ? f[i] : -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < VE; i += 2) grad_pair<ENT>(q, f[i], f[i + 1]);
        if (q.t >= j0 && q.t < j0 + VE) {
#pragma unroll
          for (int i = 0; i < VE; ++i)
            if (q.t == j0 + i) f[i] = far ? q.at : f[i] + q.at;
        }
        __stcs(dst + v, sc_pack<DT>(f));
      } else {  // a row's ends, or a result whose rows start elsewhere in their vectors
#pragma unroll 1
        for (int j = max(j0, 0); j < min(j0 + VE, a.V); ++j) {
          float y = 0.f, other = -INFINITY;
          if (!zero && legal(j)) {
            y = TY::value(row[j]);
            grad_pair<ENT>(q, y, other);
            if (j == q.t) y = far ? q.at : y + q.at;
          }
          out[j] = TY::store(y);
        }
      }
    }
  }
}

// A CTA takes up to GSTEPS steps of GT * GU vectors of its row, fewer while that
// leaves the SMs short of CTAs.  4096 x 128256 bf16: 297 us with 4 steps of 2
// vectors a thread, 354 with 1, 327 with one step of 4 vectors; 1 x 128256: 1.9
// us with 1 step, 3.5 with 4.  In place a row is one cluster, so at most GMAXC
// CTAs.
template <int DT>
int launch_grad(const GradArgs& a, int sms, cudaStream_t st) {
  constexpr int VE = DT == SMP_F32 ? 4 : 8;
  const bool in_place = a.grad == a.logits;
  const int vectors = (a.V + VE - 1) / VE + 1;  // one more than V fills: rows may start inside one
  const int steps = (vectors + GT * GU - 1) / (GT * GU);
  const long long share = (long long)a.B * steps / (4 * sms);
  int per = share < 1 ? 1 : share > GSTEPS ? GSTEPS : (int)share;
  if (in_place && (steps + per - 1) / per > GMAXC) per = (steps + GMAXC - 1) / GMAXC;
  const int seg = per * GT * GU, nc = (steps + per - 1) / per;
  if ((long long)a.B * nc > 0x7fffffffLL) return SMP_ERR_CAPACITY;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * nc));
  cfg.blockDim = dim3(GT);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)nc;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = in_place ? 2 : 1;
  const cudaError_t e = a.g_ent ? cudaLaunchKernelEx(&cfg, grad_kernel<DT, true>, a, nc, seg, in_place)
                                : cudaLaunchKernelEx(&cfg, grad_kernel<DT, false>, a, nc, seg, in_place);
  return sc_ok(e) ? SMP_OK : SMP_ERR_CUDA;
}

}  // namespace

int grad_enqueue(const GradArgs& a, int dtype, cudaStream_t st) {
  const int sms = sc_sm_count();
  if (sms < 1) return SMP_ERR_CUDA;
  switch (dtype) {
    case SMP_F32: return launch_grad<SMP_F32>(a, sms, st);
    case SMP_BF16: return launch_grad<SMP_BF16>(a, sms, st);
    default: return launch_grad<SMP_F16>(a, sms, st);
  }
}

}  // namespace smp
