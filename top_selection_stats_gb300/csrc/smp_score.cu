// smp_score.cu -- log probabilities of given tokens, entropy, rank and the n
// most likely alternatives (smp_token_logprobs), in one pass over each row.
//
// A row is cut into segments, one per CTA of a cluster.  A thread reads batches
// of SU 16-byte vectors and folds each batch, after one look at its maximum,
// into its softmax state (smp_score.cuh); the target's rank is counted only in
// batches that hold something at or above its logit.
//
// Alternatives: each thread also keeps the maximum of each of its buckets (one
// or more batches).  The k-th largest of a warp's 32 thread maxima, k = n over
// the number of warps, bounds the n-th best from below when the smallest of
// the warps' values is taken (each warp then has k values at least as large),
// and few values lie above it: 20 to 60 of 128256 for n = 20.  Only buckets
// whose maximum reaches the bound are read again, out of L2.  The values found
// are ranked by counting, in a list of SCAND; when more are found (ties, rows
// sorted by id), the n-th best of those in the list is a better bound, and the
// buckets are scanned again with it until the list holds them all.  Keys are
// (logit, smallest id first), all different, so the result is exact whatever
// the order in which candidates arrive.
#include <cooperative_groups.h>

#include "smp_score.cuh"

namespace cg = cooperative_groups;

namespace smp {
namespace {

constexpr int ST = 256;       // threads
constexpr int SW = ST / 32;   // warps
constexpr int SU = 4;         // vectors a thread has in flight
constexpr int SBUCKETS = 16;  // buckets per thread, at most
constexpr int SCAND = 512;    // candidates ranked at a time
constexpr int SMAXC = 8;      // CTAs of a row, at most

// Order key of a value: larger = earlier; 0 = none (not legal).
__device__ __forceinline__ uint32_t order32(float x) {
  if (!(x > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 folds onto +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ uint64_t order_key(uint32_t o, int id) {
  return ((uint64_t)o << 32) | (uint64_t)(0xffffffffu - (uint32_t)id);
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t b = (uint32_t)(k >> 32);
  return __uint_as_float((b & 0x80000000u) ? (b & 0x7fffffffu) : ~b);
}
__device__ __forceinline__ int key_id(uint64_t k) { return (int)(0xffffffffu - (uint32_t)k); }

// A word of a vector: one binary32 value or two 16-bit ones.
template <int DT>
struct Word {
  static constexpr uint32_t NONE = DT == SMP_F32 ? 0xff800000u : DT == SMP_BF16 ? 0xff80ff80u : 0xfc00fc00u;
  // maximum of each value; NaN wins
  static __device__ __forceinline__ uint32_t max_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (DT == SMP_F32) asm("max.NaN.f32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else if constexpr (DT == SMP_BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  // the larger value; NaN wins
  static __device__ __forceinline__ float top(uint32_t a) {
    if constexpr (DT == SMP_F32) return __uint_as_float(a);
    float x, y, r;
    if constexpr (DT == SMP_BF16) {
      x = __uint_as_float(a << 16);
      y = __uint_as_float(a & 0xffff0000u);
    } else {
      x = __half2float(__ushort_as_half((unsigned short)(a & 0xffffu)));
      y = __half2float(__ushort_as_half((unsigned short)(a >> 16)));
    }
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
  }
  // word i of a vector with the values whose bit is 0 replaced by -inf
  static __device__ __forceinline__ uint32_t keep(uint32_t a, uint32_t bits, int i) {
    if constexpr (DT == SMP_F32) return ((bits >> i) & 1u) ? a : NONE;
    const uint32_t b = bits >> (2 * i);
    const uint32_t on = ((b & 1u) ? 0x0000ffffu : 0u) | ((b & 2u) ? 0xffff0000u : 0u);
    return (a & on) | (NONE & ~on);
  }
};

// What a CTA hands to the row's first one.
struct Part {
  float m, S, U;
  int ahead, bad;
};

struct Scratch {
  uint32_t bucket[SBUCKETS * ST];
  unsigned short queue[SBUCKETS * ST];
  uint64_t cand[SCAND];
  uint64_t tops[SMAXC][SC_MAX_TOP];  // first CTA: the n best of each
  Part part[SMAXC];                  // first CTA: the states of all
  Part warp[SW];
  uint32_t kth[SW];
  uint64_t bound;
  int queued, found;
};

template <int DT, bool TOP>
__global__ void __launch_bounds__(ST, 4) score_kernel(const ScoreArgs a, const int nc, const int seg,
                                                         const int gshift) {
  using TY = ScType<DT>;
  using raw = typename TY::raw;
  using WD = Word<DT>;
  constexpr int VE = 16 / (int)sizeof(raw);
  __shared__ __align__(16) Scratch sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (nc > 1) cluster_arrive();  // waited for before the first CTA's shared memory is written
  const int r = blockIdx.x / nc, rank_c = blockIdx.x % nc;
  const raw* row = static_cast<const raw*>(a.logits) + (size_t)r * a.ld;
  const uint32_t* bm = a.bitmask ? a.bitmask + (size_t)r * a.W : nullptr;
  const float T = a.temperature ? a.temperature[r] : 1.f;
  const int t = a.targets ? a.targets[r] : -1;
  const bool valid = sc_temperature_ok(T) && t >= -1 && t < a.V;
  const float s = sc_scale(valid ? T : 1.f);
  auto legal = [&](int j) { return !bm || ((__ldg(bm + (j >> 5)) >> (j & 31)) & 1u); };
  const float xt = valid && t >= 0 && legal(t) ? TY::value(__ldg(row + t)) : -INFINITY;
  // counted: values at or above this (nothing without a target or a rank)
  const float xc = valid && t >= 0 && a.rank ? xt : INFINITY;

  // Vectors are aligned in memory: vector v has elements v VE - lead + [0, VE).
  const int lead = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(raw));
  const int vectors = (a.V + lead + VE - 1) / VE;
  const int v0 = min(vectors, rank_c * seg), v1 = min(vectors, v0 + seg);
  const uint4* src = reinterpret_cast<const uint4*>(row - lead);

  float m = -INFINITY, tmax = -INFINITY, bmax = -INFINITY;
  f32x2 S2 = pair(0.f, 0.f), U2 = pair(0.f, 0.f);
  const f32x2 s2 = pair(s, s);
  int ahead = 0, batch = 0;
  bool bad = false;
  if (TOP) {
    for (int i = tid; i < SBUCKETS * ST; i += ST) sh.bucket[i] = 0u;
  }
  const int vend = valid ? v1 : v0;
  for (int vb = v0; vb < vend; vb += ST * SU, ++batch) {
    uint4 x[SU];
    uint32_t bits[SU];
#pragma unroll
    for (int u = 0; u < SU; ++u) {
      const int v = vb + u * ST + tid, j0 = v * VE - lead;
      x[u] = make_uint4(WD::NONE, WD::NONE, WD::NONE, WD::NONE);
      bits[u] = 0xffffffffu;
      if (v < v1) {
        if (j0 >= 0 && j0 + VE <= a.V) {
          x[u] = __ldg(src + v);
          if (bm) bits[u] = __funnelshift_r(__ldg(bm + (j0 >> 5)), __ldg(bm + ((j0 + VE - 1) >> 5)), j0 & 31);
        } else {  // an end of the row
          float f[VE];
#pragma unroll
          for (int i = 0; i < VE; ++i)
            f[i] = j0 + i >= 0 && j0 + i < a.V && legal(j0 + i) ? TY::value(__ldg(row + j0 + i)) : -INFINITY;
          x[u] = sc_pack<DT>(f);
        }
      }
    }
    if (bm) {
#pragma unroll
      for (int u = 0; u < SU; ++u) {
        x[u].x = WD::keep(x[u].x, bits[u], 0);
        x[u].y = WD::keep(x[u].y, bits[u], 1);
        x[u].z = WD::keep(x[u].z, bits[u], 2);
        x[u].w = WD::keep(x[u].w, bits[u], 3);
      }
    }
    uint32_t wm = WD::NONE;
#pragma unroll
    for (int u = 0; u < SU; ++u)
      wm = WD::max_nan(wm, WD::max_nan(WD::max_nan(x[u].x, x[u].y), WD::max_nan(x[u].z, x[u].w)));
    const float top = WD::top(wm);
    bad |= !(top < INFINITY);
    if (TOP) {
      bmax = fmaxf(bmax, top);
      if (((batch + 1) & ((1 << gshift) - 1)) == 0 || vb + ST * SU >= vend) {
        sh.bucket[(batch >> gshift) * ST + tid] = order32(bmax);
        tmax = fmaxf(tmax, bmax);
        bmax = -INFINITY;
      }
    }
    if (top > -INFINITY) {
      if (top > m) {
        const float d = m == -INFINITY ? SC_DMIN : fmaxf((m - top) * s, SC_DMIN);
        const float e = sc_ex2(d);
        U2 = mul2(fma2(S2, pair(d, d), U2), pair(e, e));
        S2 = mul2(S2, pair(e, e));
        m = top;
      }
      const f32x2 mm = pair(-m, -m);
#pragma unroll
      for (int u = 0; u < SU; ++u) {
        float f[VE];
        sc_unpack<DT>(x[u], f);
#pragma unroll
        for (int i = 0; i < VE; i += 2) {
          float d0, d1;
          unpair(mul2(add2(pair(f[i], f[i + 1]), mm), s2), d0, d1);
          d0 = fmaxf(d0, SC_DMIN);
          d1 = fmaxf(d1, SC_DMIN);
          const f32x2 e = pair(sc_ex2(d0), sc_ex2(d1));
          S2 = add2(S2, e);
          U2 = fma2(e, pair(d0, d1), U2);
        }
      }
      if (top >= xc) {
#pragma unroll
        for (int u = 0; u < SU; ++u) {
          const int j0 = (vb + u * ST + tid) * VE - lead;
          float f[VE];
          sc_unpack<DT>(x[u], f);
#pragma unroll
          for (int i = 0; i < VE; ++i)
            ahead += f[i] > xt || (f[i] == xt && j0 + i < t && xt > -INFINITY);
        }
      }
    }
  }

  // the CTA's state
  Soft st;
  {
    float a0, a1, b0, b1;
    unpair(S2, a0, a1);
    unpair(U2, b0, b1);
    st.m = m;
    st.S = a0 + a1;
    st.U = b0 + b1;
  }
  for (int o = 16; o > 0; o >>= 1) {
    st = sc_merge(st, sc_shfl_xor(st, o), s);
    ahead += __shfl_xor_sync(0xffffffffu, ahead, o);
  }
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) sh.warp[warp] = Part{st.m, st.S, st.U, ahead, bad};

  // the bound: warps whose 32 threads all had vectors take part
  const int n = a.n;
  if (TOP) {
    const int full = min(SW, (min(v1 - v0, ST)) / 32);
    if (warp < full) {
      uint32_t key = order32(tmax), kth = 0u;
      for (int k = (n + full - 1) / full; k > 0; --k) {
        kth = __reduce_max_sync(0xffffffffu, key);
        const uint32_t who = __ballot_sync(0xffffffffu, key == kth);
        if (lane == __ffs(who) - 1) key = 0u;
      }
      if (lane == 0) sh.kth[warp] = kth;
    } else if (lane == 0) {
      sh.kth[warp] = full ? 0xffffffffu : 0u;
    }
    if (tid == 0) sh.queued = sh.found = 0;
  }
  __syncthreads();
  if (nc > 1) cluster_wait();
  if (tid == 0) {
    Soft b{sh.warp[0].m, sh.warp[0].S, sh.warp[0].U};
    int ah = sh.warp[0].ahead, bd = sh.warp[0].bad;
    for (int w = 1; w < SW; ++w) {
      b = sc_merge(b, Soft{sh.warp[w].m, sh.warp[w].S, sh.warp[w].U}, s);
      ah += sh.warp[w].ahead;
      bd |= sh.warp[w].bad;
    }
    Part* to = nc > 1 ? cg::this_cluster().map_shared_rank(&sh.part[rank_c], 0) : &sh.part[0];
    *to = Part{b.m, b.S, b.U, ah, bd};
  }

  if (TOP) {
    uint32_t low = sh.kth[0];
#pragma unroll
    for (int w = 1; w < SW; ++w) low = min(low, sh.kth[w]);
    if (low == 0u) low = 1u;  // any legal value
    const int buckets = min(SBUCKETS, (batch + (1 << gshift) - 1) >> gshift);
    for (int b = 0; b < buckets; ++b)
      if (sh.bucket[b * ST + tid] >= low) sh.queue[atomicAdd(&sh.queued, 1)] = (unsigned short)(b * ST + tid);
    uint64_t bound = (uint64_t)low << 32;
    __syncthreads();
    const int per = VE * SU << gshift, total = sh.queued * per;
    while (true) {
      for (int i0 = tid; i0 < total; i0 += ST * 4) {
        float x[4];
        int id[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int i = i0 + q * ST;
          x[q] = -INFINITY;
          id[q] = 0;
          if (i < total) {
            const int item = sh.queue[i / per], e = i % per;
            const int v = v0 + (item % ST) + (((item / ST) * SU << gshift) + e / VE) * ST;
            const int j = v * VE - lead + e % VE;
            if (v < v1 && j >= 0 && j < a.V && legal(j)) {
              x[q] = TY::value(__ldg(row + j));
              id[q] = j;
            }
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t o = order32(x[q]);
          const uint64_t k = order_key(o, id[q]);
          if (o && k >= bound && *reinterpret_cast<volatile int*>(&sh.found) <= SCAND) {
            const int p = atomicAdd(&sh.found, 1);
            if (p < SCAND) sh.cand[p] = k;
          }
        }
      }
      __syncthreads();
      const int found = sh.found;
      if (found <= SCAND) break;
      // the n-th best of the list bounds the n-th best of all
#pragma unroll
      for (int c = tid; c < SCAND; c += ST) {
        const uint64_t k = sh.cand[c];
        int above = 0;
        for (int i = 0; i < SCAND; ++i) above += sh.cand[i] > k;
        if (above == n - 1) sh.bound = k;
      }
      __syncthreads();
      bound = sh.bound;
      if (tid == 0) sh.found = 0;
      __syncthreads();
    }
    const int found = sh.found;
    uint64_t* tops = nc > 1 ? cg::this_cluster().map_shared_rank(&sh.tops[rank_c][0], 0) : &sh.tops[0][0];
    if (tid < n && tid >= found) tops[tid] = 0ull;
    for (int c = tid; c < found; c += ST) {
      const uint64_t k = sh.cand[c];
      int above = 0;
      for (int i = 0; i < found; ++i) above += sh.cand[i] > k;
      if (above < n) tops[above] = k;
    }
  }

  if (nc > 1) {  // the first CTA has everything; the others may go
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (rank_c) return;
  } else {
    __syncthreads();
  }
  Soft b{sh.part[0].m, sh.part[0].S, sh.part[0].U};
  ahead = sh.part[0].ahead;
  int any = sh.part[0].bad;
  for (int c = 1; c < nc; ++c) {
    b = sc_merge(b, Soft{sh.part[c].m, sh.part[c].S, sh.part[c].U}, s);
    ahead += sh.part[c].ahead;
    any |= sh.part[c].bad;
  }
  const int status = !valid ? SMP_ERR_INVALID_PARAM : any ? SMP_ERR_NONFINITE
                     : b.m == -INFINITY ? SMP_ERR_EMPTY : SMP_OK;
  const bool ok = status == SMP_OK;
  if (tid == 0) {
    a.status[r] = status;
    if (a.logprobs) a.logprobs[r] = !ok ? sc_nan() : t < 0 ? 0.f : sc_logprob(xt, b, T);
    if (a.entropy) a.entropy[r] = ok ? sc_entropy(b) : sc_nan();
    if (a.rank) a.rank[r] = ok && t >= 0 ? ahead : -1;
    if (a.stats) {
      a.stats[2 * (size_t)r] = ok ? b.m : sc_nan();
      a.stats[2 * (size_t)r + 1] = ok ? SC_LN2 * sc_log2_mass(b) : sc_nan();
    }
  }
  if (TOP) {
    int32_t* ids = a.top_ids + (size_t)r * n;
    float* lps = a.top_lp + (size_t)r * n;
    auto put = [&](int i, uint64_t k) {
      ids[i] = ok && k ? key_id(k) : -1;
      lps[i] = !ok ? sc_nan() : k ? sc_logprob(key_value(k), b, T) : -INFINITY;
    };
    if (nc == 1) {
      if (tid < n) put(tid, sh.tops[0][tid]);
    } else {
      for (int c = tid; c < nc * n; c += ST) {
        const uint64_t k = sh.tops[c / n][c % n];
        // keys of 0 (a CTA with fewer than n legal values) are all alike: by place
        int above = 0;
        for (int p = 0; p < nc; ++p)
          for (int i = 0; i < n; ++i) {
            const uint64_t o = sh.tops[p][i];
            above += o > k || (o == k && p * n + i < c);
          }
        if (above < n) put(above, k);
      }
    }
  }
}

template <int DT>
int launch_score(const ScoreArgs& a, int sms, cudaStream_t st) {
  constexpr int VE = DT == SMP_F32 ? 4 : 8;
  const int vectors = (a.V + VE - 1) / VE + 1;  // one more than V fills: rows may start inside one
  constexpr int step = ST * SU;
  int nc = 1;
  while (nc < SMAXC && (long long)a.B * nc < 4LL * sms && vectors > nc * step) nc *= 2;
  const int seg = ((vectors + nc - 1) / nc + ST - 1) / ST * ST;
  const int batches = (seg + step - 1) / step;
  int gshift = 0;
  while ((batches >> gshift) + 1 > SBUCKETS) ++gshift;
  if ((long long)a.B * nc > 0x7fffffffLL) return SMP_ERR_CAPACITY;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * nc));
  cfg.blockDim = dim3(ST);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)nc;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = nc > 1 ? 1 : 0;
  const cudaError_t e = a.n ? cudaLaunchKernelEx(&cfg, score_kernel<DT, true>, a, nc, seg, gshift)
                            : cudaLaunchKernelEx(&cfg, score_kernel<DT, false>, a, nc, seg, gshift);
  return e == cudaSuccess ? SMP_OK : SMP_ERR_CUDA;
}

}  // namespace

int score_enqueue(const ScoreArgs& a, int dtype, cudaStream_t st) {
  const int sms = sc_sm_count();
  if (sms < 1) return SMP_ERR_CUDA;
  switch (dtype) {
    case SMP_F32: return launch_score<SMP_F32>(a, sms, st);
    case SMP_BF16: return launch_score<SMP_BF16>(a, sms, st);
    default: return launch_score<SMP_F16>(a, sms, st);
  }
}

}  // namespace smp
