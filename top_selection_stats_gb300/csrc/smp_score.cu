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

#include <type_traits>

#include "smp_score.cuh"

namespace cg = cooperative_groups;

namespace smp {
namespace {

constexpr int SULOG = 2;
constexpr int SU = 1 << SULOG;  // vectors a thread has in flight
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
  // the larger of each value; NaN loses
  static __device__ __forceinline__ uint32_t max_num(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (DT == SMP_F32) asm("max.f32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else if constexpr (DT == SMP_BF16) asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  // A value to raise all smaller ones to without changing a sum: its weight
  // is 0, it is finite and so is its d.  NONE where the type has none (and for
  // binary32, where clamping d costs no more).
  static __device__ __forceinline__ uint32_t floor_of(float m, float s) {
    if constexpr (DT == SMP_F32) return NONE;
    const float want = m - __fdividef(160.f, s);
    uint32_t h;
    float f;
    if constexpr (DT == SMP_BF16) {
      h = __bfloat16_as_ushort(__float2bfloat16_rd(want));
      f = __uint_as_float(h << 16);
    } else {
      h = __half_as_ushort(__float2half_rd(want));
      f = __half2float(__ushort_as_half((unsigned short)h));
    }
    const float d = (f - m) * s;
    return f > -INFINITY && d <= -150.f && d > -1e30f ? h * 0x00010001u : NONE;
  }
  // word i of a vector with the values whose bit is 0 replaced by -inf
  static __device__ __forceinline__ uint32_t keep(uint32_t a, uint32_t bits, int i) {
    if constexpr (DT == SMP_F32) return ((bits >> i) & 1u) ? a : NONE;
    // the two bits as the signs of a byte each, spread over 16 bits each
    const uint32_t hi = bits << (30 - 2 * i);
    uint32_t on;
    asm("prmt.b32 %0, %1, %2, 0xbbff;" : "=r"(on) : "r"(hi), "r"(hi << 1));
    return (a & on) | (NONE & ~on);
  }
};

// A vector of a row that is read once (the buckets read again come out of L2).
__device__ __forceinline__ uint4 load_vector(const uint4* p) {
  uint4 q;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
               : "l"(p));
  return q;
}

// What a CTA hands to the row's first one.
struct Part {
  float m, S, U;
  int ahead, bad, kept;
};

template <int ST>
struct Scratch {
  uint32_t bucket[SBUCKETS * ST];
  unsigned short queue[SBUCKETS * ST];
  uint64_t cand[SCAND];
  uint64_t tops[SMAXC][SC_MAX_TOP];  // first CTA: the n best of each, in order
  uint64_t best[SC_MAX_TOP];
  Part part[SMAXC];                  // first CTA: the states of all
  Part warp[ST / 32];
  uint32_t kth[ST / 32];
  uint64_t bound;
  int queued, found;
};

template <int DT, int ST, bool TOP, bool MASK>
__global__ void __launch_bounds__(ST, 4 * 256 / ST) score_kernel(const ScoreArgs a, const int nc, const int seg,
                                                                     const int gshift) {
  constexpr int SW = ST / 32;
  using TY = ScType<DT>;
  using raw = typename TY::raw;
  using WD = Word<DT>;
  constexpr int VE = 16 / (int)sizeof(raw);
  __shared__ __align__(16) Scratch<ST> sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (nc > 1) cluster_arrive();  // waited for before the first CTA's shared memory is written
  const int r = blockIdx.x / nc, rank_c = blockIdx.x % nc;
  const raw* row = static_cast<const raw*>(a.logits) + (size_t)r * a.ld;
  const uint32_t* bm = MASK ? a.bitmask + (size_t)r * a.W : nullptr;
  auto legal = [&](int j) { return !MASK || ((__ldg(bm + (j >> 5)) >> (j & 31)) & 1u); };
  // Vectors are aligned in memory: vector v has elements v VE - lead + [0, VE).
  // [f0, f1) lie inside the row; what is left at its ends, fewer than 2 VE
  // values, goes one to a lane of the first CTA's first warp.
  const int lead = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(raw));
  const int f0 = lead ? 1 : 0, f1 = max(f0, (a.V + lead) / VE);
  const int v0 = min(f1, f0 + rank_c * seg), v1 = min(f1, v0 + seg);
  const uint4* src = reinterpret_cast<const uint4*>(row - lead);
  auto load = [&](uint4 (&x)[SU], int vb) {
    uint32_t bits[SU];
#pragma unroll
    for (int u = 0; u < SU; ++u) {
      const int v = vb + u * ST + tid;
      x[u] = make_uint4(WD::NONE, WD::NONE, WD::NONE, WD::NONE);
      if (MASK) bits[u] = 0xffffffffu;
      if (v < v1) {
        x[u] = load_vector(src + v);
        if (MASK) {
          const int j0 = v * VE - lead;
          bits[u] = __funnelshift_r(__ldg(bm + (j0 >> 5)), __ldg(bm + ((j0 + VE - 1) >> 5)), j0 & 31);
        }
      }
    }
    if (MASK) {
      uint32_t all = 0xffffffffu;
#pragma unroll
      for (int u = 0; u < SU; ++u) all &= bits[u];
      if ((all & ((1u << VE) - 1)) == (1u << VE) - 1) return;  // as in most rows
#pragma unroll
      for (int u = 0; u < SU; ++u) {
        x[u].x = WD::keep(x[u].x, bits[u], 0);
        x[u].y = WD::keep(x[u].y, bits[u], 1);
        x[u].z = WD::keep(x[u].z, bits[u], 2);
        x[u].w = WD::keep(x[u].w, bits[u], 3);
      }
    }
  };
  // The first batch is on its way before the row's parameters are waited for.
  uint4 x[SU];
  load(x, v0);
  const float T = a.temperature ? a.temperature[r] : 1.f;
  const int t = a.targets ? a.targets[r] : -1;
  const bool valid = sc_temperature_ok(T) && t >= -1 && t < a.V;
  const float s = sc_scale(valid ? T : 1.f);
  const float xt = valid && t >= 0 && legal(t) ? TY::value(__ldg(row + t)) : -INFINITY;
  // counted: values at or above this (nothing without a target or a rank)
  const float xc = valid && t >= 0 && a.rank ? xt : INFINITY;
  int edge = -1;
  if (rank_c == 0 && warp == 0) {
    const int head = lead ? min(a.V, VE - lead) : 0;
    const int j = lane < head ? lane : max(head, f1 * VE - lead) + lane - head;
    if (j < a.V && legal(j)) edge = j;
  }

  float m = -INFINITY, tmax = -INFINITY, bmax = -INFINITY;
  f32x2 S2 = pair(0.f, 0.f), U2 = pair(0.f, 0.f);
  const f32x2 s2 = pair(s, s);
  uint32_t low2 = WD::NONE;  // WD::floor_of(m, s)
  int ahead = 0, batch = 0;
  bool bad = false;
  auto fold = [&](uint4 (&x)[SU], int vb) {
    uint32_t wm = WD::NONE;
#pragma unroll
    for (int u = 0; u < SU; ++u)
      wm = WD::max_nan(wm, WD::max_nan(WD::max_nan(x[u].x, x[u].y), WD::max_nan(x[u].z, x[u].w)));
    const float top = WD::top(wm);
    bad |= !(top < INFINITY);
    if (TOP) {
      bmax = fmaxf(bmax, top);
      if (((batch + 1) & ((1 << gshift) - 1)) == 0 || vb + ST * SU >= v1) {
        sh.bucket[(batch >> gshift) * ST + tid] = order32(bmax);
        tmax = fmaxf(tmax, bmax);
        bmax = -INFINITY;
      }
    }
    if (!(top > -INFINITY)) return;
    if (top > m) {
      const float d = m == -INFINITY ? SC_DMIN : fmaxf((m - top) * s, SC_DMIN);
      const float e = sc_ex2(d);
      U2 = mul2(fma2(S2, pair(d, d), U2), pair(e, e));
      S2 = mul2(S2, pair(e, e));
      m = top;
      low2 = WD::floor_of(m, s);
    }
    if (top >= xc) {
#pragma unroll
      for (int u = 0; u < SU; ++u) {
        const int j0 = (vb + u * ST + tid) * VE - lead;
        float f[VE];
        sc_unpack<DT>(x[u], f);
#pragma unroll
        for (int i = 0; i < VE; ++i) ahead += f[i] > xt || (f[i] == xt && j0 + i < t && xt > -INFINITY);
      }
    }
    const f32x2 mm = pair(-m, -m);
    if (low2 != WD::NONE) {
#pragma unroll
      for (int u = 0; u < SU; ++u) {
        x[u].x = WD::max_num(x[u].x, low2);
        x[u].y = WD::max_num(x[u].y, low2);
        x[u].z = WD::max_num(x[u].z, low2);
        x[u].w = WD::max_num(x[u].w, low2);
        float f[VE];
        sc_unpack<DT>(x[u], f);
#pragma unroll
        for (int i = 0; i < VE; i += 2) {
          const f32x2 d = mul2(add2(pair(f[i], f[i + 1]), mm), s2);
          float d0, d1;
          unpair(d, d0, d1);
          const f32x2 e = pair(sc_ex2(d0), sc_ex2(d1));
          S2 = add2(S2, e);
          U2 = fma2(e, d, U2);
        }
      }
    } else {
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
    }
  };
  for (int vb = v0; vb < v1;) {
    fold(x, vb);
    ++batch;
    vb += ST * SU;
    if (vb < v1) load(x, vb);
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
  const float xe = edge >= 0 ? TY::value(__ldg(row + edge)) : -INFINITY;
  if (edge >= 0) {
    bad |= !(xe < INFINITY);
    sc_add(st, xe, s);
    ahead += xe >= xc && (xe > xt || (xe == xt && edge < t && xt > -INFINITY));
  }
  st = sc_warp_merge(st, s);
  ahead = __reduce_add_sync(0xffffffffu, ahead);
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) sh.warp[warp] = Part{st.m, st.S, st.U, ahead, bad, 0};

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
  Part* part = nc > 1 ? cg::this_cluster().map_shared_rank(&sh.part[rank_c], 0) : &sh.part[0];
  if (warp == 0) {
    const Part w = lane < SW ? sh.warp[lane] : Part{-INFINITY, 0.f, 0.f, 0, 0, 0};
    st = sc_warp_merge(Soft{w.m, w.S, w.U}, s);
    ahead = __reduce_add_sync(0xffffffffu, w.ahead);
    bad = __any_sync(0xffffffffu, w.bad != 0);
    if (lane == 0) {
      part->m = st.m;
      part->S = st.S;
      part->U = st.U;
      part->ahead = ahead;
      part->bad = bad;
    }
  }

  if (TOP) {
    uint32_t low = sh.kth[0];
#pragma unroll
    for (int w = 1; w < SW; ++w) low = min(low, sh.kth[w]);
    if (low == 0u) low = 1u;  // any legal value
    const int buckets = (batch + (1 << gshift) - 1) >> gshift;
    for (int b = 0; b < buckets; ++b)
      if (sh.bucket[b * ST + tid] >= low) sh.queue[atomicAdd(&sh.queued, 1)] = (unsigned short)(b * ST + tid);
    uint64_t bound = (uint64_t)low << 32;
    __syncthreads();
    const int lv = SULOG + gshift, total = sh.queued << lv;  // vectors of the queued buckets
    auto offer = [&](float x, int j) {
      const uint32_t o = order32(x);
      const uint64_t k = order_key(o, j);
      if (o && k >= bound && *reinterpret_cast<volatile int*>(&sh.found) <= SCAND) {
        const int p = atomicAdd(&sh.found, 1);
        if (p < SCAND) sh.cand[p] = k;
      }
    };
    int found;
    while (true) {
      if (edge >= 0) offer(xe, edge);
      for (int i0 = tid; i0 < total; i0 += ST * 2) {
        uint4 x[2];
        int j0[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int i = i0 + q * ST;
          x[q] = make_uint4(WD::NONE, WD::NONE, WD::NONE, WD::NONE);
          j0[q] = 0;
          if (i < total) {
            const int item = sh.queue[i >> lv];
            const int v = v0 + item % ST + (((item / ST) << lv) + (i & ((1 << lv) - 1))) * ST;
            if (v < v1) {
              x[q] = __ldg(src + v);
              j0[q] = v * VE - lead;
            }
          }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float f[VE];
          sc_unpack<DT>(x[q], f);
          const uint32_t wm = WD::max_num(WD::max_num(x[q].x, x[q].y), WD::max_num(x[q].z, x[q].w));
          if (order32(WD::top(wm)) < (uint32_t)(bound >> 32)) continue;
#pragma unroll
          for (int i = 0; i < VE; ++i)
            if (order32(f[i]) >= (uint32_t)(bound >> 32) && legal(j0[q] + i)) offer(f[i], j0[q] + i);
        }
      }
      __syncthreads();
      found = sh.found;
      if (found <= SCAND) break;
      // the n-th best of the list bounds the n-th best of all
#pragma unroll 1
      for (int c = tid; c < SCAND; c += ST) {
        const uint64_t k = sh.cand[c];
        int above = 0;
#pragma unroll 16
        for (int i = 0; i < SCAND; ++i) above += sh.cand[i] > k;
        if (above == n - 1) sh.bound = k;
      }
      __syncthreads();
      bound = sh.bound;
      if (tid == 0) sh.found = 0;
      __syncthreads();
    }
    uint64_t* to = nc > 1 ? cg::this_cluster().map_shared_rank(&sh.tops[rank_c][0], 0) : &sh.best[0];
    for (int c = tid; c < found; c += ST) {
      const uint64_t k = sh.cand[c];
      int above = 0;
#pragma unroll 8
      for (int i = 0; i < found; ++i) above += sh.cand[i] > k;
      if (above < n) to[above] = k;
    }
    if (tid == 0) part->kept = min(found, n);
  }

  if (nc > 1) {  // the first CTA has everything; the others may go
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (rank_c) return;
    if (TOP) {  // a key's place: how many keys of each CTA's ordered list are above it
      for (int c = tid; c < nc * SC_MAX_TOP; c += ST) {
        const int own = c / SC_MAX_TOP, i = c % SC_MAX_TOP;
        if (i >= sh.part[own].kept) continue;
        const uint64_t k = sh.tops[own][i];
        int above = i;
#pragma unroll
        for (int p = 0; p < SMAXC; ++p) {
          if (p >= nc || p == own) continue;
          const int kept = sh.part[p].kept;
          int lo = 0;
#pragma unroll
          for (int step = SC_MAX_TOP; step > 0; step >>= 1)
            if (lo + step <= kept && sh.tops[p][lo + step - 1] > k) lo += step;
          above += lo;
        }
        if (above < n) sh.best[above] = k;
      }
    }
  }
  __syncthreads();
  if (warp) return;
  const Part w = lane < nc ? sh.part[lane] : Part{-INFINITY, 0.f, 0.f, 0, 0, 0};
  st = sc_warp_merge(Soft{w.m, w.S, w.U}, s);
  ahead = __reduce_add_sync(0xffffffffu, w.ahead);
  bad = __any_sync(0xffffffffu, w.bad != 0);
  const int kept = TOP ? __reduce_add_sync(0xffffffffu, w.kept) : 0;
  const int status = !valid ? SMP_ERR_INVALID_PARAM : bad ? SMP_ERR_NONFINITE
                     : st.m == -INFINITY ? SMP_ERR_EMPTY : SMP_OK;
  const bool ok = status == SMP_OK;
  if (lane == 0) {
    a.status[r] = status;
    if (a.logprobs) a.logprobs[r] = !ok ? sc_nan() : t < 0 ? 0.f : sc_logprob(xt, st, T);
    if (a.entropy) a.entropy[r] = ok ? sc_entropy(st) : sc_nan();
    if (a.rank) a.rank[r] = ok && t >= 0 ? ahead : -1;
    if (a.stats) {
      a.stats[2 * (size_t)r] = ok ? st.m : sc_nan();
      a.stats[2 * (size_t)r + 1] = ok ? SC_LN2 * sc_log2_mass(st) : sc_nan();
    }
  }
  if (TOP && lane < n) {
    const uint64_t k = lane < kept ? sh.best[lane] : 0ull;
    a.top_ids[(size_t)r * n + lane] = ok && k ? key_id(k) : -1;
    a.top_lp[(size_t)r * n + lane] = !ok ? sc_nan() : k ? sc_logprob(key_value(k), st, T) : -INFINITY;
  }
}

// A row short enough for two batches of 64 threads takes a CTA of 64, so that
// an SM holds 16 rows.
template <int DT, int ST>
int launch_score(const ScoreArgs& a, int sms, cudaStream_t st) {
  constexpr int VE = DT == SMP_F32 ? 4 : 8;
  const int vectors = a.V / VE;
  constexpr int step = ST * SU;
  int nc = 1;
  while (nc < SMAXC && (long long)a.B * nc < 4LL * sms && vectors > nc * step) nc *= 2;
  const int seg = max(1, ((vectors + nc - 1) / nc + ST - 1) / ST) * ST;
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
  const auto kernel = a.n ? (a.bitmask ? score_kernel<DT, ST, true, true> : score_kernel<DT, ST, true, false>)
                          : (a.bitmask ? score_kernel<DT, ST, false, true> : score_kernel<DT, ST, false, false>);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a, nc, seg, gshift);
  return e == cudaSuccess ? SMP_OK : SMP_ERR_CUDA;
}

template <int DT>
int choose_score(const ScoreArgs& a, cudaStream_t st) {
  const int sms = sc_sm_count();
  if (sms < 1) return SMP_ERR_CUDA;
  return a.V <= 2 * 64 * SU * (DT == SMP_F32 ? 4 : 8) ? launch_score<DT, 64>(a, sms, st)
                                                     : launch_score<DT, 256>(a, sms, st);
}

}  // namespace

int score_enqueue(const ScoreArgs& a, int dtype, cudaStream_t st) {
  switch (dtype) {
    case SMP_F32: return choose_score<SMP_F32>(a, st);
    case SMP_BF16: return choose_score<SMP_BF16>(a, st);
    default: return choose_score<SMP_F16>(a, st);
  }
}

}  // namespace smp
