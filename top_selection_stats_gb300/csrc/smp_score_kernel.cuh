// smp_score_kernel.cuh -- log probabilities of given tokens, entropy, rank and
// the n most likely alternatives (smp_token_logprobs), in one pass over each
// row; instantiated per type in smp_score_{f32,bf16,f16}.cu.
//
// A row is cut into segments, one per CTA of a cluster of 1 to 8.  A warp takes
// chunks of 32 x NU 16-byte vectors and folds each, after one look at every
// lane's maximum, into the lanes' softmax states (smp_score.cuh); the target's
// rank is counted only by lanes that hold something at or above its logit.
//   Short segments (one chunk a warp): every load is issued at once, before the
//   row's parameters arrive, and the chunk stays in registers.
//   Long segments: each warp streams its chunks through a ring of its own in
//   shared memory (bulk copies, one mbarrier a stage), so that the bytes in
//   flight do not depend on registers and no warp waits for another.
//
// Alternatives: the warps' q largest lane maxima, 64 values over the cluster, are
// distinct elements of the row, so the n-th largest of them bounds the n-th
// best from below; hardly more than n values lie above it.  They are taken from
// the registers (short) or from the few buckets, groups of one lane's chunks,
// whose maximum reaches the bound, read again (long), and ranked by counting
// in a list of SCAND.  When more are found (ties, rows sorted by id), the n-th
// best of those in the list is a better bound, and the search is repeated with
// it until the list holds them all.  Keys are (logit, smallest id first), all
// different, so the result is exact and the same whatever the order in which
// candidates arrive.
#pragma once

#include <cooperative_groups.h>

#include "smp_device.cuh"
#include "smp_score.cuh"

namespace smp {
namespace {

constexpr int SBUCKETS = 8;   // buckets per thread, at most (long segments)
constexpr int SCAND = 512;    // candidates ranked at a time
constexpr int SMAXC = 8;      // CTAs of a row, at most
constexpr int SKEPT = 64;      // short segments: vectors with candidates kept in shared memory
constexpr int SROWS = 3;      // CTAs of 256 threads on an SM
constexpr int SSMALL = 16;    // and of 64
constexpr int SFIRST = 64;    // values the first bound is taken from
constexpr int SLNU = 3;       // long segments: log2 of a lane's vectors in a chunk
// Ring: chunks a warp has in flight.  Two where the stream of bytes is the bound (4093
// x 128256 bf16 without alternatives 152 us, 158 with one; 4000 x 128256 masked 178 and
// 185; 2000 x 128256 f32 155 and 161); one where the row's other work is, 16-bit logits
// with alternatives: what the ring leaves is cache for what is read again (512 x 151936
// masked with 8: 48.3 us, 50.4 with two; 2000 x 40000 with 5: 51.1 and 53.8).
constexpr int ring_stages(int dt, bool top) { return dt != SMP_F32 && top ? 1 : 2; }
constexpr int SMOST = 2;      // the larger of both
// Legal values of a lane in a chunk (of 64 or 32) that are taken one by one from the
// stage: 912 x 151936 bf16 with 8 alternatives, a third of the rows with one token in
// twenty legal, 72.2 us, 75.2 with every chunk taken whole; 512 rows 48.5 and 50.4.
constexpr int SFEW = 12;
constexpr float SLAG = 8.f;

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
  // the larger and the smaller of each value; NaN loses
  static __device__ __forceinline__ uint32_t max_num(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (DT == SMP_F32) asm("max.f32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else if constexpr (DT == SMP_BF16) asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ uint32_t min_num(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (DT == SMP_F32) asm("min.f32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else if constexpr (DT == SMP_BF16) asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float bottom(uint32_t a) {
    if constexpr (DT == SMP_F32) return __uint_as_float(a);
    else if constexpr (DT == SMP_BF16) return fminf(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
    else return fminf(__half2float(__ushort_as_half((unsigned short)(a & 0xffffu))),
                      __half2float(__ushort_as_half((unsigned short)(a >> 16))));
  }
  // 16-bit types: two values, each 1 where a > b, else 0; and their sums, exact up to 256
  static __device__ __forceinline__ uint32_t above(uint32_t a, uint32_t b) {
    if constexpr (DT == SMP_BF16) {
      const __nv_bfloat162 r = __hgt2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
      return *reinterpret_cast<const uint32_t*>(&r);
    } else {
      const __half2 r = __hgt2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
      return *reinterpret_cast<const uint32_t*>(&r);
    }
  }
  static __device__ __forceinline__ uint32_t sum(uint32_t a, uint32_t b) {
    if constexpr (DT == SMP_BF16) {
      const __nv_bfloat162 r = __hadd2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
      return *reinterpret_cast<const uint32_t*>(&r);
    } else {
      const __half2 r = __hadd2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
      return *reinterpret_cast<const uint32_t*>(&r);
    }
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

// A vector of a row that is read once.
__device__ __forceinline__ uint4 load_vector(const uint4* p) {
  uint4 q;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
               : "l"(p));
  return q;
}

// A chunk's words of the mask, shifted so that they start at the chunk's first value: p
// is this lane's first of them, `left` how many the row has from the chunk's first on.
template <int NW>
__device__ __forceinline__ void load_bits(uint32_t (&w)[NW], const uint32_t* p, int shift, int left) {
  const int lane = threadIdx.x & 31;
  const bool inside = left > NW * 32;  // the word after the last is the row's too
#pragma unroll
  for (int i = 0; i < NW; ++i) w[i] = inside || i * 32 + lane < left ? p[i * 32] : 0u;
  if (shift) {
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const uint32_t next = inside || i * 32 + lane + 1 < left ? p[i * 32 + 1] : 0u;
      w[i] = __funnelshift_r(w[i], next, shift);
    }
  }
}

enum { SC_NONFINITE = 1, SC_LATE = 2 };

// What a CTA hands to the row's first one.
struct Part {
  float m, S, U;
  int ahead, bad, kept;
};

// What the search for alternatives uses; long segments put it where the ring was.
template <int ST, bool LONG>
struct Lists {
  uint64_t cand[SCAND];
  uint64_t tops[SMAXC][SC_MAX_TOP];  // first CTA: the n best of each
  uint64_t all[SMAXC * SC_MAX_TOP];
  uint64_t best[SC_MAX_TOP];
  uint32_t first[SFIRST];
  // long: buckets to read again; short: vectors, the first SKEPT of them kept
  unsigned short queue[(LONG ? SBUCKETS : 8) * ST];
  uint4 kept[LONG ? 1 : SKEPT];
};

template <int ST, bool LONG, bool TOP>
struct Scratch {
  static constexpr int SW = ST / 32;
  alignas(16) unsigned char lists[TOP && !LONG ? sizeof(Lists<ST, LONG>) : 16];
  uint64_t full[LONG ? SW * SMOST : 1];
  uint32_t bucket[LONG && TOP ? SBUCKETS * ST : 1];
  Part part[SMAXC];  // first CTA: the states of all
  Part warp[SW];
  uint32_t kth[SFIRST];
  uint64_t bound;
  uint32_t low;
  int queued, found, ok;
  float m, log_mass;  // of the row, for the alternatives
};

template <int DT, int ST, bool LONG, bool TOP, bool MASK>
__global__ void __launch_bounds__(ST, ST == 64 ? SSMALL : SROWS * 256 / ST)
    score_kernel(const ScoreArgs a, const int row_ctas, const int seg, const int gshift,
                 const int r0, const bool more) {
  const int nc = ST == 256 ? row_ctas : 1;  // CTAs of 64 threads have whole rows
  using TY = ScType<DT>;
  using raw = typename TY::raw;
  using WD = Word<DT>;
  constexpr int SW = ST / 32;
  constexpr int VE = 16 / (int)sizeof(raw);
  constexpr int NU = LONG ? 1 << SLNU : 8;  // vectors of a lane in a chunk
  constexpr int CV = 32 * NU;               // vectors of a chunk
  constexpr int NW = CV * VE / 1024;        // mask words of a lane
  __shared__ __align__(16) Scratch<ST, LONG, TOP> sh;
  extern __shared__ __align__(128) uint8_t ring_raw[];
  constexpr int SSTAGES = ring_stages(DT, TOP);
  using LI = Lists<ST, LONG>;
  static_assert(!LONG || sizeof(LI) <= (ST * 16 << SLNU) * SSTAGES, "the lists fit where the ring was");
  LI& li = *reinterpret_cast<LI*>(LONG ? ring_raw : sh.lists);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = r0 + blockIdx.x / nc, rank_c = blockIdx.x % nc;
  const raw* row = static_cast<const raw*>(a.logits) + (size_t)r * a.ld;
  const uint32_t* bm = MASK ? a.bitmask + (size_t)r * a.W : nullptr;
  auto legal = [&](int j) { return !MASK || ((bm[j >> 5] >> (j & 31)) & 1u); };

  // Vectors are aligned in memory: vector v has elements v VE - lead + [0, VE).
  // [f0, f1) lie inside the row; what is left at its ends, fewer than 2 VE
  // values, goes one to a lane of the first CTA's first warp.
  const int lead = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(raw));
  const int f0 = lead ? 1 : 0, f1 = max(f0, (a.V + lead) / VE);
  const int v0 = min(f1, f0 + rank_c * seg), v1 = min(f1, v0 + seg);
  const uint4* src = reinterpret_cast<const uint4*>(row - lead);
  // this warp's first chunk; long: the next is SW * CV further; short: the segment in
  // even parts of whole rounds of 32 vectors
  const int part_v = LONG ? CV : (v1 - v0 + SW * 32 - 1) / (SW * 32) * 32;
  const int mine = v0 + warp * part_v, stop = LONG ? v1 : min(v1, mine + part_v);
  const int chunks = max(0, (stop - mine + SW * CV - 1) / (SW * CV));

  uint4 x[NU];
  uint32_t bits[MASK ? NW : 1];
  uint4* ring = reinterpret_cast<uint4*>(ring_raw) + warp * (SSTAGES * CV);
  uint64_t* full = sh.full + (LONG ? warp * SSTAGES : 0);
  // Chunk i into its stage; what it does not fill holds nothing, written by the lane that
  // reads it (only votes lie between the two, which order no memory of other lanes).
  auto fetch = [&](int i) {
    if (i >= chunks) return;
    const int c = mine + i * (SW * CV), k = min(CV, v1 - c);
    uint4* stage = ring + (i % SSTAGES) * CV;
    for (int e = k + ((lane - k) & 31); e < CV; e += 32) stage[e] = make_uint4(WD::NONE, WD::NONE, WD::NONE, WD::NONE);
    if (lane == 0) {
      fence_proxy_async_smem();
      mbar_arrive_expect_tx(&full[i % SSTAGES], k * 16);
      bulk_g2s(stage, src + c, k * 16, &full[i % SSTAGES]);
    }
  };
  if (LONG && lane == 0) {
    for (int i = 0; i < SSTAGES; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  __syncwarp();
  // A call of one launch gets ready under the end of the work before it on the stream
  // (8 x 128256: 4.3 to 4.0 us): nothing of a caller's is read or written before that
  // is complete.  It lets no other start early, whose CTAs would take their places
  // while these still have theirs, unevenly (256 x 128256 with 20 top: 26.6 us, not
  // 21.6).  Of a call of two or three launches the first starts after everything before
  // it, and each later one once all CTAs of the one before it have started: all read only
  // what was complete before the call, and their rows are their own.
  if (r0 == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (more) asm volatile("griddepcontrol.launch_dependents;");
  if (LONG) {
    for (int i = 0; i < SSTAGES; ++i) fetch(i);
    __syncwarp();
  } else {  // on its way before the row's parameters are waited for
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int v = mine + u * 32 + lane;
      x[u] = make_uint4(WD::NONE, WD::NONE, WD::NONE, WD::NONE);
      if (v < stop) x[u] = load_vector(src + v);
    }
  }
  static_assert(NW * 32 == CV * VE / 32, "a chunk has whole words for each lane");
  // the next chunk's words: their place in the row and its remainder
  const int bit0 = mine * VE - lead;
  const uint32_t* words = bm + (MASK ? (bit0 >> 5) + lane : 0);
  int words_left = a.W - (bit0 >> 5);
  if constexpr (MASK) {
    if (chunks) load_bits(bits, words, bit0 & 31, words_left);
  }

  const float T = a.temperature ? a.temperature[r] : 1.f;
  const int t = a.targets ? a.targets[r] : -1;
  const bool valid = sc_temperature_ok(T) && t >= -1 && t < a.V;
  const float s = sc_scale(valid ? T : 1.f);
  const float xt = valid && t >= 0 && legal(t) ? TY::value(row[t]) : -INFINITY;
  // counted: values at or above this (nothing without a target or a rank)
  const float xc = valid && t >= 0 && a.rank ? xt : INFINITY;
  int edge = -1;
  if (rank_c == 0 && warp == 0) {
    const int head = lead ? min(a.V, VE - lead) : 0;
    const int j = lane < head ? lane : max(head, f1 * VE - lead) + lane - head;
    if (j < a.V && legal(j)) edge = j;
  }
  const float xe = edge >= 0 ? TY::value(row[edge]) : -INFINITY;

  // The lane's sums are relative to ref, which follows its largest value mx only
  // when that has left it by a factor of 2^SLAG: most chunks have a lane with
  // a new largest value, few one that is far above.
  float ref = -INFINITY, mx = -INFINITY;
  f32x2 S2 = pair(0.f, 0.f), U2 = pair(0.f, 0.f);
  const f32x2 s2 = pair(s, s);
  // 16-bit types: the target's logit in both halves, and the next smaller one, which
  // is what a token before the target has to be above to come first
  uint32_t same2 = 0u, less2 = 0u;
  if constexpr (DT != SMP_F32) {
    const uint32_t b = TY::store(xt), prev = b == 0u ? 0x8001u : b & 0x8000u ? b + 1 : b - 1;
    same2 = b * 0x00010001u;
    less2 = (xt == -INFINITY ? b : prev) * 0x00010001u;
  }
  int ahead = 0, bad = 0;
  // x: the chunk whose first vector is c
  // The mask's bits of this lane's values in the chunk, VE for each vector: the
  // first 32 in lo, the others in hi.
  auto lane_bits = [&](uint32_t& lo, uint32_t& hi) {
    uint32_t w[NU];
#pragma unroll
    for (int u = 0; u < NU; ++u) w[u] = __shfl_sync(0xffffffffu, bits[(u * VE) / 32], (u * VE + lane * VE / 32) & 31);
    lo = hi = 0u;
    if constexpr (VE == 8) {  // byte lane % 4 of each word
      const uint32_t two = (lane & 3) * 0x11 + 0x40;
#pragma unroll
      for (int h = 0; h < NU; h += 4) {
        const uint32_t b = __byte_perm(__byte_perm(w[h], w[h + 1], two), __byte_perm(w[h + 2], w[h + 3], two), 0x5410);
        (h ? hi : lo) = b;
      }
    } else {
#pragma unroll
      for (int u = 0; u < NU; ++u) lo |= ((w[u] >> (lane * VE & 31)) & ((1u << VE) - 1)) << (u * VE);
    }
  };
  auto mask_chunk = [&](uint32_t lo, uint32_t hi) {
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const uint32_t b = (u * VE < 32 ? lo : hi) >> (u * VE & 31);
      x[u].x = WD::keep(x[u].x, b, 0);
      x[u].y = WD::keep(x[u].y, b, 1);
      x[u].z = WD::keep(x[u].z, b, 2);
      x[u].w = WD::keep(x[u].w, b, 3);
    }
  };
  auto all_legal = [&]() {  // as in most rows
    uint32_t every = bits[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) every &= bits[w];
    return (bool)__all_sync(0xffffffffu, every == 0xffffffffu);
  };
  auto chunk_top = [&]() {
    uint32_t wm = WD::NONE;
#pragma unroll
    for (int u = 0; u < NU; ++u)
      wm = WD::max_nan(wm, WD::max_nan(WD::max_nan(x[u].x, x[u].y), WD::max_nan(x[u].z, x[u].w)));
    return WD::top(wm);
  };
  auto follow = [&](float top) {  // mx and ref, before values up to top are added
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(mx) : "f"(mx), "f"(top));
    const bool raise = (top - ref) * s > SLAG;
    if (__any_sync(0xffffffffu, raise)) {
      const float d = !raise ? 0.f : ref == -INFINITY ? SC_DMIN : fmaxf((ref - top) * s, SC_DMIN);
      const float e = sc_ex2(d);
      U2 = mul2(fma2(S2, pair(d, d), U2), pair(e, e));
      S2 = mul2(S2, pair(e, e));
      if (raise) ref = top;
    }
  };
  auto fold = [&](int c, float top) {
    follow(top);
    if (__any_sync(0xffffffffu, top >= xc)) {
      uint32_t n2 = 0u;
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const int j0 = (c + u * 32 + lane) * VE - lead;
        if (DT == SMP_F32 || (j0 <= t && j0 + VE > t)) {
          float f[VE];
          sc_unpack<DT>(x[u], f);
#pragma unroll
          for (int i = 0; i < VE; ++i) ahead += f[i] > xt || (f[i] == xt && j0 + i < t && xt > -INFINITY);
        } else if constexpr (DT != SMP_F32) {
          const uint32_t b = j0 < t ? less2 : same2;
          n2 = WD::sum(n2, WD::sum(WD::sum(WD::above(x[u].x, b), WD::above(x[u].y, b)),
                                   WD::sum(WD::above(x[u].z, b), WD::above(x[u].w, b))));
        }
      }
      if constexpr (DT != SMP_F32) ahead += (int)(TY::value((raw)n2) + TY::value((raw)(n2 >> 16)));
    }
    const float base = ref == -INFINITY ? 0.f : -ref;
    const f32x2 mm = pair(base, base);
    // no -inf, and none so low that d would be: nothing to clamp
    uint32_t wm = x[0].x;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      if (!LONG && u * 32 >= part_v) break;
      wm = WD::min_num(wm, WD::min_num(WD::min_num(x[u].x, x[u].y), WD::min_num(x[u].z, x[u].w)));
    }
    if (__all_sync(0xffffffffu, (WD::bottom(wm) - ref) * s > -1.0e30f)) {
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        if (!LONG && u * 32 >= part_v) break;
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
      for (int u = 0; u < NU; ++u) {
        if (!LONG && u * 32 >= part_v) break;
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

  if (LONG) {
    float bmax = -INFINITY;
    for (int i = 0; i < chunks; ++i) {
      const int c = mine + i * (SW * CV), slot = i % SSTAGES;
      int most = SFEW + 1;  // legal values of a lane, at most
      uint32_t lo = 0u, hi = 0u;
      bool whole = true;
      if constexpr (MASK) {
        whole = all_legal();
        if (!whole) {
          lane_bits(lo, hi);
          most = __reduce_max_sync(0xffffffffu, __popc(lo) + __popc(hi));
        }
        words += SW * CV * VE / 32;
        words_left -= SW * CV * VE / 32;
        if (i + 1 < chunks) load_bits(bits, words, bit0 & 31, words_left);
      }
      if (!__all_sync(0xffffffffu, sc_wait(smem_u32(&full[slot]), (i / SSTAGES) & 1, a.wait_limit))) {
        // no copy is left in flight, into what is used for other things next; then the warp
        // goes on without the rest of its chunks
        for (int k = i; k < min(chunks, i + SSTAGES); ++k)
          sc_wait(smem_u32(&full[k % SSTAGES]), (k / SSTAGES) & 1, SC_WAIT);
        bad = SC_LATE;
        break;
      }
      float top = -INFINITY;
      if (MASK && most <= SFEW) {  // few: taken one by one, straight from the stage
        const raw* stage = reinterpret_cast<const raw*>(ring + slot * CV + lane);
        const int first = (c + lane) * VE - lead;
        float y[SFEW];
#pragma unroll
        for (int k = 0; k < SFEW; ++k) {
          if (k >= most) break;
          const bool low = lo != 0u;
          const uint32_t b = low ? lo : hi;
          const int e = (b ? __ffs(b) - 1 : 0) + (low ? 0 : 32);
          const int at = (e & ~(VE - 1)) * 32 + (e & (VE - 1));
          y[k] = b ? TY::value(stage[at]) : -INFINITY;
          (low ? lo : hi) = b & (b - 1);
          if (y[k] >= xc) ahead += y[k] > xt || (y[k] == xt && first + at < t && xt > -INFINITY);
          asm("max.NaN.f32 %0, %1, %2;" : "=f"(top) : "f"(top), "f"(y[k]));
        }
        __syncwarp();  // the stage has been read
        follow(top);
        fetch(i + SSTAGES);
        const float base = ref == -INFINITY ? 0.f : ref;
        float S = 0.f, U = 0.f;
#pragma unroll
        for (int k = 0; k < SFEW; ++k) {
          if (k >= most) break;
          const float d = fmaxf((y[k] - base) * s, SC_DMIN), e = sc_ex2(d);
          S += e;
          U = fmaf(e, d, U);
        }
        S2 = add2(S2, pair(S, 0.f));
        U2 = add2(U2, pair(U, 0.f));
      } else {
#pragma unroll
        for (int u = 0; u < NU; ++u) x[u] = ring[slot * CV + u * 32 + lane];
        if (!whole) mask_chunk(lo, hi);
        top = chunk_top();
        __syncwarp();  // the stage has been read: every lane's values have gone into its top
        fetch(i + SSTAGES);
        fold(c, top);
      }
      if constexpr (TOP) {
        bmax = fmaxf(bmax, top);
        if (((i + 1) & ((1 << gshift) - 1)) == 0 || i + 1 == chunks) {
          sh.bucket[(i >> gshift) * ST + tid] = order32(bmax);
          bmax = -INFINITY;
        }
      }
    }
  } else if (chunks) {
    if constexpr (MASK) {
      uint32_t lo, hi;
      lane_bits(lo, hi);
      if (!all_legal()) mask_chunk(lo, hi);
    }
    fold(mine, chunk_top());
  }

  // the CTA's state
  Soft st;
  {
    float a0, a1, b0, b1;
    unpair(S2, a0, a1);
    unpair(U2, b0, b1);
    const float d = mx == -INFINITY ? 0.f : (ref - mx) * s, c = sc_ex2(d);  // from ref to mx
    st.m = mx;
    st.S = (a0 + a1) * c;
    st.U = (b0 + b1 + (a0 + a1) * d) * c;
    if (!(mx < INFINITY)) bad |= SC_NONFINITE;
  }
  if (edge >= 0) {
    if (!(xe < INFINITY)) bad |= SC_NONFINITE;
    sc_add(st, xe, s);
    ahead += xe >= xc && (xe > xt || (xe == xt && edge < t && xt > -INFINITY));
  }
  st = sc_warp_merge(st, s);
  ahead = __reduce_add_sync(0xffffffffu, ahead);
  bad = __reduce_or_sync(0xffffffffu, bad);
  if (lane == 0) sh.warp[warp] = Part{st.m, st.S, st.U, ahead, bad, 0};

  const int n = a.n;
  // twice as many values as asked for, or as many as fit: hardly fewer make the bound loose
  const int q = TOP ? min(min(SFIRST, 2 * n) / (nc * SW) + 1, min(SFIRST / (nc * SW), n)) : 0;
  if constexpr (TOP) {  // the warp's q largest lane maxima
    uint32_t key = order32(mx), mineq = 0u;
    for (int k = 0; k < q; ++k) {
      const uint32_t top = __reduce_max_sync(0xffffffffu, key);
      const uint32_t who = __ballot_sync(0xffffffffu, key == top);
      if (lane == __ffs(who) - 1) key = 0u;
      if (lane == k) mineq = top;
    }
    if (lane < q) sh.kth[warp * q + lane] = mineq;
    for (int k = SW * q + tid; k < SFIRST; k += ST) sh.kth[k] = 0u;
    if (tid == 0) sh.queued = sh.found = 0;
  }
  if (nc > 1) {  // all CTAs of the row have started, and have their maxima in place
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  // One warp: the row's results from the states of its parts.
  auto finish = [&](const Part* parts, int count) {
    const Part w = lane < count ? parts[lane] : Part{-INFINITY, 0.f, 0.f, 0, 0, 0};
    const Soft b = sc_warp_merge(Soft{w.m, w.S, w.U}, s);
    const int before = __reduce_add_sync(0xffffffffu, w.ahead);
    const int wrong = __reduce_or_sync(0xffffffffu, w.bad);
    if (lane) return;
    const int status = wrong & SC_LATE ? SMP_ERR_TIMEOUT : !valid ? SMP_ERR_INVALID_PARAM : wrong ? SMP_ERR_NONFINITE
                       : b.m == -INFINITY ? SMP_ERR_EMPTY : SMP_OK;
    const bool ok = status == SMP_OK;
    const float L = sc_log_mass(b);
    a.status[r] = status;
    if (a.logprobs) a.logprobs[r] = !ok ? sc_nan() : t < 0 ? 0.f : sc_logprob(xt, b.m, L, T);
    if (a.entropy) a.entropy[r] = ok ? sc_entropy(b, L) : sc_nan();
    if (a.rank) a.rank[r] = ok && t >= 0 ? before : -1;
    if (a.stats) {
      a.stats[2 * (size_t)r] = ok ? b.m : sc_nan();
      a.stats[2 * (size_t)r + 1] = ok ? L : sc_nan();
    }
    if (TOP) {
      sh.ok = ok;
      sh.m = b.m;
      sh.log_mass = L;
    }
  };
  Part* part = nc > 1 ? cg::this_cluster().map_shared_rank(&sh.part[rank_c], 0) : &sh.part[0];
  if (TOP && nc == 1 && warp == SW - 1) finish(sh.warp, SW);  // while the others search
  if (nc > 1 && warp == SW - 1) {
    const Part w = lane < SW ? sh.warp[lane] : Part{-INFINITY, 0.f, 0.f, 0, 0, 0};
    st = sc_warp_merge(Soft{w.m, w.S, w.U}, s);
    ahead = __reduce_add_sync(0xffffffffu, w.ahead);
    bad = __reduce_or_sync(0xffffffffu, w.bad);
    if (lane == 0) {
      part->m = st.m;
      part->S = st.S;
      part->U = st.U;
      part->ahead = ahead;
      part->bad = bad;
    }
  }

  int kept = 0;
  if constexpr (TOP) {
    const uint32_t* firsts = sh.kth;
    if (nc > 1) {
      if (tid < SFIRST) {
        const int each = SW * q, owner = tid / each;
        li.first[tid] = owner < nc ? *cg::this_cluster().map_shared_rank(&sh.kth[tid % each], owner) : 0u;
      }
      firsts = li.first;
      __syncthreads();
    }
    if (tid < SFIRST) {
      const uint32_t v = firsts[tid];
      int above = 0;
#pragma unroll 16
      for (int i = 0; i < SFIRST; ++i) above += firsts[i] > v || (firsts[i] == v && i < tid);
      if (above == n - 1) sh.low = max(v, 1u);  // 0: fewer than n; any legal value
    }
    // a CTA with a late copy has not all its buckets, and its row fails: it searches nothing
    const bool late = __syncthreads_or(bad & SC_LATE);
    const uint32_t low = sh.low;
    uint64_t bound = (uint64_t)low << 32;
    auto offer = [&](float y, int j) {
      const uint32_t o = order32(y);
      const uint64_t k = order_key(o, j);
      if (o && k >= bound && *reinterpret_cast<volatile int*>(&sh.found) <= SCAND) {
        const int p = atomicAdd(&sh.found, 1);
        if (p < SCAND) li.cand[p] = k;
      }
    };
    // The vector's legal values (a bit each) at or above the bound.  Small code rather
    // than unrolled: what runs once per row pays for its fetch.
    auto offer_vector = [&](const uint4& y, int j0, uint32_t which) {
      const float least = key_value(max(bound, (uint64_t)0x00800000u << 32));  // any finite value, at least
      float f[VE];
      sc_unpack<DT>(y, f);
      uint32_t hits = 0u;
#pragma unroll
      for (int i = 0; i < VE; ++i) hits |= f[i] >= least ? 1u << i : 0u;
      hits &= which;
      while (hits) {
        const int i = __ffs(hits) - 1, w = DT == SMP_F32 ? i : i >> 1;
        hits &= hits - 1;
        const uint32_t lo = w & 1 ? y.y : y.x, hi = w & 1 ? y.w : y.z, word = w & 2 ? hi : lo;
        raw value;
        if constexpr (DT == SMP_F32) value = __uint_as_float(word);
        else value = (raw)(i & 1 ? word >> 16 : word);
        offer(TY::value(value), j0 + i);
      }
    };
    if constexpr (LONG) {
      const int buckets = late ? 0 : (chunks + (1 << gshift) - 1) >> gshift;
      for (int b = 0; b < buckets; ++b)
        if (sh.bucket[b * ST + tid] >= low) li.queue[atomicAdd(&sh.queued, 1)] = (unsigned short)(b * ST + tid);
    } else if (order32(mx) >= low) {
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        if (u * 32 >= part_v) break;
        const uint32_t wm = WD::max_num(WD::max_num(x[u].x, x[u].y), WD::max_num(x[u].z, x[u].w));
        if (order32(WD::top(wm)) >= low) {
          const int p = atomicAdd(&sh.queued, 1);
          li.queue[p] = (unsigned short)(mine - v0 + u * 32 + lane);
          if (p < SKEPT) li.kept[p] = x[u];
        }
      }
    }
    __syncthreads();
    const int lv = LONG ? SLNU + gshift : 0, total = sh.queued << lv;  // vectors to look through
    int found;
    while (true) {
      if (edge >= 0) offer(xe, edge);
#pragma unroll 1
      for (int i = tid; i < total; i += ST) {
        const int item = li.queue[i >> lv];
        int v = v0 + item;
        if constexpr (LONG) {
          const int e = i & ((1 << lv) - 1), th = item % ST;
          v = v0 + ((((item / ST) << gshift) + (e >> SLNU)) * SW + th / 32) * CV + (e % NU) * 32 + th % 32;
          if (v >= v1) continue;
        }
        const bool here = !LONG && i < SKEPT;
        const int j0 = v * VE - lead;
        uint32_t which = ~0u;  // its mask is on the way together with it
        if (MASK && !here) which = __funnelshift_r(bm[j0 >> 5], bm[(j0 + VE - 1) >> 5], j0 & 31);
        offer_vector(here ? li.kept[i] : src[v], j0, which);
      }
      __syncthreads();
      found = sh.found;
      if (found <= SCAND) break;
      // the n-th best of the list bounds the n-th best of all
#pragma unroll 1
      for (int c = tid; c < SCAND; c += ST) {
        const uint64_t k = li.cand[c];
        int above = 0;
#pragma unroll 16
        for (int i = 0; i < SCAND; ++i) above += li.cand[i] > k;
        if (above == n - 1) sh.bound = k;
      }
      __syncthreads();
      bound = sh.bound;
      if (tid == 0) sh.found = 0;
      __syncthreads();
    }
    uint64_t* to = nc > 1 ? cg::this_cluster().map_shared_rank(&li.tops[rank_c][0], 0) : &li.best[0];
    for (int c = tid; c < found; c += ST) {
      const uint64_t k = li.cand[c];
      int above = 0;
#pragma unroll 8
      for (int i = 0; i < found; ++i) above += li.cand[i] > k;
      if (above < n) to[above] = k;
    }
    kept = min(found, n);
    if (nc > 1 && tid == 0) part->kept = kept;
  }

  if (nc > 1) {  // the first CTA has everything; the others may go
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (rank_c) return;
    if constexpr (TOP) {  // the CTAs' lists in one, then each key's place in it
      const int p = tid / SC_MAX_TOP, i = tid % SC_MAX_TOP;
      int at = 0, total = 0;
      for (int o = 0; o < nc; ++o) {
        if (o < p) at += sh.part[o].kept;
        total += sh.part[o].kept;
      }
      if (p < nc && i < sh.part[p].kept) li.all[at + i] = li.tops[p][i];
      __syncthreads();
      if (warp == SW - 1) finish(sh.part, nc);
      for (int c = tid; c < total; c += ST) {
        const uint64_t k = li.all[c];
        int above = 0;
#pragma unroll 8
        for (int i = 0; i < total; ++i) above += li.all[i] > k;
        if (above < n) li.best[above] = k;
      }
      kept = min(total, n);
    }
  }
  if (TOP) __syncthreads();
  if (warp) return;
  if (!TOP) finish(nc > 1 ? sh.part : sh.warp, nc > 1 ? nc : SW);
  if (TOP && lane < n) {
    const uint64_t k = lane < kept && sh.ok ? li.best[lane] : 0ull;
    a.top_ids[(size_t)r * n + lane] = k ? key_id(k) : -1;
    a.top_lp[(size_t)r * n + lane] =
        !sh.ok ? sc_nan() : k ? sc_logprob(key_value(k), sh.m, sh.log_mass, T) : -INFINITY;
  }
  // a later launch ends only after the one it started beside, so the last ends last
  if (r0 && blockIdx.x == 0 && lane == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Rows [r0, r0 + rows).
template <int DT, int ST, bool LONG>
int launch_score(const ScoreArgs& a, int r0, int rows, int nc, cudaStream_t st) {
  const bool more = r0 + rows < a.B;
  constexpr int VE = DT == SMP_F32 ? 4 : 8, step = ST * (LONG ? 1 << SLNU : 8);
  const int seg = (a.V / VE + nc - 1) / nc;
  int gshift = 0;
  while (((seg + step - 1) / step) >> gshift >= SBUCKETS) ++gshift;
  if ((long long)rows * nc > 0x7fffffffLL) return SMP_ERR_CAPACITY;
  const auto kernel = a.n ? (a.bitmask ? score_kernel<DT, ST, LONG, true, true> : score_kernel<DT, ST, LONG, true, false>)
                          : (a.bitmask ? score_kernel<DT, ST, LONG, false, true> : score_kernel<DT, ST, LONG, false, false>);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * nc));
  cfg.blockDim = dim3(ST);
  cfg.stream = st;
  if (LONG) {
    cfg.dynamicSmemBytes = (ST * 16 << SLNU) * ring_stages(DT, a.n > 0);
    if (!sc_ok(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cfg.dynamicSmemBytes)))
      return SMP_ERR_CUDA;
  }
  cudaLaunchAttribute attr[2];
  if (nc > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = (unsigned)nc;
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs++].val.clusterDim.z = 1;
  }
  if (r0 || !more) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  return sc_ok(cudaLaunchKernelEx(&cfg, kernel, a, nc, seg, gshift, r0, more)) ? SMP_OK : SMP_ERR_CUDA;
}

// Short rows, one chunk a warp, take CTAs of 2 or 4 warps, so that an SM holds many:
// 4000 x 5000 bf16 with 5 alternatives 27.2 us in CTAs of 4 warps, 33.0 of 8.
// Rows up to four times as long as 8 warps' chunks are taken by 4 warps while they
// fill the SMs (3000 x 16000 with 5: 38.9 us, 46.9 with 8), others by 8.  The rows left
// when all others fill the SMs take a launch of their own, on what the ones before leave
// free, in clusters as large as still fit at once, while a warp has more than a
// chunk: 1024 x 256000 f16 with 32 alternatives 105 us, 112 without it; 64 x 128256
// bf16 with 20: 10.1 us in clusters of 4, 14.7 of 8 (two rounds of CTAs).  So a call
// is one launch, two or, where rows of up to four times 8 warps' chunks leave at least a
// full round of CTAs of 8 warps, three.
template <int DT>
int score_rows(const ScoreArgs& a, cudaStream_t st) {
  const int sms = sc_sm_count();
  if (sms < 1) return SMP_ERR_CUDA;
  constexpr int SHORT = 256 * 8;
  const int vectors = a.V / (DT == SMP_F32 ? 4 : 8);  // whole ones, at most
  if (vectors <= 64 * 8) return launch_score<DT, 64, false>(a, 0, a.B, 1, st);
  if (vectors <= 128 * 8) return launch_score<DT, 128, false>(a, 0, a.B, 1, st);
  int done = 0;
  if (vectors <= 8192) {
    const int load = 2 * SROWS * sms;
    done = a.B / load * load;
    if (done) {
      const int rc = launch_score<DT, 128, true>(a, 0, done, 1, st);
      if (rc != SMP_OK || done == a.B) return rc;
    }
  }
  if (vectors <= SHORT) return launch_score<DT, 256, false>(a, done, a.B - done, 1, st);
  const int slots = SROWS * sms, many = (a.B - done) / slots * slots, rows = a.B - done - many;
  if (many) {
    const int rc = launch_score<DT, 256, true>(a, done, many, 1, st);
    if (rc != SMP_OK || !rows) return rc;
    done += many;
  }
  int nc = 1;
  while (nc < SMAXC && (long long)rows * nc * 2 <= slots && vectors > nc * SHORT) nc *= 2;
  return (vectors + nc - 1) / nc <= SHORT ? launch_score<DT, 256, false>(a, done, rows, nc, st)
                                          : launch_score<DT, 256, true>(a, done, rows, nc, st);
}

}  // namespace
}  // namespace smp
