// smp_distill_kernel.cuh -- divergence of a student's distribution from a teacher's top
// tokens (smp_distill_loss), in one pass over each row; instantiated per type in
// smp_distill_{f32,bf16,f16}.cu.
//
// A row is cut into segments, one per CTA of a cluster of 1 to 8.  Each warp streams
// chunks of its segment through a ring of its own in shared memory (bulk copies, one
// mbarrier a stage) and folds them into its lanes' softmax states.  The teacher's
// tokens are kept out of these sums by writing -inf over them in the staged chunk
// before it is read: a few comparisons per chunk, where a test at each logit would
// cost more than the sums.  Their own logits are fetched one by one at the start,
// under the first copies, and enter at the end (distill_finish).  A sum has no
// second moment here, so -inf needs no clamp: 2^-inf is 0.
//
// Bound by HBM where rows fill the SMs: 4096 x 128256 bf16 with 32 slots 157 us, 6.7 TB/s (a
// copy of as many bytes: 156); 1024 x 256000 f16 with 128: 90 us (78), 2.25 rounds of rows.
// One row of 128256: 7.6 us, a launch and the chain of slots, stream, cluster and finish.
#pragma once

#include "smp_distill.cuh"
#include "smp_score_kernel.cuh"

namespace smp {
namespace {

constexpr int DI_STAGES = 2;  // chunks a warp has in flight
// Products x s below this are rounded by half a unit at most, so that a sum relative to a
// rounded one has a value next to its reference between 2^-1/2 and 2^1/2 (at 2^34 it would be
// off by up to 2^9, past what 2^x can hold).
constexpr float DI_NEAR = 0x1p24f;

struct DistillPart {
  float m, S;
  int wrong;
};

template <int ST>
struct DistillScratch {
  Slots slots;
  RowResult row;
  uint64_t full[ST / 32 * DI_STAGES];
  int seen[DI_MAX_K * 2];  // ids by open addressing; more than 32 slots
  DistillPart part[SMAXC];  // first CTA: the states of all
  DistillPart warp[ST / 32 + 1];
};

// cv: vectors of a chunk, a multiple of 32, at most 32 << SLNU.
// EXTRA: one more warp takes the slots and finishes the row, while the others stream from the
// start; without it all warps share the slots first.
template <int DT, int ST, bool MASK, bool EXTRA>
__global__ void __launch_bounds__(ST + (EXTRA ? 32 : 0), ST == 64 ? SSMALL : SROWS * 256 / ST)
    distill_kernel(const DistillArgs a, const int row_ctas, const int seg, const int cv, const int r0,
                   const bool more) {
  const int nc = ST == 256 && !EXTRA ? row_ctas : 1;
  using TY = ScType<DT>;
  using raw = typename TY::raw;
  using WD = Word<DT>;
  constexpr int SW = ST / 32;
  constexpr int VE = 16 / (int)sizeof(raw);
  constexpr int NU = 1 << SLNU;  // vectors of a lane in a chunk, at most
  constexpr int CV = 32 * NU;
  constexpr int NW = CV * VE / 1024;  // mask words of a lane
  constexpr int WF = EXTRA ? SW : 0;  // the warp that finishes the row
  __shared__ __align__(16) DistillScratch<ST> sh;
  extern __shared__ __align__(128) uint8_t ring_raw[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, K = a.K;
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
  const int mine = v0 + warp * cv;  // this warp's first chunk; the next is SW * cv further
  const bool streams = !EXTRA || warp < SW;
  const int chunks = streams ? max(0, (v1 - mine + SW * cv - 1) / (SW * cv)) : 0;
  uint4* ring = reinterpret_cast<uint4*>(ring_raw) + warp * (DI_STAGES * cv);
  uint64_t* full = sh.full + warp * DI_STAGES;
  // Chunk i into its stage; what it does not fill holds nothing, written by the lane that
  // reads it.  Every lane has read (and written -inf over) the stage's chunk before it.
  auto fetch = [&](int i) {
    if (i >= chunks) return;
    const int c = mine + i * (SW * cv), k = min(cv, v1 - c);
    uint4* stage = ring + (i % DI_STAGES) * cv;
    for (int e = k + ((lane - k) & 31); e < cv; e += 32) stage[e] = make_uint4(WD::NONE, WD::NONE, WD::NONE, WD::NONE);
    if (lane == 0) {
      fence_proxy_async_smem();
      mbar_arrive_expect_tx(&full[i % DI_STAGES], k * 16);
      bulk_g2s(stage, src + c, k * 16, &full[i % DI_STAGES]);
    }
  };
  if (lane == 0 && streams) {
    for (int i = 0; i < DI_STAGES; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (rank_c == 0 && K > 32)
    for (int i = EXTRA ? lane : tid; i < 2 * DI_MAX_K && (!EXTRA || warp == SW); i += EXTRA ? 32 : ST) sh.seen[i] = -1;
  if (EXTRA) __syncwarp();
  else __syncthreads();
  // The launches of a call follow each other, and the work before them, as those of
  // smp_token_logprobs do.
  if (r0 == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (more) asm volatile("griddepcontrol.launch_dependents;");
  for (int i = 0; i < DI_STAGES; ++i) fetch(i);
  __syncwarp();
  uint32_t bits[MASK ? NW : 1];
  const int bit0 = mine * VE - lead;  // the next chunk's words: their place in the row and its remainder
  const uint32_t* words = bm + (MASK ? (bit0 >> 5) + lane : 0);
  int words_left = a.W - (bit0 >> 5);
  if constexpr (MASK) {
    if (chunks) load_bits(bits, words, bit0 & 31, words_left);
  }

  const float T = a.temperature ? a.temperature[r] : 1.f;
  const int t = a.targets ? a.targets[r] : -1;
  int wrong = sc_temperature_ok(T) && t >= -1 && t < a.V ? 0 : DI_INVALID;
  const float s = sc_scale(wrong ? 1.f : T);
  const float xt = rank_c == 0 && !wrong && t >= 0 && legal(t) ? TY::value(row[t]) : -INFINITY;
  // the slots, 32 to a warp; those past the last are unused
  for (int k0 = EXTRA ? 0 : warp * 32; k0 < K && (!EXTRA || warp == SW); k0 += EXTRA ? 32 : ST) {
    const int k = k0 + lane, given = k < K ? a.ids[(size_t)r * K + k] : -1;
    const int id = given >= 0 && given < a.V ? given : -1;
    if (id != given) wrong |= DI_INVALID;
    sh.slots.ids[k] = id;
    if (rank_c) continue;
    const float v = id >= 0 ? a.teacher[(size_t)r * K + k] : -INFINITY;
    const float x = id >= 0 && legal(id) ? TY::value(row[id]) : -INFINITY;
    // the same id twice
    if (K <= 32) {
      if ((__match_any_sync(0xffffffffu, id) & ((1u << lane) - 1)) && id >= 0) wrong |= DI_INVALID;
    } else if (id >= 0) {
      for (unsigned h = (unsigned)id * 2654435761u >> 23;; ++h) {  // 512 entries, at most 256 ids
        const int old = atomicCAS(&sh.seen[h & (2 * DI_MAX_K - 1)], -1, id);
        if (old == id) wrong |= DI_INVALID;
        if (old == -1 || old == id) break;
      }
    }
    distill_slots(a, sh.slots, k0, id, x, v, T, s);
  }
  if (EXTRA) __syncwarp();
  else __syncthreads();
  float xe = -INFINITY;
  if (rank_c == 0 && warp == (EXTRA ? SW : 0)) {
    const int head = lead ? min(a.V, VE - lead) : 0, tail = max(head, f1 * VE - lead);
    uint32_t taken = 0u;  // lanes whose value has a slot
    for (int k = lane; k < K; k += 32) {
      const int id = sh.slots.ids[k], e = id < head ? id : id >= tail ? head + id - tail : -1;
      if (e >= 0) taken |= 1u << e;
    }
    taken = __reduce_or_sync(0xffffffffu, taken);
    const int j = lane < head ? lane : tail + lane - head;
    if (j < a.V && !((taken >> lane) & 1u) && legal(j)) xe = TY::value(row[j]);
  }

  // The lane's sum is of 2^(x s - c): one fused operation a value, rounded once whatever c
  // is.  c follows its largest value mx only when that has left it by a factor of 2^SLAG.
  // Where c would be rounded by more than half a unit (far), the sum is of 2^((x - ref) s).
  float ref = -INFINITY, c2 = 0.f, mx = -INFINITY;
  bool far = false;  // of some lane of the warp
  f32x2 S2 = pair(0.f, 0.f);
  const f32x2 s2 = pair(s, s);
  uint4 x[NU];
  auto follow = [&](float top) {  // mx and ref, before values up to top are added
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(mx) : "f"(mx), "f"(top));
    const bool raise = (top - ref) * s > SLAG;
    if (__any_sync(0xffffffffu, raise)) {
      if (raise) {
        // from what the sum is relative to (c, or ref s where that is far) to the same of top,
        // rounded once
        const float to = top * s;
        const bool was = fabsf(c2) < DI_NEAR, is = fabsf(to) < DI_NEAR;
        const float e = fmaf((was ? 0.f : ref) - (is ? 0.f : top), s, (was ? c2 : 0.f) - (is ? to : 0.f));
        const float by = ref == -INFINITY ? 0.f : sc_ex2(e);
        S2 = mul2(S2, pair(by, by));
        ref = top;
        c2 = to;
      }
      far = __any_sync(0xffffffffu, !(fabsf(c2) < DI_NEAR));
    }
  };
  for (int i = 0; i < chunks; ++i) {
    const int c = mine + i * (SW * cv), slot = i % DI_STAGES;
    uint4* stage = ring + slot * cv;
    uint32_t lo = 0u, hi = 0u;
    bool whole = true;
    if constexpr (MASK) {
      uint32_t every = bits[0];
#pragma unroll
      for (int w = 1; w < NW; ++w) every &= bits[w];
      whole = __all_sync(0xffffffffu, every == 0xffffffffu);
      if (!whole) {
        uint32_t w[NU];
#pragma unroll
        for (int u = 0; u < NU; ++u) w[u] = __shfl_sync(0xffffffffu, bits[(u * VE) / 32], (u * VE + lane * VE / 32) & 31);
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
      }
      words += SW * cv * VE / 32;
      words_left -= SW * cv * VE / 32;
      if (i + 1 < chunks) load_bits(bits, words, bit0 & 31, words_left);
    }
    if (!__all_sync(0xffffffffu, sc_wait(smem_u32(&full[slot]), (i / DI_STAGES) & 1, a.wait_limit))) {
      // no copy is left in flight; then the warp goes on without the rest of its chunks
      for (int k = i; k < min(chunks, i + DI_STAGES); ++k)
        sc_wait(smem_u32(&full[k % DI_STAGES]), (k / DI_STAGES) & 1, SC_WAIT);
      wrong |= DI_LATE;
      break;
    }
    // the teacher's tokens in this chunk
    const int first = c * VE - lead;
    raw* values = reinterpret_cast<raw*>(stage);
    bool wrote = false;
    for (int k = lane; k < K; k += 32) {
      const unsigned d = (unsigned)(EXTRA ? a.ids[(size_t)r * K + k] : sh.slots.ids[k]) - (unsigned)first;
      if (d < (unsigned)(cv * VE)) {
        if constexpr (DT == SMP_F32) values[d] = -INFINITY;
        else values[d] = (raw)(WD::NONE & 0xffffu);
        wrote = true;
      }
    }
    if (__any_sync(0xffffffffu, wrote)) fence_proxy_async_smem();
    __syncwarp();
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      x[u] = make_uint4(WD::NONE, WD::NONE, WD::NONE, WD::NONE);
      if (u * 32 < cv) x[u] = stage[u * 32 + lane];
    }
    if (MASK && !whole) {
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const uint32_t b = (u * VE < 32 ? lo : hi) >> (u * VE & 31);
        x[u].x = WD::keep(x[u].x, b, 0);
        x[u].y = WD::keep(x[u].y, b, 1);
        x[u].z = WD::keep(x[u].z, b, 2);
        x[u].w = WD::keep(x[u].w, b, 3);
      }
    }
    uint32_t wm = WD::NONE;
#pragma unroll
    for (int u = 0; u < NU; ++u)
      wm = WD::max_nan(wm, WD::max_nan(WD::max_nan(x[u].x, x[u].y), WD::max_nan(x[u].z, x[u].w)));
    const float top = WD::top(wm);
    __syncwarp();  // the stage has been read: every lane's values have gone into its top
    fetch(i + DI_STAGES);
    follow(top);
    if (!far) {
      const f32x2 cc = pair(-c2, -c2);
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        if (u * 32 >= cv) break;
        float f[VE];
        sc_unpack<DT>(x[u], f);
#pragma unroll
        for (int e = 0; e < VE; e += 2) {
          float d0, d1;
          unpair(fma2(pair(f[e], f[e + 1]), s2, cc), d0, d1);
          S2 = add2(S2, pair(sc_ex2(d0), sc_ex2(d1)));
        }
      }
    } else {
      const bool mine_far = !(fabsf(c2) < DI_NEAR);
      const float base = ref == -INFINITY ? 0.f : ref;
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        if (u * 32 >= cv) break;
        float f[VE];
        sc_unpack<DT>(x[u], f);
#pragma unroll
        for (int e = 0; e < VE; ++e)
          S2 = add2(S2, pair(sc_ex2(mine_far ? (f[e] - base) * s : fmaf(f[e], s, -c2)), 0.f));
      }
    }
  }

  // the CTA's state
  Soft st{mx, 0.f, 0.f};
  {
    float a0, a1;
    unpair(S2, a0, a1);
    // to mx
    st.S = (a0 + a1) * sc_ex2(mx == -INFINITY ? 0.f : fabsf(c2) < DI_NEAR ? -fmaf(mx, s, -c2) : (ref - mx) * s);
    if (!(mx < INFINITY) || !(xe < INFINITY)) wrong |= DI_NONFINITE;
  }
  sc_add(st, xe, s);
  st = sc_warp_merge(st, s);
  wrong = __reduce_or_sync(0xffffffffu, wrong);
  if (lane == 0) sh.warp[warp] = DistillPart{st.m, st.S, wrong};
  // One warp: the union of the states, in every lane.
  auto join = [&](const DistillPart* parts, int count) {
    const DistillPart w = lane < count ? parts[lane] : DistillPart{-INFINITY, 0.f, 0};
    st = sc_warp_merge(Soft{w.m, w.S, 0.f}, s);
    wrong = __reduce_or_sync(0xffffffffu, w.wrong);
  };
  if (nc > 1) {  // all CTAs of the row have started
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (warp == 0) {
      join(sh.warp, SW);
      if (lane == 0) *cg::this_cluster().map_shared_rank(&sh.part[rank_c], 0) = DistillPart{st.m, st.S, wrong};
      __syncwarp();
    }
    cluster_arrive();
    cluster_wait();
    if (rank_c) return;  // the first CTA has everything
    if (warp == WF) join(sh.part, nc);
  } else {
    __syncthreads();
    if (warp == WF) join(sh.warp, EXTRA ? SW + 1 : SW);
  }
  if (warp == WF) distill_finish(a, r, T, s, t, xt, wrong, st.m, st.S, sh.slots, sh.row);
  if (EXTRA || K <= 32 || (!a.slot_lp && !a.slot_g)) {
    if (warp != WF) return;
    __syncwarp();
    for (int k = lane; k < K && (a.slot_lp || a.slot_g); k += 32) distill_slot(a, r, k, sh.slots, sh.row);
  } else {
    __syncthreads();
    for (int k = tid; k < K; k += ST) distill_slot(a, r, k, sh.slots, sh.row);
  }
  // a later launch ends only after the one it started beside, so the last ends last
  if (r0 && blockIdx.x == 0 && lane == 0 && warp == WF) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Rows [r0, r0 + rows), a row in nc CTAs of ST threads.
template <int DT, int ST, bool EXTRA>
int launch_distill(const DistillArgs& a, int r0, int rows, int nc, cudaStream_t st) {
  const bool more = r0 + rows < a.B;
  constexpr int VE = DT == SMP_F32 ? 4 : 8, CV = 32 << SLNU;
  const int seg = (a.V / VE + nc - 1) / nc;
  const int even = (seg + ST - 1) / ST * 32, cv = even < 32 ? 32 : even > CV ? CV : even;
  if ((long long)rows * nc > 0x7fffffffLL) return SMP_ERR_CAPACITY;
  const auto kernel = a.bitmask ? distill_kernel<DT, ST, true, EXTRA> : distill_kernel<DT, ST, false, EXTRA>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * nc));
  cfg.blockDim = dim3(ST + (EXTRA ? 32 : 0));
  cfg.stream = st;
  cfg.dynamicSmemBytes = ST / 32 * DI_STAGES * cv * 16;
  if (!sc_ok(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ST / 32 * DI_STAGES * CV * 16)))
    return SMP_ERR_CUDA;
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
  return sc_ok(cudaLaunchKernelEx(&cfg, kernel, a, nc, seg, cv, r0, more)) ? SMP_OK : SMP_ERR_CUDA;
}

// Short rows take CTAs of 2 or 4 warps.  Long ones take CTAs of 8, and the rows left when all
// others fill the SMs a launch of their own, in clusters as large as still fit at once.  CTAs
// that fill the SMs would all be at their slots at the same time, round after round: there
// one more warp takes them while the others stream (4096 x 128256 bf16 with 32 slots 157 us,
// 180 without it), unless they take it longer than the stream takes (912 x 128256: with 64
// slots 42 and 46 us, with 192 62 and 54; 1824 x 20000: with 32 31 and 39, with 128 71 and
// 52): 96 vectors of the row to a slot, or 32 slots at most.
template <int DT>
int distill_rows(const DistillArgs& a, cudaStream_t st) {
  const int sms = sc_sm_count();
  if (sms < 1) return SMP_ERR_CUDA;
  const int vectors = a.V / (DT == SMP_F32 ? 4 : 8);
  if (vectors <= 64 * 8) return launch_distill<DT, 64, false>(a, 0, a.B, 1, st);
  if (vectors <= 128 * 8) return launch_distill<DT, 128, false>(a, 0, a.B, 1, st);
  const int slots = SROWS * sms, done = a.B / slots * slots, rows = a.B - done;
  if (done) {
    const int rc = a.K <= 32 || vectors >= 96 * a.K ? launch_distill<DT, 256, true>(a, 0, done, 1, st)
                                                    : launch_distill<DT, 256, false>(a, 0, done, 1, st);
    if (rc != SMP_OK || !rows) return rc;
  }
  int nc = 1;
  while (nc < SMAXC && (long long)rows * nc * 2 <= slots && vectors > nc * 256 * 8) nc *= 2;
  return launch_distill<DT, 256, false>(a, done, rows, nc, st);
}

}  // namespace
}  // namespace smp
