// smp_head.cu -- log probabilities and entropy straight from hidden states and
// the output head's weights (smp_head_logprobs): logits that only ever exist
// as accumulators in tensor memory.
//
// head_kernel, one persistent CTA per SM, forms tiles of states x tokens with
// tcgen05.mma (16-bit operands, binary32 accumulators): 256 x 256 on a pair of
// CTAs, each staging its 128 states and half of the weights; up to 128 states,
// where the stream of the weights is the bound, 128 x 128 on one CTA.  One
// thread feeds a ring of TMA stages (64 values of D each, 128-byte swizzle),
// one thread (of the pair) issues the products, and two groups of four warps,
// each with half of the tile's columns, read finished accumulators into
// registers: a thread owns one state's half row, folds it into a softmax state
// {m, S, U} and writes that to the workspace with the target's logit.
// 4096 x 128256 x 4096 bf16: 2360-2440 us, 1.8 PFLOP/s under the power limit; on
// single CTAs (128 x 256, half as much again from L2) 2563.  One state: 158-159
// us, 6.6 TB/s of weights, with 10 stages of 32 state rows; 163.4 with 6 of 128.
//
// The tensor cores' binary32 accumulation drops low bits instead of rounding:
// over D = 4096 in one accumulator the logits were off by 5e-6 of their size.
// So an accumulator sums HSEG stages (512 values of D) and the segments are
// added, rounded to nearest, in the epilogue's registers.  Accumulators are
// double buffered (512 columns of tensor memory): the epilogue of a segment
// or tile runs under the products of the next.
//
// Tiles are walked with the states fastest: the SMs share a few weight tiles
// at any time and every weight comes from HBM once; the hidden states stay in
// L2.  head_join merges the states of a row in a fixed order: the same bits
// each call.
//
// Every wait on a barrier is bounded.  One that expires makes all roles of the
// CTA, in a pair of both CTAs, leave; copies and products in flight are waited for
// (settle), tensor memory is freed, and all rows of the call return SMP_ERR_TIMEOUT.
#include <cuda.h>

#include "smp_score.cuh"

namespace smp {
namespace {

constexpr int HBM = 128;               // states per tile
constexpr int HBK = 64;                // values of D per stage: one 128-byte swizzle atom
constexpr int HSEG = 8;                // stages that one accumulator sums
constexpr int HEPI = 8;                // epilogue warps: two groups of four
constexpr int HTHREADS = (HEPI + 2) * 32;
constexpr int HFLAGS = 1024;           // workspace: one word per CTA, then the tiles' states

// AR: rows of states that a stage has room for.  With AR < 128 the products read on into
// the weights behind them: rows of the tile that no state has.
template <int BN, bool PAIR, int AR>
struct HeadShape {
  static constexpr int BM = PAIR ? 2 * HBM : HBM;    // states per tile
  static constexpr int B_ROWS = PAIR ? BN / 2 : BN;  // tokens that a CTA stages
  static constexpr int A_BYTES = AR * HBK * 2;
  static constexpr int B_BYTES = B_ROWS * HBK * 2;
  static constexpr int STAGES = AR < HBM ? 10 : 6;
  static_assert(A_BYTES + B_BYTES >= HBM * HBK * 2, "the last stage's products stay inside the ring");
  static constexpr int ACCS = 512 / BN;
  static constexpr int SMEM = STAGES * (A_BYTES + B_BYTES) + 1024;  // + alignment
};

// Few states: the weights' stream is the bound, and narrower tiles spread it
// more evenly over the SMs.  More states: two CTAs on a tile of 256 x 256, so
// that each stages half of the weights.
int tile_tokens(int N) { return N <= HBM ? 128 : 256; }
int tiles_of(int N, int V) { return (V - 1) / tile_tokens(N) + 1; }  // V >= 1, up to the largest int

struct HeadBars {
  uint64_t full[10], empty[10], acc_full[4], acc_empty[4], drain;
  uint32_t tmem;
  uint32_t issued[2];  // first CTA: stages that each CTA of the pair has sent copies for
  int fail;
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void bar_init(uint64_t* b, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(b)) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(b)), "r"(bytes)
               : "memory");
}
// Takes bytes that no copy will bring off what the phase still expects.
__device__ __forceinline__ void bar_deduct(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(b)), "r"(bytes)
               : "memory");
}
// The address of `p` in the pair's CTA of this rank; the first's.
__device__ __forceinline__ uint32_t pair_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t first_addr(const void* p) { return pair_addr(p, 0); }
__device__ __forceinline__ void pair_store(uint32_t addr, uint32_t v) {
  asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// Waits for the phase; false when it does not come within `limit` cycles of a first look,
// which makes all roles leave, in a pair the other CTA's as well, or when another has
// given up.  Every look parks: one that does not, before these, cost the thread that
// issues the products 1 to 4 % of the call (4096 x 128256 x 4096: 2435 to 2539 us).
template <bool PAIR>
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, int* fail, long long limit) {
  if (sc_park(smem_addr(b), parity)) return true;
  const long long t0 = clock64();
  while (!sc_park(smem_addr(b), parity)) {
    if (*(volatile int*)fail) return false;
    if (clock64() - t0 > limit) {
      *(volatile int*)fail = 1;
      if constexpr (PAIR) pair_store(pair_addr(fail, (blockIdx.x & 1) ^ 1), 1u);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ void bar_arrive_first(uint64_t* b) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(first_addr(b)) : "memory");
}
// One box into this CTA's shared memory; its bytes count on `bar`, in a pair the first CTA's.
template <bool PAIR>
__device__ __forceinline__ void tma_tile(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// Shared-memory operand: K-major, 128-byte swizzle, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3fff) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
template <bool PAIR>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  if constexpr (PAIR)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
// Arrives on `bar` when the products issued so far are done; in a pair on both CTAs'.
template <bool PAIR>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  if constexpr (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"((uint16_t)3)
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// Copies in flight when the roles have left: waits until the last phase of each stage of
// the first CTA is complete, which counts both CTAs' copies.  Where only one of the two
// got as far, the phase is made to expect that one's bytes: neither can be a whole
// ring ahead, as a stage is filled again only after products that had both halves.
template <bool PAIR, int STAGES>
__device__ __noinline__ void settle(HeadBars* bars, uint32_t bytes) {
  auto uses = [](uint32_t n, uint32_t st) { return n > st ? (n - st - 1) / STAGES + 1 : 0u; };
  for (uint32_t st = 0; st < STAGES; ++st) {
    const uint32_t u0 = uses(bars->issued[0], st), u1 = PAIR ? uses(bars->issued[1], st) : u0;
    if (u0 > u1) bar_deduct(&bars->full[st], bytes);
    if (u1 > u0) bar_expect(&bars->full[st], bytes);
    if (u0 | u1) sc_wait(smem_addr(&bars->full[st]), (max(u0, u1) - 1) & 1, SC_WAIT);
  }
}

// 32 columns of this thread's row (the warp's 32 lanes of tensor memory).
__device__ __forceinline__ void acc_load(uint32_t addr, float (&v)[32]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}

template <int BN, bool PAIR, int AR>
__global__ void __launch_bounds__(HTHREADS, 1)
    head_kernel(const HeadArgs a, const __grid_constant__ CUtensorMap map_h,
                const __grid_constant__ CUtensorMap map_w, const uint32_t idesc, const uint32_t a_bytes) {
  using SH = HeadShape<BN, PAIR, AR>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ HeadBars bars;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int peer = PAIR ? blockIdx.x & 1 : 0;  // place in the pair; the first issues the products
  const int first = PAIR ? blockIdx.x / 2 : blockIdx.x, stride = PAIR ? gridDim.x / 2 : gridDim.x;
  const int mt = (a.N + SH::BM - 1) / SH::BM, vt = (a.V + BN - 1) / BN;
  const int kt = (a.D + HBK - 1) / HBK;
  const long long tiles = (long long)mt * vt;
  int* fail = &bars.fail;
  volatile int* failed = fail;
  const long long limit = a.wait_limit;

  if (threadIdx.x == 0) {
    for (int i = 0; i < SH::STAGES; ++i) {
      bar_init(&bars.full[i], 1);
      bar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < SH::ACCS; ++i) {
      bar_init(&bars.acc_full[i], 1);
      bar_init(&bars.acc_empty[i], PAIR ? 2 * HEPI : HEPI);
    }
    bar_init(&bars.drain, 1);
    bars.fail = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == HEPI + 1) {
    if constexpr (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_addr(&bars.tmem)),
                   "r"(512u)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_addr(&bars.tmem)),
                   "r"(512u)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
  }
  __syncthreads();
  if constexpr (PAIR) {  // the other CTA's barriers and tensor memory are there
    cluster_arrive();
    cluster_wait();
  }
  fence_after();
  const uint32_t tmem = bars.tmem;
  // The launch may overlap the end of the work before it on the stream: nothing of a
  // caller's is read or written before that is complete.
  asm volatile("griddepcontrol.wait;" ::: "memory");

  if (warp == HEPI) {  // copies
    if (lane == 0) {
      uint32_t i = 0;
      for (long long tile = first; tile < tiles && !*failed; tile += stride) {
        const int m0 = (int)(tile % mt) * SH::BM + peer * HBM, v0 = (int)(tile / mt) * BN + peer * SH::B_ROWS;
        for (int k = 0; k < kt; ++k, ++i) {
          const uint32_t st = i % SH::STAGES, use = i / SH::STAGES;
          if (use && !bar_wait<PAIR>(&bars.empty[st], (use - 1) & 1, fail, limit)) break;
          uint8_t* dst = ring + st * (SH::A_BYTES + SH::B_BYTES);
          if (!peer) bar_expect(&bars.full[st], (a_bytes + SH::B_BYTES) * (PAIR ? 2 : 1));
          const uint32_t bar = PAIR ? first_addr(&bars.full[st]) : smem_addr(&bars.full[st]);
          tma_tile<PAIR>(dst, &map_h, k * HBK, m0, bar);
          tma_tile<PAIR>(dst + SH::A_BYTES, &map_w, k * HBK, v0, bar);
        }
      }
      asm volatile("griddepcontrol.launch_dependents;");  // head_join may get ready
      if (PAIR && peer) pair_store(first_addr(&bars.issued[1]), i);
      else bars.issued[0] = i;
      // the last use of each stage: its products are done before the CTA ends
      for (uint32_t j = i > SH::STAGES ? i - SH::STAGES : 0; j < i; ++j)
        if (!bar_wait<PAIR>(&bars.empty[j % SH::STAGES], (j / SH::STAGES) & 1, fail, limit)) break;
    }
  } else if (warp == HEPI + 1) {  // products
    if (lane == 0 && !peer) {
      uint32_t i = 0, sg = 0;
      for (long long tile = first; tile < tiles && !*failed; tile += stride) {
        for (int k0 = 0; k0 < kt && !*failed; k0 += HSEG, ++sg) {
          const uint32_t b = sg % SH::ACCS, use = sg / SH::ACCS;
          if (use && !bar_wait<PAIR>(&bars.acc_empty[b], (use - 1) & 1, fail, limit)) break;
          fence_after();
          const int k1 = min(kt, k0 + HSEG);
          for (int k = k0; k < k1; ++k, ++i) {
            const uint32_t st = i % SH::STAGES;
            if (!bar_wait<PAIR>(&bars.full[st], (i / SH::STAGES) & 1, fail, limit)) break;
            fence_after();
            const uint32_t base = smem_addr(ring + st * (SH::A_BYTES + SH::B_BYTES));
            const uint64_t da = operand_desc(base), db = operand_desc(base + SH::A_BYTES);
#pragma unroll
            for (int q = 0; q < HBK / 16; ++q)  // 16 values of D: 32 bytes further in the atom
              mma<PAIR>(tmem + b * BN, da + 2 * q, db + 2 * q, idesc, k > k0 || q > 0);
            mma_commit<PAIR>(&bars.empty[st]);
          }
          if (!*failed) mma_commit<PAIR>(&bars.acc_full[b]);
        }
      }
    }
  } else {  // epilogue: group warp / 4 has half of the tile's columns
    constexpr int NC = BN / 2;
    uint32_t sg = 0;
    bool gone = false;
    for (long long tile = first; tile < tiles; tile += stride) {
      f32x2 x2[NC / 2];
#pragma unroll
      for (int j = 0; j < NC / 2; ++j) x2[j] = pair(0.f, 0.f);
      const int c0 = (warp >> 2) * NC;
      for (int k = 0; k < kt; k += HSEG, ++sg) {
        const uint32_t b = sg % SH::ACCS;
        // the warp leaves or stays as one: the loads below are the whole warp's
        gone = !__all_sync(0xffffffffu, bar_wait<PAIR>(&bars.acc_full[b], (sg / SH::ACCS) & 1, fail, limit));
        if (gone) break;
        fence_after();
        const uint32_t acc = tmem + b * BN + c0 + ((uint32_t)(warp & 3) * 32u << 16);
#pragma unroll
        for (int c = 0; c < NC; c += 32) {
          float v[32];
          acc_load(acc + c, v);
#pragma unroll
          for (int j = 0; j < 16; ++j) x2[c / 2 + j] = add2(x2[c / 2 + j], pair(v[2 * j], v[2 * j + 1]));
        }
        fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR) bar_arrive_first(&bars.acc_empty[b]);
          else bar_arrive(&bars.acc_empty[b]);
        }
      }
      if (gone) break;
      const int vtile = (int)(tile / mt), v0 = vtile * BN + c0;
      const int row = (int)(tile % mt) * SH::BM + peer * HBM + (warp & 3) * 32 + lane;
      const bool mine = row < a.N;
      const float T = mine && a.temperature ? a.temperature[row] : 1.f;
      const float s = sc_scale(sc_temperature_ok(T) ? T : 1.f);
      const int t = (mine && a.targets ? a.targets[row] : -1) - v0;  // the target's column, if any
      float x[NC];
#pragma unroll
      for (int j = 0; j < NC / 2; ++j) unpair(x2[j], x[2 * j], x[2 * j + 1]);
      if (v0 + NC > a.V) {
#pragma unroll
        for (int j = 0; j < NC; ++j)
          if (v0 + j >= a.V) x[j] = -INFINITY;
      }
      float xt = -INFINITY;
      if (__any_sync(0xffffffffu, t >= 0 && t < NC)) {
#pragma unroll
        for (int j = 0; j < NC; ++j)
          if (t == j) xt = x[j];
      }
      float m = x[0], low = x[0];
#pragma unroll
      for (int j = 1; j < NC; ++j) {
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(m), "f"(x[j]));
        low = fminf(low, x[j]);
      }
      // Usually there is no -inf or NaN, and nothing so low that its d would be -inf: nothing
      // to clamp.  Both ways add the same values in the same order.  Lanes without a
      // state hold what earlier work left and have no say.
      const float mm = m == -INFINITY ? 0.f : m;
      const f32x2 base = pair(-mm, -mm), ss = pair(s, s);
      f32x2 S2[2] = {pair(0.f, 0.f), pair(0.f, 0.f)}, U2[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
      auto add = [&](int j, bool clamp) {
        f32x2 d = mul2(add2(pair(x[2 * j], x[2 * j + 1]), base), ss);
        float d0, d1;
        unpair(d, d0, d1);
        if (clamp) {
          d0 = fmaxf(d0, SC_DMIN);
          d1 = fmaxf(d1, SC_DMIN);
          d = pair(d0, d1);
        }
        const f32x2 e = pair(sc_ex2(d0), sc_ex2(d1));
        S2[j & 1] = add2(S2[j & 1], e);
        U2[j & 1] = fma2(e, d, U2[j & 1]);
      };
      if (__all_sync(0xffffffffu, !mine || (low - m) * s > -1.0e30f)) {
#pragma unroll
        for (int j = 0; j < NC / 2; ++j) add(j, false);
      } else {
#pragma unroll
        for (int j = 0; j < NC / 2; ++j) add(j, true);
      }
      float a0, a1, b0, b1;
      unpair(add2(S2[0], S2[1]), a0, a1);
      unpair(add2(U2[0], U2[1]), b0, b1);
      const float S = a0 + a1, U = b0 + b1;
      if (mine)
        a.part[HFLAGS / 4 + ((size_t)row * vt + vtile) * 2 + (warp >> 2)] =
            make_float4(m < INFINITY ? m : INFINITY, S, U, xt);
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if constexpr (PAIR) {  // neither CTA's memory is used by the other any more
    cluster_arrive();
    cluster_wait();
  }
  if (*failed) {  // in a pair both CTAs see it, or neither: all roles have left
    if (lane == 0 && warp == HEPI + 1) {
      if (!peer) mma_commit<PAIR>(&bars.drain);  // by the thread that issued the products
      sc_wait(smem_addr(&bars.drain), 0, SC_WAIT);
    }
    if (lane == 0 && warp == HEPI && !peer) settle<PAIR, SH::STAGES>(&bars, a_bytes + SH::B_BYTES);
    __syncwarp();
    __syncthreads();
    if constexpr (PAIR) {
      cluster_arrive();
      cluster_wait();
    }
  }
  if (warp == HEPI + 1) {
    fence_after();
    if constexpr (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
  if (threadIdx.x == 0) reinterpret_cast<int*>(a.part)[blockIdx.x] = bars.fail;
}

// One CTA per row: the tiles' states merged, the outputs written.  A row has
// 2 V / BN states: with one warp a row, the load latency of a single row's 2004
// states took 23 of 196 us (1 x 128256 x 4096).
constexpr int HJOIN = 128;
__global__ void __launch_bounds__(HJOIN) head_join(const HeadArgs a, int parts, int ctas) {
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ float4 sw[HJOIN / 32];
  asm volatile("griddepcontrol.launch_dependents;");  // a next call's head_kernel may get ready
  // head_kernel's states are complete, and what was written before it is visible here too
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float T = a.temperature ? a.temperature[row] : 1.f;
  const int t = a.targets ? a.targets[row] : -1;
  const bool valid = sc_temperature_ok(T) && t >= -1 && t < a.V;
  const float s = sc_scale(valid ? T : 1.f);
  Soft st{-INFINITY, 0.f, 0.f};
  float xt = -INFINITY;
  bool bad = false, late = false;
  for (int c = tid; c < ctas; c += HJOIN) late |= reinterpret_cast<const int*>(a.part)[c] != 0;
  const float4* part = a.part + HFLAGS / 4 + (size_t)row * parts;
  for (int c = tid; c < parts; c += 8 * HJOIN) {
    float4 p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      p[i] = c + i * HJOIN < parts ? part[c + i * HJOIN] : make_float4(-INFINITY, 0.f, 0.f, -INFINITY);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (p[i].x == INFINITY) bad = true;
      else st = sc_merge(st, Soft{p[i].x, p[i].y, p[i].z}, s);
      xt = fmaxf(xt, p[i].w);
    }
  }
  for (int o = 16; o > 0; o >>= 1) {
    st = sc_merge(st, sc_shfl_xor(st, o), s);
    xt = fmaxf(xt, __shfl_xor_sync(0xffffffffu, xt, o));
  }
  if (lane == 0) sw[warp] = make_float4(st.m, st.S, st.U, xt);
  bad = __syncthreads_or(bad);
  late = __syncthreads_or(late);
  if (tid) return;
  for (int w = 1; w < HJOIN / 32; ++w) {
    st = sc_merge(st, Soft{sw[w].x, sw[w].y, sw[w].z}, s);
    xt = fmaxf(xt, sw[w].w);
  }
  const int status = late ? SMP_ERR_TIMEOUT : !valid ? SMP_ERR_INVALID_PARAM : bad ? SMP_ERR_NONFINITE
                     : st.m == -INFINITY ? SMP_ERR_EMPTY : SMP_OK;
  const bool ok = status == SMP_OK;
  const float L = sc_log_mass(st);
  a.status[row] = status;
  if (a.logprobs) a.logprobs[row] = !ok ? sc_nan() : t < 0 ? 0.f : sc_logprob(xt, st.m, L, T);
  if (a.entropy) a.entropy[row] = ok ? sc_entropy(st, L) : sc_nan();
  if (a.stats) {
    a.stats[2 * (size_t)row] = ok ? st.m : sc_nan();
    a.stats[2 * (size_t)row + 1] = ok ? L : sc_nan();
  }
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                 CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                 CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (!sc_ok(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q)) ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// Rows of D values; boxes of 64 values x `box` rows.  What lies past D or past
// the last row reads as zero.
bool tile_map(CUtensorMap* map, const void* base, int dtype, int rows, int D, long long ld, int box) {
  const EncodeTiled fn = encoder();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t boxes[2] = {HBK, (cuuint32_t)box}, ones[2] = {1, 1};
  return fn(map, dtype == SMP_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
            const_cast<void*>(base), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, bool PAIR, int AR>
int launch_head(const HeadArgs& a, int dtype, int sms, cudaStream_t st, int* ctas) {
  using SH = HeadShape<BN, PAIR, AR>;
  // 8-row granules: of a state tile that N does not fill, only the rows there are are copied
  const int rows = a.N < AR ? (a.N + 7) / 8 * 8 : AR;
  CUtensorMap mh, mw;
  if (!tile_map(&mh, a.hidden, dtype, a.N, a.D, a.ldh, rows) ||
      !tile_map(&mw, a.weight, dtype, a.V, a.D, a.ldw, SH::B_ROWS))
    return SMP_ERR_CUDA;
  const uint32_t type = dtype == SMP_BF16 ? 1u : 0u;
  // binary32 accumulators, both operands of `type` and K-major, N = BN, M = BM
  const uint32_t idesc = (1u << 4) | (type << 7) | (type << 10) | ((uint32_t)(BN >> 3) << 17) |
                         ((uint32_t)(SH::BM >> 4) << 24);
  if (!sc_ok(cudaFuncSetAttribute(head_kernel<BN, PAIR, AR>, cudaFuncAttributeMaxDynamicSharedMemorySize, SH::SMEM)))
    return SMP_ERR_CUDA;
  constexpr int each = PAIR ? 2 : 1;
  const long long tiles = (long long)((a.N + SH::BM - 1) / SH::BM) * ((a.V + BN - 1) / BN);
  const int grid = (int)(tiles < sms / each ? tiles : sms / each) * each;
  *ctas = grid;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(HTHREADS);
  cfg.dynamicSmemBytes = SH::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = each;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  return sc_ok(cudaLaunchKernelEx(&cfg, head_kernel<BN, PAIR, AR>, a, mh, mw, idesc, (uint32_t)(rows * HBK * 2)))
             ? SMP_OK : SMP_ERR_CUDA;
}

}  // namespace

int64_t head_workspace(int N, int V) {
  return HFLAGS * 4 + (int64_t)tiles_of(N, V) * 2 * N * (int64_t)sizeof(float4);
}

int head_enqueue(const HeadArgs& a, int dtype, cudaStream_t st) {
  int ctas = 0;
  const int sms = sc_sm_count();
  if (sms < 2 || sms > HFLAGS) return SMP_ERR_CUDA;
  const int rc = a.N <= 32 ? launch_head<128, false, 32>(a, dtype, sms, st, &ctas)
                 : a.N <= HBM ? launch_head<128, false, HBM>(a, dtype, sms, st, &ctas)
                              : launch_head<256, true, HBM>(a, dtype, sms, st, &ctas);
  if (rc != SMP_OK) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.N);
  cfg.blockDim = dim3(HJOIN);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return sc_ok(cudaLaunchKernelEx(&cfg, head_join, a, 2 * tiles_of(a.N, a.V), ctas)) ? SMP_OK : SMP_ERR_CUDA;
}

}  // namespace smp
