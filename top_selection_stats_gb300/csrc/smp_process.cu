// smp_process.cu -- penalties for repeated tokens, biases and grammar masks on
// logits (smp_process_logits).
//
// A row is cut into segments of whole 16-byte vectors, one per CTA.  A CTA looks
// through the row's history and biases for the tokens of its segment (its cells), and
// keeps in shared memory
//   touched  one bit a cell: in the history or biased;
//   table    the touched cells, by open addressing: copies among the generated tokens,
//            whether the token was seen, and its bias (a token with several slots is
//            marked, and its biases are then looked up in slot order);
//   count    for long histories, in place of their part of the table: a word for each cell.
// Integer atomics only, so that results do not depend on the order of arrival.  Then the
// segment streams from the logits to the result with its mask, and the few touched tokens
// of a vector are computed from its registers and written over it by the same thread, while
// its line is in L2.  In place only vectors with something masked or touched are read, and
// those without a legal token are written without being read.
//
// Bound by HBM where rows are long and many: 1024 x 256000 f16 to binary32 248 us, 6.3 TB/s
// (a copy of as many bytes: 233).  A result aligned unlike its logits, whose vectors are put
// together from two, takes 1.4 to 1.7 times as long: 1000 x 128257 bf16 133 us, 88 alike.
// Small calls are bound by the chain of a launch, parameters, history, table and logits (1 x
// 128256 with 1000 entries 3.6 us), long histories by the instructions that look through them
// in every CTA of the row.
#include "smp_score_kernel.cuh"
#include "smp_train.cuh"

namespace smp {
namespace {

constexpr int PSMALL = 256;    // threads, usually
constexpr int PLARGE = 1024;   // and of a CTA that counts by cell, at most
constexpr int PCTAS = 5;       // CTAs of the former on an SM (four with the largest tables and segments, 53 KB)
constexpr int PDENSECTAS = 1;  // CTAs of the latter
constexpr int PEARLY = 4;      // history entries that a thread loads before anything else
constexpr int PBATCH = 8;      // and those that it has in flight later
constexpr int PU = 4;          // vectors a lane has in flight, at most
constexpr int PENDS = 16;      // values of a row outside its whole vectors, at most
constexpr int PDENSE = 32768;  // cells of a segment that counts by cell, at most
constexpr int PMOST = 131072;  // and of one that counts in the table, at most
constexpr int PSHORT = 2048;   // entries of history and biases that go into a table, at most
constexpr int PSETUP = 2048;   // cells that are streamed in the time that a CTA takes before it streams
constexpr int PSPARSE = 512;   // threads of a row that changes in place without a mask
constexpr int PEACH = PSHORT / PSPARSE;
constexpr uint32_t PSEEN = 0x80000000u, PBIAS = 0x40000000u, PMULTI = 0x20000000u, PCOUNT = 0x1fffffffu;

// How a call is cut, and a CTA's shared memory in 32-bit words.
struct ProcessPlan {
  int nc, seg, each;  // CTAs of a row, vectors of a segment, vectors of a lane in a chunk
  int counts;         // cells counted by themselves (0: in the table)
  int table;          // entries of the table
  int bits;           // words of touched
};

// The row's numbers, and what becomes of a touched token.  Penalties are finite, but their product
// with a count (2^24 at most) may not be: those from 2^100 on are taken, like the logits, 2^26
// times smaller, where only bits below 2^-124 are lost.
struct ProcessRow {
  float theta, presence, frequency, scale;
};
__device__ __forceinline__ ProcessRow process_row(const ProcessArgs& a, int r) {
  ProcessRow p{a.repetition ? a.repetition[r] : 1.f, a.presence ? a.presence[r] : 0.f, a.frequency ? a.frequency[r] : 0.f, 1.f};
  if (fmaxf(fabsf(p.presence), fabsf(p.frequency)) >= 0x1p100f) p.scale = 0x1p-26f;
  p.presence *= p.scale;
  p.frequency *= p.scale;
  return p;
}
__device__ __forceinline__ float process_penalty(const ProcessRow& p, float v, uint32_t n) {
  if (n & (PSEEN | PCOUNT)) {
    v = v > 0.f ? __fdiv_rn(v, p.theta) : __fmul_rn(v, p.theta);
    const float copies = (float)(n & PCOUNT), take = __fadd_rn(__fmul_rn(p.frequency, copies), copies > 0.f ? p.presence : 0.f);
    v = __fsub_rn(__fmul_rn(v, p.scale), take);
    if (p.scale != 1.f) v = __fmul_rn(v, 0x1p26f);
  }
  return v;
}
__device__ __forceinline__ float process_bias(float v, float b) {
  return v == -INFINITY || b == -INFINITY ? -INFINITY : __fadd_rn(v, b);
}

__device__ __forceinline__ bool process_valid(const ProcessRow& p, int length, int prompt, int H) {
  return p.theta > 0.f && p.theta < INFINITY && fabsf(p.presence) < INFINITY && fabsf(p.frequency) < INFINITY &&
         length >= 0 && length <= H && prompt >= 0 && prompt <= length;
}
// The entry of a key in a table of `size` entries, more than there are keys: where it is,
// or (add) where it is put.
__device__ __forceinline__ int process_entry(int* keys, int size, int key, bool add) {
  int at = (int)__umulhi((uint32_t)key * 2654435761u, (uint32_t)size);
  while (true) {
    int old = *reinterpret_cast<volatile int*>(&keys[at]);
    if (add && old == -1) old = atomicCAS(&keys[at], -1, key);
    if (old == key || old == -1) return at;
    if (++at == size) at = 0;
  }
}
// A touched token's result from its logit, its number and its only bias.  A token with several
// biases looks through all of the row's for them, one thread for itself: 64 x 128256 bf16 with 512
// biases takes 11 us, 73 when every id is there twice, with 4096 20 and 1170.
__device__ __forceinline__ float process_token(const ProcessArgs& a, const ProcessRow& p, float v, uint32_t n, float only,
                                               int id, const int32_t* bias_ids, const float* bias) {
  if (v == -INFINITY) return v;
  v = process_penalty(p, v, n);
  if (n & PMULTI) {
    for (int i = 0; i < a.NB; ++i)
      if (bias_ids[i] == id) v = process_bias(v, bias[i]);
  } else if (n & PBIAS) {
    v = process_bias(v, only);
  }
  return v;
}

enum { PR_COPY = 0, PR_ACROSS = 1, PR_IN_PLACE = 2 };

// In place and without a mask only the tokens of a short history and the biases change: a
// CTA has a row, and all its tokens in a table.
template <int DT>
__global__ void __launch_bounds__(PSPARSE, 2) process_sparse_kernel(const ProcessArgs a, const int size) {
  using TY = ScType<DT>;
  using raw = typename TY::raw;
  extern __shared__ __align__(16) uint32_t words[];
  int* keys = reinterpret_cast<int*>(words);  // tokens; -1: none
  uint32_t* numbers = words + size;
  float* biases = reinterpret_cast<float*>(numbers + size);  // of tokens with one; only with biases
  const int r = blockIdx.x, tid = threadIdx.x;
  raw* row = static_cast<raw*>(a.out) + (size_t)r * a.old;
  for (int i = tid; i < size; i += PSPARSE) {
    keys[i] = -1;
    numbers[i] = 0u;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int32_t* history = a.history + (size_t)r * a.hld;
  const int32_t* bias_ids = a.bias_ids + (size_t)r * a.NB;
  const float* bias = a.bias + (size_t)r * a.NB;
  // all loads at once: PSHORT entries are at most PEACH for a thread
  int t[PEACH], id[PEACH];
  float b[PEACH];
#pragma unroll
  for (int k = 0; k < PEACH; ++k) {
    const int i = tid + k * PSPARSE;
    t[k] = i < a.H ? history[i] : -1;
    id[k] = i < a.NB ? bias_ids[i] : -1;
    b[k] = i < a.NB ? bias[i] : 0.f;
  }
  const ProcessRow p = process_row(a, r);
  const int length = a.lengths ? a.lengths[r] : a.H, prompt = a.prompts ? a.prompts[r] : 0;
  bool bad = !process_valid(p, length, prompt, a.H);
#pragma unroll
  for (int k = 0; k < PEACH; ++k) {
    if (tid + k * PSPARSE >= length || (unsigned)t[k] >= (unsigned)a.V) t[k] = -1;
    if ((unsigned)id[k] >= (unsigned)a.V) id[k] = -1;
    // on their way into the cache while the table is filled
    if (t[k] >= 0) asm volatile("prefetch.global.L1 [%0];" ::"l"(row + t[k]));
    if (id[k] >= 0) asm volatile("prefetch.global.L1 [%0];" ::"l"(row + id[k]));
    bad |= id[k] >= 0 && !(b[k] < INFINITY);
  }
  bad = __syncthreads_or(bad);
  if (tid == 0) a.status[r] = bad ? SMP_ERR_INVALID_PARAM : SMP_OK;
  if (bad) return;
#pragma unroll
  for (int k = 0; k < PEACH; ++k) {
    if (t[k] >= 0) {
      uint32_t* n = &numbers[process_entry(keys, size, t[k], true)];
      if (tid + k * PSPARSE < prompt) atomicOr(n, PSEEN);
      else atomicAdd(n, 1u);
    }
    if (id[k] >= 0) {
      const int at = process_entry(keys, size, id[k], true);
      if (atomicOr(&numbers[at], PBIAS) & PBIAS) atomicOr(&numbers[at], PMULTI);
      else biases[at] = b[k];
    }
  }
  __syncthreads();
  for (int i = tid; i < size; i += PSPARSE) {
    const int j = keys[i];
    if (j < 0) continue;
    const uint32_t n = numbers[i];
    row[j] = TY::store(process_token(a, p, TY::value(row[j]), n, n & PBIAS ? biases[i] : 0.f, j, bias_ids, bias));
  }
}

// HOW: to a result that starts alike in its vectors, to one that starts otherwise, in place.
template <int DT, int OT, int HOW, bool MASK, int PT>
__global__ void __launch_bounds__(PT, PT == PSMALL ? PCTAS : PDENSECTAS) process_kernel(const ProcessArgs a, const ProcessPlan plan) {
  using TI = ScType<DT>;
  using TO = ScType<OT>;
  using WD = Word<DT>;
  using raw = typename TI::raw;
  using out_t = typename TO::raw;
  constexpr int VE = 16 / (int)sizeof(raw), SW = PT / 32;
  constexpr uint32_t ALL = (1u << VE) - 1;
  extern __shared__ __align__(16) uint32_t words[];
  constexpr bool DENSE = PT == PLARGE;
  const int nc = plan.nc, r = blockIdx.x / nc, c = blockIdx.x % nc, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const raw* row = static_cast<const raw*>(a.logits) + (size_t)r * a.ld;
  out_t* out = static_cast<out_t*>(a.out) + (size_t)r * a.old;
  // Vector v has elements v VE - lead + [0, VE) of the row, aligned in the result, and
  // (unless across) in the logits.  This CTA has vectors [v0, v1), of which [w0, w1) lie
  // inside the row; the values of the others, one at each end of the row, go one to a thread.
  const int lead = HOW == PR_ACROSS ? (int)((reinterpret_cast<uintptr_t>(out) & 15) / sizeof(out_t))
                                    : (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(raw));
  const int v0 = c * plan.seg, v1 = min((a.V + lead + VE - 1) / VE, v0 + plan.seg);
  const int w0 = max(v0, lead ? 1 : 0), w1 = min(v1, (a.V + lead) / VE);
  const char* first = reinterpret_cast<const char*>(row - lead);  // of vector 0
  const int off = HOW == PR_ACROSS ? (int)(reinterpret_cast<uintptr_t>(first) & 15) : 0;
  const uint4* src = reinterpret_cast<const uint4*>(first - off);
  uint32_t* touched = words;
  uint32_t* count = touched + plan.bits;
  int* keys = reinterpret_cast<int*>(count + plan.counts);  // cells; -1: none
  uint32_t* numbers = reinterpret_cast<uint32_t*>(keys + plan.table);
  float* biases = reinterpret_cast<float*>(numbers + plan.table);  // of cells with one; only with biases
  // The launch gets ready under the end of the work before it on the stream: nothing of
  // a caller's is read or written before that is complete.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // This warp's chunks of 32 * each vectors.
  const int each = plan.each, chunk = 32 * each;
  uint4 x[PU];
  auto load = [&](int vb) {
#pragma unroll
    for (int u = 0; u < PU; ++u) {
      const int v = vb + u * 32 + lane;
      if (u < each && v >= w0 && v < w1) x[u] = HOW == PR_ACROSS ? vector_across(src + v, off) : __ldcs(src + v);
    }
  };
  if (HOW != PR_IN_PLACE) load(v0 + warp * chunk);
  // The mask's words of a chunk, one to a lane, shifted so that they start at the chunk's first
  // value; values past the chunk count as legal.
  const uint32_t* bm = MASK ? a.bitmask + (size_t)r * a.W : nullptr;
  auto mask_words = [&](int vb, uint32_t& lo, uint32_t& hi) {
    // the first chunk of a row may start before it
    const int j0 = vb * VE - lead, k = (j0 >> 5) + lane;
    lo = k >= 0 && k < a.W ? bm[k] : ~0u;
    hi = (j0 & 31) && (j0 >> 5) + 32 < a.W ? bm[(j0 >> 5) + 32] : ~0u;
  };
  uint32_t mask_lo = ~0u, mask_hi = ~0u;  // of the next chunk
  if (MASK && v0 + warp * chunk < w1) mask_words(v0 + warp * chunk, mask_lo, mask_hi);

  const int32_t* history = a.history + (size_t)r * a.hld;
  const int32_t* bias_ids = a.bias_ids + (size_t)r * a.NB;
  const float* bias = a.bias + (size_t)r * a.NB;
  const ProcessRow p = process_row(a, r);
  const int length = a.lengths ? a.lengths[r] : a.H, prompt = a.prompts ? a.prompts[r] : 0;
  // the first of the history and the biases, on their way with the parameters
  int early[PEARLY], bias_id = -1;
  float first_bias = 0.f;
#pragma unroll
  for (int k = 0; k < PEARLY; ++k) early[k] = !DENSE && tid + k * PT < a.H ? history[tid + k * PT] : -1;
  bool bad = !process_valid(p, length, prompt, a.H);
  for (int i = tid; i < a.NB; i += PT) {
    const int id = bias_ids[i];
    const float b = bias[i];
    if (i == tid) {
      bias_id = id;
      first_bias = b;
    }
    if ((unsigned)id < (unsigned)a.V && !(b < INFINITY)) bad = true;
  }
  const bool any = a.H > 0 || a.NB > 0;
  if (any) {
    const int clear = plan.bits + plan.counts;  // a multiple of 4
    for (int i = tid * 4; i < clear; i += PT * 4) *reinterpret_cast<uint4*>(words + i) = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < plan.table; i += PT) {
      keys[i] = -1;
      numbers[i] = 0u;
    }
    bad = __syncthreads_or(bad);
  } else {
    bad = __any_sync(0xffffffffu, bad);  // the same in all threads
  }
  if (c == 0 && tid == 0) a.status[r] = bad ? SMP_ERR_INVALID_PARAM : SMP_OK;
  // tokens [j0, j1) are this CTA's; a token's cell is its distance from `base`
  const int base = v0 * VE - lead, j0 = max(0, base), j1 = min(a.V, v1 * VE - lead);
  const unsigned span = (unsigned)max(0, j1 - j0);
  if (any && !bad) {
    if constexpr (DENSE) {
      // entries [i0, i1): nothing but a subtraction and a comparison for most
      auto scan = [&](int i0, int i1, bool generated) {
        for (; i0 < i1; i0 += PT * PBATCH) {
          int t[PBATCH];
          if (i0 + PT * PBATCH <= i1) {
#pragma unroll
            for (int k = 0; k < PBATCH; ++k) t[k] = history[i0 + tid + k * PT];
          } else {
#pragma unroll
            for (int k = 0; k < PBATCH; ++k) t[k] = i0 + tid + k * PT < i1 ? history[i0 + tid + k * PT] : -1;
          }
#pragma unroll
          for (int k = 0; k < PBATCH; ++k) {
            if ((unsigned)t[k] - (unsigned)j0 < span) {
              if (generated) atomicAdd(&count[t[k] - base], 1u);
              else atomicOr(&count[t[k] - base], PSEEN);
            }
          }
        }
      };
      scan(0, prompt, false);
      scan(prompt, length, true);
    } else {
      auto seen = [&](int t, int i) {  // entry i of the history
        if (i >= length || (unsigned)t - (unsigned)j0 >= span) return;
        const int u = t - base;
        uint32_t* n = &numbers[process_entry(keys, plan.table, u, true)];
        if (i < prompt) atomicOr(n, PSEEN);
        else atomicAdd(n, 1u);
        atomicOr(&touched[u >> 5], 1u << (u & 31));
      };
#pragma unroll
      for (int k = 0; k < PEARLY; ++k)
        if (k * PT < length) seen(early[k], tid + k * PT);
      for (int i0 = PEARLY * PT; i0 < length; i0 += PT * PBATCH) {
        int t[PBATCH];
#pragma unroll
        for (int k = 0; k < PBATCH; ++k) t[k] = i0 + tid + k * PT < length ? history[i0 + tid + k * PT] : -1;
#pragma unroll
        for (int k = 0; k < PBATCH; ++k) {
          if (i0 + k * PT >= length) break;
          seen(t[k], i0 + tid + k * PT);
        }
      }
    }
    for (int i = tid; i < a.NB; i += PT) {
      const int id = i == tid ? bias_id : bias_ids[i];
      if ((unsigned)id - (unsigned)j0 >= span) continue;
      const int u = id - base;
      const int at = process_entry(keys, plan.table, u, true);
      if (atomicOr(&numbers[at], PBIAS) & PBIAS) atomicOr(&numbers[at], PMULTI);
      else biases[at] = i == tid ? first_bias : bias[i];
      if (DENSE && a.H) atomicOr(&count[u], PBIAS);
      if (!(DENSE && a.H)) atomicOr(&touched[u >> 5], 1u << (u & 31));
    }
    __syncthreads();
    if (DENSE && a.H) {  // a byte of touched from eight counts
      for (int i = tid; i < plan.counts / 8; i += PT) {
        const uint4 lo = reinterpret_cast<const uint4*>(count)[2 * i], hi = reinterpret_cast<const uint4*>(count)[2 * i + 1];
        const uint32_t b = (lo.x ? 1 : 0) | (lo.y ? 2 : 0) | (lo.z ? 4 : 0) | (lo.w ? 8 : 0) | (hi.x ? 16 : 0) |
                           (hi.y ? 32 : 0) | (hi.z ? 64 : 0) | (hi.w ? 128 : 0);
        reinterpret_cast<uint8_t*>(touched)[i] = (uint8_t)b;
      }
      __syncthreads();
    }
  }
  // A touched token's result from its logit.
  auto changed = [&](float v, int u, int id) {
    const bool by_cell = DENSE && a.H > 0;
    uint32_t n = by_cell ? count[u] : 0u;
    float only = 0.f;
    if (!by_cell || (n & PBIAS)) {
      const int at = process_entry(keys, plan.table, u, false);
      n |= numbers[at];
      if (n & PBIAS) only = biases[at];
    }
    return process_token(a, p, v, n, only, id, bias_ids, bias);
  };
  const bool look = any && !bad, masked = MASK && !bad;
  for (int vb = v0 + warp * chunk; vb < w1; vb += SW * chunk) {
    // the mask's bits of this lane's vectors, and those touched, VE for each vector
    uint32_t legal = ~0u, hits = 0u;
    bool some = false;  // something masked in the chunk
    if constexpr (MASK) {
      if (masked) {
        const uint32_t next = __shfl_down_sync(0xffffffffu, mask_lo, 1);
        uint32_t w = __funnelshift_r(mask_lo, lane < 31 ? next : mask_hi, (vb * VE - lead) & 31);
        const int valid = min(chunk, w1 - vb) * VE - lane * 32;
        if (valid < 32) w |= valid > 0 ? ~0u << valid : ~0u;
        if (vb < w0 && lane == 0) w |= (1u << (w0 - vb) * VE) - 1;  // of a vector that is not whole
        if (vb + SW * chunk < w1) mask_words(vb + SW * chunk, mask_lo, mask_hi);
        some = __any_sync(0xffffffffu, w != ~0u);
        if (some) {
          legal = 0u;
#pragma unroll
          for (int u = 0; u < PU; ++u) {
            const uint32_t b = __shfl_sync(0xffffffffu, w, (u * 32 + lane) * VE / 32 & 31) >> (lane * VE & 31);
            legal |= (b & ALL) << (u * VE);
          }
        }
      }
    }
    if (look) {  // a word of touched to a lane, VE bits of it for each of 32 / VE vectors
      const uint32_t w = lane < each * VE ? touched[(vb - v0) * VE / 32 + lane] : 0u;
      if (__any_sync(0xffffffffu, w != 0u)) {
#pragma unroll
        for (int u = 0; u < PU; ++u)
          hits |= ((__shfl_sync(0xffffffffu, w, (u * 32 + lane) * VE / 32 & 31) >> (lane * VE & 31)) & ALL) << (u * VE);
        hits &= legal;
        if (vb < w0 && lane < w0 - vb) hits &= ~ALL;
        if (vb + chunk > w1) {
#pragma unroll
          for (int u = 0; u < PU; ++u)
            if (vb + u * 32 + lane >= w1) hits &= ~(ALL << (u * VE));
        }
      }
    }
    if (HOW == PR_IN_PLACE && !some && !__any_sync(0xffffffffu, hits != 0u)) continue;
    if (HOW == PR_IN_PLACE) {
#pragma unroll
      for (int u = 0; u < PU; ++u) {
        const uint32_t b = (legal >> (u * VE)) & ALL;
        const int v = vb + u * 32 + lane;
        if (u < each && v >= w0 && v < w1 && b && (b != ALL || ((hits >> (u * VE)) & ALL))) x[u] = src[v];
      }
    }
#pragma unroll
    for (int u = 0; u < PU; ++u) {
      const int v = vb + u * 32 + lane, j = v * VE - lead;
      if (u >= each || v < w0 || v >= w1) continue;
      const uint32_t b = (legal >> (u * VE)) & ALL;
      if (HOW != PR_IN_PLACE || b != ALL) {
        uint4 y = x[u];
        if (MASK && some) {
          y.x = WD::keep(y.x, b, 0);
          y.y = WD::keep(y.y, b, 1);
          y.z = WD::keep(y.z, b, 2);
          y.w = WD::keep(y.w, b, 3);
        }
        if constexpr (DT == OT) {
          __stcs(reinterpret_cast<uint4*>(out + j), y);
        } else {
          float f[VE];
          sc_unpack<DT>(y, f);
          float4* to = reinterpret_cast<float4*>(out + j);
          __stcs(to, make_float4(f[0], f[1], f[2], f[3]));
          __stcs(to + 1, make_float4(f[4], f[5], f[6], f[7]));
        }
      }
    }
    while (hits) {  // over what was just written
      const int k = __ffs(hits) - 1, u = k / VE, e = k % VE, w = DT == SMP_F32 ? e : e >> 1;
      hits &= hits - 1;
      const uint4 y = u & 2 ? (u & 1 ? x[3] : x[2]) : (u & 1 ? x[1] : x[0]);
      const uint32_t word = w & 2 ? (w & 1 ? y.w : y.z) : (w & 1 ? y.y : y.x);
      raw value;
      if constexpr (DT == SMP_F32) value = __uint_as_float(word);
      else value = (raw)(e & 1 ? word >> 16 : word);
      const int j = (vb + u * 32 + lane) * VE - lead + e;
      out[j] = TO::store(changed(TI::value(value), j - base, j));
    }
    if (HOW != PR_IN_PLACE) load(vb + SW * chunk);
  }
  // the values outside whole vectors
  const int head = v0 < w0 ? min(a.V, VE - lead) : 0, tail = v1 > w1 ? max(head, w1 * VE - lead) : a.V;
  const int j = tid < head ? tid : tail + tid - head;
  if (v0 < v1 && tid < PENDS && j < a.V && (tid < head || v1 > w1)) {
    const int u = j - base;
    const bool hit = look && ((touched[u >> 5] >> (u & 31)) & 1u);
    const bool none = masked && !((bm[j >> 5] >> (j & 31)) & 1u);
    float v = none ? -INFINITY : TI::value(row[j]);
    if (hit && !none) v = changed(v, u, j);
    if (HOW != PR_IN_PLACE || hit || none) out[j] = TO::store(v);
  }
}

// Entries of a table for as many tokens.
constexpr int process_table(int held) { return held + held / 2 + 8; }

// Histories and biases of up to PSHORT entries go into a table, and a segment is as long
// as the batch allows: rounds of CTAs times what each has to do, its set-up counted as
// PSETUP cells (in place, where a cell is less work, as twice that).  1024 x 256000 f16 to
// binary32 with 512 entries: 248 us with PSETUP 1024 or 2048, 273 with 4096; 512 x 151936
// masked in place: 42, 33 and 30.  Longer ones are counted by cell, by CTAs of 1024 threads, as
// nearly all the work is to look through the history: 64 x 32000 with 4096 entries 16 us, 18
// with 512 threads; 16 x 50001 with 65536 entries 12.7, and 41 where the CTAs of a row share
// the entries and count into each other's shared memory.  Up to 2048 entries the table is
// faster: 128 x 128256 with 1500 entries 18 us, 36 counted by cell.  What counts is what the
// buffers hold, as the host does not know a row's length: 128 x 128256 bf16 with 500 entries in use
// takes 15.3 us from a buffer of up to 2048, 26.1 from a longer one (in place 6.7 and 21.0).
template <int DT, int OT, int HOW>
int launch_process(const ProcessArgs& a, int sms, cudaStream_t st) {
  constexpr int VE = DT == SMP_F32 ? 4 : 8;
  ProcessPlan plan;
  const bool dense = a.H + a.NB > PSHORT;
  const int threads = dense ? PLARGE : PSMALL;
  const int vectors = (a.V + VE - 1) / VE + 1, unit = threads;  // a row may start inside one; a vector to each thread
  const int most = (dense ? PDENSE : PMOST) / VE;
  plan.seg = most;
  const long long resident = (long long)(dense ? PDENSECTAS : PCTAS) * sms;
  const long long setup = HOW == PR_IN_PLACE ? 2 * PSETUP : PSETUP;  // a cell is less work there
  long long least = -1;
  for (int steps = 1; steps * unit <= most; steps += dense ? steps : steps < 4 ? 1 : 4) {
    const int seg = steps * unit;
    const long long ctas = (long long)a.B * ((vectors + seg - 1) / seg), rounds = (ctas + resident - 1) / resident;
    const long long cost = rounds * (setup + a.H + seg * VE);
    if (least < 0 || cost < least) {
      least = cost;
      plan.seg = seg;
    }
    if (seg >= vectors) break;
  }
  plan.nc = (vectors + plan.seg - 1) / plan.seg;
  plan.each = plan.seg < unit ? 1 : plan.seg / unit < PU ? plan.seg / unit : PU;  // never 0: a step is that long
  const int words = (plan.seg * VE + 31) / 32;
  plan.bits = (words + 3) & ~3;
  plan.counts = dense && a.H ? plan.seg * VE : 0;
  const int held = (dense && a.H ? 0 : a.H) + a.NB;
  plan.table = held ? process_table(held) : 0;
  if ((long long)a.B * plan.nc > 0x7fffffffLL) return SMP_ERR_CAPACITY;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * plan.nc));
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cfg.dynamicSmemBytes = (size_t)(plan.bits + plan.counts + plan.table * (a.NB ? 3 : 2)) * 4;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto kernel = dense ? (a.bitmask ? process_kernel<DT, OT, HOW, true, PLARGE> : process_kernel<DT, OT, HOW, false, PLARGE>)
                            : (a.bitmask ? process_kernel<DT, OT, HOW, true, PSMALL> : process_kernel<DT, OT, HOW, false, PSMALL>);
  // The limit is the kernel's, for all threads of the process: always the most that a plan may
  // have, as a call with less could set it between another's setting and its launch.
  constexpr int by_cell = (PDENSE / 32 + PDENSE + 3 * process_table(PR_MAX_NB)) * 4;
  constexpr int by_table = (PMOST / 32 + 3 * process_table(PSHORT)) * 4;
  static_assert(by_cell <= 227 * 1024 && by_table <= 227 * 1024, "every plan fits an SM");
  if (cfg.dynamicSmemBytes > 48 * 1024 &&
      !sc_ok(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, dense ? by_cell : by_table)))
    return SMP_ERR_CUDA;
  return sc_ok(cudaLaunchKernelEx(&cfg, kernel, a, plan)) ? SMP_OK : SMP_ERR_CUDA;
}

template <int DT>
int launch_sparse(const ProcessArgs& a, cudaStream_t st) {
  const int size = process_table(a.H + a.NB);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.B);
  cfg.blockDim = dim3(PSPARSE);
  cfg.stream = st;
  cfg.dynamicSmemBytes = (size_t)size * (a.NB ? 3 : 2) * 4;
  static_assert(process_table(PSHORT) * 12 <= 48 * 1024, "the table needs no opt-in");
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return sc_ok(cudaLaunchKernelEx(&cfg, process_sparse_kernel<DT>, a, size)) ? SMP_OK : SMP_ERR_CUDA;
}

template <int DT, int OT>
int launch_to(const ProcessArgs& a, cudaStream_t st) {
  const int sms = sc_sm_count();
  if (sms < 1) return SMP_ERR_CUDA;
  if constexpr (DT == OT) {
    if (a.out == a.logits && !a.bitmask && a.H + a.NB <= PSHORT) return launch_sparse<DT>(a, st);
    if (a.out == a.logits) return launch_process<DT, DT, PR_IN_PLACE>(a, sms, st);
  }
  // whether a place that is aligned in the logits is so in the result, in all rows
  constexpr int in = DT == SMP_F32 ? 4 : 2, to = OT == SMP_F32 ? 4 : 2;
  const long long d0 = (long long)(reinterpret_cast<uintptr_t>(a.logits) / in) - (long long)(reinterpret_cast<uintptr_t>(a.out) / to);
  const bool alike = ((d0 | (a.ld - a.old)) & (16 / to - 1)) == 0;
  return alike ? launch_process<DT, OT, PR_COPY>(a, sms, st) : launch_process<DT, OT, PR_ACROSS>(a, sms, st);
}

}  // namespace

int process_enqueue(const ProcessArgs& a, int dtype, int out_dtype, cudaStream_t st) {
  if (dtype == SMP_F32) return launch_to<SMP_F32, SMP_F32>(a, st);
  if (dtype == SMP_BF16)
    return out_dtype == SMP_F32 ? launch_to<SMP_BF16, SMP_F32>(a, st) : launch_to<SMP_BF16, SMP_BF16>(a, st);
  return out_dtype == SMP_F32 ? launch_to<SMP_F16, SMP_F32>(a, st) : launch_to<SMP_F16, SMP_F16>(a, st);
}

}  // namespace smp
