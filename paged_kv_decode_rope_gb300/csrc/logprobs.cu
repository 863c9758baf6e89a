// logprobs.cu -- log-probabilities of given tokens, with the entropy of each
// row's distribution and its most likely tokens, in one pass over the logits.
//
// With y_v = scale x_v, M = max y, S = sum e^(y-M) and Z = sum (y-M) e^(y-M):
//     lse = M + log S,   logp_t = y_t - lse,   H = log S - Z / S.
// The logits are read once from memory: a thread streams 16-byte vectors of
// its row, keeping S and Z against a reference that it moves only when a
// logit passes it by more than kSlack (base 2, so a term stays below 2^kSlack
// and the sums lose nothing), in fp32 with paired arithmetic. CTAs stay and
// take row after row; a warp of its own issues bulk copies into a ring of
// shared-memory stages and runs ahead into the next row while the others pick
// the alternatives of this one, so that the memory never idles (a CTA a row,
// loading as it went: 128 us for 2048 rows of 128256 bf16, 60% of the copy
// bandwidth). What bounds it
// is that stream; the arithmetic (unpack, difference, product, exp2, two sums an
// element) is the next limit, about half of it.
//
// The most likely tokens come without sorting the row. Every thread's vectors
// are a group; a group's best logit is known after the stream. The K groups
// with the best ones (ties: the group whose best comes first) hold the row's K
// best logits, since the K group bests are K logits that no logit outside
// these groups beats. So only K groups of the CTA's threads are read again
// (from L2: K / kLogThreads of the row), and of them only the logits not below
// the K-th group best are kept, about K of them. Keys are 64-bit: the logit as
// an ordered integer above, the complement of its index below, so that equal
// logits rank by index and all keys differ; any number of ties (a row of equal
// logits, or masked to -inf) costs no more than others.
//
// Few rows are split over several CTAs each, as many as give every SM work;
// the last CTA of a row to finish (a ticket in the workspace) merges the
// pieces in their order, so the result does not depend on which one it is.
#include <atomic>
#include <cerrno>
#include <cmath>

#include "f32x2.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kLogThreads = 256;
constexpr int kLogCtas = 4;         // CTAs a SM
constexpr int kLogWarps = kLogThreads / 32;
constexpr int kTop = PKV_MAX_TOP;
constexpr int kUnroll = 4;          // vectors a thread takes from a stage
constexpr int kLogStages = 3;
constexpr int kStageVectors = kUnroll * kLogThreads;
constexpr int kLogBlock = kLogThreads + 32;  // and the copying warp
constexpr int kCandidates = 256;    // keys the second look keeps at once
constexpr int kMaxSplits = 64;
#ifndef KMIN
#define KMIN 4
#endif
constexpr int kMinSplitVectors = KMIN * kLogThreads;  // smallest piece of a split row
constexpr float kLogSlack = 8.f;
// In the stream a logit below kLowest counts as kLowest, so that -inf makes
// e^y = 0 and 0 * y = 0, not NaN; only a logit above kFloor sets the reference
// (100 times smaller, so that e^y of kLowest is 0 for any scale in kMinScale
// .. 1 / kMinScale). A CTA whose logits are all at or below kFloor (masked by
// the type's lowest value) takes its sums again without these limits.
constexpr float kLowest = -1e30f, kFloor = -1e28f;
constexpr float kMinScale = 1e-6f;
static_assert(kTop == 32, "a sorted list is one key a lane");
static_assert(kCandidates == kLogThreads, "a warp sorts 32 candidates");

struct LogprobsParams {
  const uint8_t* logits;
  long long row_bytes;
  int rows, vocab;
  float c2;     // scale * log2 e
  float scale;
  const int32_t* targets;
  int top;
  float* logprobs;
  float* entropy;
  int32_t* top_ids;
  float* top_logprobs;
  int splits;          // CTAs a row
  int split_vectors;   // vectors of each
  int* tickets;        // [rows], zero between calls
  float4* sums;        // [rows][splits] {M, S, Z, -} (base 2)
  uint64_t* keys;      // [rows][splits][kTop]
};

// A logit as an integer of the same order (-0 as +0, NaN as -inf), and back.
__device__ __forceinline__ uint32_t ordered(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint64_t key_of(float x, int index) {
  return static_cast<uint64_t>(ordered(x)) << 32 | (0xffffffffu - static_cast<uint32_t>(index));
}
__device__ __forceinline__ int index_of(uint64_t key) {
  return static_cast<int>(0xffffffffu - static_cast<uint32_t>(key));
}

// One compare-exchange of a bitonic network over the warp's keys: lane and
// lane ^ j, the larger one to the lane that `first` says.
__device__ __forceinline__ uint64_t exchange(uint64_t key, int j, bool larger) {
  const uint64_t o = __shfl_xor_sync(kFull, key, j);
  return (key > o) == larger ? key : o;
}
// The warp's 32 keys, largest first.
__device__ __forceinline__ uint64_t sort32(uint64_t key, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j; j >>= 1) key = exchange(key, j, ((lane & j) == 0) == ((lane & k) == 0));
  return key;
}
// The 32 largest of two lists sorted largest first, sorted again.
__device__ __forceinline__ uint64_t merge32(uint64_t a, uint64_t b, int lane) {
  b = __shfl_sync(kFull, b, 31 - lane);
  uint64_t key = a > b ? a : b;  // bitonic
#pragma unroll
  for (int j = 16; j; j >>= 1) key = exchange(key, j, (lane & j) == 0);
  return key;
}
// A barrier of the CTA's computing warps.
__device__ __forceinline__ void compute_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kLogThreads) : "memory");
}
// The 32 largest of the first `lists` warps' sorted lists, in warp 0 (all
// computing threads call it; s_list is free again after the caller's next
// barrier).
__device__ __forceinline__ uint64_t merge_warps(uint64_t key, uint64_t (*s_list)[32], int lists) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int half = 1;
  while (2 * half < lists) half *= 2;
  if (warp < lists) s_list[warp][lane] = key;
  for (; half >= 1; half >>= 1) {
    compute_sync();
    if (warp < half && warp + half < lists) {
      key = merge32(key, s_list[warp + half][lane], lane);
      s_list[warp][lane] = key;
    }
    lists = min(lists, half);
  }
  return key;
}

template <typename T>
struct Vec;
template <>
struct Vec<uint16_t> {  // 8 bf16
  static constexpr int kElems = 8;
  __device__ static float get(const uint4& w, int e) {
    const uint32_t u = e < 2 ? w.x : e < 4 ? w.y : e < 6 ? w.z : w.w;
    return __uint_as_float(e & 1 ? u & 0xffff0000u : u << 16);
  }
  __device__ static uint16_t raw(const uint8_t* p) { return *reinterpret_cast<const uint16_t*>(p); }
  __device__ static float value(uint16_t r) { return __uint_as_float(static_cast<uint32_t>(r) << 16); }
  // the largest element, NaN ignored
  __device__ static float max(const uint4& w) {
    uint32_t a, b;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(w.x), "r"(w.y));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(w.z), "r"(w.w));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
    const float2 f = bf16x2_to_float2(a);
    return fmaxf(f.x, f.y);
  }
  // pair i, -inf as kLowest, NaN kept
  __device__ static float2 pair(const uint4& w, int i) {
    uint32_t u = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(u) : "r"(0xf149f149u));  // bf16 -9.95e29
    return bf16x2_to_float2(u);
  }
};
template <>
struct Vec<float> {  // 4 fp32
  static constexpr int kElems = 4;
  __device__ static float get(const uint4& w, int e) {
    return __uint_as_float(e == 0 ? w.x : e == 1 ? w.y : e == 2 ? w.z : w.w);
  }
  __device__ static float raw(const uint8_t* p) { return *reinterpret_cast<const float*>(p); }
  __device__ static float value(float r) { return r; }
  __device__ static float max(const uint4& w) {
    return fmaxf(fmaxf(get(w, 0), get(w, 1)), fmaxf(get(w, 2), get(w, 3)));
  }
  __device__ static float2 pair(const uint4& w, int i) {
    float a = get(w, 2 * i), b = get(w, 2 * i + 1);
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(kLowest));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(b) : "f"(kLowest));
    return make_float2(a, b);
  }
};

// What one side has seen: its reference logit m, S = sum e^(y - y_m) and
// Z = sum of (y - y_m) e^(y - y_m), y in base 2 (y = c2 x). m = -inf: no logit
// that set a reference (then s is 0, or NaN).
struct Sums {
  float m, s, z;
  __device__ void join(const Sums& o, float c2) {
    const float mm = fmaxf(m, o.m);
    // a side without logits keeps its 0 (or NaN); with a logit of +inf the
    // difference of infinities makes the NaN that such a row has
    const float da = m == -INFINITY ? 0.f : (m - mm) * c2, db = o.m == -INFINITY ? 0.f : (o.m - mm) * c2;
    const float wa = exp2f(da), wb = exp2f(db);
    z = (wa > 0.f ? wa * (z + s * da) : wa * s) + (wb > 0.f ? wb * (o.z + o.s * db) : wb * o.s);
    s = wa * s + wb * o.s;
    m = mm;
  }
};

// A piece of a row, as 16-byte vectors at 16-byte addresses: vector v holds
// elements v kE - off .. + kE - 1 of the row; the row's first and last vector
// may be partly outside it.
template <typename T>
struct Piece {
  static constexpr int kE = Vec<T>::kElems;
  const uint8_t* base;   // element 0
  const uint8_t* vbase;  // vector 0
  int row, off, vocab;
  int v0, v1;            // the piece's vectors
  int whole0, whole1;    // vectors that lie inside the row
  __device__ Piece(const LogprobsParams& p, int piece) {
    row = piece / p.splits;
    const int split = piece - row * p.splits;
    base = p.logits + static_cast<size_t>(row) * p.row_bytes;
    off = static_cast<int>((reinterpret_cast<uintptr_t>(base) & 15u) / sizeof(T));
    vbase = base - off * sizeof(T);
    vocab = p.vocab;
    const int nv = static_cast<int>((static_cast<long long>(off) + vocab + kE - 1) / kE);
    v0 = split * p.split_vectors;
    v1 = min(nv, v0 + p.split_vectors);
    whole0 = off ? 1 : 0;
    whole1 = (off + vocab) % kE ? nv - 1 : nv;
  }
  // Vector v from memory; elements outside the row are -inf and never read.
  __device__ uint4 load(int v) const {
    if (v >= whole0 && v < whole1) return __ldg(reinterpret_cast<const uint4*>(vbase) + v);
    union {
      T t[kE];
      uint4 w;
    } u;
    const float none = -INFINITY;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const int i = v * kE - off + e;
      if (i >= 0 && i < vocab) {
        u.t[e] = Vec<T>::raw(base + static_cast<size_t>(i) * sizeof(T));
      } else if constexpr (sizeof(T) == 2) {
        u.t[e] = 0xff80u;
      } else {
        u.t[e] = none;
      }
    }
    return u.w;
  }
};

template <typename T>
__global__ void __launch_bounds__(kLogBlock, kLogCtas) logprobs_kernel(const LogprobsParams p) {
  using V = Vec<T>;
  constexpr int kE = V::kElems;
  extern __shared__ __align__(128) uint8_t s_ring[];
  __shared__ __align__(8) uint64_t full[kLogStages], empty[kLogStages];
  __shared__ uint64_t s_list[kLogWarps][32];
  __shared__ uint64_t s_cand[kCandidates];
  __shared__ Sums s_sums[kLogWarps];
  __shared__ int s_group[kTop];
  __shared__ uint64_t s_bound;
  __shared__ int s_count, s_last;
  __shared__ uint32_t s_top;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int pieces = p.rows * p.splits;
  if (tid == 0) {
    for (int s = 0; s < kLogStages; ++s) {
      mbar_init(smem_addr(&full[s]), 1);
      mbar_init(smem_addr(&empty[s]), kLogWarps);
    }
  }
  fence_mbar_init();
  __syncthreads();
  int chunk = 0;  // stages used so far

  if (warp == kLogWarps) {
    // ---- the copies: every piece's whole vectors, kStageVectors a stage ----
    if (lane != 0) return;
    bool failed = false;
    for (int piece = blockIdx.x; piece < pieces && !failed; piece += gridDim.x) {
      const Piece<T> r(p, piece);
      for (int c = r.v0; c < r.v1; c += kStageVectors, ++chunk) {
        const int st = chunk % kLogStages, use = chunk / kLogStages;
        if (use > 0 && !mbar_wait_bounded(smem_addr(&empty[st]), (use - 1) & 1)) {
          failed = true;
          break;
        }
        const int a = max(c, r.whole0), b = min(min(c + kStageVectors, r.v1), r.whole1);
        const uint32_t bar = smem_addr(&full[st]);
        if (a < b) {
          const uint32_t bytes = static_cast<uint32_t>(b - a) * 16u;
          mbar_arrive_expect_tx(bar, bytes);
          bulk_g2s(smem_addr(s_ring) + (st * kStageVectors + (a - c)) * 16, r.vbase + static_cast<size_t>(a) * 16, bytes,
                   bar);
        } else {
          mbar_arrive(bar);
        }
      }
    }
    // let the copies still in flight land before shared memory goes away
    for (int k = max(0, chunk - kLogStages); k < chunk; ++k)
      mbar_wait_bounded(smem_addr(&full[k % kLogStages]), (k / kLogStages) & 1);
    return;
  }

  for (int piece = blockIdx.x; piece < pieces; piece += gridDim.x) {
    const Piece<T> r(p, piece);
    const int row = r.row, v0 = r.v0, v1 = r.v1;
    // ---- the stream ----
    // The reference is a logit, so that x - ref is exact where it matters (near
    // the largest logits) whatever the scale; it moves when a logit passes
    // limit = ref + kLogSlack / c2.
    float ref = -INFINITY, limit = kFloor;
    const float slack = kLogSlack / p.c2;
    float best = -INFINITY;
    int best_v = v0 + tid;
    uint64_t s2 = f32x2(0.f, 0.f), z2 = s2;
    const uint64_t cc = f32x2(p.c2, p.c2);
    auto take = [&](const uint4& w, int v) {
      const float m = V::max(w);
      if (m > best) {
        best = m;
        best_v = v;
      }
      if (m > limit) {  // move the reference: the first logit, or one far above it
        if (ref != -INFINITY) {
          const float d = (ref - m) * p.c2, f = fast_exp2(d);
          const float2 s = unpack_f32x2(s2), z = unpack_f32x2(z2);
          s2 = f32x2(s.x * f, s.y * f);
          z2 = f32x2((z.x + s.x * d) * f, (z.y + s.y * d) * f);
        }
        ref = m;
        limit = m + slack;
      }
      const float nref = ref == -INFINITY ? 0.f : -ref;
      const uint64_t nr = f32x2(nref, nref);
#pragma unroll
      for (int i = 0; i < kE / 2; ++i) {
        const float2 x = V::pair(w, i);
        const uint64_t y2 = mul_f32x2(add_f32x2(f32x2(x.x, x.y), nr), cc);
        const float2 y = unpack_f32x2(y2);
        const uint64_t e2 = f32x2(fast_exp2(y.x), fast_exp2(y.y));
        s2 = add_f32x2(s2, e2);
        z2 = fma_f32x2(e2, y2, z2);
      }
    };
    bool late = false;  // a copy did not come: its vectors count as NaN
    for (int c = v0; c < v1; c += kStageVectors, ++chunk) {
      const int st = chunk % kLogStages;
      if (!mbar_wait_bounded(smem_addr(&full[st]), (chunk / kLogStages) & 1)) late = true;
      const uint32_t src = smem_addr(s_ring) + (st * kStageVectors + tid) * 16;
      if (c >= r.whole0 && c + kStageVectors <= min(v1, r.whole1)) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) take(lds128(src + u * kLogThreads * 16), c + tid + u * kLogThreads);
      } else {  // a stage at the row's or the piece's end
#pragma unroll 1
        for (int u = 0; u < kUnroll; ++u) {
          const int v = c + tid + u * kLogThreads;
          if (v >= v1) break;
          take(v >= r.whole0 && v < r.whole1 ? lds128(src + u * kLogThreads * 16) : r.load(v), v);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&empty[st]));
    }

    // ---- the sums of the CTA ----
    Sums all;
    {
      const float2 s = unpack_f32x2(s2), z = unpack_f32x2(z2);
      all = Sums{ref, late ? NAN : s.x + s.y, z.x + z.y};
    }
    auto share_sums = [&]() {  // of each warp
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        Sums t;
        t.m = __shfl_xor_sync(kFull, all.m, o);
        t.s = __shfl_xor_sync(kFull, all.s, o);
        t.z = __shfl_xor_sync(kFull, all.z, o);
        all.join(t, p.c2);
      }
      if (lane == 0) s_sums[warp] = all;
      compute_sync();
    };
    if (tid == 0) s_top = 0u;
    share_sums();
    bool any = false;
#pragma unroll
    for (int w = 0; w < kLogWarps; ++w) any |= s_sums[w].m != -INFINITY;
    if (!any) {  // nothing above kFloor: rare
      atomicMax(&s_top, ordered(best));
      compute_sync();
      const float top = unordered(s_top);
      if (top != -INFINITY) {
        all = Sums{top, 0.f, 0.f};
        for (int u = v0 + tid; u < v1; u += kLogThreads) {
          const uint4 w = r.load(u);
#pragma unroll
          for (int e = 0; e < kE; ++e) {
            const float y = (V::get(w, e) - top) * p.c2, f = exp2f(y);
            all.s += f;
            if (f > 0.f) all.z += f * y;
          }
        }
        share_sums();
      }
    }

    // ---- the K best of the CTA's piece ----
    uint64_t key = 0;
    if (p.top > 0) {
      // each group by its best logit and the vector that holds it
      key = v0 + tid < v1 ? key_of(best, best_v) : 0;
      key = merge_warps(sort32(key, lane), s_list, kLogWarps);
      if (warp == 0) {
        s_group[lane] = key && lane < p.top ? (index_of(key) - v0) % kLogThreads : -1;
        if (lane == p.top - 1) {
          // no logit below the K-th group's best is needed (index: the last one
          // its vector can hold)
          s_bound = key ? (key >> 32 << 32 | (0xffffffffu - static_cast<uint32_t>(index_of(key) * kE - r.off + kE - 1)))
                        : 1;
        }
        if (lane == 0) s_count = 0;
      }
      compute_sync();
      for (;;) {
        const uint64_t bound = s_bound;
        const float least = unordered(static_cast<uint32_t>(bound >> 32));
        for (int g = warp; g < p.top; g += kLogWarps) {
          if (s_group[g] < 0) continue;
          for (int u = v0 + s_group[g] + lane * kLogThreads; u < v1; u += 32 * kLogThreads) {
            const uint4 w = r.load(u);
            if (bound > 1 && V::max(w) < least) continue;
#pragma unroll
            for (int e = 0; e < kE; ++e) {
              const int i = u * kE - r.off + e;
              const uint64_t k = key_of(V::get(w, e), i);
              if (i >= 0 && i < p.vocab && k >= bound) {
                const int at = atomicAdd(&s_count, 1);
                if (at < kCandidates) s_cand[at] = k;
              }
            }
          }
        }
        compute_sync();
        const int n = s_count;
        const int lists = min((min(n, kCandidates) + 31) / 32, kLogWarps);
        key = tid < min(n, kCandidates) ? s_cand[tid] : 0;
        if (warp < lists) key = sort32(key, lane);
        key = merge_warps(key, s_list, lists);
        if (n <= kCandidates) break;
        // More than fit: the K-th of those kept is a higher bound (all keys
        // differ, and more than K were kept), so look again.
        compute_sync();
        if (tid == p.top - 1) s_bound = key;
        if (tid == 0) s_count = 0;
        compute_sync();
      }
    }

    // ---- the row's result: from this piece, or from all of them ----
    if (warp == 0) {
      all = lane < kLogWarps ? s_sums[lane] : Sums{-INFINITY, 0.f, 0.f};
#pragma unroll
      for (int o = kLogWarps / 2; o; o >>= 1) {
        Sums t;
        t.m = __shfl_down_sync(kFull, all.m, o);
        t.s = __shfl_down_sync(kFull, all.s, o);
        t.z = __shfl_down_sync(kFull, all.z, o);
        all.join(t, p.c2);
      }
    }
    bool mine = true;  // this CTA writes the row's result
    if (p.splits > 1) {
      if (warp == 0) {
        if (lane < p.top) p.keys[static_cast<size_t>(piece) * kTop + lane] = key;
        if (lane == 0) p.sums[piece] = make_float4(all.m, all.s, all.z, 0.f);
        __threadfence();
        __syncwarp();
        if (lane == 0) s_last = atomicAdd(&p.tickets[row], 1) == p.splits - 1;
      }
      compute_sync();
      mine = s_last;
      if (mine) {
        __threadfence();
        const size_t first = static_cast<size_t>(row) * p.splits;
        if (p.top > 0) {
          const int lists = min(p.splits, kLogWarps);
          key = 0;
          for (int q = warp; q < p.splits; q += kLogWarps) {
            const uint64_t k =
                lane < p.top ? __ldcg(reinterpret_cast<const unsigned long long*>(p.keys + (first + q) * kTop + lane)) : 0;
            key = q == warp ? k : merge32(key, k, lane);
          }
          key = merge_warps(key, s_list, lists);
        }
        if (warp == 0) {
          all = Sums{-INFINITY, 0.f, 0.f};
          for (int q = lane; q < p.splits; q += 32) {
            const float4 t = __ldcg(p.sums + first + q);
            all.join(Sums{t.x, t.y, t.z}, p.c2);
          }
#pragma unroll
          for (int o = 16; o; o >>= 1) {
            Sums t;
            t.m = __shfl_down_sync(kFull, all.m, o);
            t.s = __shfl_down_sync(kFull, all.s, o);
            t.z = __shfl_down_sync(kFull, all.z, o);
            all.join(t, p.c2);
          }
          if (lane == 0) p.tickets[row] = 0;
        }
      }
    }
    if (mine && warp == 0) {
      const float m = __shfl_sync(kFull, all.m, 0), s = __shfl_sync(kFull, all.s, 0), z = __shfl_sync(kFull, all.z, 0);
      // without a finite logit there is no distribution
      const float log_s = m == -INFINITY ? NAN : logf(s);
      constexpr float kLn2f = 0.6931471805599453f;
      auto logp = [&](float x) { return (x - m) * p.scale - log_s; };
      if (lane == 0) {
        if (p.targets) {
          const int t = p.targets[row];
          p.logprobs[row] =
              t >= 0 && t < p.vocab ? logp(V::value(V::raw(r.base + static_cast<size_t>(t) * sizeof(T)))) : NAN;
        }
        if (p.entropy) p.entropy[row] = log_s - z / s * kLn2f;
      }
      if (lane < p.top) {
        p.top_ids[static_cast<size_t>(row) * p.top + lane] = index_of(key);
        p.top_logprobs[static_cast<size_t>(row) * p.top + lane] = logp(unordered(static_cast<uint32_t>(key >> 32)));
      }
    }
    compute_sync();  // the shared arrays are free for the next piece
  }
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// CTAs a row: as many as run at once (rounded down: a few CTAs of a second
// round would double the time), none smaller than kMinSplitVectors.
int splits_for(int rows, long long vectors, int sms) {
  const long long want = static_cast<long long>(kLogCtas) * sms / rows;
  long long n = vectors / kMinSplitVectors;
  if (n > want) n = want;
  if (n > kMaxSplits) n = kMaxSplits;
  return n < 1 ? 1 : static_cast<int>(n);
}

}  // namespace
}  // namespace pkv

extern "C" {

size_t token_logprobs_workspace_bytes(int rows, int vocab, int top) {
  using namespace pkv;
  if (rows < 1 || vocab < 1 || top < 0 || top > PKV_MAX_TOP || top > vocab) return 0;
  // room for either type: fp32 rows have more vectors, so at least as many pieces
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return 0;
  const int sms = device_sm_count(device);
  if (sms < 1) return 0;
  const size_t pieces = static_cast<size_t>(rows) * splits_for(rows, static_cast<long long>(vocab) / 4 + 2, sms);
  return align256(sizeof(int) * static_cast<size_t>(rows)) + align256(sizeof(float4) * pieces) +
         sizeof(uint64_t) * kTop * pieces;
}

int token_logprobs(const void* logits, int logits_type, long long row_stride, int rows, int vocab,
                   float scale, const int32_t* targets, int top, float* logprobs, float* entropy,
                   int32_t* top_ids, float* top_logprobs, void* workspace, size_t workspace_bytes,
                   void* stream) {
  using namespace pkv;
  if ((logits_type != PKV_BF16 && logits_type != PKV_F32) || rows < 0 || vocab < 1 || vocab > (1 << 30) ||
      row_stride < 0 || top < 0 || top > PKV_MAX_TOP || top > vocab || !(scale >= kMinScale) || !(scale <= 1.f / kMinScale))
    return -EINVAL;
  if (rows == 0) return 0;
  const size_t size = logits_type == PKV_BF16 ? 2 : 4;
  if (!logits || reinterpret_cast<uintptr_t>(logits) % size || !targets != !logprobs ||
      (top > 0 && (!top_ids || !top_logprobs)) || !workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return -EINVAL;
  const size_t need = token_logprobs_workspace_bytes(rows, vocab, top);
  if (need == 0 || workspace_bytes < need) return -EINVAL;
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return -EIO;
  }
  const int elems = static_cast<int>(16 / size);
  const long long vectors = (static_cast<long long>(vocab) + elems - 1) / elems + 1;
  LogprobsParams p;
  p.logits = static_cast<const uint8_t*>(logits);
  p.row_bytes = row_stride * static_cast<long long>(size);
  p.rows = rows;
  p.vocab = vocab;
  p.c2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.scale = scale;
  p.targets = targets;
  p.top = top;
  p.logprobs = logprobs;
  p.entropy = entropy;
  p.top_ids = top_ids;
  p.top_logprobs = top_logprobs;
  p.splits = splits_for(rows, vectors, device_sm_count(device));
  p.split_vectors = static_cast<int>((vectors + p.splits - 1) / p.splits);
  const size_t pieces = static_cast<size_t>(rows) * p.splits;
  if (pieces > 0x7fff0000u) return -EINVAL;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.tickets = reinterpret_cast<int*>(ws);
  ws += align256(sizeof(int) * static_cast<size_t>(rows));
  p.sums = reinterpret_cast<float4*>(ws);
  ws += align256(sizeof(float4) * pieces);
  p.keys = reinterpret_cast<uint64_t*>(ws);
  auto kernel = logits_type == PKV_BF16 ? logprobs_kernel<uint16_t> : logprobs_kernel<float>;
  constexpr int kSmem = kLogStages * kStageVectors * 16;
  static std::atomic<bool> ready[2];
  if (!ready[logits_type].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess) ready[logits_type].store(true, std::memory_order_relaxed);
  }
  if (e == cudaSuccess) {
    const size_t most = static_cast<size_t>(kLogCtas) * device_sm_count(device);
    kernel<<<static_cast<unsigned>(pieces < most ? pieces : most), kLogBlock, kSmem, static_cast<cudaStream_t>(stream)>>>(p);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return -EIO;
  }
  return 0;
}

}  // extern "C"
