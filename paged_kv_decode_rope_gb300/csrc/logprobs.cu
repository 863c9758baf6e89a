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
// bandwidth; now 114 us, 4.63 TB/s, 68%). Rows are handed out from a counter:
// with a fixed share for every CTA the slowest SM's memory path set the time
// (33% over the median's). What bounds it is that stream together with the
// issue slots of its arithmetic (unpack, difference, product, exp2, two sums
// an element) and of the selection. 64 rows of 151936 fp32 take 15.9 us, one
// row of 128256 bf16 9.7 us: launch, stream, selection and merge, one latency
// after the other (12.1 and 5.7 us where no alternatives are asked for).
//
// The most likely tokens come without sorting the row. Every thread's vectors
// are a group; a group's best logit is known after the stream. The K groups
// with the best ones (ties: the group whose best comes first) hold the row's K
// best logits, since the K group bests are K logits that no logit outside
// these groups beats. Of these groups only the logits not below the K-th group
// best are wanted, about K in all; unless a group's second best vector reaches
// that bound too, they are all in the vector of its best, which its thread
// keeps; in the few other cases the group is read again. Keys are 64-bit:
// the logit as an ordered integer above, the complement of its index below, so
// that equal logits rank by index and all keys differ; any number of ties (a
// row of equal logits, or masked to -inf) is resolved by the same steps.
//
// This selection is a chain of short steps, and its latency is what the copies
// running ahead into the CTA's next row must cover. First done by sorting the
// group bests and the candidates in bitonic networks and reading the K groups
// again, it took 25,000 cycles a row next to the stream's 42,000. So the K-th
// group best is found in two steps (a bound from the ceil(K / warps)-th best of
// each warp, by warp-wide maxima, leaves about twice K groups; those, and later
// the candidates, are ranked by counting).
//
// Few rows, and the rows left over when the CTAs have taken whole rounds, are
// split over several CTAs each; the last CTA of a row to finish (a ticket in the
// workspace) merges the pieces in their order, so the result does not depend
// on which one it is.
//
// Every wait is bounded. When one gives up, the computing warps of its CTA leave
// together (a barrier tells all of them), the workspace's error word says so and
// the CTA makes every row NaN; other CTAs may write theirs later. The counter and
// the tickets are then left as they are, so a call that finds the error word set
// writes NaN everywhere and touches neither. (All this takes 1.5% of the 2048
// rows: 113.6 us against 111.9.)
#include <atomic>
#include <cerrno>
#include <climits>
#include <cmath>

#include "f32x2.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kLogThreads = 256;
constexpr int kLogCtas = 3;         // CTAs a SM
constexpr int kLogWarps = kLogThreads / 32;
constexpr int kTop = PKV_MAX_TOP;
constexpr int kUnroll = 4;          // vectors a thread takes from a stage
constexpr int kLogStages = 4;
constexpr int kStageVectors = kUnroll * kLogThreads;
constexpr int kLogBlock = kLogThreads + 32;  // and the copying warp
constexpr int kCandidates = 256;    // keys ranked at once
constexpr int kMaxSplits = 64;
constexpr int kMinSplitVectors = 4 * kLogThreads;  // smallest piece of a split row
constexpr float kLogSlack = 8.f;
// In the stream a logit below kLowest counts as kLowest, so that -inf makes
// e^y = 0 and 0 * y = 0, not NaN; only a logit above kFloor sets the reference
// (100 times smaller, so that e^y of kLowest is 0 for any scale in kMinScale
// .. 1 / kMinScale). A CTA whose logits are all at or below kFloor (masked by
// the type's lowest value), or whose reference is above kHuge (so that a
// difference could overflow when scaled), takes its sums again without these
// limits.
constexpr float kLowest = -1e30f, kFloor = -1e28f, kHuge = 1e32f;
constexpr float kMinScale = 1e-6f;
static_assert(kTop == 32, "a sorted list is one key a lane");
static_assert(kCandidates == kLogThreads, "every group can be a candidate");

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
  int whole;           // rows 0 .. whole - 1 are a piece each
  int splits;          // pieces of each row after them
  int split_vectors;   // vectors of such a piece
  int pieces;          // of all rows
  int* error;          // PKV_ERR_TIMEOUT, from this call or one before it
  uint32_t polls;      // bound of the waits
  int* counter;        // pieces handed out past the first round, zero between calls
  int* tickets;        // [split rows], zero between calls
  float4* sums;        // [split pieces] {m, S, Z, -}
  uint64_t* keys;      // [split pieces][kTop]
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
// The same; true if `mine` is true in all of their threads.
__device__ __forceinline__ bool compute_all(bool mine) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(static_cast<uint32_t>(mine)), "n"(kLogThreads)
      : "memory");
  return all != 0;
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
  int row, split_row, off, vocab;  // split_row: among the split rows, -1 for a whole one
  int v0, v1;            // the piece's vectors
  int whole0, whole1;    // vectors that lie inside the row
  __device__ Piece(const LogprobsParams& p, int piece) {
    const int rest = piece - p.whole;
    split_row = rest < 0 ? -1 : rest / p.splits;
    const int split = rest < 0 ? 0 : rest - split_row * p.splits;
    row = rest < 0 ? piece : p.whole + split_row;
    base = p.logits + static_cast<size_t>(row) * p.row_bytes;
    off = static_cast<int>((reinterpret_cast<uintptr_t>(base) & 15u) / sizeof(T));
    vbase = base - off * sizeof(T);
    vocab = p.vocab;
    const int nv = static_cast<int>((static_cast<long long>(off) + vocab + kE - 1) / kE);
    v0 = rest < 0 ? 0 : min(nv, split * p.split_vectors);
    v1 = rest < 0 ? nv : min(nv, v0 + p.split_vectors);
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
  __shared__ __align__(8) uint64_t full[kLogStages], empty[kLogStages], piece_full[2], piece_empty[2];
  __shared__ int s_piece[2];  // the pieces to work on, in turns; -1: no more
  __shared__ uint64_t s_list[kLogWarps][32];  // merging pieces
  __shared__ __align__(16) uint64_t s_cand[kCandidates];
  __shared__ uint64_t s_best[kTop];           // the piece's best, in order
  __shared__ float s_ref[kLogWarps];
  __shared__ uint32_t s_least[kLogWarps];
  __shared__ float2 s_sums[kLogWarps];
  __shared__ int s_group[kTop];  // groups to read again: thread, best vector
  __shared__ int s_group_best[kTop], s_group_end[kTop];
  __shared__ int s_groups;
  __shared__ uint64_t s_bound;
  __shared__ int s_count, s_last;
  __shared__ uint32_t s_top;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int pieces = p.pieces;
  if (tid == 0) {
    for (int s = 0; s < kLogStages; ++s) {
      mbar_init(smem_addr(&full[s]), 1);
      mbar_init(smem_addr(&empty[s]), kLogWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&piece_full[i]), 1);
      mbar_init(smem_addr(&piece_empty[i]), kLogWarps);
    }
  }
  fence_mbar_init();
  __syncthreads();
  // The launch overlaps the end of the kernel before it, and the next one's
  // this one's end; logits, workspace and outputs are touched from here on.
  // The next kernel is let go only after the wait: what it reads before its
  // own wait may come from a kernel before this one.
  grid_dependency_wait();
  grid_launch_dependents();
  int chunk = 0;  // stages used so far

  if (warp == kLogWarps) {
    // ---- the copies: every piece's whole vectors, kStageVectors a stage ----
    if (lane != 0) return;
    bool failed = false;
    for (int n = 0; !failed; ++n) {
      int piece = blockIdx.x;
      if (n > 0) {
        if (n == 1 && __ldcg(p.error) != 0) break;  // (the computing warps leave after the first piece)
        const int v = atomicAdd(p.counter, 1);
        piece = static_cast<int>(gridDim.x) + v;
        if (v == pieces - 1) *p.counter = 0;  // every CTA has had its last answer: ready for the next call
      }
      if (piece >= pieces) piece = -1;
      if (n >= 2 && !mbar_wait_bounded(smem_addr(&piece_empty[n & 1]), ((n >> 1) - 1) & 1, p.polls)) {
        failed = true;
        break;
      }
      s_piece[n & 1] = piece;
      mbar_arrive(smem_addr(&piece_full[n & 1]));
      if (piece < 0) break;
      const Piece<T> r(p, piece);
      for (int c = r.v0; c < r.v1; c += kStageVectors, ++chunk) {
        const int st = chunk % kLogStages, use = chunk / kLogStages;
        if (use > 0 && !mbar_wait_bounded(smem_addr(&empty[st]), (use - 1) & 1, p.polls)) {
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
    if (failed) atomicOr(p.error, PKV_ERR_TIMEOUT);
    // let the copies still in flight land before shared memory goes away
    for (int k = max(0, chunk - kLogStages); k < chunk; ++k)
      mbar_wait_bounded(smem_addr(&full[k % kLogStages]), (k / kLogStages) & 1);
    return;
  }

  // The computing warps leave together, at a barrier after a piece's stream, so
  // what a warp finds on its own (that no piece or no copy came) only lets it run
  // through to there without waiting again.
  bool good;
  for (int n = 0;; ++n) {
    const bool lost =
        __any_sync(kFull, !mbar_wait_bounded(smem_addr(&piece_full[n & 1]), (n >> 1) & 1, p.polls));
    const int piece = lost ? static_cast<int>(blockIdx.x) : s_piece[n & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&piece_empty[n & 1]));
    if (piece < 0) {  // no more
      good = compute_all(true);
      break;
    }
    const Piece<T> r(p, piece);
    const int row = r.row, v0 = r.v0, v1 = r.v1;
    // ---- the stream ----
    // The reference is a logit, so that x - ref is exact where it matters (near
    // the largest logits) whatever the scale; it moves when a logit passes
    // limit = ref + kLogSlack / c2.
    float ref = -INFINITY, limit = kFloor;
    const float slack = kLogSlack / p.c2;
    float best = -INFINITY, next = -INFINITY;  // the largest logit, and of the vectors without it
    int best_v = v0 + tid;
    uint4 best_w = make_uint4(0u, 0u, 0u, 0u);
    // the error word and the target's logit, wanted at the end (by reading the word
    // there 1 row took 9.9 us instead of 9.6)
    const int error = tid == 0 ? __ldcg(p.error) : 0;
    const int target = p.targets && tid == 0 ? p.targets[row] : -1;
    const float target_x =
        target >= 0 && target < p.vocab ? V::value(V::raw(r.base + static_cast<size_t>(target) * sizeof(T))) : NAN;
    uint64_t s2 = f32x2(0.f, 0.f), z2 = s2, nr = s2;  // nr: -ref, 0 while there is none
    const uint64_t cc = f32x2(p.c2, p.c2);
    auto take = [&](const uint4& w, int v) {
      const float m = V::max(w);
      next = fmaxf(next, fminf(m, best));
      if (m > best) {
        best = m;
        best_v = v;
        best_w = w;
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
        nr = f32x2(-m, -m);
      }
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
    uint32_t polls = lost ? 0 : p.polls;  // 0: a copy did not come, stages are not given back
    for (int c = v0; c < v1; c += kStageVectors, ++chunk) {
      const int st = chunk % kLogStages;
      if (!mbar_wait_bounded(smem_addr(&full[st]), (chunk / kLogStages) & 1, polls)) polls = 0;
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
      if (lane == 0 && polls > 0) mbar_arrive(smem_addr(&empty[st]));
    }

    // ---- the sums and the K best of the CTA's piece ----
    // One exchange for both: the warps' largest references, and their
    // ceil(K / warps)-th best groups, the least of which bounds the K-th best
    // group of all from below.
    const uint32_t mine = v0 + tid < v1 ? ordered(best) : 0u;  // 0: no group
    {
      const float wref = unordered(__reduce_max_sync(kFull, ordered(ref)));
      uint32_t left = mine, nth = 0u;
      for (int k = 0; k < p.top; k += kLogWarps) {
        nth = __reduce_max_sync(kFull, left);
        const unsigned who = __ballot_sync(kFull, left == nth);
        if (lane == __ffs(who) - 1) left = 0u;
      }
      if (lane == 0) {
        s_ref[warp] = wref;
        s_least[warp] = nth;
      }
      if (tid == 0) {
        s_top = 0u;
        s_count = 0;
      }
    }
    good = compute_all(polls > 0 && error == 0);
    if (!good) break;
    Sums all;
    all.m = s_ref[0];
    uint32_t least = s_least[0];
#pragma unroll
    for (int w = 1; w < kLogWarps; ++w) {
      all.m = fmaxf(all.m, s_ref[w]);
      least = min(least, s_least[w]);
    }
    {
      const float2 s = unpack_f32x2(s2), z = unpack_f32x2(z2);
      all.s = s.x + s.y;
      all.z = z.x + z.y;
      if (all.m == -INFINITY || all.m > kHuge) {  // rare
        atomicMax(&s_top, mine);
        compute_sync();
        const float top = unordered(s_top);
        if (s_top != 0u && top != -INFINITY) {
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
        }
      } else if (ref != -INFINITY) {  // to the CTA's reference; a thread without one has 0 (or NaN)
        const float d = (ref - all.m) * p.c2, f = fast_exp2(d);
        all.z = f > 0.f ? f * (all.z + all.s * d) : f * all.s;
        all.s *= f;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        all.s += __shfl_xor_sync(kFull, all.s, o);
        all.z += __shfl_xor_sync(kFull, all.z, o);
      }
      if (lane == 0) s_sums[warp] = make_float2(all.s, all.z);
    }
    // the number of the n keys of s_cand above this one
    auto rank = [&](uint64_t key, int n) {
      int above = 0;
      for (int i = 0; i < n; i += 4) {  // (zeros fill up a last four)
        const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(s_cand + i);
        const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(s_cand + i + 2);
        above += (a.x > key) + (a.y > key) + (b.x > key) + (b.y > key);
      }
      return above;
    };
    if (p.top > 0) {
      // the groups not below the bound, each by its best logit and the vector
      // that holds it; of these the K best
      const uint64_t key = mine ? static_cast<uint64_t>(mine) << 32 | (0xffffffffu - static_cast<uint32_t>(best_v)) : 0;
      // (of a warp's groups of nothing but -inf only the first K can count: they
      // rank by thread)
      bool in = mine && mine >= least;
      const unsigned nothing = __ballot_sync(kFull, in && best == -INFINITY);
      if (best == -INFINITY && __popc(nothing & ((1u << lane) - 1)) >= p.top) in = false;
      const unsigned who = __ballot_sync(kFull, in);
      int at = 0;
      if (lane == 0) at = atomicAdd(&s_count, __popc(who));
      at = __shfl_sync(kFull, at, 0) + __popc(who & ((1u << lane) - 1));
      if (in) s_cand[at] = key;
      if (tid < p.top) s_best[tid] = 0;  // (a piece may hold fewer than K)
      if (tid == 0) s_bound = 1;
      compute_sync();
      const int groups = s_count;
      if (tid >= groups && tid < ((groups + 3) & ~3)) s_cand[tid] = 0;
      compute_sync();
      int place = p.top;  // of this thread's group among the K best
      if (in) {
        if (best == -INFINITY) best_w = r.load(best_v);  // (all -inf or NaN: its first vector)
        place = rank(key, groups);
        // no logit below the K-th group's best is needed (index: the last one
        // its vector can hold)
        if (place == p.top - 1)
          s_bound = key >> 32 << 32 | (0xffffffffu - static_cast<uint32_t>(best_v * kE - r.off + kE - 1));
      }
      for (;;) {
        if (tid == 0) s_count = s_groups = 0;
        compute_sync();
        const uint64_t bound = s_bound;
        const float low = bound > 1 ? unordered(static_cast<uint32_t>(bound >> 32)) : -INFINITY;
        const int last_v = bound > 1 ? (index_of(bound) + r.off) / kE : INT_MAX;  // logits equal to low count up to here
        // the logit at place e of vector v, if it is one and not below the bound
        auto look = [&](float x, int v, int e) {
          const int index = v * kE - r.off + e;
          const uint64_t k = index >= 0 && index < p.vocab ? key_of(x, index) : 0;
          if (k < bound) return;
          const int slot = atomicAdd(&s_count, 1);
          if (slot < kCandidates) s_cand[slot] = k;
        };
        if (place < p.top) {
#pragma unroll
          for (int e = 0; e < kE; ++e)
            if (!(V::get(best_w, e) < low)) look(V::get(best_w, e), best_v, e);
          if (!(next < low)) {  // the group may hold more
            const int slot = atomicAdd(&s_groups, 1);
            s_group[slot] = tid;
            s_group_best[slot] = best_v;
            s_group_end[slot] = next > low || last_v >= v1 ? v1 : last_v + 1;  // nothing past it counts
          }
        }
        compute_sync();
        for (int g = warp; g < s_groups; g += kLogWarps) {
          constexpr int kAhead = 2;  // vectors a lane loads at once
          for (int u0 = v0; u0 < s_group_end[g]; u0 += kAhead * 32 * kLogThreads) {
            uint4 w[kAhead];
            bool maybe[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
              const int u = u0 + s_group[g] + (lane + 32 * i) * kLogThreads;
              maybe[i] = u < s_group_end[g] && u != s_group_best[g];
              w[i] = make_uint4(0u, 0u, 0u, 0u);
              if (maybe[i]) w[i] = r.load(u);
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
              // a vector with a logit not below the bound is taken apart, a logit a
              // lane (one of NaN has no largest: taken apart as well)
              const int u = u0 + s_group[g] + (lane + 32 * i) * kLogThreads;
              const float m = V::max(w[i]);
              for (unsigned hit = __ballot_sync(kFull, maybe[i] && (u <= last_v ? !(m < low) : m > low)); hit;
                   hit &= hit - 1) {
                const int src = __ffs(hit) - 1;
                const uint4 x = make_uint4(__shfl_sync(kFull, w[i].x, src), __shfl_sync(kFull, w[i].y, src),
                                           __shfl_sync(kFull, w[i].z, src), __shfl_sync(kFull, w[i].w, src));
                if (lane < kE) look(V::get(x, lane % kE), u0 + s_group[g] + (src + 32 * i) * kLogThreads, lane);
              }
            }
          }
        }
        compute_sync();
        const int n = s_count, kept = min(n, kCandidates);
        if (tid >= kept && tid < ((kept + 3) & ~3)) s_cand[tid] = 0;
        compute_sync();
        if (tid < kept) {
          const uint64_t k = s_cand[tid];
          const int above = rank(k, kept);
          if (above < p.top) s_best[above] = k;
          if (above == p.top - 1) s_bound = k;
        }
        compute_sync();
        if (n <= kCandidates) break;
        // More than fit: the K-th of those kept is a higher bound (all keys
        // differ, and more than K were kept), so look again.
      }
    } else {
      compute_sync();
    }
    uint64_t key = lane < p.top ? s_best[lane] : 0;  // (only warp 0's is used)

    // ---- the row's result: from this piece, or from all of them ----
    if (warp == 0) {
      all.s = all.z = 0.f;
#pragma unroll
      for (int w = 0; w < kLogWarps; ++w) {
        all.s += s_sums[w].x;
        all.z += s_sums[w].y;
      }
    }
    bool writes = true;  // this CTA writes the row's result
    if (r.split_row >= 0) {
      const int slot = piece - p.whole;
      if (warp == 0) {
        if (lane < p.top) p.keys[static_cast<size_t>(slot) * kTop + lane] = key;
        if (lane == 0) p.sums[slot] = make_float4(all.m, all.s, all.z, 0.f);
        __threadfence();
        __syncwarp();
        if (lane == 0) s_last = atomicAdd(&p.tickets[r.split_row], 1) == p.splits - 1;
      }
      compute_sync();
      writes = s_last;
      if (writes) {
        __threadfence();
        const size_t first = static_cast<size_t>(r.split_row) * p.splits;
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
          if (lane == 0) p.tickets[r.split_row] = 0;
        }
      }
    }
    if (writes && warp == 0) {
      const float m = __shfl_sync(kFull, all.m, 0), s = __shfl_sync(kFull, all.s, 0), z = __shfl_sync(kFull, all.z, 0);
      // without a finite logit there is no distribution
      const float log_s = m == -INFINITY ? NAN : logf(s);
      constexpr float kLn2f = 0.6931471805599453f;
      auto logp = [&](float x) { return (x - m) * p.scale - log_s; };
      if (lane == 0) {
        if (p.targets) p.logprobs[row] = logp(target_x);
        if (p.entropy) p.entropy[row] = log_s - z / s * kLn2f;
      }
      if (lane < p.top) {
        p.top_ids[static_cast<size_t>(row) * p.top + lane] = index_of(key);
        p.top_logprobs[static_cast<size_t>(row) * p.top + lane] = logp(unordered(static_cast<uint32_t>(key >> 32)));
      }
    }
    compute_sync();  // the shared arrays are free for the next piece
  }
  if (!good) {
    if (tid == 0) atomicOr(p.error, PKV_ERR_TIMEOUT);
    for (long long i = tid; i < p.rows; i += kLogThreads) {
      if (p.targets) p.logprobs[i] = NAN;
      if (p.entropy) p.entropy[i] = NAN;
    }
    for (long long i = tid; i < static_cast<long long>(p.rows) * p.top; i += kLogThreads) {
      p.top_ids[i] = 0;  // a token's id all the same, so that what looks it up stays in range
      p.top_logprobs[i] = NAN;
    }
  }
}

// The workspace: error word, counter and tickets, then the split pieces' sums
// and keys. Its places depend on the GPU alone (fewer rows are split than CTAs
// run at once, into no more pieces than that), not on a call's sizes, so a call
// finds its counter and tickets where every other call left them at zero.
struct Workspace {
  size_t sums, keys, bytes;  // offsets; error word, counter and tickets from 0 on
  explicit Workspace(int ctas) {
    auto align256 = [](size_t n) { return (n + 255) / 256 * 256; };
    sums = align256(sizeof(int) * (static_cast<size_t>(ctas) + 2));
    keys = sums + align256(sizeof(float4) * ctas);
    bytes = keys + sizeof(uint64_t) * kTop * ctas;
  }
};

// How the rows are cut for `ctas` CTAs: whole rounds of a row a CTA first; the
// rows left over (or all, when they are fewer) are split over as many CTAs as
// run at once, rounded down (a few pieces of a further round would double the
// time), no piece smaller than kMinSplitVectors. `vectors` as for a row that
// starts anywhere.
struct Cut {
  int whole, splits;
};
Cut cut(int rows, long long vectors, int ctas) {
  const int rest = rows % ctas;
  if (rest == 0) return {rows, 1};
  long long n = vectors / kMinSplitVectors;
  if (n > ctas / rest) n = ctas / rest;
  if (n > kMaxSplits) n = kMaxSplits;
  return n < 2 ? Cut{rows, 1} : Cut{rows - rest, static_cast<int>(n)};
}

// A poll that finds nothing takes 4 us, so about a second.
std::atomic<uint32_t> g_wait_polls{1u << 18};

}  // namespace
}  // namespace pkv

extern "C" {

int token_logprobs_set_wait_limit(uint32_t polls, uint32_t* previous) {
  const uint32_t before = pkv::g_wait_polls.exchange(polls);
  if (previous) *previous = before;
  return 0;
}

int token_logprobs_get_error(void* workspace, int* bits, int reset) {
  using namespace pkv;
  if (!workspace || !bits || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return -EINVAL;
  int device = 0, v = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(&v, workspace, sizeof(int), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && reset) {
    const int sms = device_sm_count(device);
    if (sms < 1) return -EIO;
    e = cudaMemset(workspace, 0, Workspace(kLogCtas * sms).sums);
  }
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return -EIO;
  }
  *bits = v;
  return 0;
}

size_t token_logprobs_workspace_bytes(int rows, int vocab, int top) {
  using namespace pkv;
  if (rows < 1 || vocab < 1 || top < 0 || top > PKV_MAX_TOP || top > vocab) return 0;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return 0;
  const int sms = device_sm_count(device);
  return sms < 1 ? 0 : Workspace(kLogCtas * sms).bytes;
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
  const int ctas = kLogCtas * device_sm_count(device);
  const Cut c = cut(rows, vectors, ctas);
  p.whole = c.whole;
  p.splits = c.splits;
  p.split_vectors = static_cast<int>((vectors + c.splits - 1) / c.splits);
  const long long pieces = c.whole + static_cast<long long>(rows - c.whole) * c.splits;
  if (pieces > 0x7fff0000ll) return -EINVAL;
  p.pieces = static_cast<int>(pieces);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.error = reinterpret_cast<int*>(ws);
  p.polls = g_wait_polls.load(std::memory_order_relaxed);
  p.counter = p.error + 1;
  p.tickets = p.counter + 1;
  const Workspace at(ctas);
  p.sums = reinterpret_cast<float4*>(ws + at.sums);
  p.keys = reinterpret_cast<uint64_t*>(ws + at.keys);
  auto kernel = logits_type == PKV_BF16 ? logprobs_kernel<uint16_t> : logprobs_kernel<float>;
  constexpr int kSmem = kLogStages * kStageVectors * 16;
  static DeviceSetup setup[2];
  e = setup[logits_type]([&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem); });
  if (e == cudaSuccess) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(pieces < ctas ? pieces : ctas));
    cfg.blockDim = dim3(kLogBlock);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, p);
  }
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return -EIO;
  }
  return 0;
}

}  // extern "C"
