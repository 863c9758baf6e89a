// decode_shared.cu -- decode attention of sequences that share their first pages:
// these are read once for a group of sequences, not once for each.
//
// The formula is the scored decode's: with i = n_b - 1 the position of sequence
// b's token and j a key's,
//     t = scale q.k,  s = cap tanh(t / cap) - slope |i - j|,
//     out = softmax(s) V over the keys that the window leaves.
// Sums over keys join by their maxima: over any pieces x of the keys, each with a
// reference m_x, l_x = sum e^(s - m_x) and O_x = sum e^(s - m_x) v,
//     out = sum_x e^(m_x - M) O_x / sum_x e^(m_x - M) l_x,  M = max m_x.
//
// The kernel here takes the shared pages. A tile is up to 128 rows (the query heads
// of one kv head, of up to 128 / G members of a group) against the group's shared
// keys, 64 a step:
//   S = Q_hi K^T + Q_lo K^T      (tensor memory, 128 x 64 fp32, two buffers)
//   P = exp2(S - m)              (softmax warps: 16 rows each; a warp without rows
//                                 does nothing, so a step of few rows is short)
//   O += P V (+ P_lo V),  l += P 1
// Q enters as bf16 with its bf16 remainder, as everywhere in this library, P too
// where the output is fp32 (kPair); with a bf16 output P is rounded once and its
// row sums come from a product with ones, of the rounded P. That makes an error of 1.2e-3
// to 1.5e-3 of the output's norm beside the 1.66e-3 of rounding the output, and saves 13%
// (256 sequences behind three documents 144 us against 166).
//
// All steps of all tiles form one line (kv head by kv head, tile by tile), which is
// cut evenly over the CTAs, two an SM: every CTA works the line's prefix sums out
// itself from the lengths, and walks its share. A tile that is cut leaves pieces;
// every piece puts its rows' m, l and O into the workspace. A piece's place needs no
// counting: tile and CTA only ever go up along the line, so (first row of the tile)
// + 128 * CTA is free. The sequences' own pages are the second kernel's, which joins
// the pieces too (decode_rest.cu). Under a window a tile's rows see different keys, and a
// value that is not finite makes NaN of the rows whose weight for it is 0: the second
// kernel works rows that are not finite out from their own keys alone.
//
// Warps 0-7 run the softmax and the epilogue; of 8-11, which hand registers to
// them, 8 copies keys (and finds the tiles), 11 values, 9 issues the score
// products, 10 the P V products. Every wait is bounded.
//
// Measured in graph replays with the second kernel, bf16 out (fp32): 256 rows behind
// one prompt of 32768 tokens, 8 kv heads, 123 us (146), 151 (185) with a cap; with every
// sequence reading all of it, 1630 us for 256 behind three documents that take 144
// here. A step takes an SM 850 cycles (1000), of 128 rows or 16: what bounds it is
// neither the tensor core alone (600 cycles of products of N = 64, which take their A
// operand at half the rate that N = 128 would) nor the issue of the softmax (some 250
// instructions a warp), but the chain of one after the other in each of the SM's two
// CTAs: scores, their load from tensor memory, weights, their store, P V, and back to
// the buffer of two steps before. Fewer products at the price of more instructions (the
// row sums in registers: 930 cycles) lost, fewer instructions won: a kernel for each
// form of the scores (1020 to 910), an arrival a warp on the barriers instead of one a
// thread (910 to 850, with the row sums as 16 columns more of the P V product instead of
// products of their own). Around the steps lie 5 us until the first scores (the line,
// the tile, page ids, keys, one latency after the other) and a few for every further
// piece.
#include <climits>

#include "f32x2.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "score_cap.cuh"
#include "shared_line.cuh"
#include "tc05.cuh"

namespace pkv {
namespace {

constexpr float kSlack = 8.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kSBufs = 2;
constexpr uint32_t kTmemCols = 256;  // two S buffers of 64 columns, O (64), l (16 equal columns)
constexpr int kCtas = 2;             // CTAs a SM
constexpr int kMaxBatch = PKV_SHARED_MAX_BATCH;
// tanh(x) on |x| <= kPolyMax where the output is bf16: x (c0 + c1 x^2 + c2 x^4)
// with the smallest largest error (1.7e-7), as in prefill_scored.cu; where it is
// fp32 (kPair) the polynomial of score_cap.cuh. Elsewhere cap tanh(x) = cap - 2 cap
// / (2^t + 1) with t = 2 log2(e) x.
constexpr double kPolyMax = 0.3;
constexpr double kPoly[3] = {0.999996010, -0.332974797, 0.125225911};

struct SharedParams {
  const float* q_rot;  // [B][hq][64]
  const int32_t* block_tables;
  int max_blocks;
  const int32_t* seq_lens;
  int batch;
  const int32_t* cu_groups;    // [groups + 1]
  const int32_t* shared_lens;  // [groups]
  int groups;
  int hkv, hq, group;
  long long num_pages;
  float qscale;        // what a query is multiplied by: scores in base 2, or t when capped
  float cap;           // softcap * log2(e), 0: none
  float poly[4];       // cap tanh as a polynomial of t
  const float* slopes;  // [hq] or null
  int window;           // 0: none
  SharedPieces to;      // the workspace
  int* err;
};

// A piece of a tile as the key warp publishes it. Positions count from key0;
// n_steps = 0: no more.
struct Piece {
  int b, members, h;          // its first member, whose table it is, and how many
  int key0, lo, last;         // first key any row sees, last key of the piece
  int n_pages, n_steps;
  long long at;               // its first row in the workspace
};

struct Cfg {
  static constexpr int kStages = 4;
  static constexpr int kSoftmaxThreads = 256;
  static constexpr int kThreads = kSoftmaxThreads + 128;
  // registers a thread after the split (setmaxnreg): the launch gives 80 to
  // each of the 384 threads; 128 x 56 + 256 x 88 <= 384 x 80
  static constexpr int kIssueRegs = 56;
  static constexpr int kSoftmaxRegs = 88;
  static_assert(128 * kIssueRegs + kSoftmaxThreads * kSoftmaxRegs <= kThreads * 80,
                "the register shares exceed what two CTAs an SM give a CTA");
  static constexpr uint32_t kTile = 128 * 128;  // a 128-row x 128-byte operand tile
  static constexpr uint32_t kStep = 64 * 128;   // 64 K rows (or V rows) of one step
  // dynamic shared memory: Q_hi, Q_lo, per stage K and V, then 16 rows of ones,
  // then the line (line, blocks, lengths); the stages serve its making
  static constexpr uint32_t kQhi = 0, kQlo = kTile;
  static constexpr uint32_t kStage0 = 2 * kTile;
  static constexpr uint32_t kOnes = kStage0 + kStages * 2 * kStep;
  static constexpr uint32_t kLine = kOnes + 16 * 128;
  static constexpr uint32_t bytes(int batch) { return kLine + (3 * batch + 1) * sizeof(int); }
};

// A sequence's length, 0 where it cannot be served.
__device__ __forceinline__ int served_length(int n, int max_blocks) {
  return n >= 1 && n <= static_cast<long long>(max_blocks) * kPage ? n : 0;
}
__device__ __forceinline__ int first_key(int n, int window) { return window > 0 ? max(n - window, 0) : 0; }

// Inclusive prefix sum over a CTA of kThreads threads (s_warp: a word a warp).
template <int kThreads>
__device__ __forceinline__ int cta_scan(int x, int* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += t;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w)
    if (w < warp) x += s_warp[w];
  __syncthreads();
  return x;
}

// kCap, kSlopes: whether scores are capped and biased (apart, so that the steps that
// need neither have no branches around the registers that hold a row's scores: those
// cost a copy of all of them each).
template <bool kPair, bool kCap, bool kSlopes>
__global__ void __launch_bounds__(Cfg::kThreads, kCtas)
    decode_shared_kernel(const __grid_constant__ CUtensorMap kv16_map, const SharedParams p) {
  using C = Cfg;
  const int G = p.group, most_members = 128 / G;
  extern __shared__ __align__(1024) uint8_t dsmem[];
  __shared__ __align__(8) uint64_t k_full[C::kStages], k_empty[C::kStages];
  __shared__ __align__(8) uint64_t v_full[C::kStages], v_empty[C::kStages];
  __shared__ __align__(8) uint64_t s_full[kSBufs], p_full[kSBufs], pv_done[kSBufs], q_ready, drain[2];
  __shared__ __align__(8) uint64_t piece_full[2], piece_empty[2];
  __shared__ Piece s_piece[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_warp[C::kThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_addr(dsmem) + 1023u) & ~1023u;
  uint8_t* gbase = dsmem + (base - smem_addr(dsmem));
  int* s_line = reinterpret_cast<int*>(gbase + C::kLine);
  int* s_blocks = s_line + p.batch + 1;
  int* s_len = s_blocks + p.batch;
  auto kst = [&](int st) { return base + C::kStage0 + st * 2 * C::kStep; };
  auto vst = [&](int st) { return base + C::kStage0 + st * 2 * C::kStep + C::kStep; };

  if (warp == 0) {
    tmem_alloc(smem_addr(&s_tmem), kTmemCols);
    tmem_relinquish();
  }
  if (tid == 32) {
    for (int st = 0; st < C::kStages; ++st) {
      mbar_init(smem_addr(&k_full[st]), 1);
      mbar_init(smem_addr(&k_empty[st]), 1);
      mbar_init(smem_addr(&v_full[st]), 1);
      mbar_init(smem_addr(&v_empty[st]), 1);
    }
    mbar_init(smem_addr(&q_ready), C::kSoftmaxThreads / 32);
    // S done, P ready and P V done, one barrier each per buffer (step % kSBufs):
    // a wait for a step never sees its barrier two phases on
    for (int i = 0; i < kSBufs; ++i) {
      mbar_init(smem_addr(&s_full[i]), 1);
      mbar_init(smem_addr(&p_full[i]), C::kSoftmaxThreads / 32);
      mbar_init(smem_addr(&pv_done[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&drain[i]), 1);
      mbar_init(smem_addr(&piece_full[i]), 1);
      mbar_init(smem_addr(&piece_empty[i]), 11);  // every warp but the key warp
    }
  }
  for (int i = tid; i < 16 * 128 / 4; i += C::kThreads)
    reinterpret_cast<uint32_t*>(gbase + C::kOnes)[i] = 0x3F803F80u;  // (the same in any swizzle)
  fence_proxy_async_smem();
  fence_mbar_init();
  // The second kernel is let go only after the wait: what it reads before its own
  // may come from a kernel before this one.
  grid_dependency_wait();
  grid_launch_dependents();

  // ---- the line, the same in every CTA (see Cfg: in the stages, until the first copies) ----
  {
    int* s_cu = reinterpret_cast<int*>(gbase + C::kStage0);  // [groups + 1]
    int* s_shared = s_cu + kMaxBatch + 1;                    // [groups]
    int* s_least = s_shared + kMaxBatch;                     // [groups] least length of the members
    int* s_group = s_least + kMaxBatch;                      // [B] a sequence's group, -1: none
    int* s_tile = s_group + kMaxBatch;                       // [B] least length of the tile that begins here
    static_assert((5 * kMaxBatch + 1) * sizeof(int) <= C::kStages * 2 * C::kStep, "the stages hold what makes the line");
    for (int i = tid; i <= p.batch; i += C::kThreads) {
      if (i < p.batch) {
        s_len[i] = p.seq_lens[i];
        s_tile[i] = INT_MAX;
      }
      if (i <= p.groups) s_cu[i] = p.cu_groups[i];
      if (i < p.groups) {
        s_shared[i] = p.shared_lens[i];
        s_least[i] = INT_MAX;
      }
    }
    __syncthreads();
    // A sequence that no group holds shares nothing; nor does any when the groups
    // do not follow one another.
    bool bad = false;
    for (int g = tid; g < p.groups; g += C::kThreads) bad |= s_cu[g] < 0 || s_cu[g + 1] < s_cu[g] || s_cu[g + 1] > p.batch;
    const bool grouped = !__syncthreads_or(bad) && p.groups > 0;
    for (int b = tid; b < p.batch; b += C::kThreads) {
      const int n = served_length(s_len[b], p.max_blocks);
      s_len[b] = n;
      int g = -1;
      if (grouped && b >= s_cu[0] && b < s_cu[p.groups]) {
        g = 0;  // the last group that begins at or before b
        for (int hi = p.groups - 1; g < hi;) {
          const int mid = (g + hi + 1) >> 1;
          if (s_cu[mid] <= b) g = mid; else hi = mid - 1;
        }
        if (n > 0) atomicMin(&s_least[g], n);
      }
      s_group[b] = g;
    }
    // (the second kernel reports bad lengths)
    if (__syncthreads_or(bad && !grouped && p.groups > 0) && blockIdx.x == 0 && tid == 0) atomicOr(p.err, PKV_ERR_SEQ_LEN);
    for (int b = tid; b < p.batch; b += C::kThreads) {
      const int g = s_group[b];
      int word = 0;
      if (g >= 0 && s_cu[g + 1] - s_cu[g] > 1) {
        const int shared = max(min(s_shared[g], s_least[g]), 0) / kPage;
        const int place = (b - s_cu[g]) % most_members;
        if (shared > 0 && s_least[g] != INT_MAX) {
          word = shared | place << kPlaceShift;
          if (s_len[b] > 0) atomicMin(&s_tile[b - place], s_len[b]);
        }
      }
      s_blocks[b] = word;
    }
    __syncthreads();
    int before = 0;
    for (int at = 0; at < p.batch; at += C::kThreads) {
      const int b = at + tid;
      int cost = 0;
      if (b < p.batch) {
        const int shared = shared_of(s_blocks[b]);
        if (shared > 0 && place_of(s_blocks[b]) == 0 && s_tile[b] != INT_MAX) {
          // the tile's pages from the first that a member sees, in whole steps from page 0
          const int from = first_key(s_tile[b], p.window) / kPage;
          if (from < shared) cost = kUnitCost + (shared + kStepPages - 1) / kStepPages - from / kStepPages;
        }
      }
      const int upto = before + cta_scan<C::kThreads>(cost, s_warp);
      if (b < p.batch) s_line[b + 1] = upto;
      if (tid == C::kThreads - 1) s_warp[0] = upto;
      __syncthreads();
      before = s_warp[0];
      __syncthreads();
    }
    if (tid == 0) s_line[0] = 0;
    fence_proxy_async_smem();  // before the copies into the stages
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (blockIdx.x == 0) {  // for the second kernel
    for (int b = tid; b <= p.batch; b += C::kThreads) {
      int4 tile = make_int4(s_line[b], 0, 0, 0);
      if (b < p.batch) {
        const int place = place_of(s_blocks[b]), start = s_line[b - place];
        tile = make_int4(start, s_line[b - place + 1] - start, shared_of(s_blocks[b]), place);
      }
      p.to.tiles[b] = tile;
    }
  }

  const uint32_t tmem = s_tmem, tO = tmem + 64 * kSBufs, tL = tO + 64;
  // steps are numbered through, piece after piece
  auto tS = [&](int g) { return tmem + 64 * (g % kSBufs); };  // S, then P (hi: +0, lo: +32)
  auto buf = [](int g) { return g % kSBufs; };
  auto par = [](int g) { return static_cast<uint32_t>((g / kSBufs) & 1); };
  // Step j of a piece takes the 64 keys of block key_block(j). With a distance
  // bias the last block comes first (the largest scores are there, and the
  // reference found in the first step stands), without one the first. Page ids
  // come in windows of 32, eight steps: lane i of window m holds page
  // window_page(m) + i, and step j's four pages are lanes window_lane(j) .. + 3.
  constexpr bool down = kSlopes;
  auto key_block = [&](int j, int n_steps) { return down ? n_steps - 1 - j : j; };
  auto window_page = [&](int m, int n_steps) { return down ? 4 * n_steps - 32 * (m + 1) : 32 * m; };
  auto window_lane = [&](int j) { return down ? 28 - ((4 * j) & 31) : (4 * j) & 31; };
  // (pages before the first visible key are no part of the piece)
  auto is_page = [](const Piece& t, int pg) { return pg >= t.lo / kPage && pg < t.n_pages; };
  auto page_id = [&](const Piece& t, int pg) {
    return is_page(t, pg) ? p.block_tables[static_cast<size_t>(t.b) * p.max_blocks + t.key0 / kPage + pg] : -1;
  };
  // Piece n's entry, for every warp but the key warp; release() when it is read.
  auto piece_wait = [&](int n) { return mbar_wait_bounded(smem_addr(&piece_full[n & 1]), (n >> 1) & 1); };
  auto release = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&piece_empty[n & 1]));
  };
  bool failed = false;

  if (warp >= 8) {
    // the copy and product warps (one warpgroup) give registers to the softmax
    // warpgroups, first thing and unconditionally, so the softmax warps'
    // increase (the shares add up to the launch's total) never waits for more
    regs_dec<C::kIssueRegs>();
    if (warp == 8 || warp == 11) {
      // ---- TMA producers: a step's four pages' K rows (warp 8) or V rows (warp
      // 11) into its stage. A warp reads the page ids 32 at a time, the next 32
      // while it issues the current ones. ----
      const int kind = warp == 8 ? 0 : 1;
      uint64_t* full = kind ? v_full : k_full;
      uint64_t* empty = kind ? v_empty : k_empty;
      int g = 0;  // steps issued
      // The key warp's own: the next piece of this CTA's share, published as entry n.
      const int all = s_line[p.batch];
      const long long total = static_cast<long long>(all) * p.hkv;
      const long long share = share_of(total, p.to.ctas);
      long long x = share * blockIdx.x;
      const long long end = min(x + share, total);
      auto fetch = [&](int n) {
        Piece t = {};
        while (x < end) {
          t.h = static_cast<int>(x / all);
          const int off = static_cast<int>(x - static_cast<long long>(t.h) * all);
          int b = 0;  // the last sequence that begins at or before off
          for (int hi = p.batch - 1; b < hi;) {
            const int mid = (b + hi + 1) >> 1;
            if (s_line[mid] <= off) b = mid; else hi = mid - 1;
          }
          const int start = s_line[b], cost = s_line[b + 1] - start, shared = shared_of(s_blocks[b]);
          const int upto = static_cast<int>(min(static_cast<long long>(start + cost), end - static_cast<long long>(t.h) * all));
          const int s0 = steps_before(off - start), s1 = steps_before(upto - start);
          x = static_cast<long long>(t.h) * all + upto;
          if (s1 <= s0) continue;
          t.b = b;
          for (int i0 = b + 1;; i0 += 32) {  // its members follow its first one
            const int i = i0 + lane;
            const unsigned other = __ballot_sync(kFull, i >= p.batch || place_of(s_blocks[i]) == 0);
            if (other) {
              t.members = i0 + __ffs(other) - 1 - b;
              break;
            }
          }
          const int page0 = ((shared + kStepPages - 1) / kStepPages - steps_before(cost) + s0) * kStepPages;
          const int page_end = min(shared, page0 + (s1 - s0) * kStepPages);
          t.key0 = page0 * kPage;
          t.n_pages = page_end - page0;
          t.n_steps = s1 - s0;
          t.at = (static_cast<long long>(t.h) * p.batch + b) * G + 128ll * blockIdx.x;
          t.last = t.n_pages * kPage - 1;
          int lo = t.last;
          for (int i = lane; i < t.members; i += 32) {
            if (s_len[b + i] > 0) lo = min(lo, first_key(s_len[b + i], p.window) - t.key0);
            // its query rows, to L2
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                             p.q_rot + (static_cast<size_t>(b + i) * p.hq + t.h * G) * kHeadDim),
                         "r"(G * kHeadDim * 4)
                         : "memory");
          }
          t.lo = max(__reduce_min_sync(kFull, lo), 0);
          break;
        }
        if (n >= 2 && !mbar_wait_idle(smem_addr(&piece_empty[n & 1]), ((n >> 1) - 1) & 1)) failed = true;
        if (__any_sync(kFull, failed)) failed = true;
        if (lane == 0 && !failed) {
          s_piece[n & 1] = t;
          mbar_arrive(smem_addr(&piece_full[n & 1]));
        }
        return t;
      };
      Piece t, next = {};
      if (kind == 0) next = fetch(0);
      for (int n = 0; !failed; ++n) {
        if (kind == 0) {
          t = next;
        } else {
          if (!piece_wait(n)) failed = true;
          if (__any_sync(kFull, failed)) {
            failed = true;
            break;
          }
          t = s_piece[n & 1];
          release(n);
        }
        if (t.n_steps == 0) break;
        // lane i: the copy's row coordinate for page window_page(m) + i (-1: no
        // page of the piece, or a bad id), and the window's valid pages as a mask
        uint32_t valid = 0;
        auto window = [&](int pid, int m) {
          const bool in = is_page(t, window_page(m, t.n_steps) + lane);
          const bool ok = in && pid >= 0 && static_cast<long long>(pid) < p.num_pages;
          if (kind == 0 && __any_sync(kFull, in && !ok) && lane == 0) atomicOr(p.err, PKV_ERR_PAGE_ID);
          valid = __ballot_sync(kFull, ok);
          return ok ? (pid * p.hkv + t.h) * (2 * kPage) + kind * kPage : -1;
        };
        int row = window(page_id(t, window_page(0, t.n_steps) + lane), 0);
        int pid_next = page_id(t, window_page(1, t.n_steps) + lane);
        for (int j = 0; j < t.n_steps; ++j, ++g) {
          const int st = g % C::kStages, use = g / C::kStages;
          if (j > 0 && (j & 7) == 0) {  // the next 32 pages
            row = window(pid_next, j >> 3);
            pid_next = page_id(t, window_page((j >> 3) + 1, t.n_steps) + lane);
          }
          const int l0 = window_lane(j);
          const uint32_t vbits = (valid >> l0) & 0xFu;
          int rows[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) rows[q] = __shfl_sync(kFull, row, l0 + q);
          // the stage is free once its scores (K) or its P V product (V) are done
          if (use > 0 && !mbar_wait_idle(smem_addr(&empty[st]), (use - 1) & 1)) failed = true;
          if (__any_sync(kFull, failed)) {
            failed = true;
            break;
          }
          const uint32_t dst = (kind ? vst(st) : kst(st)), bar = smem_addr(&full[st]);
          mbar_arrive_expect_tx_elect(bar, static_cast<uint32_t>(__popc(vbits)) * kHalfBytes);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if ((vbits >> q) & 1u) tma_load_2d_elect(dst + q * kHalfBytes, &kv16_map, 0, rows[q], bar);
          // the next piece, once this one's first stages are on their way
          if (kind == 0 && j == min(t.n_steps, C::kStages) - 1) next = fetch(n + 1);
        }
      }
      // let the copies still in flight (the last kStages steps at most) land
      // before shared memory goes away
      if (failed && lane == 0)
        for (int k = max(0, g - C::kStages); k < g; ++k)
          mbar_wait_bounded(smem_addr(&full[k % C::kStages]), (k / C::kStages) & 1);
    } else {
      // ---- MMA issuers, each a whole warp, converged: warp 9 the score
      // products, warp 10 the P V products. A commit covers only its own warp's
      // products. ----
      auto wait_all = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(kFull, mbar_wait_bounded(bar, parity)) != 0;
      };
      constexpr uint32_t idS = idesc_bf16_f32(128, 64, false), idPV = idesc_bf16_f32(128, kPair ? 64 : 80, true);
      const uint64_t dQhi = smem_desc_sw128(base + C::kQhi), dQlo = smem_desc_sw128(base + C::kQlo);
      int g = 0;
      for (int n = 0; !failed; ++n) {
        if (!wait_all(smem_addr(&piece_full[n & 1]), (n >> 1) & 1)) {
          failed = true;
          break;
        }
        const int n_steps = s_piece[n & 1].n_steps;
        release(n);
        if (n_steps == 0) break;
        if (warp == 9) {
          if (!wait_all(smem_addr(&q_ready), n & 1)) failed = true;
          for (int j = 0; j < n_steps && !failed; ++j, ++g) {
            const int st = g % C::kStages;
            // S goes into the buffer of the P kSBufs steps before: once its P V is done
            if (g >= kSBufs && !wait_all(smem_addr(&pv_done[buf(g)]), par(g - kSBufs))) failed = true;
            if (failed || !wait_all(smem_addr(&k_full[st]), (g / C::kStages) & 1)) {
              failed = true;
              break;
            }
            tc_fence_after();
            const uint64_t dK = smem_desc_sw128(kst(st));
            // K-major tiles: a 16-element K step is 32 bytes along the swizzled
            // row (+2 in the descriptor's 16-byte address units)
#pragma unroll
            for (int k = 0; k < 4; ++k) umma_bf16(tS(g), dQhi + 2 * k, dK + 2 * k, idS, k > 0);
#pragma unroll
            for (int k = 0; k < 4; ++k) umma_bf16(tS(g), dQlo + 2 * k, dK + 2 * k, idS, true);
            umma_commit(smem_addr(&k_empty[st]));
            umma_commit(smem_addr(&s_full[buf(g)]));
          }
        } else {
          for (int j = 0; j < n_steps && !failed; ++j, ++g) {
            const int st = g % C::kStages;
            if (!wait_all(smem_addr(&p_full[buf(g)]), par(g)) ||
                !wait_all(smem_addr(&v_full[st]), (g / C::kStages) & 1)) {
              failed = true;
              break;
            }
            tc_fence_after();
            // P from tensor memory (a 16-key K step is 8 columns); V is MN-major:
            // a 16-key K step is 16 rows = 2048 bytes (+128). Without kPair the
            // product has 16 columns more, of ones, for the row sums: the 64 columns
            // after V's 64 are the leading byte offset away, which is made the
            // distance to the tile of ones.
            uint64_t dV = smem_desc_sw128(vst(st));
            if constexpr (!kPair) {
              dV &= ~(static_cast<uint64_t>(0x3FFFu) << 16);
              dV |= static_cast<uint64_t>((base + C::kOnes - vst(st)) >> 4) << 16;
            }
            constexpr uint64_t kNext = kPair ? 128 : 128 - (static_cast<uint64_t>(128) << 16);
#pragma unroll
            for (int k = 0; k < 4; ++k) umma_bf16_tmem_a(tO, tS(g) + 8 * k, dV + kNext * k, idPV, j > 0 || k > 0);
            if constexpr (kPair) {
#pragma unroll
              for (int k = 0; k < 4; ++k) umma_bf16_tmem_a(tO, tS(g) + 32 + 8 * k, dV + 128 * k, idPV, true);
            }
            umma_commit(smem_addr(&v_empty[st]));
            umma_commit(smem_addr(&pv_done[buf(g)]));
          }
        }
      }
      if (failed) {  // let this warp's products already issued finish before the memory goes away
        umma_commit(smem_addr(&drain[warp - 9]));
        mbar_wait_bounded(smem_addr(&drain[warp - 9]), 0);
      }
    }
  } else {
    regs_inc<C::kSoftmaxRegs>();
    // ---- softmax and epilogue. Warp w has rows 16 w .. + 15 of a piece (row r:
    // member r / G, head r % G), in tensor-memory lanes L .. L + 15, L = 32 (w % 4)
    // + 16 (w / 4), so that few rows spread over the SM's four parts. Its thread t
    // holds rows t / 4 (hh = 0) and t / 4 + 8 (hh = 1) of them and, of each, the key
    // pairs 8 i + 2 q and 8 i + 2 q + 1 (i = 0..7, q = t % 4): the 16x256b layout,
    // in which S word 4 i + 2 hh + e is key 8 i + 2 q + e of row hh. ----
    const int q = lane & 3;
    const int lrow = 32 * (warp & 3) + 16 * (warp >> 2);
    const uint32_t lane_addr = static_cast<uint32_t>(lrow) << 16;
    auto row_of = [&](int hh) { return 16 * warp + (lane >> 2) + 8 * hh; };
    // this thread's share of a piece's query rows: dims 16 q .. 16 q + 15 of its two rows
    float4 qv[2][4];
    auto load_q = [&](const Piece& t) {
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const bool in = row_of(hh) < t.members * G;
        const float* qr = p.q_rot + (static_cast<size_t>(t.b + (in ? row_of(hh) / G : 0)) * p.hq + t.h * G +
                                     row_of(hh) % G) * kHeadDim + 16 * q;
#pragma unroll
        for (int d = 0; d < 4; ++d)
          qv[hh][d] = in ? *reinterpret_cast<const float4*>(qr + 4 * d) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    };
    // scaled, as bf16 high part and remainder, 128-byte swizzled (chunks 2 q and 2 q + 1 of the row)
    auto store_q = [&]() {
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int rw = lrow + (lane >> 2) + 8 * hh;
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 v = qv[hh][2 * cc + (e >> 1)];
            const float a0 = ((e & 1) ? v.z : v.x) * p.qscale, a1 = ((e & 1) ? v.w : v.y) * p.qscale;
            hi[e] = pack_bf16x2(a0, a1);
            const float2 f = bf16x2_to_float2(hi[e]);
            lo[e] = pack_bf16x2(a0 - f.x, a1 - f.y);
          }
          const uint32_t off = rw * 128 + (((2 * q + cc) ^ (rw & 7)) << 4);
          *reinterpret_cast<uint4*>(gbase + C::kQhi + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(gbase + C::kQlo + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
    };
    // the piece's rows' positions (from key0) and slopes (base 2), and its first
    // window of page ids
    int pos[2], pid = 0;
    // keys that all of the warp's rows see
    int clean_from = 0, clean_to = 0;
    [[maybe_unused]] float slope[2] = {0.f, 0.f};
    auto load_rows = [&](const Piece& t) {
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int len = s_len[t.b + min(row_of(hh) / G, t.members - 1)];
        pos[hh] = len - 1 - t.key0;
        if constexpr (kSlopes) slope[hh] = p.slopes[t.h * G + row_of(hh) % G] * kLog2e;
      }
      clean_from = p.window > 0 ? __reduce_max_sync(kFull, max(pos[0], pos[1])) - p.window + 1 : 0;
      clean_to = min(__reduce_min_sync(kFull, min(pos[0], pos[1])), t.last);
      pid = page_id(t, window_page(0, t.n_steps) + lane);
    };
    // (a warp arrives once: 256 threads' arrivals on one word follow one another)
    auto arrive = [&](uint64_t& bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&bar));
    };
    auto ready_q = [&]() {
      fence_proxy_async_smem();
      arrive(q_ready);
    };
    auto has_rows = [&](const Piece& t) { return 16 * warp < t.members * G; };  // this warp

    // A wait that gives up leaves 0 polls to those after it: what is left is run
    // through without waiting, to the piece's end.
    uint32_t polls = kWaitPolls;
    auto wait = [&](uint64_t& bar, uint32_t parity) {
      if (!mbar_wait_bounded(smem_addr(&bar), parity, polls)) polls = 0;
    };
    if (!piece_wait(0)) failed = true;
    int n = 0, g = 0;
    const bool some = !failed && s_piece[0].n_steps > 0;
    if (some) {
      if (has_rows(s_piece[0])) {
        load_q(s_piece[0]);
        load_rows(s_piece[0]);
        store_q();
      }
      ready_q();
    }
    for (; some && !failed; ++n) {
      const Piece& t = s_piece[n & 1];
      const int n_steps = t.n_steps;
      const bool active = has_rows(t);
      // the rows' references (0 until a row has seen a key: `set`), and with
      // kPair their sums
      float m_ref[2] = {0.f, 0.f};
      [[maybe_unused]] float l_sum[2] = {0.f, 0.f};
      bool set[2] = {false, false};
      // which pages have a bad id: bit i of bad_win for page window_page(m) + i,
      // the next window loaded while this one is used
      auto bad_bits = [&](int id, int m) {
        return __ballot_sync(kFull, is_page(t, window_page(m, n_steps) + lane) &&
                                        (id < 0 || static_cast<long long>(id) >= p.num_pages));
      };
      auto window_id = [&](int m) { return page_id(t, window_page(m, n_steps) + lane); };
      if (!active) pid = window_id(0);
      uint32_t bad_win = bad_bits(pid, 0);
      int next_id = n_steps > 8 ? window_id(1) : 0;
      for (int j = 0; j < n_steps; ++j, ++g) {
        const int st = g % C::kStages;
        const int k0 = 64 * key_block(j, n_steps);  // the step's first key position
        const int kb = k0 + 2 * q;                  // this thread's first
        if (j > 0 && (j & 7) == 0) {
          bad_win = bad_bits(next_id, j >> 3);
          next_id = j + 8 < n_steps ? window_id((j >> 3) + 1) : 0;
        }
        const int bad_pages = static_cast<int>((bad_win >> window_lane(j)) & 0xFu);
        wait(s_full[buf(g)], par(g));
        if (active) {
          tc_fence_after();
          // S, capped and biased, less the row's reference as it stands, with the
          // keys that get no weight at -inf
          float sv[32];
          // what is taken off this thread's scores of each row: the reference less
          // the part of the bias that is common to the step
          uint64_t off[2];
          auto set_off = [&]() {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              float x = -m_ref[hh];
              if constexpr (kSlopes) x += slope[hh] * static_cast<float>(kb - pos[hh]);
              off[hh] = f32x2(x, x);
            }
          };
          set_off();
          auto take_off = [&]() {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 v = unpack_f32x2(add_f32x2(f32x2(sv[2 * i], sv[2 * i + 1]), off[i & 1]));
              sv[2 * i] = v.x;
              sv[2 * i + 1] = v.y;
            }
          };
          auto scores = [&]() {
            tmem_ld_16x256b_x8(tS(g) + lane_addr, sv);
            tmem_wait_ld();
            if constexpr (kCap) {
              const uint64_t c0 = f32x2(p.poly[0], p.poly[0]), c1 = f32x2(p.poly[1], p.poly[1]);
              const uint64_t c2 = f32x2(p.poly[2], p.poly[2]);
              [[maybe_unused]] const uint64_t c3 = f32x2(p.poly[3], p.poly[3]);
              float um = 0.f;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const uint64_t x = f32x2(sv[2 * i], sv[2 * i + 1]), u = mul_f32x2(x, x);
                const float2 uf = unpack_f32x2(u);
                um = fmax3(um, uf.x, uf.y);
                uint64_t h = c2;
                if constexpr (kPair) h = fma_f32x2(c3, u, c2);
                const float2 v = unpack_f32x2(fma_f32x2(fma_f32x2(fma_f32x2(h, u, c1), u, c0), x, off[i & 1]));
                sv[2 * i] = v.x;
                sv[2 * i + 1] = v.y;
              }
              constexpr double kMostT = 2.0 * 1.4426950408889634 * kPolyMax;
              if (__any_sync(kFull, !(um <= static_cast<float>(kMostT * kMostT)))) {
                // the exact cap where it is due, in place in tensor memory, 8 columns
                // at a time; a score keeps the form and the roundings that it has above
#pragma unroll 1
                for (int c = 0; c < 64; c += 8) {
                  float x[4];
                  tmem_ld_16x256b_x1(tS(g) + lane_addr + c, x);
                  tmem_wait_ld();
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const float u = x[i] * x[i], o = unpack_f32x2(off[i >> 1]).x;
                    const float h = kPair ? fmaf(p.poly[3], u, p.poly[2]) : p.poly[2];
                    const float near = fmaf(fmaf(fmaf(h, u, p.poly[1]), u, p.poly[0]), x[i], o);
                    const float far = fmaf(-2.f * p.cap, fast_rcp(fast_exp2(x[i]) + 1.f), p.cap) + o;
                    x[i] = u <= static_cast<float>(kMostT * kMostT) ? near : far;
                  }
                  tmem_st_16x256b_x1(tS(g) + lane_addr + c, x);
                }
                tmem_wait_st();
                tmem_ld_16x256b_x8(tS(g) + lane_addr, sv);
                tmem_wait_ld();
              }
            } else {
              take_off();
            }
            if constexpr (kSlopes) {
              // Keys after the query are masked, so the distance of key 8 i + e is
              // -(kb - pos + 8 i + e); slope (kb - pos) is in `off`.
#pragma unroll
              for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                  for (int e = 0; e < 2; ++e) sv[4 * i + 2 * hh + e] += slope[hh] * static_cast<float>(8 * i + e);
            }
            if (k0 < clean_from || k0 + 63 > clean_to || bad_pages) {
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
                const int most = min(pos[hh], t.last) - kb, least = p.window > 0 ? pos[hh] - p.window + 1 - kb : -64;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const int key = 8 * (i >> 1) + (i & 1);
                  if (key > most || key < least || ((bad_pages >> (i >> 2)) & 1))
                    sv[4 * (i >> 1) + 2 * hh + (i & 1)] = -INFINITY;
                }
              }
            }
          };
          // P = exp2 of that, as bf16 (and remainder) (16x128b: word 2 i + hh is
          // column 4 i + q, the pair 8 i + 2 q, + 1 of row hh)
          uint32_t ph[16], pl[16];
          [[maybe_unused]] uint64_t lp[2];
          auto weights = [&]() {
            lp[0] = lp[1] = f32x2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float p0 = fast_exp2(sv[2 * i]), p1 = fast_exp2(sv[2 * i + 1]);
              ph[i] = pack_bf16x2(p0, p1);
              if constexpr (kPair) {
                lp[i & 1] = add_f32x2(lp[i & 1], f32x2(p0, p1));
                const float2 rem = bf16x2_remainder(ph[i], p0, p1);
                pl[i] = pack_bf16x2(rem.x, rem.y);
              }
            }
          };
          scores();
          // this thread's maxima above the rows' references
          float mx[2];
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            mx[hh] = -INFINITY;
#pragma unroll
            for (int i = 0; i < 8; ++i) mx[hh] = fmax3(mx[hh], sv[4 * i + 2 * hh], sv[4 * i + 2 * hh + 1]);
          }
          auto above = [&](int hh) { return set[hh] ? mx[hh] > kSlack : mx[hh] != -INFINITY; };
          // The weights are made against the references as they stand before it is
          // known that they do, and again from the scores where they do not. (Not
          // under a cap, whose exact form has taken the scores' place.)
          if constexpr (!kCap) weights();
          // Move the reference to a row's first maximum, and up where a score passed
          // it by more than kSlack; O and l follow, once the last product into them
          // is done. The tensor-memory loads and stores are warp-wide, so a warp
          // rescales them when any of its rows moves, the other rows by exactly 1.
          if (__any_sync(kFull, above(0) || above(1))) {
            bool moves[2], resc[2];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {  // the row's four threads (lanes 4 (t / 4) .. + 3)
              mx[hh] = fmaxf(mx[hh], __shfl_xor_sync(kFull, mx[hh], 1));
              mx[hh] = fmaxf(mx[hh], __shfl_xor_sync(kFull, mx[hh], 2));
              moves[hh] = above(hh);
              resc[hh] = moves[hh] && set[hh];
            }
            if (__any_sync(kFull, resc[0] || resc[1])) {
              wait(pv_done[buf(g - 1)], par(g - 1));
              tc_fence_after();
              float alpha[2];
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
                alpha[hh] = resc[hh] ? fast_exp2(-mx[hh]) : 1.f;
                if constexpr (kPair) l_sum[hh] *= alpha[hh];
              }
#pragma unroll 1
              for (int c = 0; c < (kPair ? 64 : 72); c += 8) {  // 8 columns at a time: all of them at once would spill
                float o[4];
                tmem_ld_16x256b_x1(tO + lane_addr + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] *= alpha[i >> 1];
                tmem_st_16x256b_x1(tO + lane_addr + c, o);
              }
              tmem_wait_st();
            }
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              if (moves[hh]) {
                m_ref[hh] += mx[hh];
                set[hh] = true;
              }
              if constexpr (kCap) {
                const float x = moves[hh] ? -mx[hh] : 0.f;
                off[hh] = f32x2(x, x);
              }
            }
            if constexpr (kCap) {
              take_off();
            } else {
              set_off();
              scores();
              weights();
            }
          }
          if constexpr (kCap) weights();
          tmem_st_16x128b_x8(tS(g) + lane_addr, ph);
          if constexpr (kPair) tmem_st_16x128b_x8(tS(g) + lane_addr + 32, pl);
          tmem_wait_st();
          if constexpr (kPair) {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const float2 a = unpack_f32x2(lp[hh]);
              l_sum[hh] += a.x + a.y;
            }
          }
        }
        // V rows that hold no key of the piece (outside its first and last key, or
        // of a page with a bad id) are zeroed once the stage's V copies have
        // landed, so that their bits cannot reach O
        if (k0 + 63 > t.last || bad_pages || k0 < t.lo) {
          wait(v_full[st], (g / C::kStages) & 1);
          uint8_t* vrow = gbase + (vst(st) - base);
          for (int idx = tid; idx < 64 * 8; idx += C::kSoftmaxThreads) {
            const int key = idx >> 3;
            if (k0 + key > t.last || ((bad_pages >> (key >> 4)) & 1) || k0 + key < t.lo)
              *reinterpret_cast<uint4*>(vrow + key * 128 + (idx & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();  // the zeroed rows, before the tensor core reads V
        }
        tc_fence_before();
        arrive(p_full[buf(g)]);
      }
      // The next piece's queries go to the tensor core before this one's rows
      // are written: its scores are made meanwhile. (Every score product of this
      // piece is done, so Q's shared memory is free.)
      if (__any_sync(kFull, polls == 0) || !piece_wait(n + 1)) failed = true;
      const Piece& nt = s_piece[(n + 1) & 1];
      const bool more = !failed && nt.n_steps > 0;
      if (more) {
        if (has_rows(nt)) {
          load_q(nt);
          load_rows(nt);
          store_q();
        }
        ready_q();
      }
      // m, l and O of the rows (with kPair l is summed over the row's four threads
      // here). The decision is warp-uniform: the tensor-memory load is warp-wide.
      const bool done = !failed && mbar_wait_bounded(smem_addr(&pv_done[buf(g - 1)]), par(g - 1));
      if (__all_sync(kFull, done)) {
        if (active) {
          tc_fence_after();
          float o[32], sums[4];
          tmem_ld_16x256b_x8(tO + lane_addr, o);
          if constexpr (!kPair) tmem_ld_16x256b_x1(tL + lane_addr, sums);
          tmem_wait_ld();
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            float l;
            if constexpr (kPair) {
              l = l_sum[hh];
              l += __shfl_xor_sync(kFull, l, 1);
              l += __shfl_xor_sync(kFull, l, 2);
            } else {
              l = sums[2 * hh];
            }
            if (row_of(hh) < t.members * G) {
              const long long at = t.at + row_of(hh);
              float* dst = p.to.o + at * kHeadDim + 2 * q;
#pragma unroll
              for (int i = 0; i < 8; ++i)
                *reinterpret_cast<float2*>(dst + 8 * i) = make_float2(o[4 * i + 2 * hh], o[4 * i + 2 * hh + 1]);
              if (q == 0) p.to.ml[at] = make_float2(set[hh] ? m_ref[hh] : -INFINITY, l);
            }
          }
        }
      } else {
        failed = true;
      }
      release(n);
      if (!more) break;
    }
  }
  if (failed && lane == 0) atomicOr(p.err, PKV_ERR_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Places of the workspace.
struct SharedWorkspace {
  size_t ml, o, bytes;
  SharedWorkspace(int batch, int hq, int ctas) {
    auto align256 = [](size_t n) { return (n + 255) / 256 * 256; };
    const size_t rows = static_cast<size_t>(batch) * hq + 128 * static_cast<size_t>(ctas);
    ml = align256(sizeof(int4) * (static_cast<size_t>(batch) + 1));
    o = ml + align256(sizeof(float2) * rows);
    bytes = o + sizeof(float) * kHeadDim * rows;
  }
};
SharedPieces pieces_in(void* workspace, int batch, int hq, int ctas) {
  const SharedWorkspace at(batch, hq, ctas);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  SharedPieces to;
  to.tiles = reinterpret_cast<int4*>(ws);
  to.ml = reinterpret_cast<float2*>(ws + at.ml);
  to.o = reinterpret_cast<float*>(ws + at.o);
  to.ctas = ctas;
  return to;
}

template <bool kPair, bool kCap, bool kSlopes>
cudaError_t launch(const SharedLaunch& a, const SharedPieces& to, cudaStream_t stream) {
  using C = Cfg;
  const auto kernel = decode_shared_kernel<kPair, kCap, kSlopes>;
  static DeviceSetup setup;
  cudaError_t e = setup([&] {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(C::bytes(kMaxBatch) + 1024));
    if (e != cudaSuccess) return e;
    // The warpgroups' register shares must fit in what the launch gives the
    // CTA (the compiler's count a thread x its threads), or the softmax
    // warps' increase would wait for registers that never come: refuse.
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return e;
    return 128 * C::kIssueRegs + C::kSoftmaxThreads * C::kSoftmaxRegs > C::kThreads * fa.numRegs
               ? cudaErrorInvalidConfiguration
               : cudaSuccess;
  });
  if (e != cudaSuccess) return e;
  constexpr double log2e = 1.4426950408889634;
  SharedParams p = {};
  p.q_rot = a.q_rot;
  p.block_tables = a.block_tables;
  p.max_blocks = a.max_blocks;
  p.seq_lens = a.seq_lens;
  p.batch = a.batch;
  p.cu_groups = a.cu_groups;
  p.shared_lens = a.shared_lens;
  p.groups = a.groups;
  p.hkv = a.num_kv_heads;
  p.hq = a.num_q_heads;
  p.group = a.num_q_heads / a.num_kv_heads;
  p.num_pages = a.num_pages;
  p.qscale = static_cast<float>(a.softcap > 0.f ? 2.0 * a.scale / a.softcap * log2e : a.scale * log2e);
  p.cap = static_cast<float>(a.softcap * log2e);
  if constexpr (kPair) {
    const ScoreCap cap = make_score_cap(a.softcap);
    for (int i = 0; i < 4; ++i) p.poly[i] = cap.c[i];
  } else {
    double step = 1.0 / (2.0 * log2e);  // x = t / (2 log2 e)
    for (int i = 0; i < 3; ++i, step /= 4.0 * log2e * log2e)
      p.poly[i] = static_cast<float>(a.softcap * log2e * kPoly[i] * step);
  }
  p.slopes = a.slopes;
  p.window = a.window;
  p.to = to;
  p.err = a.err;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(to.ctas);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::bytes(a.batch) + 1024;  // + alignment to 1 KiB
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, *a.kv16_map, p);
}

template <bool kPair>
cudaError_t launch_scores(const SharedLaunch& a, const SharedPieces& to, cudaStream_t stream) {
  if (a.softcap > 0.f) return a.slopes ? launch<kPair, true, true>(a, to, stream) : launch<kPair, true, false>(a, to, stream);
  return a.slopes ? launch<kPair, false, true>(a, to, stream) : launch<kPair, false, false>(a, to, stream);
}

}  // namespace

size_t shared_workspace_bytes(int batch, int num_q_heads, int sm_count) {
  return SharedWorkspace(batch, num_q_heads, kCtas * sm_count).bytes;
}

cudaError_t launch_decode_shared(const SharedLaunch& a, cudaStream_t stream) {
  // Little work is done without sharing, by the scored decode's kernel for it: reading
  // it all takes no longer than the two kernels' latencies. Calls measured there and with
  // the shared kernels, us, tables filled, half of the tokens shared by all of 4, 16 and 64
  // sequences:
  //   32 + 8 heads, 20000 pages in all  14.2 / 25.2  13.9 / 20.0  16.9 / 18.0
  //                 25000               16.8 / 29.9  16.4 / 21.6  18.3 / 18.9
  // and over 60 batches of 4 to 256, 32 + 8, 14 + 2 and 8 + 8 heads, half to nine tenths
  // shared, by one group or many, the shared kernels' time in the other's (the mean, least
  // and most): 32000 pages 1.12 (0.70 to 1.62), 40000 1.02 (0.60 to 1.49), 50000 0.92 (0.54
  // to 1.38); with tables half filled 40000 1.37 (0.87 to 1.84), 65000 1.12 (0.69 to 1.62).
  constexpr long long kMostPages = 32768;
  DecodeLaunch all = {};
  all.pool = a.pool;
  all.num_pages = a.num_pages;
  all.num_kv_heads = a.num_kv_heads;
  all.q_rot = a.q_rot;
  all.out = static_cast<float*>(a.out);
  all.block_tables = a.block_tables;
  all.max_blocks = a.max_blocks;
  all.seq_lens = a.seq_lens;
  all.batch = a.batch;
  all.num_q_heads = a.num_q_heads;
  all.scale = a.scale;
  all.softcap = a.softcap;
  all.slopes = a.slopes;
  all.window = a.window;
  all.out_bf16 = a.out_bf16;
  all.err = a.err;
  if (decode_small_fits(all, kMostPages)) return launch_decode_small(all, stream);
  SharedPieces to = pieces_in(a.workspace, a.batch, a.num_q_heads, kCtas * a.sm_count);
  if (a.groups == 0) {
    to.ctas = 0;  // no pieces
    return launch_decode_rest(a, to, stream);
  }
  const cudaError_t e = a.out_bf16 ? launch_scores<false>(a, to, stream) : launch_scores<true>(a, to, stream);
  return e == cudaSuccess ? launch_decode_rest(a, to, stream) : e;
}

}  // namespace pkv
