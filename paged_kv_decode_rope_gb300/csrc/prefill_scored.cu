// prefill_scored.cu -- attention of chunks whose keys are already in the pool,
// with scores that are capped, biased by distance, and limited to a window, a
// document or a prefix.
//
// With i the query's position and j the key's, t = scale q.k,
//     s = cap tanh(t / cap),  s -= slope |i - j|,
// and the row sees the keys lo <= j <= hi that its window, its document's start
// and its sequence's prefix leave it; out = softmax(s) V over those, zero where
// there are none.
//
// A tile is 128 / G chunk tokens x G query heads = up to 128 rows of one kv
// head (row R = token R / G, head R % G): the M = 128 of one tcgen05 MMA. Keys
// go in steps of 64 (four pages) from the page of the tile's first visible key
// to its last. Per step:
//   S = Q_hi K^T + Q_lo K^T          (tensor memory, 128 x 64 fp32, two buffers)
//   softmax warps: P = exp2(S - m)   row R = tensor-memory lane R
//   O += P V (+ P_lo V)              (tensor memory, 128 x 64 fp32; P over its own S)
//   l += P 1                         (tensor memory; the row sums, as a product with a tile of ones)
// Q enters as bf16 plus its bf16 rounding remainder (about 16 bits), as
// everywhere in this library, and so does P where the output is fp32 (kPair).
// Where the output is bf16, P is rounded to bf16 once, and the tensor core sums
// the rounded P, so that the weights still sum to one (and no instruction of the
// softmax is spent on the sums); what is left (1.1 to 1.35 times the error of
// rounding the output alone, over 16 to 2048 keys) costs a quarter less of the
// softmax's arithmetic and half the P V products. Scores, sums and O are fp32.
// The reference maximum of a row moves only when a score passes it by more than
// kSlack (base 2), so P <= 2^kSlack.
//
// Measured in graph replays, 4 chunks of 2048 tokens, 32 + 8 heads, bf16 out and
// (fp32 out): with a window of 1024 (51.6 GFLOP) 130 us (152) with a cap, 396
// TFLOP/s, 114 (127) without; 234 (265) with a cap of 50 and scores of a standard
// deviation of 16, most steps of which hold one past kPolyMax; over all keys 133
// us (150), 153 (182) with a cap, 141 with a distance bias, 144 with a two-way
// prefix of 512, 164 with both.
//
// What bounds it: the softmax warps. A step of 128 x 64 scores takes an SM some
// 1450 cycles with a cap and 1280 without, about 420 instructions a warp; 62% of
// the cycles issue one (the special-function pipe is 18% busy), and in the others
// the warps wait, for tensor memory and for one another's barriers (1.38 are
// ready in a cycle). Around the steps come those of a tile's start and end, some
// 3700 cycles. With
// a CTA a tile these took 13,000 of the 20,000 cycles of a
// tile of three steps (window 128): launch, tensor memory, tile, query rows,
// first keys, last product, epilogue, one after the other. So CTAs stay, two on
// an SM, and everything but the softmax runs ahead into the next tile: the key
// warp fetches tiles from a counter, publishes what the others need of them,
// asks for their query rows to come to L2 and starts their key copies; the
// softmax warps load, split and hand over the next tile's queries before they
// write this one's rows out. Tiles with the most steps are handed out first.
//
// Warps 0-7 (two warpgroups) run the softmax and the epilogue, 16 rows a warp
// and four threads a row (the 16x256b tensor-memory layout). Warps 8-11, which
// hand registers to them, issue: 8 the K copies, 11 the V copies, 9 the score
// products, 10 the P V products, each as soon as its operands and buffers are
// free. Every wait is bounded.
#include <climits>

#include "f32x2.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "score_cap.cuh"
#include "tc05.cuh"

namespace pkv {
namespace {

constexpr float kSlack = 8.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kSBufs = 2;
constexpr uint32_t kTmemCols = 256;  // two S buffers of 64 columns, O (64), l (16 equal columns)
constexpr int kCtas = 2;             // CTAs a SM

// tanh(x) on |x| <= kPolyMax. Where the output is bf16, as x (c0 + c1 x^2 + c2
// x^4) with the smallest largest error (1.7e-7, found by exchanging the error's
// extrema): four paired fp32 operations for two scores. That is up to 4e-6 of
// a score, all in one direction, which shows where the output is fp32 (kPair), so
// there it is the polynomial of score_cap.cuh with a term more (1e-8 of a score).
// Elsewhere cap tanh(x) = cap - 2 cap / (2^t + 1) with t = 2 log2(e) x, two
// special-function operations a score.
constexpr double kPolyMax = 0.3;
constexpr double kPoly[3] = {0.999996010, -0.332974797, 0.125225911};

struct ScoredParams {
  const float* q_rot;  // [T][hq][64]
  void* out;           // [T][hq][64], fp32 or bf16
  const int32_t* block_tables;
  int max_blocks;
  long long pos_cap;   // positions at or past this are past the block table
  const int4* tiles;   // {sequence, first chunk row, tokens, position of the first token}
  int* counts;         // {tiles, next (tile, kv head) to hand out}
  int hkv, hq;
  long long num_pages;
  float qscale;        // what a query is multiplied by: scores in base 2, or t when capped
  float cap;           // softcap * log2(e), 0: none
  float poly[4];       // cap tanh as a polynomial of t: t (poly[0] + poly[1] t^2 + poly[2] t^4 + poly[3] t^6)
  const int32_t* cu_tokens;    // [batch + 1]
  const int32_t* start_pos;    // [batch]
  const int32_t* prefix_lens;  // [batch] or null
  const int32_t* doc_starts;   // [T] or null
  const float* slopes;         // [hq] or null
  int window;                  // 0: none
  int* err;
};

// A tile as the key warp publishes it. Positions count from key0, a multiple
// of 64; n_steps = 0: no more tiles.
struct Tile {
  int b, row0, n_ok, h;
  int pos0, end, key0, lo;  // first token's position; end of the prefix; first visible key
  int n_pages, n_steps, last, pad;
};

template <int G>
struct Cfg {
  static constexpr int kTokens = 128 / G;
  static constexpr int kRows = kTokens * G;  // <= 128; rows past it are padding
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
  // dynamic shared memory: Q_hi, Q_lo, per stage K and V, then 16 rows of ones
  static constexpr uint32_t kQhi = 0, kQlo = kTile;
  static constexpr uint32_t kStage0 = 2 * kTile;
  static constexpr uint32_t kOnes = kStage0 + kStages * 2 * kStep;
  static constexpr uint32_t kBytes = kOnes + 16 * 128;
};

template <int G, bool kPair>
__global__ void __launch_bounds__(Cfg<G>::kThreads, kCtas)
    prefill_scored_kernel(const __grid_constant__ CUtensorMap kv16_map, const ScoredParams p) {
  using C = Cfg<G>;
  extern __shared__ __align__(1024) uint8_t dsmem[];
  __shared__ __align__(8) uint64_t k_full[C::kStages], k_empty[C::kStages];
  __shared__ __align__(8) uint64_t v_full[C::kStages], v_empty[C::kStages];
  __shared__ __align__(8) uint64_t s_full[kSBufs], p_full[kSBufs], pv_done[kSBufs], q_ready, drain[2];
  __shared__ __align__(8) uint64_t tile_full[2], tile_empty[2];
  __shared__ Tile s_tile[2];
  __shared__ uint32_t s_tmem;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_addr(dsmem) + 1023u) & ~1023u;
  uint8_t* gbase = dsmem + (base - smem_addr(dsmem));
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
    mbar_init(smem_addr(&q_ready), C::kSoftmaxThreads);
    // S done, P ready and P V done, one barrier each per buffer (step % kSBufs):
    // a wait for a step never sees its barrier two phases on
    for (int i = 0; i < kSBufs; ++i) {
      mbar_init(smem_addr(&s_full[i]), 1);
      mbar_init(smem_addr(&p_full[i]), C::kSoftmaxThreads);
      mbar_init(smem_addr(&pv_done[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&drain[i]), 1);
      mbar_init(smem_addr(&tile_full[i]), 1);
      mbar_init(smem_addr(&tile_empty[i]), 11);  // every warp but the key warp
    }
  }
  for (int i = tid; i < 16 * 128 / 4; i += C::kThreads)
    reinterpret_cast<uint32_t*>(gbase + C::kOnes)[i] = 0x3F803F80u;  // (the same in any swizzle)
  fence_proxy_async_smem();
  fence_mbar_init();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // The plan is the kernel before this one: the set-up overlaps its end.
  grid_dependency_wait();
  const uint32_t tmem = s_tmem, tO = tmem + 64 * kSBufs, tL = tO + 64;
  // steps are numbered through, tile after tile
  auto tS = [&](int g) { return tmem + 64 * (g % kSBufs); };  // S, then P (hi: +0, lo: +32)
  auto buf = [](int g) { return g % kSBufs; };
  auto par = [](int g) { return static_cast<uint32_t>((g / kSBufs) & 1); };
  // Step j of a tile takes the 64 keys of block key_block(j). With a distance
  // bias the last block comes first: the largest scores are there, and the
  // reference maximum found in the first step stands (from the first block on
  // it moved in nearly every step: 1.6 times the time for 4 x 2048 tokens).
  // Without one the first block comes first, a full one where the last one
  // holds few keys of the early rows, so that their first maximum is soon
  // passed (0.88 of the time with a window of 1024). Page ids come in windows
  // of 32, eight steps: lane i of window m holds page window_page(m) + i, and
  // step j's four pages are lanes window_lane(j) .. + 3.
  const bool down = p.slopes != nullptr;
  auto key_block = [&](int j, int n_steps) { return down ? n_steps - 1 - j : j; };
  auto window_page = [&](int m, int n_steps) { return down ? 4 * n_steps - 32 * (m + 1) : 32 * m; };
  auto window_lane = [&](int j) { return down ? 28 - ((4 * j) & 31) : (4 * j) & 31; };
  // (pages before the first visible key are no part of the tile)
  auto is_page = [](const Tile& t, int pg) { return pg >= t.lo / kPage && pg < t.n_pages; };
  auto table = [&](const Tile& t) {
    return p.block_tables + static_cast<size_t>(t.b) * p.max_blocks + t.key0 / kPage;
  };
  auto page_id = [&](const Tile& t, int pg) { return is_page(t, pg) ? table(t)[pg] : -1; };
  // first key (position) that the token in chunk row r at position pos sees
  auto first_key = [&](int r, int pos) {
    int lo = p.doc_starts ? max(p.doc_starts[r], 0) : 0;
    if (p.window > 0) lo = max(lo, pos - p.window + 1);
    return lo;
  };
  // Tile n's entry, for every warp but the key warp; release() when it is read.
  auto tile_wait = [&](int n) { return mbar_wait_bounded(smem_addr(&tile_full[n & 1]), (n >> 1) & 1); };
  auto release = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&tile_empty[n & 1]));
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
      bool first = true;
      // The key warp's own: the next tile that sees a key, published as entry n.
      auto fetch = [&](int n) {
        Tile t = {};
        const int total = p.counts[0] * p.hkv;
        for (;;) {
          int x = first ? static_cast<int>(blockIdx.x) : 0;
          if (!first && lane == 0) x = atomicAdd(&p.counts[1], 1);
          x = __shfl_sync(kFull, x, 0);
          first = false;
          if (x >= total) {
            t.n_steps = 0;
            break;
          }
          const int ti = x / p.hkv;
          const int4 tile = p.tiles[ti];
          t.h = x - ti * p.hkv;
          t.b = tile.x;
          t.row0 = tile.y;
          const int c0 = p.cu_tokens[t.b], c1 = p.cu_tokens[t.b + 1], start = p.start_pos[t.b];
          const int prefix = p.prefix_lens ? p.prefix_lens[t.b] : 0;
          const long long room = p.pos_cap - tile.w;
          t.n_ok = start < 0 || tile.w < 0 ? 0 : static_cast<int>(min(static_cast<long long>(tile.z), max(room, 0ll)));
          // keys past the chunk's end exist for no query; a prefix reaches up to it
          t.end = static_cast<int>(min(static_cast<long long>(max(prefix, 0)),
                                       min(static_cast<long long>(start) + (c1 - c0), p.pos_cap)));
          if (t.n_ok < tile.z && lane == 0) atomicOr(p.err, PKV_ERR_SEQ_LEN);
          // the least first key and the last key of the tokens that see one
          int lo = INT_MAX, hi = -1;
          for (int i = lane; i < t.n_ok; i += 32) {
            const int l = first_key(t.row0 + i, tile.w + i);
            const int last = max(tile.w + i, t.end - 1);
            if (l <= last) {
              lo = min(lo, l);
              hi = max(hi, last);
            }
            // its query rows, to L2
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                             p.q_rot + (static_cast<size_t>(t.row0 + i) * p.hq + t.h * G) * kHeadDim),
                         "r"(G * kHeadDim * 4)
                         : "memory");
          }
          lo = __reduce_min_sync(kFull, lo);
          hi = __reduce_max_sync(kFull, hi);
          if (lo == INT_MAX) t.n_ok = 0;  // no row sees a key
          // rows past n_ok, all of them when no row sees a key
          const int words = G * kHeadDim / (kPair ? 1 : 2);
          for (int e = t.n_ok * words + lane; e < tile.z * words; e += 32) {
            const int i = e / words, rest = e - i * words;
            static_cast<uint32_t*>(p.out)[static_cast<size_t>(t.row0 + i) * (p.hq / G) * words + t.h * words + rest] = 0u;
          }
          if (t.n_ok == 0) continue;
          t.key0 = lo / 64 * 64;
          t.lo = lo - t.key0;
          t.pos0 = tile.w - t.key0;
          t.end -= t.key0;
          t.last = hi - t.key0;
          t.n_pages = t.last / kPage + 1;
          t.n_steps = (t.n_pages + 3) / 4;
          break;
        }
        if (n >= 2 && !mbar_wait_idle(smem_addr(&tile_empty[n & 1]), ((n >> 1) - 1) & 1)) failed = true;
        if (__any_sync(kFull, failed)) failed = true;
        if (lane == 0 && !failed) {
          s_tile[n & 1] = t;
          mbar_arrive(smem_addr(&tile_full[n & 1]));
        }
        return t;
      };
      Tile t, next = {};
      if (kind == 0) next = fetch(0);
      for (int n = 0; !failed; ++n) {
        if (kind == 0) {
          t = next;
        } else {
          if (!tile_wait(n)) failed = true;
          if (__any_sync(kFull, failed)) {
            failed = true;
            break;
          }
          t = s_tile[n & 1];
          release(n);
        }
        if (t.n_steps == 0) break;
        // lane i: the copy's row coordinate for page window_page(m) + i (-1: no
        // page of the tile, or a bad id), and the window's valid pages as a mask
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
          // the next tile, once this one's first stages are on their way
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
        return __all_sync(kFull, mbar_wait_idle(bar, parity)) != 0;
      };
      constexpr uint32_t idS = idesc_bf16_f32(128, 64, false), idPV = idesc_bf16_f32(128, 64, true);
      constexpr uint32_t idL = idesc_bf16_f32(128, 16, false);
      const uint64_t dOnes = smem_desc_sw128(base + C::kOnes);
      const uint64_t dQhi = smem_desc_sw128(base + C::kQhi), dQlo = smem_desc_sw128(base + C::kQlo);
      int g = 0;
      for (int n = 0; !failed; ++n) {
        if (!wait_all(smem_addr(&tile_full[n & 1]), (n >> 1) & 1)) {
          failed = true;
          break;
        }
        const int n_steps = s_tile[n & 1].n_steps;
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
            const uint64_t dV = smem_desc_sw128(vst(st));
            // P from tensor memory (a 16-key K step is 8 columns); V is MN-major:
            // a 16-key K step is 16 rows = 2048 bytes (+128)
#pragma unroll
            for (int k = 0; k < 4; ++k) umma_bf16_tmem_a(tO, tS(g) + 8 * k, dV + 128 * k, idPV, j > 0 || k > 0);
            if constexpr (kPair) {
#pragma unroll
              for (int k = 0; k < 4; ++k) umma_bf16_tmem_a(tO, tS(g) + 32 + 8 * k, dV + 128 * k, idPV, true);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) umma_bf16_tmem_a(tL, tS(g) + 8 * k, dOnes + 2 * k, idL, j > 0 || k > 0);
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
    // ---- softmax and epilogue. Warp w owns rows L .. L + 15, L = 32 (w % 4)
    // + 16 (w / 4) (tensor-memory lanes). Its thread t holds rows L + t / 4
    // (hh = 0) and L + t / 4 + 8 (hh = 1) and, of each, the key pairs
    // 8 i + 2 q and 8 i + 2 q + 1 (i = 0..7, q = t % 4): the 16x256b layout,
    // in which S word 4 i + 2 hh + e is key 8 i + 2 q + e of row hh. ----
    const int q = lane & 3;
    const int lrow = 32 * (warp & 3) + 16 * (warp >> 2);  // the warp's first row
    const uint32_t lane_addr = static_cast<uint32_t>(lrow) << 16;
    // its rows' tokens and heads (kTokens: a padding row), worked out where they
    // are used: the steps' registers are full
    auto tok = [&](int hh) {
      const int rw = lrow + (lane >> 2) + 8 * hh;
      return rw < C::kRows ? rw / G : C::kTokens;
    };
    auto gix = [&](int hh) { return (lrow + (lane >> 2) + 8 * hh) % G; };
    // this thread's share of a tile's query rows: dims 16 q .. 16 q + 15 of its two rows
    float4 qv[2][4];
    auto load_q = [&](const Tile& t) {
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const bool in = tok(hh) < t.n_ok;
        const float* qr = p.q_rot +
                          (static_cast<size_t>(t.row0 + (in ? tok(hh) : 0)) * p.hq + t.h * G + gix(hh)) * kHeadDim +
                          16 * q;
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
      fence_proxy_async_smem();
      mbar_arrive(smem_addr(&q_ready));
    };
    // what a tile's rows see (positions from key0: lo to the larger of pos and
    // the prefix's last), their slopes (base 2), and the tile's first window of
    // page ids
    int lo[2], pos[2], pid = 0;
    float slope[2] = {0.f, 0.f};
    auto load_rows = [&](const Tile& t) {
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int i = min(tok(hh), t.n_ok - 1);
        pos[hh] = t.pos0 + i;
        lo[hh] = first_key(t.row0 + i, pos[hh] + t.key0) - t.key0;
        if (p.slopes) slope[hh] = p.slopes[t.h * G + gix(hh)] * kLog2e;
      }
      pid = page_id(t, window_page(0, t.n_steps) + lane);
    };

    if (!tile_wait(0)) failed = true;
    int n = 0, g = 0;
    const bool some = !failed && s_tile[0].n_steps > 0;
    if (some) {
      load_q(s_tile[0]);
      load_rows(s_tile[0]);
      store_q();
    }
    for (; some && !failed; ++n) {
      const Tile& t = s_tile[n & 1];
      const int n_steps = t.n_steps;
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
      auto window_id = [&](int m) {
        const int pg = window_page(m, n_steps) + lane;
        return page_id(t, pg);
      };
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
        const int bad = static_cast<int>((bad_win >> window_lane(j)) & 0xFu);
        if (!mbar_wait_bounded(smem_addr(&s_full[buf(g)]), par(g))) failed = true;
        tc_fence_after();
        // S, capped and biased, less the row's reference as it stands, with the
        // keys that get no weight at -inf
        float sv[32];
        // what is taken off this thread's scores of each row: the reference less
        // the part of the bias that is common to the step
        uint64_t off[2];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          float x = -m_ref[hh];
          if (p.slopes && !p.prefix_lens) x += slope[hh] * static_cast<float>(kb - pos[hh]);
          off[hh] = f32x2(x, x);
        }
        auto take_off = [&]() {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 v = unpack_f32x2(add_f32x2(f32x2(sv[2 * i], sv[2 * i + 1]), off[i & 1]));
            sv[2 * i] = v.x;
            sv[2 * i + 1] = v.y;
          }
        };
        {
          tmem_ld_16x256b_x8(tS(g) + lane_addr, sv);
          tmem_wait_ld();
          if (p.cap > 0.f) {
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
              // The exact cap where it is due, in place in tensor memory, 8 columns
              // at a time (with both forms over all 32 scores of a thread in one
              // path its registers spilled, and every step took 1.5 times as
              // long). A score keeps the form and the roundings that it has above:
              // rows of keys that are not the tile's hold anything, and what they
              // score must not show in the others.
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
          if (p.slopes) {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const float d0 = static_cast<float>(kb - pos[hh]);  // of the first key from the query
              if (!p.prefix_lens) {
                // Keys after the query are masked, so the distance of key
                // 8 i + e is -(d0 + 8 i + e); slope d0 is in `off`.
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                  for (int e = 0; e < 2; ++e) sv[4 * i + 2 * hh + e] += slope[hh] * static_cast<float>(8 * i + e);
              } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                  for (int e = 0; e < 2; ++e)
                    sv[4 * i + 2 * hh + e] -= slope[hh] * fabsf(d0 + static_cast<float>(8 * i + e));
              }
            }
          }
          // (an end at a time: two instructions a score, and a step seldom has both)
          if (k0 + 63 > min(pos[0], pos[1]) && k0 + 63 >= t.end) {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const int most = max(pos[hh], t.end - 1) - kb;
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (8 * (i >> 1) + (i & 1) > most) sv[4 * (i >> 1) + 2 * hh + (i & 1)] = -INFINITY;
            }
          }
          if (k0 < max(lo[0], lo[1])) {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const int least = lo[hh] - kb;
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (8 * (i >> 1) + (i & 1) < least) sv[4 * (i >> 1) + 2 * hh + (i & 1)] = -INFINITY;
            }
          }
          if (bad) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if ((bad >> (i >> 3)) & 1) sv[i] = -INFINITY;
          }
        }
        // each row's maximum above its reference: the row's four threads (lanes
        // 4 (t / 4) .. + 3)
        float mx[2];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          float m = -INFINITY;
#pragma unroll
          for (int i = 0; i < 8; ++i) m = fmax3(m, sv[4 * i + 2 * hh], sv[4 * i + 2 * hh + 1]);
          m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
          mx[hh] = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
        }
        // Move the reference to a row's first maximum, and up where a score passed
        // it by more than kSlack; O and l follow, once the last product into them
        // is done. The tensor-memory loads and stores are warp-wide, so a warp
        // rescales them when any of its rows moves, the other rows by exactly 1.
        bool moves[2], resc[2];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          moves[hh] = set[hh] ? mx[hh] > kSlack : mx[hh] != -INFINITY;
          resc[hh] = moves[hh] && set[hh];
        }
        if (__any_sync(kFull, moves[0] || moves[1])) {
          if (__any_sync(kFull, resc[0] || resc[1])) {
            if (!mbar_wait_bounded(smem_addr(&pv_done[buf(g - 1)]), par(g - 1))) failed = true;
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
            const float x = moves[hh] ? -mx[hh] : 0.f;
            off[hh] = f32x2(x, x);
          }
          take_off();
        }
        // P = exp2 of that, as bf16 (and remainder) (16x128b: word 2 i + hh is
        // column 4 i + q, the pair 8 i + 2 q, + 1 of row hh)
        uint32_t ph[16], pl[16];
        [[maybe_unused]] uint64_t lp[2] = {f32x2(0.f, 0.f), f32x2(0.f, 0.f)};
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
        // V rows that hold no key of the tile (outside its first and last key, or
        // of a page with a bad id) are zeroed once the stage's V copies have
        // landed, so that their bits cannot reach O
        if (k0 + 63 > t.last || bad || k0 < t.lo) {
          if (!mbar_wait_bounded(smem_addr(&v_full[st]), (g / C::kStages) & 1)) failed = true;
          uint8_t* vrow = gbase + (vst(st) - base);
          for (int idx = tid; idx < 64 * 8; idx += C::kSoftmaxThreads) {
            const int key = idx >> 3;
            if (k0 + key > t.last || ((bad >> (key >> 4)) & 1) || k0 + key < t.lo)
              *reinterpret_cast<uint4*>(vrow + key * 128 + (idx & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();  // the zeroed rows, before the tensor core reads V
        }
        tc_fence_before();
        mbar_arrive(smem_addr(&p_full[buf(g)]));
        if (failed) break;
      }
      // The next tile's queries go to the tensor core before this one's rows
      // are written: its scores are made meanwhile. (Every score product of this
      // tile is done, so Q's shared memory is free.)
      if (!failed && !tile_wait(n + 1)) failed = true;
      const Tile& nt = s_tile[(n + 1) & 1];
      const bool more = !failed && nt.n_steps > 0;
      if (more) {
        load_q(nt);
        load_rows(nt);
        store_q();
      }
      // O / l for the live rows (with kPair l is summed over the row's four
      // threads here). The decision is warp-uniform: the tensor-memory load is warp-wide.
      const bool done = !failed && mbar_wait_bounded(smem_addr(&pv_done[buf(g - 1)]), par(g - 1));
      if (__all_sync(kFull, done)) {
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
          if (tok(hh) < t.n_ok) {
            const float inv = l > 0.f ? 1.f / l : 0.f;
            const size_t at =
                (static_cast<size_t>(t.row0 + tok(hh)) * p.hq + t.h * G + gix(hh)) * kHeadDim + 2 * q;
            if constexpr (!kPair) {
              uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + at);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                dst[4 * i] = pack_bf16x2(o[4 * i + 2 * hh] * inv, o[4 * i + 2 * hh + 1] * inv);
            } else {
              float* dst = static_cast<float*>(p.out) + at;
#pragma unroll
              for (int i = 0; i < 8; ++i)
                *reinterpret_cast<float2*>(dst + 8 * i) =
                    make_float2(o[4 * i + 2 * hh] * inv, o[4 * i + 2 * hh + 1] * inv);
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

// Lists the tiles: sequence b's chunk gives ceil(len / tokens) of them. One
// CTA. The tiles are ordered by the 64-key steps they take, most first (a
// counting sort over kBuckets buckets, the last one shared by every tile of
// that many steps or more; the order within a bucket is arbitrary), so that
// the tiles handed out last are the short ones. Rows are clipped to
// [0, total); tiles past `capacity` (only possible when chunks overlap) are
// dropped and flagged.
constexpr int kPlanThreads = 1024;
constexpr int kBuckets = kPlanThreads;
__global__ void __launch_bounds__(kPlanThreads)
    prefill_scored_plan_kernel(const int32_t* __restrict__ cu_tokens, const int32_t* __restrict__ start_pos,
                               int batch, int total, int tokens_per_tile, int capacity, int window,
                               const int32_t* __restrict__ doc_starts, int grid, int4* __restrict__ tiles,
                               int* __restrict__ counts, int* __restrict__ err) {
  grid_launch_dependents();  // the attention waits for this kernel itself
  __shared__ int s_hist[kBuckets];  // tiles per bucket, then the bucket's next slot
  __shared__ int s_warp[kPlanThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  s_hist[tid] = 0;
  __syncthreads();
  // a warp per sequence, its lanes over the sequence's tiles; a tile's steps
  // from the keys before its last token that its first one sees
  auto for_tiles = [&](auto visit) {
    for (int b = warp; b < batch; b += kPlanThreads / 32) {
      const int c0 = max(cu_tokens[b], 0), c1 = min(cu_tokens[b + 1], total), start = start_pos[b];
      for (int r = c0 + lane * tokens_per_tile; r < c1; r += 32 * tokens_per_tile) {
        const int n = min(tokens_per_tile, c1 - r);
        const long long pos = static_cast<long long>(start) + (r - c0);
        int bucket = kBuckets - 1;  // no work: last
        if (start >= 0 && pos <= INT_MAX) {
          long long lo = window > 0 ? max(pos - window, 0ll) : 0ll;
          if (doc_starts) lo = max(lo, min(static_cast<long long>(doc_starts[r]), pos));
          bucket = kBuckets - 1 - static_cast<int>(min((pos + n - 1 - lo) / 64 + 1, static_cast<long long>(kBuckets - 1)));
        }
        visit(bucket, make_int4(b, r, n, start < 0 || pos > INT_MAX ? -1 : static_cast<int>(pos)));
      }
    }
  };
  for_tiles([&](int bucket, int4) { atomicAdd(&s_hist[bucket], 1); });
  __syncthreads();
  const int mine = s_hist[tid];
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(kFull, upto, o);
    if (lane >= o) upto += t;
  }
  if (lane == 31) s_warp[warp] = upto;
  __syncthreads();
  int before = lane < warp ? s_warp[lane] : 0;
#pragma unroll
  for (int o = 16; o; o >>= 1) before += __shfl_xor_sync(kFull, before, o);
  s_hist[tid] = before + upto - mine;
  if (tid == kPlanThreads - 1) {
    const int all = before + upto;
    if (all > capacity) atomicOr(err, PKV_ERR_SEQ_LEN);
    counts[0] = min(all, capacity);
    counts[1] = grid;  // every CTA's first is its own index
  }
  __syncthreads();
  for_tiles([&](int bucket, int4 tile) {
    const int slot = atomicAdd(&s_hist[bucket], 1);
    if (slot < capacity) tiles[slot] = tile;
  });
}

template <int G, bool kPair>
cudaError_t launch(const PrefillLaunch& a, int4* tiles, int* counts, cudaStream_t stream) {
  using C = Cfg<G>;
  const int smem = static_cast<int>(C::kBytes + 1024);  // + alignment to 1 KiB
  static DeviceSetup setup;
  cudaError_t e = setup([&] {
    cudaError_t e = cudaFuncSetAttribute(prefill_scored_kernel<G, kPair>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // The warpgroups' register shares must fit in what the launch gives the
    // CTA (the compiler's count a thread x its threads), or the softmax
    // warps' increase would wait for registers that never come: refuse.
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, prefill_scored_kernel<G, kPair>);
    if (e != cudaSuccess) return e;
    return 128 * C::kIssueRegs + C::kSoftmaxThreads * C::kSoftmaxRegs > C::kThreads * fa.numRegs
               ? cudaErrorInvalidConfiguration
               : cudaSuccess;
  });
  if (e != cudaSuccess) return e;
  const size_t capacity = static_cast<size_t>(a.total_tokens + C::kTokens - 1) / C::kTokens + a.batch;
  const size_t units = capacity * static_cast<size_t>(a.num_kv_heads);
  if (units > 0x7fff0000u) return cudaErrorInvalidValue;
  const size_t most = static_cast<size_t>(kCtas) * a.sm_count;
  const int grid = static_cast<int>(units < most ? units : most);
  prefill_scored_plan_kernel<<<1, kPlanThreads, 0, stream>>>(
      a.cu_tokens, a.start_pos, a.batch, a.total_tokens, C::kTokens, static_cast<int>(capacity), a.window,
      a.doc_starts, grid, tiles, counts, a.err);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  constexpr double log2e = 1.4426950408889634;
  ScoredParams p = {};
  p.q_rot = a.q_rot;
  p.out = a.out;
  p.block_tables = a.block_tables;
  p.max_blocks = a.max_blocks;
  p.pos_cap = static_cast<long long>(a.max_blocks) * kPage;
  p.tiles = tiles;
  p.counts = counts;
  p.hkv = a.num_kv_heads;
  p.hq = a.num_q_heads;
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
  p.cu_tokens = a.cu_tokens;
  p.start_pos = a.start_pos;
  p.prefix_lens = a.prefix_lens;
  p.doc_starts = a.doc_starts;
  p.slopes = a.slopes;
  p.window = a.window;
  p.err = a.err;
  // programmatic dependent launch: the kernel's set-up overlaps the plan
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefill_scored_kernel<G, kPair>, *a.kv16_map, p);
}

template <int G>
cudaError_t launch_group(const PrefillLaunch& a, int4* tiles, int* counts, cudaStream_t stream) {
  return a.out_bf16 ? launch<G, false>(a, tiles, counts, stream) : launch<G, true>(a, tiles, counts, stream);
}

}  // namespace

// The workspace of a prefill (prefill_workspace_bytes) holds more tiles than
// these: the counts go first, then the tile list.
cudaError_t launch_prefill_scored(const PrefillLaunch& a, cudaStream_t stream) {
  if (a.total_tokens == 0) return cudaSuccess;
  int* counts = static_cast<int*>(a.workspace);
  int4* tiles = reinterpret_cast<int4*>(static_cast<uint8_t*>(a.workspace) + 256);
  switch (a.num_q_heads / a.num_kv_heads) {
    case 1: return launch_group<1>(a, tiles, counts, stream);
    case 2: return launch_group<2>(a, tiles, counts, stream);
    case 3: return launch_group<3>(a, tiles, counts, stream);
    case 4: return launch_group<4>(a, tiles, counts, stream);
    case 5: return launch_group<5>(a, tiles, counts, stream);
    case 6: return launch_group<6>(a, tiles, counts, stream);
    case 7: return launch_group<7>(a, tiles, counts, stream);
    case 8: return launch_group<8>(a, tiles, counts, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pkv
