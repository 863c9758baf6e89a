// decode_rest.cu -- the second kernel of paged_gqa_decode_shared: every sequence's own
// pages, and the join with the pieces of the pages it shares (decode_shared.cu).
//
// A segment is a sequence and a kv head: G query rows, the pages from the end of the
// shared ones on. As in decode_small.cu a segment is a cluster of 1 to 16 CTAs, as
// many (a power of two) as keep all clusters on the GPU at once, whose warps take its pages in turn and
// whose sums meet in shared memory, then across the cluster. The own pages need nothing
// of the first kernel (what a sequence shares is worked out here again, from the
// lengths), so they are read before it is complete, on the SMs that it has left;
// only then come the pieces of the shared pages, also in turn (16 x 4 beams 28.7 -> 24.6
// us, 3 documents 150 -> 145). A page and kv head (4 KB, keys and values) comes by one
// bulk tensor copy into the warp's own ring of kStages, 128-byte swizzled, from which
// the operands of the products are read without conflicts of banks: lane (g, t) takes
// dims 16 t .. + 15 of keys g and g + 8, and dims 8 g .. + 7 of tokens 2 t, 2 t + 1,
// 2 t + 8 and 2 t + 9 (both contractions may take their index in any order). Q (rows
// 0-7: heads) and P enter as bf16 with their remainders in rows 8-15.
//
// Measured in graph replays, own pages alone, 32 + 8 heads: 256 sequences of 4096 tokens
// 316 us, 6.8 TB/s, the rate of a copy; 64 of up to 600 tokens 11.5 us, of one token
// 6.0 us. With pages loaded straight into registers, two in flight a warp (as
// decode_small.cu does, for less work), the first took 413 us. 16 x 4 beams (both
// kernels) take 24.6 us, 64 answers behind 8192 tokens 31: the many small segments wait
// for latencies (lengths, page ids, pages, pieces), so four CTAs an SM with rings of
// three pages beat three with rings of four (before the own pages came first, 29.0 against
// 30.9 and 31.8 against 35.2). The first kernel on half of its CTAs, to leave room
// beside it, took 30.7 and 31.5 (256 sequences behind three documents 156 against 126).
#include <atomic>
#include <climits>

#include <cooperative_groups.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "score_cap.cuh"
#include "shared_line.cuh"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kCtas = 4;  // CTAs a SM
constexpr int kStages = 3;
constexpr int kMaxCluster = 16;
constexpr int kShortPages = 160;  // tables of up to this many blocks take clusters of at most 8 CTAs (decode_small.cu)
constexpr int kMaxGroup = PKV_MAX_GROUP;
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kRing = kWarps * kStages * kHeadPageBytes;
static_assert(kMaxGroup * kHeadDim * sizeof(float) <= kStages * kHeadPageBytes, "a warp's sums go into its ring");

struct RestParams {
  const uint8_t* pool;
  long long num_pages;
  int hkv, group;
  const float* q_rot;  // [batch][hq][64]
  void* out;           // [batch][hq][64], fp32 or bf16
  const int32_t* block_tables;
  int max_blocks;
  const int32_t* seq_lens;
  int batch;
  const float* slopes;  // [hq] or null
  int window;           // 0: none
  float qscale;         // scores in base 2, or 2 log2(e) x when capped
  ScoreCap cap;
  int out_bf16;
  SharedPieces pieces;  // ctas = 0: nothing is shared
  const int32_t* cu_groups;    // [groups + 1]
  const int32_t* shared_lens;  // [groups]
  int groups;
  int* err;
};

// Elements e0 .. e1 - 1 of a segment's rows from the sequence's own keys alone, key by
// key in plain arithmetic, a row a warp. Under a window a tile's rows see different keys,
// and a value that is not finite makes NaN of the rows whose weight for it is 0, so this
// is for rows that are not finite. Small and inlined: as a function that is called, or as
// the loop over the ring a second time, it made every call with a window 3% slower.
__device__ __forceinline__ void finish_alone(const RestParams& p, int b, int h, int e0, int e1) {
  const int lane = threadIdx.x & 31, n = p.seq_lens[b], lo = max(n - p.window, 0);
  const int32_t* bt = p.block_tables + static_cast<size_t>(b) * p.max_blocks;
  for (int g = e0 / kHeadDim + (threadIdx.x >> 5); g * kHeadDim < e1; g += kWarps) {
    const size_t row = (static_cast<size_t>(b) * p.hkv + h) * p.group + g;
    const float2 q = *reinterpret_cast<const float2*>(p.q_rot + row * kHeadDim + 2 * lane);
    const float slope = p.slopes ? p.slopes[h * p.group + g] * kLog2e : 0.f;
    float m = -INFINITY, l = 0.f, o[2] = {0.f, 0.f};  // dims 2 lane and 2 lane + 1
    for (int key = lo; key < n; ++key) {
      const int page = bt[key / kPage];
      if (page < 0 || page >= p.num_pages) continue;  // (reported where it was met first)
      const uint8_t* at = p.pool + (static_cast<size_t>(page) * p.hkv + h) * kHeadPageBytes + key % kPage * kRowBytes + 4 * lane;
      const float2 k = bf16x2_to_float2(*reinterpret_cast<const uint32_t*>(at));
      const float2 v = bf16x2_to_float2(*reinterpret_cast<const uint32_t*>(at + kHalfBytes));
      float s = q.x * p.qscale * k.x + q.y * p.qscale * k.y;
#pragma unroll
      for (int i = 16; i; i >>= 1) s += __shfl_xor_sync(kFull, s, i);
      if (p.cap.cap > 0.f) s = capped_score(p.cap, s);
      s -= slope * static_cast<float>(n - 1 - key);
      const float up = fmaxf(m, s), ref = up == -INFINITY ? 0.f : up;
      const float keep = fast_exp2(m - ref), w = fast_exp2(s - ref);
      m = up;
      l = l * keep + w;
      o[0] = o[0] * keep + w * v.x;
      o[1] = o[1] * keep + w * v.y;
    }
    for (int i = 0; i < 2; ++i) {
      const int d = 2 * lane + i, e = g * kHeadDim + d;
      if (e < e0 || e >= e1) continue;
      const float y = l == 0.f ? 0.f : o[i] / l;
      if (p.out_bf16) {
        static_cast<uint16_t*>(p.out)[row * kHeadDim + d] = static_cast<uint16_t>(pack_bf16x2(y, 0.f));
      } else {
        static_cast<float*>(p.out)[row * kHeadDim + d] = y;
      }
    }
  }
}

// kWindow: whether there is one (p.window > 0).
template <bool kWindow>
__global__ void __launch_bounds__(kThreads, kCtas)
    decode_rest_kernel(const __grid_constant__ CUtensorMap kv_map, const RestParams p) {
  extern __shared__ __align__(1024) uint8_t dsmem[];
  __shared__ __align__(8) uint64_t s_bar[kWarps][kStages];
  __shared__ int3 s_group;  // of the sequence: its members and what they share
  __shared__ int s_least;   // their least length
  __shared__ float s_m[kWarps][kMaxGroup], s_l[kWarps][kMaxGroup];
  __shared__ float c_acc[kMaxGroup][kHeadDim], c_m[kMaxGroup], c_l[kMaxGroup];  // the CTA's sums
  const cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), ctas = static_cast<int>(cluster.num_blocks());
  const int G = p.group;
  const int sg = blockIdx.x / ctas, b = sg / p.hkv, h = sg - b * p.hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g8 = lane >> 2, t4 = lane & 3;
  const size_t row0 = static_cast<size_t>(sg) * G;  // b hq + h G
  const uint32_t base = (smem_addr(dsmem) + 1023u) & ~1023u;
  const uint32_t ring = base + warp * kStages * kHeadPageBytes;
  uint8_t* gbase = dsmem + (base - smem_addr(dsmem));
  // a warp's sums, where its ring was
  auto acc = [&](int w) { return reinterpret_cast<float*>(gbase + w * kStages * kHeadPageBytes); };
  if (lane == 0)
    for (int s = 0; s < kStages; ++s) mbar_init(smem_addr(&s_bar[warp][s]), 1);
  fence_mbar_init();
  __syncwarp();
  // The first kernel lets this one go when all kernels before it are complete, so the
  // sequence's own pages are read without waiting for it; its pieces come after them.
  // (Where it is not launched, what is before is waited for here.)
  if (p.pieces.ctas == 0) {
    grid_dependency_wait();
    grid_launch_dependents();
  }
  const int n = p.seq_lens[b];
  int first = 0;
  if (p.pieces.ctas > 0) {  // shared blocks, as the first kernel counts them
    int bad_groups = 0;
    if (tid == 0) s_group = make_int3(0, 0, 0), s_least = INT_MAX;
    __syncthreads();
    for (int g = tid; g < p.groups; g += kThreads) {
      const int c0 = p.cu_groups[g], c1 = p.cu_groups[g + 1], shared = p.shared_lens[g];
      bad_groups |= c0 < 0 || c1 < c0 || c1 > p.batch;
      if (c0 <= b && b < c1) s_group = make_int3(c0, c1, shared);
    }
    if (!__syncthreads_or(bad_groups) && s_group.y - s_group.x > 1) {
      int least = INT_MAX;
      for (int i = s_group.x + tid; i < s_group.y; i += kThreads) {
        const int len = p.seq_lens[i];
        if (len >= 1 && len <= p.max_blocks * kPage) least = min(least, len);
      }
      least = __reduce_min_sync(kFull, least);
      if (lane == 0 && least != INT_MAX) atomicMin(&s_least, least);
      __syncthreads();
      if (s_least != INT_MAX) first = max(min(s_group.z, s_least), 0) / kPage;
    }
  }
  const bool bad = n < 1 || n > p.max_blocks * kPage, shares = first > 0 && !bad;
  // Q as the A operand of the four steps: head g8's dims 16 t4 + 4 s .. + 3
  uint32_t aq[4][4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (g8 < G) x = *reinterpret_cast<const float4*>(p.q_rot + (row0 + g8) * kHeadDim + 16 * t4 + 4 * s);
    x.x *= p.qscale;
    x.y *= p.qscale;
    x.z *= p.qscale;
    x.w *= p.qscale;
    aq[s][0] = pack_bf16x2(x.x, x.y);
    aq[s][2] = pack_bf16x2(x.z, x.w);
    const float2 r0 = bf16x2_to_float2(aq[s][0]), r1 = bf16x2_to_float2(aq[s][2]);
    aq[s][1] = pack_bf16x2(x.x - r0.x, x.y - r0.y);
    aq[s][3] = pack_bf16x2(x.z - r1.x, x.w - r1.y);
  }
  const float slope = p.slopes && g8 < G ? p.slopes[h * G + g8] * kLog2e : 0.f;
  if (bad && rank == 0 && tid == 0) atomicOr(p.err, PKV_ERR_SEQ_LEN);
  const int lo = kWindow ? max(n - p.window, 0) : 0;
  // pages first .. last - 1; none for a bad length
  first = max(first, lo / kPage);
  const int last = bad ? first : max((n + kPage - 1) / kPage, first);
  const bool alone = ctas == 1 || (last - first <= kWarps && !shares);
  if (alone && rank > 0) return;
  const int stride = alone ? kWarps : kWarps * ctas, turn = alone ? warp : rank * kWarps + warp;

  // This warp's pages, k = 0 .. count - 1: page first + turn + k stride. Their ids come
  // 32 at a time, the next 32 before they are due.
  const int count = first + turn < last ? (last - first - turn + stride - 1) / stride : 0;
  const int32_t* bt = p.block_tables + static_cast<size_t>(b) * p.max_blocks;
  auto ids_from = [&](int k) { return k + lane < count ? bt[first + turn + (k + lane) * stride] : -1; };
  int ids = ids_from(0), ids_next = ids_from(32);
  uint32_t there = 0, phase = 0;  // by stage: whether a copy was made; the phase to wait for
  auto issue = [&](int k) {  // (the whole warp)
    if (k >= count) return;
    if (k > 0 && (k & 31) == 0) {
      ids = ids_next;
      ids_next = ids_from(k + 32);
    }
    const int st = k % kStages, page = __shfl_sync(kFull, ids, k & 31);
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) atomicOr(p.err, PKV_ERR_PAGE_ID);
      there &= ~(1u << st);
      return;
    }
    there |= 1u << st;
    const uint32_t bar = smem_addr(&s_bar[warp][st]);
    mbar_arrive_expect_tx_elect(bar, kHeadPageBytes);
    tma_load_2d_elect(ring + st * kHeadPageBytes, &kv_map, 0, (page * p.hkv + h) * 2 * kPage, bar);
  };
#pragma unroll
  for (int k = 0; k < kStages; ++k) issue(k);

  float m_run = -INFINITY, l_run = 0.f;  // head g8: the maximum, and this lane's share of the sum
  float o[8][4];
#pragma unroll
  for (int d = 0; d < 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
  bool failed = false;
  for (int k = 0; k < count; ++k) {
    const int st = k % kStages;
    if ((there >> st) & 1u) {
      if (!mbar_wait_bounded(smem_addr(&s_bar[warp][st]), (phase >> st) & 1u)) failed = true;
      if (__any_sync(kFull, failed)) {
        failed = true;
        break;
      }
      phase ^= 1u << st;
      const int pg = first + turn + k * stride;
      const int from = lo - pg * kPage, to = n - pg * kPage;  // the page's visible slots: from .. to - 1
      const uint32_t page = ring + st * kHeadPageBytes;
      // 16-byte chunk c of row r of the page (K rows 0-15, V rows 16-31): swizzled
      auto chunk = [&](int r, int c) { return lds128(page + r * kRowBytes + ((c ^ (r & 7)) << 4)); };
      float sc[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
        const uint4 k0 = chunk(8 * j + g8, 2 * t4), k1 = chunk(8 * j + g8, 2 * t4 + 1);
        const uint32_t w[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
#pragma unroll
        for (int s = 0; s < 4; ++s) mma_bf16_16816(sc[j], aq[s], w[2 * s], w[2 * s + 1]);
      }
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = chunk(kPage + 2 * t4 + (i & 1) + 8 * (i >> 1), g8);
      // head g8, tokens 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9
      float x[4] = {sc[0][0] + sc[0][2], sc[0][1] + sc[0][3], sc[1][0] + sc[1][2], sc[1][1] + sc[1][3]};
      if (p.cap.cap > 0.f) {  // the scores are 2 log2(e) x
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = capped_score(p.cap, x[i]);
      }
      bool seen[4];
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int slot = 2 * t4 + (i & 1) + 8 * (i >> 1);
        seen[i] = slot >= from && slot < to;
        x[i] = seen[i] ? x[i] - slope * static_cast<float>(to - 1 - slot) : -INFINITY;
        mx = fmaxf(mx, x[i]);
      }
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
      const float mn = fmaxf(m_run, mx);
      const float keep = mn == m_run ? 1.f : fast_exp2(m_run - mn);
      const float ref = mn == -INFINITY ? 0.f : mn;
      float pr[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) pr[i] = fast_exp2(x[i] - ref);
      l_run = l_run * keep + ((pr[0] + pr[1]) + (pr[2] + pr[3]));
      m_run = mn;
      if (__any_sync(kFull, keep != 1.f)) {
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          o[d][0] *= keep;
          o[d][1] *= keep;
          o[d][2] *= keep;
          o[d][3] *= keep;
        }
      }
      uint32_t ap[4];
      ap[0] = pack_bf16x2(pr[0], pr[1]);
      ap[2] = pack_bf16x2(pr[2], pr[3]);
      const float2 f0 = bf16x2_to_float2(ap[0]), f1 = bf16x2_to_float2(ap[2]);
      ap[1] = pack_bf16x2(pr[0] - f0.x, pr[1] - f0.y);
      ap[3] = pack_bf16x2(pr[2] - f1.x, pr[3] - f1.y);
      if (from > 0 || to < kPage) {  // a slot that is not visible may hold anything
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!seen[i]) v[i] = make_uint4(0u, 0u, 0u, 0u);
      }
      const uint32_t v0[4] = {v[0].x, v[0].y, v[0].z, v[0].w}, v1[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
      const uint32_t v2[4] = {v[2].x, v[2].y, v[2].z, v[2].w}, v3[4] = {v[3].x, v[3].y, v[3].z, v[3].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // dims 2 i and 2 i + 1 of the lane's eight
        mma_bf16_16816(o[2 * i], ap, __byte_perm(v0[i], v1[i], 0x5410), __byte_perm(v2[i], v3[i], 0x5410));
        mma_bf16_16816(o[2 * i + 1], ap, __byte_perm(v0[i], v1[i], 0x7632), __byte_perm(v2[i], v3[i], 0x7632));
      }
    }
    __syncwarp();  // the stage is read
    issue(k + kStages);
  }
  if (failed) {  // the copies in flight land before shared memory goes away; the rows get what there is
    if (lane == 0) {
      atomicOr(p.err, PKV_ERR_TIMEOUT);
      for (int st = 0; st < kStages; ++st)
        if ((there >> st) & 1u) mbar_wait_bounded(smem_addr(&s_bar[warp][st]), (phase >> st) & 1u);
    }
    __syncwarp();
  }

  if (p.pieces.ctas > 0) {
    grid_dependency_wait();
    grid_launch_dependents();
  }
  if (shares) {
    // The shared pages' pieces: head g8's dims 16 t4 .. + 15, kAhead pieces asked for
    // together.
    const int4 tile = __ldcg(p.pieces.tiles + b);
    const PieceRange pieces = pieces_of(tile, __ldcg(&p.pieces.tiles[p.batch].x), p.pieces.ctas, p.hkv, h);
    constexpr int kAhead = 2;
    const long long at = (static_cast<long long>(h) * p.batch + b) * G + min(g8, G - 1);
    const float2* ml = p.pieces.ml + at;
    const float* po = p.pieces.o + at * kHeadDim + 16 * t4;
    for (int c = pieces.c0 + turn; c <= pieces.c1; c += kAhead * stride) {
      float2 t[kAhead];
      float4 v[kAhead][4];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        t[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
        const int ci = c + i * stride;
        if (ci <= pieces.c1 && has_piece(pieces, ci)) {
          t[i] = __ldcg(ml + 128ll * ci);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[i][j] = __ldcg(reinterpret_cast<const float4*>(po + 128ll * kHeadDim * ci) + j);
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float mn = fmaxf(m_run, t[i].x), ref = mn == -INFINITY ? 0.f : mn;
        const float a = fast_exp2(m_run - ref), w = fast_exp2(t[i].x - ref);
        m_run = mn;
        l_run = l_run * a + (t4 == 0 ? t[i].y * w : 0.f);
#pragma unroll
        for (int d = 0; d < 8; ++d) {
          const float4 x = v[i][d >> 2], y = v[i][2 + (d >> 2)];
          const float x0 = (d & 3) == 0 ? x.x : (d & 3) == 1 ? x.y : (d & 3) == 2 ? x.z : x.w;
          const float y0 = (d & 3) == 0 ? y.x : (d & 3) == 1 ? y.y : (d & 3) == 2 ? y.z : y.w;
          o[d][0] = o[d][0] * a + x0 * w;
          o[d][1] = o[d][1] * a + y0 * w;
          o[d][2] *= a;
          o[d][3] *= a;
        }
      }
    }
  }


  // the warps' sums, then the CTAs': o[d] holds dims 16 t4 + d and 16 t4 + 8 + d
  l_run += __shfl_xor_sync(kFull, l_run, 1);
  l_run += __shfl_xor_sync(kFull, l_run, 2);
  if (g8 < G) {
    if (t4 == 0) {
      s_m[warp][g8] = m_run;
      s_l[warp][g8] = l_run;
    }
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      acc(warp)[g8 * kHeadDim + 16 * t4 + d] = o[d][0] + o[d][2];
      acc(warp)[g8 * kHeadDim + 16 * t4 + 8 + d] = o[d][1] + o[d][3];
    }
  }
  __syncthreads();
  // element i of the segment's G rows: head g = i / 64, dim i % 64
  [[maybe_unused]] bool lost = false;
  auto finish = [&](int i, float sum, float total) {
    const float y = total == 0.f ? 0.f : sum / total;  // (a NaN score makes the row NaN)
    if constexpr (kWindow) lost |= !isfinite(y);
    if (p.out_bf16) {
      static_cast<uint16_t*>(p.out)[row0 * kHeadDim + i] = static_cast<uint16_t>(pack_bf16x2(y, 0.f));
    } else {
      static_cast<float*>(p.out)[row0 * kHeadDim + i] = y;
    }
  };
  for (int i = tid; i < G * kHeadDim; i += kThreads) {
    const int g = i / kHeadDim, d = i % kHeadDim;
    float mx = -INFINITY, sum = 0.f, total = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][g]);
    const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = fast_exp2(s_m[w][g] - ref);
      sum += f * acc(w)[i];
      total += f * s_l[w][g];
    }
    if (alone) {
      finish(i, sum, total);
    } else {
      c_acc[g][d] = sum;
      if (d == 0) {
        c_m[g] = mx;
        c_l[g] = total;
      }
    }
  }
  // whether elements e0 .. e1 - 1, this CTA's, need finish_alone, and that
  auto finish_lost = [&](int e0, int e1) {
    if constexpr (kWindow)
      if (__syncthreads_or(lost && shares)) finish_alone(p, b, h, e0, e1);
  };
  if (alone) {
    finish_lost(0, G * kHeadDim);
    return;
  }
  cluster.sync();
  // each CTA finishes its share of the rows
  const int share = (G * kHeadDim + ctas - 1) / ctas;
  for (int i = rank * share + tid; i < min((rank + 1) * share, G * kHeadDim); i += kThreads) {
    const int g = i / kHeadDim;
    float cm[kMaxCluster], cl[kMaxCluster], ca[kMaxCluster];
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      cm[r] = -INFINITY;
      cl[r] = ca[r] = 0.f;
      if (r < ctas) {
        cm[r] = cluster.map_shared_rank(c_m, r)[g];
        cl[r] = cluster.map_shared_rank(c_l, r)[g];
        ca[r] = cluster.map_shared_rank(&c_acc[0][0], r)[i];
      }
    }
    float mx = -INFINITY, sum = 0.f, total = 0.f;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) mx = fmaxf(mx, cm[r]);
    const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      const float f = fast_exp2(cm[r] - ref);
      sum += f * ca[r];
      total += f * cl[r];
    }
    finish(i, sum, total);
  }
  finish_lost(rank * share, min((rank + 1) * share, G * kHeadDim));
  cluster.sync();  // no CTA leaves while another reads its sums
}

cudaLaunchConfig_t config(cudaLaunchAttribute (&attr)[2], int segments, int ctas, cudaStream_t stream) {
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(segments * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kRing + 1024;  // + alignment to 1 KiB
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

// Clusters of `ctas` CTAs that run at once (fewer than the CTAs that fit over
// `ctas`: see decode_small.cu); -1: a CUDA call failed.
template <bool kWindow>
int clusters_at_once(int device, int ctas) {
  static std::atomic<int> cache[64][kMaxCluster + 1];  // found + 1
  std::atomic<int>& known = cache[device & 63][ctas];
  int n = known.load(std::memory_order_relaxed) - 1;
  if (n >= 0) return n;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = config(attr, 1, ctas, nullptr);
  cfg.numAttrs = 1;  // the cluster's
  if (cudaOccupancyMaxActiveClusters(&n, decode_rest_kernel<kWindow>, &cfg) != cudaSuccess) return -1;
  known.store(n + 1, std::memory_order_relaxed);
  return n;
}

template <bool kWindow>
cudaError_t launch(const CUtensorMap& kv_map, const RestParams& p, cudaStream_t stream) {
  static DeviceSetup setup;
  cudaError_t e = setup([] {
    cudaError_t e = cudaFuncSetAttribute(decode_rest_kernel<kWindow>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing + 1024);
    if (e != cudaSuccess) return e;
    // more CTAs a cluster than every GPU has to grant
    return cudaFuncSetAttribute(decode_rest_kernel<kWindow>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  int device = 0;
  if (e == cudaSuccess) e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const int segments = p.batch * p.hkv;
  // the most CTAs a segment with which all segments run at once, a power of two: 24
  // sequences of 2240 tokens in 2 CTAs a segment 19.0 us, in 3 23.0; 5 of 16040 in 8 20.7, in
  // 15 26.5; 20 of 2300 in 2 19.2, in 3 18.1 (32 + 8 heads, one prompt, both kernels)
  int ctas = p.max_blocks > kShortPages ? kMaxCluster : 8;
  for (; ctas > 1; ctas /= 2) {
    const int most = clusters_at_once<kWindow>(device, ctas);
    if (most < 0) return cudaGetLastError();
    if (segments <= most) break;
  }
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = config(attr, segments, ctas, stream);
  return cudaLaunchKernelEx(&cfg, decode_rest_kernel<kWindow>, kv_map, p);
}

}  // namespace

cudaError_t launch_decode_rest(const SharedLaunch& a, const SharedPieces& pieces, cudaStream_t stream) {
  constexpr double log2e = 1.4426950408889634;
  RestParams p = {};
  p.pool = a.pool;
  p.pool = a.pool;
  p.num_pages = a.num_pages;
  p.hkv = a.num_kv_heads;
  p.group = a.num_q_heads / a.num_kv_heads;
  p.q_rot = a.q_rot;
  p.out = a.out;
  p.block_tables = a.block_tables;
  p.max_blocks = a.max_blocks;
  p.seq_lens = a.seq_lens;
  p.batch = a.batch;
  p.slopes = a.slopes;
  p.window = a.window;
  p.qscale = static_cast<float>(a.softcap > 0.f ? 2.0 * a.scale / a.softcap * log2e : a.scale * log2e);
  p.cap = make_score_cap(a.softcap);
  p.out_bf16 = a.out_bf16;
  p.pieces = pieces;
  p.cu_groups = a.cu_groups;
  p.shared_lens = a.shared_lens;
  p.groups = a.groups;
  p.err = a.err;
  return a.window > 0 ? launch<true>(*a.kv_map, p, stream) : launch<false>(*a.kv_map, p, stream);
}

}  // namespace pkv
