// decode_small.cu -- the scored decode (paged_gqa_decode_scored) for little work:
// few (sequence, kv head) segments of few pages, where latency counts.
//
// The same formula as gqa_decode.cu's scored mode. There a launch passes through
// some 2000 instructions once (lengths, prefix sums, partition, TMA ring, merges
// in shared memory, then through the workspace), one latency after the other:
// 12 us for eight sequences of up to 2048 tokens and 32 + 8 heads, 6 us for
// sequences of one token. Here a segment is a cluster of 1 to 16 CTAs, as many as
// keep all clusters on the GPU at once; its warps take its pages in turn, and their
// pieces meet in shared memory, then across the cluster through distributed
// shared memory: no partition, no workspace, no spinning. A segment that one
// CTA's warps cover is done by its first CTA alone.
//
// A warp and a page: the operands of the tensor-core products come straight from
// global memory, 16 bytes a lane and load, because both contractions may take
// their index in any order. For S = Q K^T lane (g, t) loads dims 16 t .. + 15 of
// keys g and g + 8: step s of the contraction takes dims 16 t + 4 s .. + 3, in Q
// as in K. For O = P V it loads dims 8 g .. + 7 of tokens 2 t, 2 t + 1, 2 t + 8
// and 2 t + 9, and column n of product d is dim 8 n + d. Q (rows 0-7: heads) and
// P enter as bf16 with their remainders in rows 8-15, as in gqa_decode.cu. The
// next page's loads are in flight while a page is worked on.
#include <atomic>

#include <cooperative_groups.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "score_cap.cuh"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCluster = 16;
// Segments of up to this many pages take clusters of at most 8 CTAs: one
// sequence of 1024 tokens (64 pages) 4.8 us against 5.2 with 16, of 2048 6.0
// against 5.7, of 8192 12.0 against 9.3 (32 + 8 heads; with 14 + 2 5.0 / 4.9, 6.2 /
// 5.2, 12.1 / 8.3, but eight sequences of 2048 7.2 / 7.5).
constexpr int kShortPages = 160;
constexpr int kCtas = 3;  // CTAs a SM
constexpr float kLog2e = 1.4426950408889634f;

struct SmallParams {
  const uint8_t* pool;
  long long num_pages;
  int hkv;
  const float* q_rot;  // [batch][hq][64]
  void* out;           // [batch][hq][64], fp32 or bf16
  const int32_t* block_tables;
  int max_blocks;
  const int32_t* seq_lens;
  const int32_t* first_keys;  // [batch] or null
  const float* slopes;        // [hq] or null
  int window;                 // 0: none
  float qscale;               // scores in base 2, or 2 log2(e) x when capped
  ScoreCap cap;
  int out_bf16;
  int* err;
};

// What a lane holds of a page: keys g and g + 8 (dims 16 t .. + 15), and the
// four value rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9 (dims 8 g .. + 7).
struct PageRegs {
  uint4 k[2][2], v[4];
};

template <int G>
__global__ void __launch_bounds__(kThreads, kCtas) decode_small_kernel(const SmallParams p) {
  __shared__ float s_acc[kWarps][G][kHeadDim], s_m[kWarps][G], s_l[kWarps][G];
  __shared__ float c_acc[G][kHeadDim], c_m[G], c_l[G];  // the CTA's piece
  const cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), ctas = static_cast<int>(cluster.num_blocks());
  const int sg = blockIdx.x / ctas, b = sg / p.hkv, h = sg - b * p.hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g8 = lane >> 2, t4 = lane & 3;
  const size_t row0 = static_cast<size_t>(sg) * G;  // b hq + h G
  // the next kernel may start once every kernel before this one is complete
  grid_dependency_wait();
  grid_launch_dependents();
  const int n = p.seq_lens[b];
  int lo = p.window > 0 ? max(n - p.window, 0) : 0;
  if (p.first_keys) lo = max(lo, p.first_keys[b]);
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
  const bool bad = n < 1 || n > p.max_blocks * kPage;
  if (bad && rank == 0 && tid == 0) atomicOr(p.err, PKV_ERR_SEQ_LEN);
  // pages first .. last - 1; none for a bad length or when no key is visible
  const int first = lo / kPage, last = bad || lo >= n ? first : (n + kPage - 1) / kPage;
  const bool alone = last - first <= kWarps || ctas == 1;
  if (alone && rank > 0) return;

  float m_run = -INFINITY, l_run = 0.f;  // head g8: the maximum, and this lane's share of the sum
  float o[8][4];
#pragma unroll
  for (int d = 0; d < 8; ++d) o[d][0] = o[d][1] = o[d][2] = o[d][3] = 0.f;
  const int32_t* bt = p.block_tables + static_cast<size_t>(b) * p.max_blocks;
  const int stride = alone ? kWarps : kWarps * ctas;
  auto page_at = [&](int pg) { return pg < last ? bt[pg] : -1; };
  auto usable = [&](int page) { return page >= 0 && page < p.num_pages; };
  auto load = [&](int page, PageRegs& r) {
    if (!usable(page)) return;
    const uint8_t* base = p.pool + (static_cast<size_t>(page) * p.hkv + h) * kHeadPageBytes;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        r.k[j][i] = *reinterpret_cast<const uint4*>(base + (8 * j + g8) * kRowBytes + 32 * t4 + 16 * i);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r.v[i] = *reinterpret_cast<const uint4*>(base + kHalfBytes + (2 * t4 + (i & 1) + 8 * (i >> 1)) * kRowBytes + 16 * g8);
  };
  auto work = [&](int pg, int page, PageRegs& r) {
    if (!usable(page)) {
      if (lane == 0) atomicOr(p.err, PKV_ERR_PAGE_ID);
      return;
    }
    const int from = lo - pg * kPage, to = n - pg * kPage;  // the page's visible slots: from .. to - 1
    float sc[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
      const uint32_t w[8] = {r.k[j][0].x, r.k[j][0].y, r.k[j][0].z, r.k[j][0].w,
                             r.k[j][1].x, r.k[j][1].y, r.k[j][1].z, r.k[j][1].w};
#pragma unroll
      for (int s = 0; s < 4; ++s) mma_bf16_16816(sc[j], aq[s], w[2 * s], w[2 * s + 1]);
    }
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
        if (!seen[i]) r.v[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    const uint32_t v0[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w}, v1[4] = {r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
    const uint32_t v2[4] = {r.v[2].x, r.v[2].y, r.v[2].z, r.v[2].w}, v3[4] = {r.v[3].x, r.v[3].y, r.v[3].z, r.v[3].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // dims 2 i and 2 i + 1 of the lane's eight
      mma_bf16_16816(o[2 * i], ap, __byte_perm(v0[i], v1[i], 0x5410), __byte_perm(v2[i], v3[i], 0x5410));
      mma_bf16_16816(o[2 * i + 1], ap, __byte_perm(v0[i], v1[i], 0x7632), __byte_perm(v2[i], v3[i], 0x7632));
    }
  };
  {
    int pg = first + (alone ? warp : rank * kWarps + warp);
    int page = page_at(pg), next = page_at(pg + stride);
    PageRegs r[2];
    load(page, r[0]);
    while (pg < last) {  // two pages a turn, so that the register sets stay where they are
      int after = page_at(pg + 2 * stride);
      load(next, r[1]);
      work(pg, page, r[0]);
      pg += stride;
      if (pg >= last) break;
      page = after;
      after = page_at(pg + 2 * stride);
      load(page, r[0]);
      work(pg, next, r[1]);
      pg += stride;
      next = after;
    }
  }

  // the warps' pieces, then the CTAs': o[d] holds dims 16 t4 + d and 16 t4 + 8 + d
  l_run += __shfl_xor_sync(kFull, l_run, 1);
  l_run += __shfl_xor_sync(kFull, l_run, 2);
  if (g8 < G) {
    if (t4 == 0) {
      s_m[warp][g8] = m_run;
      s_l[warp][g8] = l_run;
    }
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      s_acc[warp][g8][16 * t4 + d] = o[d][0] + o[d][2];
      s_acc[warp][g8][16 * t4 + 8 + d] = o[d][1] + o[d][3];
    }
  }
  __syncthreads();
  // element i of the segment's G rows: head g = i / 64, dim i % 64
  auto finish = [&](int i, float sum, float total) {
    const float y = total == 0.f ? 0.f : sum / total;  // (a NaN score makes the row NaN)
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
      sum += f * s_acc[w][g][d];
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
  if (alone) return;
  cluster.sync();
  // each CTA finishes its share of the rows
  const int share = (G * kHeadDim + ctas - 1) / ctas;
  for (int i = rank * share + tid; i < min((rank + 1) * share, G * kHeadDim); i += kThreads) {
    const int g = i / kHeadDim, d = i % kHeadDim;
    float cm[kMaxCluster], cl[kMaxCluster], ca[kMaxCluster];
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      cm[r] = -INFINITY;
      cl[r] = ca[r] = 0.f;
      if (r < ctas) {
        cm[r] = cluster.map_shared_rank(c_m, r)[g];
        cl[r] = cluster.map_shared_rank(c_l, r)[g];
        ca[r] = cluster.map_shared_rank(&c_acc[0][0], r)[g * kHeadDim + d];
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
  cluster.sync();  // no CTA leaves while another reads its piece
}

// Clusters of `ctas` CTAs that run at once. (SMs come in groups of which a
// cluster takes one, so this is less than the CTAs that fit over `ctas`: 64
// clusters of 7 do not fit beside one another although their CTAs would, and
// take 13 us where 64 of 4 take 10.)
template <int G>
int clusters_at_once(int device, int ctas) {
  static std::atomic<int> cache[64][kMaxCluster + 1];  // found + 1
  std::atomic<int>& known = cache[device & 63][ctas];
  int n = known.load(std::memory_order_relaxed) - 1;
  if (n >= 0) return n;
  if (ctas > 8) {  // more than every GPU has to grant
    const cudaError_t e =
        cudaFuncSetAttribute(decode_small_kernel<G>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return -1;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, decode_small_kernel<G>, &cfg) != cudaSuccess) return -1;
  known.store(n + 1, std::memory_order_relaxed);
  return n;
}

template <int G>
cudaError_t launch(const SmallParams& p, int segments, int most_ctas, int device, cudaStream_t stream) {
  // the most CTAs a segment with which all segments run at once
  int ctas = most_ctas;
  for (; ctas > 1; --ctas) {
    const int most = clusters_at_once<G>(device, ctas);
    if (most < 0) return cudaGetLastError();
    if (segments <= most) break;
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(segments * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, decode_small_kernel<G>, p);
}

}  // namespace

// Little work, as far as the host can tell: the pages that the block tables (or
// the window) can hold, over all segments, and of one segment. Measured against
// the general kernel (lengths between half and all of what the tables hold), 32 +
// 8 heads: 3.9 against 6.2 us for 8 sequences of one token, 9.3 / 12.6 for 8 of
// 2048 (8192 pages in all), 12.3 / 15.8 for 16 of 2048 and 13.4 / 15.6 for 32 of
// 1024 (16384), but 26.2 / 21.8 for 32 of 2048 (32768), where an even partition of
// all pages counts. 14 + 2 heads, 2048 pages a segment: 20.0 / 53.5 for one
// sequence, 21.8 / 28.2 for four; 4096 pages: 35.4 / 43.9 and 48.9 / 37.0.
constexpr long long kMostPages = 20480, kMostSegmentPages = 2048;
static int segment_pages(const DecodeLaunch& a) {
  return a.window > 0 && a.window / kPage + 2 < a.max_blocks ? a.window / kPage + 2 : a.max_blocks;
}
bool decode_small_fits(const DecodeLaunch& a) {
  const long long pages = segment_pages(a);
  return pages <= kMostSegmentPages && pages * a.batch * a.num_kv_heads <= kMostPages;
}

cudaError_t launch_decode_small(const DecodeLaunch& a, cudaStream_t stream) {
  constexpr double log2e = 1.4426950408889634;
  SmallParams p;
  p.pool = a.pool;
  p.num_pages = a.num_pages;
  p.hkv = a.num_kv_heads;
  p.q_rot = a.q_rot;
  p.out = a.out;
  p.block_tables = a.block_tables;
  p.max_blocks = a.max_blocks;
  p.seq_lens = a.seq_lens;
  p.first_keys = a.first_keys;
  p.slopes = a.slopes;
  p.window = a.window;
  p.qscale = static_cast<float>(a.softcap > 0.f ? 2.0 * a.scale / a.softcap * log2e : a.scale * log2e);
  p.cap = make_score_cap(a.softcap);
  p.out_bf16 = a.out_bf16;
  p.err = a.err;
  const int segments = a.batch * a.num_kv_heads;
  int device = 0;
  const cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const int most_ctas = segment_pages(a) > kShortPages ? kMaxCluster : 8;
  switch (a.num_q_heads / a.num_kv_heads) {
    case 1: return launch<1>(p, segments, most_ctas, device, stream);
    case 2: return launch<2>(p, segments, most_ctas, device, stream);
    case 3: return launch<3>(p, segments, most_ctas, device, stream);
    case 4: return launch<4>(p, segments, most_ctas, device, stream);
    case 5: return launch<5>(p, segments, most_ctas, device, stream);
    case 6: return launch<6>(p, segments, most_ctas, device, stream);
    case 7: return launch<7>(p, segments, most_ctas, device, stream);
    case 8: return launch<8>(p, segments, most_ctas, device, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pkv
