// step_tables.cu -- a step's block tables, slot maps and positions, built on
// the GPU from the requests' lengths.
//
// Sequence b has s_b cached tokens and brings n_b new ones. Its pages reach
// block ceil(s/16) and must reach ceil((s+n)/16): need_b blocks more in every
// layer. With base_b the sum of need over the sequences before b, block
// ceil(s_b/16) + i of (layer l, sequence b) takes entry
//     head + base_b * L + l * need_b + i
// of the list of free pages, and token t of the step (sequence b, position
// p = s_b + t - cu_b) goes to slot table[l][b][p / 16] * 16 + p % 16 of layer l.
//
// The work is a few KB to a few MB of writes behind two prefix sums over the
// batch, so it is bound by latency: one launch, in which every CTA repeats the
// two sums in shared memory (2 B integers, a few hundred cycles) instead of
// waiting for one CTA to publish them. No CTA reads what another writes: a
// slot of a new page takes its page from the free list, by the formula above,
// not from the table entry that another CTA stores, and arrays that overlap one
// that is written are refused. Measured in graph
// replays (and as calls one after the other, which the host's 3 us a call and
// the launch set): 3.3 us (5.1) for 64 decoding sequences and 16 layers, 4.0 us
// (6.1) for 256 sequences (12 of them prompts), 24 layers and 12000 tokens.
#include <cerrno>
#include <climits>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kTablesThreads = 256;
constexpr int kTablesWarps = kTablesThreads / 32;
constexpr int kMostTokens = (1 << 30) - 1;  // token counts stop here
constexpr int kAtOnce = 4;                  // layers whose pages a token asks for together

struct TablesParams {
  long long num_pages;
  const int32_t* start_pos;
  const int32_t* new_tokens;
  int batch, num_layers;
  const int32_t* free_pages;
  int num_free;
  const int32_t* free_head;
  int32_t* free_head_out;
  int32_t* block_tables;  // [L][B][max_blocks]
  int max_blocks;
  int32_t* cu_tokens;  // [B + 1]
  int32_t* seq_lens;   // [B]
  int32_t* positions;  // [capacity]
  int32_t* slot_map;   // [L][capacity]
  int capacity;
  int layers_per_cta;
  int* err;
};

// Inclusive prefix sum over the CTA of one value a thread, sums above `cap`
// held at cap (adding non-negative numbers with saturation is associative).
// Either cap is below 2^30 or the sums are below 2^31 by themselves, so
// nothing overflows.
__device__ __forceinline__ int block_scan(int x, int cap, int* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x = min(x + t, cap);
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int w = 0; w < kTablesWarps; ++w)
    if (w < warp) before = min(before + s_warp[w], cap);
  __syncthreads();
  return min(x + before, cap);
}

// Largest i in [0, n) with a[i] <= x (a[0] <= x, a non-decreasing).
__device__ __forceinline__ int last_at_most(const int* a, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kTablesThreads) step_tables_kernel(const TablesParams p) {
  extern __shared__ int s_tab[];
  int* s_start = s_tab;              // [B] cached tokens; -1: the sequence is refused
  int* s_cu = s_start + p.batch;     // [B + 1] first token of each sequence
  int* s_base = s_cu + p.batch + 1;  // [B + 1] new pages (of one layer) before each sequence
  __shared__ int s_warp[kTablesWarps];
  const int tid = threadIdx.x;
  const bool first_cta = blockIdx.x == 0 && blockIdx.y == 0;
  const int head = *p.free_head;
  const bool head_ok = head >= 0 && head <= p.num_free;
  const int room = head_ok ? (p.num_free - head) / p.num_layers : 0;
  const long long cap = static_cast<long long>(p.max_blocks) * kPage;

  // The two prefix sums, kTablesThreads sequences at a time.
  int tokens = 0, pages = 0, bits = head_ok ? 0 : PKV_ERR_NO_PAGES;
  for (int b0 = 0; b0 < p.batch; b0 += kTablesThreads) {
    const int b = b0 + tid;
    const bool in = b < p.batch;
    const int s = in ? p.start_pos[b] : 0, raw = in ? p.new_tokens[b] : 0;
    const int n = min(max(raw, 0), kMostTokens);
    const int end = block_scan(min(n + (tid == 0 ? tokens : 0), kMostTokens), kMostTokens, s_warp);
    const bool ok = s >= 0 && raw >= 0 && static_cast<long long>(s) + raw <= cap && end <= p.capacity;
    const int need = ok ? (s + n + kPage - 1) / kPage - (s + kPage - 1) / kPage : 0;
    const int upto = block_scan(need + (tid == 0 ? pages : 0), INT_MAX, s_warp);
    // sequences are served in order while their pages fit
    const bool fits = need == 0 || upto <= room;
    if (in) {
      s_start[b] = ok && fits ? s : -1;
      s_cu[b + 1] = end;
      s_base[b + 1] = upto;
      if (!ok) bits |= PKV_ERR_SEQ_LEN;
      if (!fits) bits |= PKV_ERR_NO_PAGES;
      if (first_cta) {
        p.cu_tokens[b + 1] = end;
        p.seq_lens[b] = ok && fits ? s + n : max(s, 0);
      }
    }
    if (tid == kTablesThreads - 1) {  // the running totals, to the next round's first thread
      s_warp[0] = end;
      s_warp[1] = upto;
    }
    __syncthreads();
    tokens = s_warp[0];
    pages = s_warp[1];
    __syncthreads();
  }
  if (tid == 0) {
    s_cu[0] = 0;
    s_base[0] = 0;
  }
  __syncthreads();
  // Pages handed out: all of them, or those of the served sequences, which
  // come before the first one that did not fit.
  int served = pages;
  if (pages > room) {
    const int b = last_at_most(s_base, p.batch + 1, room);
    served = s_base[b];
  }
  if (first_cta) {
    if (tid == 0) {
      p.cu_tokens[0] = 0;
      *p.free_head_out = head_ok ? head + served * p.num_layers : head;
    }
    if (bits) atomicOr(p.err, bits);
  }

  // Entry r of the pages handed out goes to the tables, all CTAs together, after
  // the slots below; this thread's first one is asked for now.
  const int ctas = gridDim.x * gridDim.y, handed = served * p.num_layers;
  const int r0 = (blockIdx.y * gridDim.x + blockIdx.x) * kTablesThreads + tid;
  const int given = r0 < handed ? __ldg(p.free_pages + head + r0) : 0;
  auto checked = [&](int page) {  // -1 (reported) for an id outside the pool
    const bool good = page >= 0 && page < p.num_pages;
    if (!good) atomicOr(p.err, PKV_ERR_PAGE_ID);
    return good ? page : -1;
  };

  // Positions and slots: one token a thread, its layers in a loop, the pages of
  // kAtOnce of them asked for together (one after the other they took 5.5 us
  // instead of 4.2, in replays, for 256 sequences, 24 layers and 12000 tokens).
  const int t = blockIdx.x * kTablesThreads + tid;
  if (t < p.capacity) {
    const int l0 = blockIdx.y * p.layers_per_cta, l1 = min(l0 + p.layers_per_cta, p.num_layers);
    int b = -1, s = -1;
    if (p.batch > 0 && t < s_cu[p.batch]) {
      b = last_at_most(s_cu, p.batch, t);
      s = s_start[b];
    }
    const int pos = s < 0 ? 0 : s + (t - s_cu[b]);
    // layer l's page: a new one, or the table's
    const int32_t* pages_of = nullptr;
    size_t stride = 0;
    if (s >= 0) {
      const int fresh = pos / kPage - (s + kPage - 1) / kPage;  // the page's place among the sequence's new ones
      if (fresh >= 0) {
        pages_of = p.free_pages + head + s_base[b] * p.num_layers + fresh;
        stride = s_base[b + 1] - s_base[b];
      } else {
        pages_of = p.block_tables + static_cast<size_t>(b) * p.max_blocks + pos / kPage;
        stride = static_cast<size_t>(p.batch) * p.max_blocks;
      }
    }
    for (int l = l0; l < l1; l += kAtOnce) {
      int page[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) page[i] = s >= 0 && l + i < l1 ? pages_of[(l + i) * stride] : -1;
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        if (l + i >= l1) break;
        const int good = s >= 0 ? checked(page[i]) : -1;
        p.slot_map[static_cast<size_t>(l + i) * p.capacity + t] = good >= 0 ? good * kPage + pos % kPage : -1;
      }
    }
    if (blockIdx.y == 0) p.positions[t] = pos;
  }

  for (int r = r0; r < handed; r += ctas * kTablesThreads) {
    const int b = last_at_most(s_base, p.batch, r / p.num_layers);
    const int need = s_base[b + 1] - s_base[b], off = r - s_base[b] * p.num_layers;
    const int layer = off / need, i = off - layer * need;
    p.block_tables[(static_cast<size_t>(layer) * p.batch + b) * p.max_blocks + (s_start[b] + kPage - 1) / kPage + i] =
        checked(r == r0 ? given : __ldg(p.free_pages + head + r));
  }
}

// Whether one of the arrays that a step writes shares a word with another of
// its arrays. Every CTA reads all lengths, at its own time, while the first one
// writes the new lengths (and all read free_head), so none may be updated in
// place.
bool tables_overlap(const TablesParams& p) {
  struct Range {
    const int32_t* first;
    long long n;
  };
  const long long layers = p.num_layers;
  const Range r[] = {{p.free_head_out, 1},
                     {p.block_tables, layers * p.batch * p.max_blocks},
                     {p.cu_tokens, p.batch + 1ll},
                     {p.seq_lens, p.batch},
                     {p.positions, p.capacity},
                     {p.slot_map, layers * p.capacity},
                     {p.start_pos, p.batch},  // the rest is only read
                     {p.new_tokens, p.batch},
                     {p.free_pages, p.num_free},
                     {p.free_head, 1}};
  constexpr int kWritten = 6, kAll = sizeof(r) / sizeof(r[0]);
  for (int i = 0; i < kWritten; ++i)
    for (int j = i + 1; j < kAll; ++j) {
      const uintptr_t a = reinterpret_cast<uintptr_t>(r[i].first), b = reinterpret_cast<uintptr_t>(r[j].first);
      if (r[i].n > 0 && r[j].n > 0 && a < b + sizeof(int32_t) * r[j].n && b < a + sizeof(int32_t) * r[i].n) return true;
    }
  return false;
}

size_t tables_smem(int batch) { return sizeof(int) * (3 * static_cast<size_t>(batch) + 2); }

}  // namespace
}  // namespace pkv

extern "C" int paged_tables_build(pkv_pool_t* pool, const int32_t* start_pos, const int32_t* new_tokens,
                                  int batch, int num_layers, const int32_t* free_pages, int num_free,
                                  const int32_t* free_head, int32_t* free_head_out, int32_t* block_tables,
                                  int max_blocks, int32_t* cu_tokens, int32_t* seq_lens, int32_t* positions,
                                  int32_t* slot_map, int capacity, void* stream) {
  using namespace pkv;
  if (!pool || batch < 0 || batch > PKV_TABLES_MAX_BATCH || num_layers < 1 || num_free < 0 || max_blocks < 1 ||
      capacity < 0 || capacity >= (1 << 29))
    return -EINVAL;
  if (static_cast<long long>(batch) * max_blocks >= (1ll << 31) ||
      static_cast<long long>(max_blocks) * kPage >= (1ll << 31))
    return -EINVAL;
  if (!free_head || !free_head_out || !cu_tokens) return -EINVAL;
  if ((num_free > 0 && !free_pages) || (capacity > 0 && (!positions || !slot_map))) return -EINVAL;
  if (batch > 0 && (!start_pos || !new_tokens || !block_tables || !seq_lens)) return -EINVAL;
  TablesParams p;
  p.num_pages = pool->num_pages;
  p.start_pos = start_pos;
  p.new_tokens = new_tokens;
  p.batch = batch;
  p.num_layers = num_layers;
  p.free_pages = free_pages;
  p.num_free = num_free;
  p.free_head = free_head;
  p.free_head_out = free_head_out;
  p.block_tables = block_tables;
  p.max_blocks = max_blocks;
  p.cu_tokens = cu_tokens;
  p.seq_lens = seq_lens;
  p.positions = positions;
  p.slot_map = slot_map;
  p.capacity = capacity;
  p.err = pool->d_err;
  if (tables_overlap(p)) return -EINVAL;
  if (const int rc = check_pool_device(pool)) return rc;
  const size_t smem = tables_smem(batch);
  if (smem > 48u * 1024u) {
    const cudaError_t e = cudaFuncSetAttribute(step_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(tables_smem(PKV_TABLES_MAX_BATCH)));
    if (e != cudaSuccess) {
      record_cuda_error(e);
      return -EIO;
    }
  }
  // A layer to each CTA while that leaves no SM with more than about two,
  // then several layers to a CTA, so that the prefix sums are not repeated
  // more often than they need be.
  const int sms = device_sm_count(pool->device);
  const int gx = capacity > 0 ? (capacity + kTablesThreads - 1) / kTablesThreads : 1;
  const long long all = static_cast<long long>(gx) * num_layers;
  const long long want = sms > 0 ? 2ll * sms : 1;
  p.layers_per_cta = static_cast<int>((all + want - 1) / want);
  if (p.layers_per_cta > num_layers) p.layers_per_cta = num_layers;
  const int gy = (num_layers + p.layers_per_cta - 1) / p.layers_per_cta;
  if (gy > 65535) return -EINVAL;
  step_tables_kernel<<<dim3(gx, gy), kTablesThreads, smem, static_cast<cudaStream_t>(stream)>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return -EIO;
  }
  return 0;
}
