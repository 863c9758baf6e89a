// page_moves.cu -- sequences that go on from others, and held pages moved to the
// front of the pool: block tables, reference counts, free list and page contents,
// all on the GPU.
//
// shares[p] is the number of holders of page p beyond its first: 0 for a page
// that one sequence holds and for one that nobody does.
//
// Fork. Child b goes on from sequence a(b) of n_a tokens. It shares a's full pages
// by reference. A part-filled last page stays with a's first child; every other
// child gets a copy of its n_a % 16 filled slots in a page of its own. With c_a
// the children of a,
//     shares'[p] = shares[p] + sum over a holding p of (c_a - 1)
// (for a's part-filled page: -1 where c_a = 0, else 0), and a page where that
// comes to -1 has lost its last holder: it goes back to the list, in the order of
// the ids, before the list's next entry. Three launches: tables, copies and the
// changes of the counts (commutative sums, so their order does not show); the
// pages given back, counted by chunks; counts and list written. Little work in a
// small pool is one launch of one cluster, which meets where a launch would end.
//
// Compaction. U pages are held. The k-th held page with an id of U or more moves
// to the k-th listed page with an id below U. Four launches: pages marked; marks
// counted by chunks; movers and places ranked; contents, tables, counts and list
// written. Here too the first three are one cluster for little work.
//
// Measured in graph replays: a fork of 4 beams in a pool of 2500 pages 6.3 us (in others:
// see kForkUnits), of 64 x 4 (16 layers, 8 kv heads; 40 MB of tables, counts and copies)
// 14.9, of 16 prompts into 8 each (24 layers) 11.9: launches and, in each kernel, two or
// three reads one after the other. What the list kernel reads is asked for together, and the list is copied by CTAs of its own beside
// those that write the counts (one after the other in the same CTAs: 9.1, 18.8 and 15.1
// us). Compaction of half a pool (18144 pages held, 11400 of 32 KB moved) 128 us, of
// which the contents are 113 (5.9 TB/s read and written, 88% of a copy's rate); of 8
// sequences 16.
#include <atomic>
#include <cerrno>
#include <climits>

#include <cooperative_groups.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

namespace cg = cooperative_groups;

constexpr int kMoveThreads = 256;
constexpr int kMoveWarps = kMoveThreads / 32;
constexpr int kMoveCtas = 4;     // CTAs a SM of the launches that copy
constexpr int kWarpPages = 256;  // consecutive pages that a warp looks at: a ballot for each 32
constexpr int kBallots = kWarpPages / 32;
constexpr int kRoundPages = kMoveWarps * kWarpPages;  // 2048
constexpr int kMaxChunks = 1024;
constexpr int kCluster = 16;  // CTAs of the launches that are one cluster
constexpr int kMaxLayers = 4096;  // (rows of the tables are counted in 32 bits)

// The pages cut into at most kMaxChunks chunks of whole rounds.
struct Chunks {
  long long pages;
  int rounds, n;
  explicit Chunks(long long num_pages) : pages(num_pages) {
    rounds = static_cast<int>((num_pages + static_cast<long long>(kRoundPages) * kMaxChunks - 1) /
                              (static_cast<long long>(kRoundPages) * kMaxChunks));
    const long long size = static_cast<long long>(rounds) * kRoundPages;
    n = static_cast<int>((num_pages + size - 1) / size);
  }
};

// The workspace: a word, a word's chunk counts and what each operation keeps a
// page. `change`, and the marks, are zero between calls; nothing else is, and they are
// counted from the front, the rest from the back. So calls for pools of any sizes (of n
// and N pages, n < N) leave what the others need at zero alone: zero up to a place that
// grows with the pages, anything from one that falls with them, and those of N do not meet.
struct PagesWorkspace {
  size_t head, counts, change, marks, ranks, movers, places, bytes;
  // `given`: the bytes that the caller has, the least where it is 0.
  explicit PagesWorkspace(long long pages, size_t given = 0) {
    auto align256 = [](size_t n) { return (n + 255) / 256 * 256; };
    const size_t n = static_cast<size_t>(pages), words = align256(sizeof(int) * n);
    head = 0;
    counts = 256;
    change = counts + sizeof(int2) * kMaxChunks;
    marks = change + words;
    bytes = marks + align256(2 * n) + 3 * words;
    places = (given > bytes ? given / 256 * 256 : bytes) - words;
    movers = places - words;
    ranks = movers - words;
  }
};

// The rows of the tables are taken in parts of 128 entries, a part a warp at a time,
// four entries a lane asked for together (a long sequence's row by one warp: 70 us
// for the 2500 blocks of a compaction's only one, 22 for a fork of 30000 tokens).
constexpr int kPart = 128, kPartLoads = kPart / 32;
struct RowPart {
  int row, at;  // its first entry
  __device__ RowPart(long long u, int parts) : row(static_cast<int>(u / parts)), at(kPart * static_cast<int>(u % parts)) {}
};
__host__ __device__ __forceinline__ int parts_of(int entries) { return static_cast<int>((static_cast<uint32_t>(entries) + kPart - 1) / kPart); }

// Exclusive prefix sum over the CTA of one value a thread, and the total (s_warp
// is free again when all threads have returned and met).
__device__ __forceinline__ int block_before(int x, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int upto = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(kFull, upto, o);
    if (lane >= o) upto += t;
  }
  if (lane == 31) s_warp[warp] = upto;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kMoveWarps; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
  __syncthreads();
  return before + upto - x;
}

// `bytes` (a multiple of 128) from one place of the pool to another, by a warp.
__device__ __forceinline__ void warp_copy(uint8_t* to, const uint8_t* from, int bytes, int lane) {
  constexpr int kAhead = 8;
  for (int at = 16 * lane; at < bytes; at += 512 * kAhead) {
    uint4 w[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (at + 512 * i < bytes) w[i] = __ldcs(reinterpret_cast<const uint4*>(from + at + 512 * i));
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (at + 512 * i < bytes) __stcs(reinterpret_cast<uint4*>(to + at + 512 * i), w[i]);
  }
}

// ---------------------------------------------------------------------------
// fork

struct ForkParams {
  uint8_t* pool;
  long long num_pages;
  int hkv;
  const int32_t* parents;  // [children]
  int children;
  const int32_t* seq_lens;  // [batch]
  int batch, num_layers;
  const int32_t* tables;  // [L][batch][max_blocks]
  int max_blocks;
  const int32_t* shares;  // [num_pages]
  const int32_t* free_pages;
  int num_free;
  const int32_t* free_head;
  int32_t* tables_out;  // [L][children][max_blocks]
  int32_t* lens_out;    // [children]
  int32_t* shares_out;
  int32_t* list_out;
  int32_t* head_out;
  int* taken;   // pages taken off the list by the first launch
  int* counts;  // pages given back, by chunk
  int chunks, rounds;
  int* change;  // of a page's count; zero between calls
  int* err;
};

// The two halves of a barrier of the cluster.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait;" ::: "memory"); }

__device__ __forceinline__ int blocks_of(int tokens) { return tokens / kPage + (tokens % kPage != 0); }

__device__ __forceinline__ void fork_tables(const ForkParams& p, int* s_fork) {
  int* s_first = s_fork;               // [batch] a parent's first child
  int* s_count = s_first + p.batch;    // [batch] its children
  int* s_len = s_count + p.batch;      // [batch] tokens, -1: bad
  int* s_rank = s_len + p.batch;       // [children] a child's place among those that get a copy, -1: none, -2: not served
  int* s_copy = s_rank + p.children;   // [children] the parents of the children that get one, in order
  int* s_parent = s_copy + p.children;  // [children]
  __shared__ int s_warp[kMoveWarps];
  const int tid = threadIdx.x, lane = tid & 31;
  const bool first_cta = blockIdx.x == 0;
  // (what the first rounds read is asked for together)
  const int head = *p.free_head, len0 = tid < p.batch ? p.seq_lens[tid] : 0, parent0 = tid < p.children ? p.parents[tid] : 0;
  const bool head_ok = head >= 0 && head <= p.num_free;
  const int room = head_ok ? (p.num_free - head) / p.num_layers : 0;
  int bits = head_ok ? 0 : PKV_ERR_NO_PAGES;
  for (int a = tid; a < p.batch; a += kMoveThreads) {
    const int n = a == tid ? len0 : p.seq_lens[a];
    const bool ok = n >= 0 && n <= static_cast<long long>(p.max_blocks) * kPage;
    if (!ok) bits |= PKV_ERR_SEQ_LEN;
    s_len[a] = ok ? n : -1;
    s_first[a] = INT_MAX;
    s_count[a] = 0;
  }
  __syncthreads();
  for (int b = tid; b < p.children; b += kMoveThreads) {
    const int a = b == tid ? parent0 : p.parents[b];
    if (a < -1 || a >= p.batch) bits |= PKV_ERR_PARENT;
    if (a >= 0 && a < p.batch) atomicMin(&s_first[a], b);
    s_parent[b] = a;
  }
  __syncthreads();
  int copies = 0;  // of the children before this round's
  for (int b0 = 0; b0 < p.children; b0 += kMoveThreads) {
    const int b = b0 + tid;
    const int a = b < p.children ? s_parent[b] : -1;
    const bool there = a >= 0 && a < p.batch && s_len[a] >= 0;
    const bool copy = there && s_len[a] % kPage != 0 && s_first[a] != b;
    int total;
    const int rank = copies + block_before(copy, s_warp, total);
    const bool served = there && (!copy || rank < room);
    if (there && !served) bits |= PKV_ERR_NO_PAGES;
    if (b < p.children) {
      s_rank[b] = !served ? -2 : copy ? rank : -1;
      if (served && copy) s_copy[rank] = a;
      if (served) atomicAdd(&s_count[a], 1);
      if (first_cta) p.lens_out[b] = served ? s_len[a] : 0;
    }
    copies += total;
  }
  __syncthreads();
  copies = min(copies, room);
  if (first_cta) {
    if (tid == 0) *p.taken = copies * p.num_layers;
    if (bits) atomicOr(p.err, bits);
  }

  const int w0 = blockIdx.x * kMoveWarps + (tid >> 5), warps = gridDim.x * kMoveWarps;
  auto usable = [&](int page) { return page >= 0 && page < p.num_pages; };
  auto row = [&](int layer, int a) { return p.tables + (static_cast<size_t>(layer) * p.batch + a) * p.max_blocks; };
  // The copies, a kv head's slots a warp, keys and values; the next one's pages are
  // asked for before this one's slots.
  const int units = copies * p.num_layers * p.hkv;
  struct Copy {
    int from, to, h, bytes;
  };
  auto copy_of = [&](int u) {
    Copy c = {-1, -1, 0, 0};
    if (u < units) {
      const int rest = u / p.hkv, rank = rest / p.num_layers, layer = rest - rank * p.num_layers;
      const int a = s_copy[rank], n = s_len[a];
      c.h = u - rest * p.hkv;
      c.from = row(layer, a)[n / kPage];
      c.to = p.free_pages[head + rest];
      c.bytes = n % kPage * kRowBytes;
    }
    return c;
  };
  Copy next = copy_of(w0);
  for (int u = w0; u < units; u += warps) {
    const Copy c = next;
    next = copy_of(u + warps);
    if (!usable(c.from) || !usable(c.to)) {
      if (lane == 0 && (c.from != -1 || !usable(c.to))) atomicOr(p.err, PKV_ERR_PAGE_ID);
      continue;
    }
    const uint8_t* src = p.pool + (static_cast<size_t>(c.from) * p.hkv + c.h) * kHeadPageBytes;
    uint8_t* dst = p.pool + (static_cast<size_t>(c.to) * p.hkv + c.h) * kHeadPageBytes;
    uint4 k[4], v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = 16 * lane + 512 * i;
      if (at < c.bytes) {
        k[i] = __ldcs(reinterpret_cast<const uint4*>(src + at));
        v[i] = __ldcs(reinterpret_cast<const uint4*>(src + kHalfBytes + at));
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = 16 * lane + 512 * i;
      if (at < c.bytes) {
        *reinterpret_cast<uint4*>(dst + at) = k[i];
        *reinterpret_cast<uint4*>(dst + kHalfBytes + at) = v[i];
      }
    }
  }
  // What the parents' holders come to: none where one child takes over.
  const int parts = parts_of(p.max_blocks);
  for (long long u = w0; u < static_cast<long long>(p.batch) * p.num_layers * parts; u += warps) {
    const RowPart part(u, parts);
    const int layer = part.row / p.batch, a = part.row - layer * p.batch;
    const int n = s_len[a], d = s_count[a] - 1;
    if (n <= 0 || d == 0) continue;
    const int32_t* from = row(layer, a);
    const int upto = d < 0 ? blocks_of(n) : n / kPage;  // (a part-filled page: only where nobody takes it over)
    int page[kPartLoads];
#pragma unroll
    for (int i = 0; i < kPartLoads; ++i) {
      const int at = part.at + 32 * i + lane;
      page[i] = at < upto ? from[at] : -1;
    }
#pragma unroll
    for (int i = 0; i < kPartLoads; ++i)
      if (usable(page[i])) atomicAdd(p.change + page[i], d);
  }
  // The children's tables.
  for (long long u = w0; u < static_cast<long long>(p.children) * p.num_layers * parts; u += warps) {
    const RowPart part(u, parts);
    const int layer = part.row / p.children, b = part.row - layer * p.children, rank = s_rank[b];
    int32_t* to = p.tables_out + static_cast<size_t>(part.row) * p.max_blocks;
    const int a = rank == -2 ? -1 : s_parent[b];
    const int n = a < 0 ? 0 : s_len[a], upto = blocks_of(n);
    const int32_t* from = row(layer, max(a, 0));
    const int fresh = rank >= 0 ? p.free_pages[head + rank * p.num_layers + layer] : -1;
    int page[kPartLoads];
#pragma unroll
    for (int i = 0; i < kPartLoads; ++i) {
      const int at = part.at + 32 * i + lane;
      page[i] = at < upto ? (rank >= 0 && at == upto - 1 ? fresh : from[at]) : -1;
    }
#pragma unroll
    for (int i = 0; i < kPartLoads; ++i) {
      const int at = part.at + 32 * i + lane;
      if (page[i] != -1 && !usable(page[i])) {
        atomicOr(p.err, PKV_ERR_PAGE_ID);
        page[i] = -1;
      }
      if (at < p.max_blocks) to[at] = page[i];
    }
  }
}

// A warp's pages: their counts now, and which have lost their last holder, a bit a
// page. `change`: of the counts, in this call.
__device__ __forceinline__ void counts_of(const ForkParams& p, long long page0, int lane, int (&change)[kBallots],
                                          int (&now)[kBallots]) {
#pragma unroll
  for (int i = 0; i < kBallots; ++i) {
    const long long page = page0 + 32 * i + lane;
    change[i] = page < p.num_pages ? __ldcg(p.change + page) : 0;
    now[i] = page < p.num_pages ? p.shares[page] : 0;
  }
#pragma unroll
  for (int i = 0; i < kBallots; ++i) now[i] += change[i];
}

__global__ void __launch_bounds__(kMoveThreads, kMoveCtas) fork_tables_kernel(const ForkParams p) {
  extern __shared__ int s_fork[];
  grid_dependency_wait();
  grid_launch_dependents();
  fork_tables(p, s_fork);
}

__global__ void __launch_bounds__(kMoveThreads) fork_count_kernel(const ForkParams p) {
  __shared__ int s_warp[kMoveWarps];
  grid_dependency_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int mine = 0;
  for (int r = 0; r < p.rounds; ++r) {
    const long long page0 = (static_cast<long long>(blockIdx.x) * p.rounds + r) * kRoundPages + warp * kWarpPages;
    int change[kBallots], now[kBallots];
    counts_of(p, page0, lane, change, now);
#pragma unroll
    for (int i = 0; i < kBallots; ++i) mine += __popc(__ballot_sync(kFull, now[i] < 0));
  }
  if (lane == 0) s_warp[warp] = mine;
  __syncthreads();
  if (threadIdx.x == 0) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kMoveWarps; ++w) sum += s_warp[w];
    p.counts[blockIdx.x] = sum;
  }
}

// The first `chunks` CTAs write the counts of a chunk each, and put its pages given
// back into the list; the others copy what stays of the list. kFew: all CTAs are a
// cluster, count the chunks themselves and copy the list together.
template <bool kFew>
__device__ __forceinline__ void fork_list(const ForkParams& p) {
  __shared__ int s_warp[kMoveWarps], s_sums[2], s_mine;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, chunk = blockIdx.x;
  const bool lists = !kFew && chunk >= p.chunks;
  const int head = *p.free_head, taken = __ldcg(p.taken);
  auto page_at = [&](int r) { return (static_cast<long long>(chunk) * p.rounds + r) * kRoundPages + warp * kWarpPages; };
  int change[kBallots], now[kBallots];
  if (!lists) counts_of(p, page_at(0), lane, change, now);
  // pages given back by the chunks before this one, and by all
  int before = 0, all = 0;
  if constexpr (kFew) {
    int mine = 0;
#pragma unroll
    for (int i = 0; i < kBallots; ++i) mine += __popc(__ballot_sync(kFull, now[i] < 0));
    if (tid == 0) s_mine = 0;
    __syncthreads();
    if (lane == 0) atomicAdd(&s_mine, mine);
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    for (int c = 0; c < p.chunks; ++c) {
      const int n = *cluster.map_shared_rank(&s_mine, c);
      all += n;
      if (c < chunk) before += n;
    }
    cluster_arrive();
  } else {
    for (int c = tid; c < p.chunks; c += kMoveThreads) {
      const int n = __ldcg(p.counts + c);
      all += n;
      if (c < chunk) before += n;
    }
    before = __reduce_add_sync(kFull, before);
    all = __reduce_add_sync(kFull, all);
    if (tid < 2) s_sums[tid] = 0;
    __syncthreads();
    if (lane == 0) {
      atomicAdd(&s_sums[0], before);
      atomicAdd(&s_sums[1], all);
    }
    __syncthreads();
    before = s_sums[0];
    all = s_sums[1];
  }
  const bool head_ok = head >= 0 && head <= p.num_free;
  const int next = head_ok ? head + taken : 0;  // the list's next entry before pages come back
  const int first = next - all;                 // and after
  if (kFew || lists) {
    const int skip = kFew ? 0 : p.chunks, lister = chunk - skip, listers = static_cast<int>(gridDim.x) - skip;
    for (long long j = static_cast<long long>(lister) * kMoveThreads + tid; j < p.num_free;
         j += static_cast<long long>(listers) * kMoveThreads)
      if (j < first || j >= next) p.list_out[j] = p.free_pages[j];
    if (!kFew) return;
  }
  if (chunk == 0 && tid == 0) {
    *p.head_out = head_ok ? max(first, 0) : head;
    if (first < 0) atomicOr(p.err, PKV_ERR_FREE_LIST);
  }
  for (int r = 0; r < p.rounds; ++r) {
    if (r > 0) counts_of(p, page_at(r), lane, change, now);
    uint32_t bits[kBallots];
    int mine = 0;
#pragma unroll
    for (int i = 0; i < kBallots; ++i) {
      bits[i] = __ballot_sync(kFull, now[i] < 0);
      mine += __popc(bits[i]);
    }
    __syncthreads();
    if (lane == 0) s_warp[warp] = mine;
    __syncthreads();
    int at = first + before;
#pragma unroll
    for (int w = 0; w < kMoveWarps; ++w) {
      if (w < warp) at += s_warp[w];
      before += s_warp[w];
    }
#pragma unroll
    for (int i = 0; i < kBallots; ++i) {
      const long long page = page_at(r) + 32 * i + lane;
      if (page < p.num_pages) {
        const int slot = at + __popc(bits[i] & ((1u << lane) - 1));
        if (now[i] < 0 && slot >= 0 && slot < next) p.list_out[slot] = static_cast<int32_t>(page);
        p.shares_out[page] = max(now[i], 0);
        if (change[i] != 0) p.change[page] = 0;
      }
      at += __popc(bits[i]);
    }
  }
  if constexpr (kFew) cluster_wait();  // no CTA leaves while another reads its count
}

__global__ void __launch_bounds__(kMoveThreads) fork_list_kernel(const ForkParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  fork_list<false>(p);
}

// All of it in one cluster. (No kernel after this one starts early, as after
// compact_move_kernel.)
__global__ void __launch_bounds__(kMoveThreads) fork_kernel(const ForkParams p) {
  extern __shared__ int s_fork[];
  grid_dependency_wait();
  fork_tables(p, s_fork);
  __threadfence();
  cg::this_cluster().sync();
  fork_list<true>(p);
}

// ---------------------------------------------------------------------------
// compaction

struct CompactParams {
  uint8_t* pool;
  long long num_pages;
  int hkv;
  const int32_t* seq_lens;  // [batch]
  int batch, num_layers;
  const int32_t* tables;  // [L][batch][max_blocks]
  int max_blocks;
  const int32_t* shares;  // [num_pages]
  const int32_t* free_pages;
  int num_free;
  const int32_t* free_head;
  int32_t* tables_out;
  int32_t* shares_out;
  int32_t* list_out;
  int32_t* used_out;  // [1]
  uint8_t* held;    // [num_pages] marks, zero between calls
  uint8_t* listed;  // [num_pages] the same
  int2* counts;     // by chunk: pages held; pages listed and not held
  int chunks, rounds;
  int* moves;   // [1] pages that move
  int* rank;    // [num_pages] of a mover, or of a place: its number; -1: neither
  int* movers;  // [num_pages] the movers in order
  int* places;  // [num_pages] the places in order
  int* err;
};

// First entry of the list that counts.
__device__ __forceinline__ int list_from(const CompactParams& p) {
  const int head = *p.free_head;
  return head >= 0 && head <= p.num_free ? head : p.num_free;
}

__device__ __forceinline__ void compact_mark(const CompactParams& p) {
  const int tid = threadIdx.x, lane = tid & 31;
  const int w0 = blockIdx.x * kMoveWarps + (tid >> 5), warps = gridDim.x * kMoveWarps;
  const int parts = parts_of(p.max_blocks);
  for (long long u = w0; u < static_cast<long long>(p.batch) * p.num_layers * parts; u += warps) {
    const RowPart part(u, parts);
    const int n = p.seq_lens[part.row % p.batch];
    const int32_t* from = p.tables + static_cast<size_t>(part.row) * p.max_blocks;
    int page[kPartLoads];  // asked for before the length is known
#pragma unroll
    for (int i = 0; i < kPartLoads; ++i) {
      const int at = part.at + 32 * i + lane;
      page[i] = at < p.max_blocks ? from[at] : -1;
    }
    const bool ok = n >= 0 && n <= static_cast<long long>(p.max_blocks) * kPage;
    if (!ok && lane == 0) atomicOr(p.err, PKV_ERR_SEQ_LEN);
    const int upto = ok ? blocks_of(n) : 0;
#pragma unroll
    for (int i = 0; i < kPartLoads; ++i) {
      if (part.at + 32 * i + lane >= upto) break;
      if (page[i] >= 0 && page[i] < p.num_pages)
        p.held[page[i]] = 1;
      else if (page[i] != -1)
        atomicOr(p.err, PKV_ERR_PAGE_ID);
    }
  }
  if (*p.free_head != list_from(p) && w0 == 0 && lane == 0) atomicOr(p.err, PKV_ERR_NO_PAGES);
  for (long long j = list_from(p) + static_cast<long long>(blockIdx.x) * kMoveThreads + tid; j < p.num_free;
       j += static_cast<long long>(gridDim.x) * kMoveThreads) {
    const int page = p.free_pages[j];
    if (page >= 0 && page < p.num_pages)
      p.listed[page] = 1;
    else
      atomicOr(p.err, PKV_ERR_PAGE_ID);
  }
}

__global__ void __launch_bounds__(kMoveThreads) compact_mark_kernel(const CompactParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  compact_mark(p);
}

// A warp's pages: held, and listed without being held, a bit a page.
__device__ __forceinline__ void marks_of(const CompactParams& p, long long page0, int lane, uint32_t (&held)[kBallots],
                                         uint32_t (&open)[kBallots]) {
  int h[kBallots], l[kBallots];
#pragma unroll
  for (int i = 0; i < kBallots; ++i) {
    const long long page = page0 + 32 * i + lane;
    h[i] = page < p.num_pages ? __ldcg(p.held + page) : 0;
    l[i] = page < p.num_pages ? __ldcg(p.listed + page) : 0;
  }
#pragma unroll
  for (int i = 0; i < kBallots; ++i) {
    held[i] = __ballot_sync(kFull, h[i] != 0);
    open[i] = __ballot_sync(kFull, l[i] != 0) & ~held[i];
  }
}

__global__ void __launch_bounds__(kMoveThreads) compact_count_kernel(const CompactParams p) {
  __shared__ int2 s_warp[kMoveWarps];
  grid_dependency_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int2 mine = make_int2(0, 0);
  for (int r = 0; r < p.rounds; ++r) {
    uint32_t held[kBallots], open[kBallots];
    marks_of(p, (static_cast<long long>(blockIdx.x) * p.rounds + r) * kRoundPages + warp * kWarpPages, lane, held, open);
#pragma unroll
    for (int i = 0; i < kBallots; ++i) {
      mine.x += __popc(held[i]);
      mine.y += __popc(open[i]);
    }
  }
  if (lane == 0) s_warp[warp] = mine;
  __syncthreads();
  if (threadIdx.x == 0) {
    int2 sum = make_int2(0, 0);
#pragma unroll
    for (int w = 0; w < kMoveWarps; ++w) {
      sum.x += s_warp[w].x;
      sum.y += s_warp[w].y;
    }
    p.counts[blockIdx.x] = sum;
  }
}

// Ranks: chunk by chunk, as the counts say what is before it. The chunk that
// holds page U is in part below it, so every CTA counts that part itself. kFew: all
// CTAs are a cluster and count the chunks themselves.
template <bool kFew>
__device__ __forceinline__ void compact_rank(const CompactParams& p) {
  __shared__ int2 s_warp[kMoveWarps];
  __shared__ int s_sums[5];
  __shared__ int2 s_mine;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long size = static_cast<long long>(p.rounds) * kRoundPages;
  const int chunk = blockIdx.x;
  auto page_at = [&](int c, int r) { return c * size + r * kRoundPages + warp * kWarpPages; };
  uint32_t held[kBallots], open[kBallots];
  marks_of(p, page_at(chunk, 0), lane, held, open);
  if (tid < 5) s_sums[tid] = 0;
  if (tid == 0) s_mine = make_int2(0, 0);
  __syncthreads();
  constexpr int kCounts = kFew ? 1 : kMaxChunks / kMoveThreads;
  int2 counts[kCounts];
  int used = 0;
  if constexpr (kFew) {
    int2 mine = make_int2(0, 0);
#pragma unroll
    for (int i = 0; i < kBallots; ++i) {
      mine.x += __popc(held[i]);
      mine.y += __popc(open[i]);
    }
    if (lane == 0) {
      atomicAdd(&s_mine.x, mine.x);
      atomicAdd(&s_mine.y, mine.y);
    }
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    counts[0] = tid < p.chunks ? *cluster.map_shared_rank(&s_mine, tid) : make_int2(0, 0);
    used = counts[0].x;
    cluster_arrive();
  } else {
#pragma unroll
    for (int i = 0; i < kCounts; ++i) {
      const int c = tid + i * kMoveThreads;
      counts[i] = c < p.chunks ? __ldcg(&p.counts[c]) : make_int2(0, 0);
      used += counts[i].x;
    }
  }
  used = __reduce_add_sync(kFull, used);
  if (lane == 0) atomicAdd(&s_sums[0], used);
  __syncthreads();
  used = s_sums[0];
  const int border = static_cast<int>(used / size);  // the chunk of page U
  // movers before this chunk and in all; places before it and in all
  int m0 = 0, m1 = 0, h0 = 0, h1 = 0;
#pragma unroll
  for (int i = 0; i < kCounts; ++i) {
    const int c = tid + i * kMoveThreads;
    if (c > border) {
      m1 += counts[i].x;
      if (c < chunk) m0 += counts[i].x;
    }
    if (c < border) {
      h1 += counts[i].y;
      if (c < chunk) h0 += counts[i].y;
    }
  }
  if (border < p.chunks) {
    for (int r = 0; r < p.rounds; ++r) {
      const long long page0 = page_at(border, r);
      uint32_t held_b[kBallots], open_b[kBallots];
      marks_of(p, page0, lane, held_b, open_b);
      if (lane == 0) {
#pragma unroll
        for (int i = 0; i < kBallots; ++i) {
          const long long below = used - (page0 + 32 * i);  // pages of these 32 that are below U
          const uint32_t low = below <= 0 ? 0u : below >= 32 ? ~0u : (1u << below) - 1;
          const int m = __popc(held_b[i] & ~low), h = __popc(open_b[i] & low);
          m1 += m;
          h1 += h;
          if (border < chunk) {
            m0 += m;
            h0 += h;
          }
        }
      }
    }
  }
  m0 = __reduce_add_sync(kFull, m0);
  m1 = __reduce_add_sync(kFull, m1);
  h0 = __reduce_add_sync(kFull, h0);
  h1 = __reduce_add_sync(kFull, h1);
  if (lane == 0) {
    atomicAdd(&s_sums[1], m0);
    atomicAdd(&s_sums[2], m1);
    atomicAdd(&s_sums[3], h0);
    atomicAdd(&s_sums[4], h1);
  }
  __syncthreads();
  int m = s_sums[1], h = s_sums[3];
  const int moves = min(s_sums[2], s_sums[4]);
  if (chunk == 0 && tid == 0) {
    *p.used_out = used;
    *p.moves = moves;
  }
  for (int r = 0; r < p.rounds; ++r) {
    const long long page0 = page_at(chunk, r);
    if (r > 0) marks_of(p, page0, lane, held, open);
    int2 mine = make_int2(0, 0);
#pragma unroll
    for (int i = 0; i < kBallots; ++i) {
      const long long below = used - (page0 + 32 * i);
      const uint32_t low = below <= 0 ? 0u : below >= 32 ? ~0u : (1u << below) - 1;
      held[i] &= ~low;  // movers
      open[i] &= low;   // places
      mine.x += __popc(held[i]);
      mine.y += __popc(open[i]);
    }
    __syncthreads();
    if (lane == 0) s_warp[warp] = mine;
    __syncthreads();
    int2 at = make_int2(m, h);
#pragma unroll
    for (int w = 0; w < kMoveWarps; ++w) {
      if (w < warp) {
        at.x += s_warp[w].x;
        at.y += s_warp[w].y;
      }
      m += s_warp[w].x;
      h += s_warp[w].y;
    }
#pragma unroll
    for (int i = 0; i < kBallots; ++i) {
      const long long page = page0 + 32 * i + lane;
      const uint32_t lower = (1u << lane) - 1;
      if (page < p.num_pages) {
        int rank = -1;
        if ((held[i] >> lane) & 1u) {
          rank = at.x + __popc(held[i] & lower);
          if (rank < moves) p.movers[rank] = static_cast<int>(page);
        } else if ((open[i] >> lane) & 1u) {
          rank = at.y + __popc(open[i] & lower);
          if (rank < moves) p.places[rank] = static_cast<int>(page);
        }
        p.rank[page] = rank < moves ? rank : -1;
      }
      at.x += __popc(held[i]);
      at.y += __popc(open[i]);
    }
  }
  if constexpr (kFew) cluster_wait();  // no CTA leaves while another reads its counts
}

__global__ void __launch_bounds__(kMoveThreads) compact_rank_kernel(const CompactParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  compact_rank<false>(p);
}

// Marks, counts and ranks in one cluster.
__global__ void __launch_bounds__(kMoveThreads) compact_plan_kernel(const CompactParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  compact_mark(p);
  __threadfence();
  cg::this_cluster().sync();
  compact_rank<true>(p);
}

__global__ void __launch_bounds__(kMoveThreads, kMoveCtas) compact_move_kernel(const CompactParams p) {
  // (no kernel after this one starts early: a decode step reads tables and pages
  // before its own wait. A fork's tables and pages are complete when its last kernel
  // lets go.)
  grid_dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31;
  const int w0 = blockIdx.x * kMoveWarps + (tid >> 5), warps = gridDim.x * kMoveWarps;
  const long long t0 = static_cast<long long>(blockIdx.x) * kMoveThreads + tid;
  const long long threads = static_cast<long long>(gridDim.x) * kMoveThreads;
  const int moves = __ldcg(p.moves), used = *p.used_out;
  // where a held page goes, and what a listed page makes room for
  auto to = [&](int page) {
    const int r = page >= used ? __ldcg(p.rank + page) : -1;
    return r >= 0 ? __ldcg(p.places + r) : page;
  };
  auto of = [&](int page) {
    const int r = page < used ? __ldcg(p.rank + page) : -1;
    return r >= 0 ? __ldcg(p.movers + r) : page;
  };
  // Contents, a kv head's 4 KB a warp.
  const int units = moves * p.hkv;  // (of 4 KB each: fewer than 2^31 in any memory)
  for (int u = w0; u < units; u += warps) {
    const int k = u / p.hkv, h = u - k * p.hkv;
    warp_copy(p.pool + (static_cast<size_t>(__ldcg(p.places + k)) * p.hkv + h) * kHeadPageBytes,
              p.pool + (static_cast<size_t>(__ldcg(p.movers + k)) * p.hkv + h) * kHeadPageBytes, kHeadPageBytes, lane);
  }
  const int parts = parts_of(p.max_blocks);
  for (long long u = w0; u < static_cast<long long>(p.batch) * p.num_layers * parts; u += warps) {
    const RowPart part(u, parts);
    const int n = p.seq_lens[part.row % p.batch];
    const int upto = n >= 0 && n <= static_cast<long long>(p.max_blocks) * kPage ? blocks_of(n) : 0;
    const size_t at = static_cast<size_t>(part.row) * p.max_blocks;
    int page[kPartLoads];
#pragma unroll
    for (int i = 0; i < kPartLoads; ++i) {
      const int k = part.at + 32 * i + lane;
      page[i] = k < upto ? p.tables[at + k] : -1;
    }
#pragma unroll
    for (int i = 0; i < kPartLoads; ++i) page[i] = page[i] >= 0 && page[i] < p.num_pages ? to(page[i]) : -1;
#pragma unroll
    for (int i = 0; i < kPartLoads; ++i) {
      const int k = part.at + 32 * i + lane;
      if (k < p.max_blocks) p.tables_out[at + k] = page[i];
    }
  }
  const int from = list_from(p);
  for (long long j = t0; j < p.num_free; j += threads) {
    const int page = p.free_pages[j];
    p.list_out[j] = j >= from && page >= 0 && page < p.num_pages ? of(page) : page;
  }
  // a place takes its mover's count, the mover is left with none
  for (long long page = t0; page < p.num_pages; page += threads) {
    const int r = __ldcg(p.rank + page);
    p.shares_out[page] = r < 0 ? p.shares[page] : page < used ? p.shares[__ldcg(p.movers + r)] : 0;
    p.held[page] = 0;
    p.listed[page] = 0;
  }
}

// ---------------------------------------------------------------------------

// Launch with programmatic stream serialization, as one cluster or without clusters.
cudaLaunchConfig_t config(cudaLaunchAttribute (&attr)[2], int grid, size_t smem, cudaStream_t stream, bool one_cluster) {
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = grid;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = one_cluster ? 2 : 1;
  return cfg;
}
template <typename P>
cudaError_t launch_after(void (*kernel)(P), int grid, size_t smem, cudaStream_t stream, const P& p, bool one_cluster = false) {
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = config(attr, grid, smem, stream, one_cluster);
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Whether `device`, the current one, runs a cluster of kCluster CTAs of `kernel`, the
// only one asked for of its type P. (Eight are what every GPU grants; a part of a GPU may
// have no 16 SMs that a cluster can take.)
template <typename P>
bool cluster_runs(void (*kernel)(P), size_t smem, int device) {
  static std::atomic<int> known[64];  // by device: 1 yes, -1 no; any further device is asked in every call
  if (device < 64)
    if (const int k = known[device].load(std::memory_order_relaxed)) return k > 0;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = config(attr, kCluster, smem, nullptr, true);
  cfg.attrs = attr + 1;  // the cluster's
  cfg.numAttrs = 1;
  int n = 0;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
  if (e != cudaSuccess) return cudaGetLastError(), false;  // the launches by grids say what there is to say
  if (device < 64) known[device].store(n > 0 ? 1 : -1, std::memory_order_relaxed);
  return n > 0;
}

int failed(cudaError_t e) {
  record_cuda_error(e);
  return -EIO;
}

// CTAs for `warps` units of a warp, at most `most` a SM.
int grid_for(long long warps, int most, int sms) {
  const long long n = (warps + kMoveWarps - 1) / kMoveWarps;
  return static_cast<int>(n < 1 ? 1 : n < static_cast<long long>(most) * sms ? n : static_cast<long long>(most) * sms);
}

// When a call is one cluster: by the pool's chunks and a warp's pieces of work (a fork's
// copies and parts of rows, five a warp; a compaction's parts of rows and of the list).
// Measured, one cluster against a grid a kernel, graph replays / calls in a row, us, all
// of the pool listed:
//   fork, 2048 pages       16 pieces  6.3 /  6.3 against  7.0 /  8.0; 640  6.9 /  6.9 against  7.5 /  8.4
//        12000             16         7.3 /  7.3          7.0 /  7.8  640  7.7 /  7.7          7.5 /  8.3
//                                                                     800  8.7 /  8.7          7.6 /  8.3
//        25000             16         8.0 /  8.0          7.0 /  7.9  640  8.3 /  8.5          7.6 /  8.4
//        30000             16         8.7 /  8.7          7.0 /  7.9  640  9.2 /  9.2          7.6 /  8.5
//   compaction, 2048       17        10.3 / 10.7         11.9 / 13.2  112 10.6 / 10.9         11.3 / 12.2
//        12000             95        11.2 / 11.6         11.9 / 12.7  214 14.0 / 14.3         13.8 / 15.0
//                         286        15.2 / 15.4         14.9 / 15.6  350 15.4 / 15.7         14.9 / 15.9
//        25000            197        12.7 / 13.1         12.2 / 13.3  292 15.1 / 15.5         14.7 / 15.6
//        30000            236        13.4 / 13.7         12.3 / 13.2  331 15.5 / 15.8         14.7 / 15.8
// so that calls gain up to some 25000 pages, replays up to some 8000.
constexpr int kClusterChunks = 12;
constexpr long long kForkUnits = 5 * kCluster * kMoveWarps, kPlanUnits = 256;
static_assert(kClusterChunks <= kCluster, "a chunk a CTA at most");
bool one_cluster(const Chunks& cut, long long units, long long most) {
  return cut.n <= kClusterChunks && units <= most;
}

size_t fork_smem(int batch, int children) { return sizeof(int) * (3 * static_cast<size_t>(batch) + 3 * static_cast<size_t>(children)); }

}  // namespace
}  // namespace pkv

extern "C" {

size_t paged_pages_workspace_bytes(const pkv_pool_t* pool) {
  return pool ? pkv::PagesWorkspace(pool->num_pages).bytes : 0;
}

int paged_tables_fork(pkv_pool_t* pool, const int32_t* parents, int children, const int32_t* seq_lens, int batch,
                      int num_layers, const int32_t* block_tables, int max_blocks, const int32_t* shares,
                      const int32_t* free_pages, int num_free, const int32_t* free_head, int32_t* block_tables_out,
                      int32_t* seq_lens_out, int32_t* shares_out, int32_t* free_pages_out, int32_t* free_head_out,
                      void* workspace, size_t workspace_bytes, void* stream) {
  using namespace pkv;
  if (!pool || children < 0 || children > PKV_TABLES_MAX_BATCH || batch < 0 || batch > PKV_TABLES_MAX_BATCH ||
      num_layers < 1 || num_layers > kMaxLayers || max_blocks < 1 || max_blocks > (1 << 23) || num_free < 0)
    return -EINVAL;
  if ((children > 0 && (!parents || !block_tables_out || !seq_lens_out)) || (batch > 0 && (!seq_lens || !block_tables)) ||
      !shares || !free_head || (num_free > 0 && (!free_pages || !free_pages_out)) || !shares_out || !free_head_out ||
      !workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return -EINVAL;
  // (rows and copies are counted in 32 bits)
  if (static_cast<long long>(children) * num_layers * pool->num_kv_heads >= (1ll << 30)) return -EINVAL;
  const PagesWorkspace at(pool->num_pages, workspace_bytes);
  if (workspace_bytes < at.bytes) return -EINVAL;
  const long long rows = static_cast<long long>(num_layers) * max_blocks;
  const ByteRange ranges[] = {{block_tables_out, 4 * rows * children},
                              {seq_lens_out, 4ll * children},
                              {shares_out, 4 * pool->num_pages},
                              {free_pages_out, 4ll * num_free},
                              {free_head_out, 4},
                              {workspace, static_cast<long long>(workspace_bytes)},
                              {pool->storage, static_cast<long long>(pool->storage_bytes)},
                              {parents, 4ll * children},  // the rest is only read
                              {seq_lens, 4ll * batch},
                              {block_tables, 4 * rows * batch},
                              {shares, 4 * pool->num_pages},
                              {free_pages, 4ll * num_free},
                              {free_head, 4}};
  if (ranges_overlap(ranges, 7, sizeof(ranges) / sizeof(ranges[0]))) return -EINVAL;
  if (const int rc = check_pool_device(pool)) return rc;
  const int sms = device_sm_count(pool->device);
  if (sms < 1) return -EINVAL;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const Chunks cut(pool->num_pages);
  ForkParams p;
  p.pool = static_cast<uint8_t*>(pool->storage);
  p.num_pages = pool->num_pages;
  p.hkv = pool->num_kv_heads;
  p.parents = parents;
  p.children = children;
  p.seq_lens = seq_lens;
  p.batch = batch;
  p.num_layers = num_layers;
  p.tables = block_tables;
  p.max_blocks = max_blocks;
  p.shares = shares;
  p.free_pages = free_pages;
  p.num_free = num_free;
  p.free_head = free_head;
  p.tables_out = block_tables_out;
  p.lens_out = seq_lens_out;
  p.shares_out = shares_out;
  p.list_out = free_pages_out;
  p.head_out = free_head_out;
  p.taken = reinterpret_cast<int*>(ws + at.head);
  p.counts = reinterpret_cast<int*>(ws + at.counts);
  p.chunks = cut.n;
  p.rounds = cut.rounds;
  p.change = reinterpret_cast<int*>(ws + at.change);
  p.err = pool->d_err;
  const cudaStream_t on = static_cast<cudaStream_t>(stream);
  static DeviceSetup setup;
  cudaError_t e = setup([&] {
    return cudaFuncSetAttribute(fork_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(fork_smem(PKV_TABLES_MAX_BATCH, PKV_TABLES_MAX_BATCH)));
  });
  if (e != cudaSuccess) return failed(e);
  const long long copies = static_cast<long long>(children) * num_layers * pool->num_kv_heads;  // at most
  const long long units = copies + (static_cast<long long>(batch) + children) * num_layers * parts_of(max_blocks);
  if (one_cluster(cut, units, kForkUnits) && cluster_runs(fork_kernel, fork_smem(kForkUnits, 0), pool->device)) {
    e = launch_after(fork_kernel, kCluster, fork_smem(batch, children), on, p, true);
    return e == cudaSuccess ? 0 : failed(e);
  }
  e = launch_after(fork_tables_kernel, grid_for(units, kMoveCtas, sms), fork_smem(batch, children), on, p);
  if (e == cudaSuccess) e = launch_after(fork_count_kernel, cut.n, 0, on, p);
  if (e == cudaSuccess) e = launch_after(fork_list_kernel, cut.n + grid_for(num_free / 32, 2, sms), 0, on, p);
  return e == cudaSuccess ? 0 : failed(e);
}

int paged_pages_compact(pkv_pool_t* pool, const int32_t* seq_lens, int batch, int num_layers, const int32_t* block_tables,
                        int max_blocks, const int32_t* shares, const int32_t* free_pages, int num_free,
                        const int32_t* free_head, int32_t* block_tables_out, int32_t* shares_out,
                        int32_t* free_pages_out, int32_t* used, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace pkv;
  if (!pool || batch < 0 || batch > PKV_TABLES_MAX_BATCH || num_layers < 1 || num_layers > kMaxLayers || max_blocks < 1 ||
      max_blocks > (1 << 23) || num_free < 0)
    return -EINVAL;
  if ((batch > 0 && (!seq_lens || !block_tables || !block_tables_out)) || !shares || !free_head ||
      (num_free > 0 && (!free_pages || !free_pages_out)) || !shares_out || !used || !workspace ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return -EINVAL;
  const PagesWorkspace at(pool->num_pages, workspace_bytes);
  if (workspace_bytes < at.bytes) return -EINVAL;
  const long long rows = static_cast<long long>(num_layers) * max_blocks;
  const ByteRange ranges[] = {{block_tables_out, 4 * rows * batch},
                              {shares_out, 4 * pool->num_pages},
                              {free_pages_out, 4ll * num_free},
                              {used, 4},
                              {workspace, static_cast<long long>(workspace_bytes)},
                              {pool->storage, static_cast<long long>(pool->storage_bytes)},
                              {seq_lens, 4ll * batch},  // the rest is only read
                              {block_tables, 4 * rows * batch},
                              {shares, 4 * pool->num_pages},
                              {free_pages, 4ll * num_free},
                              {free_head, 4}};
  if (ranges_overlap(ranges, 6, sizeof(ranges) / sizeof(ranges[0]))) return -EINVAL;
  if (const int rc = check_pool_device(pool)) return rc;
  const int sms = device_sm_count(pool->device);
  if (sms < 1) return -EINVAL;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const Chunks cut(pool->num_pages);
  CompactParams p;
  p.pool = static_cast<uint8_t*>(pool->storage);
  p.num_pages = pool->num_pages;
  p.hkv = pool->num_kv_heads;
  p.seq_lens = seq_lens;
  p.batch = batch;
  p.num_layers = num_layers;
  p.tables = block_tables;
  p.max_blocks = max_blocks;
  p.shares = shares;
  p.free_pages = free_pages;
  p.num_free = num_free;
  p.free_head = free_head;
  p.tables_out = block_tables_out;
  p.shares_out = shares_out;
  p.list_out = free_pages_out;
  p.used_out = used;
  p.held = ws + at.marks;
  p.listed = p.held + pool->num_pages;
  p.counts = reinterpret_cast<int2*>(ws + at.counts);
  p.chunks = cut.n;
  p.rounds = cut.rounds;
  p.moves = reinterpret_cast<int*>(ws + at.head);
  p.rank = reinterpret_cast<int*>(ws + at.ranks);
  p.movers = reinterpret_cast<int*>(ws + at.movers);
  p.places = reinterpret_cast<int*>(ws + at.places);
  p.err = pool->d_err;
  const cudaStream_t on = static_cast<cudaStream_t>(stream);
  const long long units = static_cast<long long>(num_layers) * batch * parts_of(max_blocks), list_units = parts_of(num_free);
  cudaError_t e = cudaSuccess;
  if (one_cluster(cut, units + list_units, kPlanUnits) && cluster_runs(compact_plan_kernel, 0, pool->device)) {
    e = launch_after(compact_plan_kernel, kCluster, 0, on, p, true);
  } else {
    e = launch_after(compact_mark_kernel, grid_for(units > list_units ? units : list_units, 4, sms), 0, on, p);
    if (e == cudaSuccess) e = launch_after(compact_count_kernel, cut.n, 0, on, p);
    if (e == cudaSuccess) e = launch_after(compact_rank_kernel, cut.n, 0, on, p);
  }
  if (e == cudaSuccess) e = launch_after(compact_move_kernel, kMoveCtas * sms, 0, on, p);
  return e == cudaSuccess ? 0 : failed(e);
}

}  // extern "C"
