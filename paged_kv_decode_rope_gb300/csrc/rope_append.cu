// rope_append.cu -- RoPE of a step's q and k in either pairing, of all or part
// of the head, with the append of k and v into the pool by slot.
//
// Pair j < r/2 of a head is dims (j, j + r/2), or (2j, 2j + 1) when
// interleaved; with c, s the cos and sin of the token's row of the RoPE table,
//     y0 = x0 c - x1 s,   y1 = x1 c + x0 s,
// dims from r on unchanged. q is rotated in fp32 and kept in fp32; k is rounded
// to bf16 once, exactly as the fp64 rotation rounds it, as every other append of
// this library: in fp32 where the result is far enough from a rounding boundary
// (rotated_bf16_quick, all but about one in two thousand), else in fp32 double
// words (rotated_bf16_fast), else in fp64. v is copied.
//
// The kernel moves (Hq + 2 Hkv) * 128 bytes in and Hq * 256 + Hkv * 256 out a
// token and computes next to nothing, so memory bounds it, and what it takes
// is bytes in flight: the cos and sin of a token depend on its position, and a
// CTA a token spent its life waiting for that chain (48 us for 8192 tokens of
// 32 + 8 heads, 42% of the copy bandwidth; now 25.4 us in graph replays, 5.36
// TB/s, 79%, and 27 as calls). So
// CTAs stay and stream units (a token, up to kUnitRows of its rows) through a
// ring of kRopeStages shared-memory stages: one warp issues bulk copies of the
// units' rows, reads their positions and slots ahead, and copies their table
// rows when it knows them; kRopeWarps warps rotate and store. Eight threads
// hold a head's row, 8 dims each: 4 whole pairs (rot_dim is a multiple of 8),
// the same ones in every row it takes, or 8 dims that pass through. Every wait
// is bounded. 64 tokens of 14 + 2 heads take 3.2 us in replays, 4.6 as calls: a
// launch and that chain.
#include <cerrno>
#include <initializer_list>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kHalfDim = kHeadDim / 2;
constexpr int kPieces = kHeadDim / 8;          // threads a row
constexpr int kWarpRows = 32 / kPieces;
// Consumer warps: six, so that 48 rows (32 + 2 * 8 heads) are two even passes:
// 25.1 us for 8192 tokens, against 28.6 with eight (a pass and a half) and 27.0
// with four.
constexpr int kRopeWarps = 6;                 // consumers
constexpr int kRopeThreads = 32 * (kRopeWarps + 1);
constexpr int kUnitRows = 64;                  // rows of a unit at most
constexpr int kRopeStages = 4;
constexpr int kTrigBytes = kHalfDim * 16;      // a row of the table's fp32 pairs
constexpr int kStageBytes = kUnitRows * kRowBytes + kTrigBytes;
constexpr int kRopeCtas = 4;                   // CTAs a SM

struct RopeAppendParams {
  uint16_t* pool;
  long long num_pages;
  int hkv, hq;
  const uint16_t *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  float* q_rot;
  const int32_t* slot_map;
  const int32_t* positions;
  const float4* rope_ff;   // [rows][32] {cos_hi, cos_lo, sin_hi, sin_lo}
  const double2* rope_dd;  // [rows][32] {cos, sin}
  int rope_positions;
  int rot_dim;
  int tokens;
  int unit_rows, units;  // rows of a unit; units a token
  int* err;
};

// a c - b s rounded to bf16 as the exact value rounds, in plain fp32: f has
// the errors of c and s (2^-24 relative each), of the product a c and of the
// fma, at most 5 * 2^-24 of the larger product in all, so where the rounding
// boundary in f's bf16 interval (and the next one, at least 2^-9 |f| away) is
// farther than 2^-20 of it, f and the exact value round to the same bf16.
// Returns whether it is (false for zeros, tiny, huge and non-finite values).
__device__ __forceinline__ bool rotated_bf16_quick(float a, float b, float c, float s, uint32_t& y) {
  const float pa = __fmul_rn(a, c), f = __fmaf_rn(-b, s, pa);
  const float m = fmaxf(fabsf(pa), fabsf(__fmul_rn(b, s))), af = fabsf(f);
  const uint32_t u = __float_as_uint(f);
  const float mid = __uint_as_float((u & 0x7fff0000u) | 0x8000u);  // same binade as af: exact difference
  y = (u + 0x8000u) >> 16;
  return fabsf(__fsub_rn(mid, af)) > __fmul_rn(m, 0x1p-20f) && af >= 0x1p-100f && m <= 0x1p120f &&
         __fmul_rn(af, 0x1p-10f) > __fmul_rn(m, 0x1p-20f);
}

// The same where the quick form cannot tell: bf16 of fl64(a c) - fl64(b s).
__device__ __noinline__ uint32_t rotated_bf16_slow(float a, float b, float4 cs, const double2* cd) {
  uint16_t y;
  if (rotated_bf16_fast(a, b, cs.x, cs.y, cs.z, cs.w, y)) return y;
  const double2 c = *cd;
  return double_to_bf16_rne(__dsub_rn(__dmul_rn(static_cast<double>(a), c.x),
                                      __dmul_rn(static_cast<double>(b), c.y)));
}

template <bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_append_kernel(const RopeAppendParams p) {
  extern __shared__ __align__(128) uint8_t s_ring[];
  __shared__ __align__(8) uint64_t full[kRopeStages], empty[kRopeStages];
  __shared__ int2 s_token[kRopeStages];  // position (-1: none in the table) and slot (-1: not stored)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rows = p.hq + 2 * p.hkv;  // q heads, then k heads, then v heads
  // unit i of this CTA: part `part` of token t, in steps of the grid
  const int t_step = gridDim.x / p.units, part_step = gridDim.x % p.units;
  int t = blockIdx.x / p.units, part = blockIdx.x % p.units;
  auto next_unit = [&]() {
    t += t_step;
    part += part_step;
    if (part >= p.units) {
      part -= p.units;
      ++t;
    }
  };
  if (tid == 0) {
    for (int s = 0; s < kRopeStages; ++s) {
      mbar_init(smem_addr(&full[s]), 1);
      mbar_init(smem_addr(&empty[s]), kRopeWarps);
    }
  }
  fence_mbar_init();
  __syncthreads();
  bool failed = false;

  if (warp == kRopeWarps) {
    // ---- the producer: lane 0 issues; positions and slots are read 32 units
    // ahead, a unit a lane ----
    int pos = 0, slot = 0;
    int i = 0;
    for (; t < p.tokens; next_unit(), ++i) {
      const int st = i % kRopeStages, use = i / kRopeStages;
      if (i % 32 == 0) {
        const long long mine = t + (part + static_cast<long long>(lane) * gridDim.x) / p.units;
        if (mine < p.tokens) {
          pos = p.positions[mine];
          slot = p.slot_map[mine];
          int bits = 0;
          if (pos < 0 || pos >= p.rope_positions) {
            bits |= PKV_ERR_POSITION;
            pos = slot = -1;
          }
          if (slot >= 0 && slot / kPage >= p.num_pages) {
            bits |= PKV_ERR_PAGE_ID;
            slot = -1;
          }
          if (bits) atomicOr(p.err, bits);
        }
      }
      if (use > 0 && !mbar_wait_bounded(smem_addr(&empty[st]), (use - 1) & 1)) failed = true;
      if (__any_sync(kFull, failed)) {
        failed = true;
        break;
      }
      // the rows first: they do not wait for the position
      const uint32_t bar = smem_addr(&full[st]), dst = smem_addr(s_ring) + st * kStageBytes;
      if (lane == 0) {
        const int r0 = part * p.unit_rows, r1 = min(r0 + p.unit_rows, rows);
        mbar_expect_tx(bar, static_cast<uint32_t>((r1 - r0) * kRowBytes));
        auto copy = [&](const uint16_t* src, int first, int last) {  // rows first .. last - 1 of the unit's q, k or v
          const int a = max(r0, first), b = min(r1, last);
          if (a < b)
            bulk_g2s(dst + (a - r0) * kRowBytes, src + static_cast<size_t>(a - first) * kHeadDim,
                     static_cast<uint32_t>((b - a) * kRowBytes), bar);
        };
        copy(p.q + t * p.q_stride, 0, p.hq);
        copy(p.k + t * p.k_stride, p.hq, p.hq + p.hkv);
        copy(p.v + t * p.v_stride, p.hq + p.hkv, rows);
      }
      const int ps = __shfl_sync(kFull, pos, i % 32), sl = __shfl_sync(kFull, slot, i % 32);
      if (lane == 0) {
        s_token[st] = make_int2(ps, sl);
        mbar_arrive_expect_tx(bar, kTrigBytes);
        bulk_g2s(dst + kUnitRows * kRowBytes, p.rope_ff + static_cast<size_t>(max(ps, 0)) * kHalfDim, kTrigBytes, bar);
      }
      __syncwarp();
    }
    // let the copies still in flight land before shared memory goes away
    if (failed && lane == 0)
      for (int k = max(0, i - kRopeStages); k < i; ++k)
        mbar_wait_bounded(smem_addr(&full[k % kRopeStages]), (k / kRopeStages) & 1);
  } else {
    // ---- the consumers ----
    // This thread's pairs: j0 .. j0 + 3 of the table row; their dims are
    // d0 .. d0 + 3 and d1 .. d1 + 3 (half pairs), or the eight from d0 on
    // (interleaved, and where nothing turns).
    const int piece = tid % kPieces, j0 = 4 * piece;
    const bool turns = 8 * piece < p.rot_dim, apart = !kInterleaved && turns;
    const int d0 = apart ? j0 : 8 * piece, d1 = apart ? j0 + p.rot_dim / 2 : d0 + 4;
    int i = 0;
    for (; t < p.tokens; next_unit(), ++i) {
      const int st = i % kRopeStages;
      if (!mbar_wait_bounded(smem_addr(&full[st]), (i / kRopeStages) & 1)) failed = true;
      if (__any_sync(kFull, failed)) {
        failed = true;
        break;
      }
      const int r0 = part * p.unit_rows;
      const int n = min(p.unit_rows, rows - r0);
      const uint32_t src = smem_addr(s_ring) + st * kStageBytes;
      const int2 token = s_token[st];
      float4 cs[4];  // {cos_hi, cos_lo, sin_hi, sin_lo} of the thread's pairs
#pragma unroll
      for (int e = 0; e < 4; ++e)
        cs[e] = turns ? lds128f(src + kUnitRows * kRowBytes + 16 * (j0 + e)) : make_float4(1.f, 0.f, 0.f, 0.f);
      uint16_t* page = p.pool +
                       static_cast<size_t>(max(token.y, 0) / kPage) * p.hkv * (kHeadPageBytes / 2) +
                       (max(token.y, 0) % kPage) * kHeadDim;
      // kWarpRows rows a warp; the warps take turns, so that the key rows, the
      // most work, do not always fall to the same ones
      for (int r = kWarpRows * ((warp + i) % kRopeWarps); r < n; r += kWarpRows * kRopeWarps) {
        const int local = r + lane / kPieces, row = r0 + local;
        if (local >= n) continue;
        const uint2 w0 = lds64u(src + local * kRowBytes + 2 * d0), w1 = lds64u(src + local * kRowBytes + 2 * d1);
        float a[4], b[4];  // the pairs' first and second dims
        {
          const float2 f0 = bf16x2_to_float2(w0.x), f1 = bf16x2_to_float2(w0.y);
          const float2 f2 = bf16x2_to_float2(w1.x), f3 = bf16x2_to_float2(w1.y);
          const float x[8] = {f0.x, f0.y, f1.x, f1.y, f2.x, f2.y, f3.x, f3.y};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[e] = kInterleaved ? x[2 * e] : x[e];
            b[e] = kInterleaved ? x[2 * e + 1] : x[4 + e];
          }
        }
        if (row < p.hq) {
          float y[8];  // dims d0 .. + 3, d1 .. + 3
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float y0 = a[e] * cs[e].x - b[e] * cs[e].z, y1 = b[e] * cs[e].x + a[e] * cs[e].z;
            if (!turns) {
              y0 = a[e];
              y1 = b[e];
            }
            if (token.x < 0) y0 = y1 = 0.f;
            y[kInterleaved ? 2 * e : e] = y0;
            y[kInterleaved ? 2 * e + 1 : 4 + e] = y1;
          }
          float* dst = p.q_rot + (static_cast<size_t>(t) * p.hq + row) * kHeadDim;
          *reinterpret_cast<float4*>(dst + d0) = make_float4(y[0], y[1], y[2], y[3]);
          *reinterpret_cast<float4*>(dst + d1) = make_float4(y[4], y[5], y[6], y[7]);
        } else if (token.y >= 0) {
          const bool key = row < p.hq + p.hkv;
          const int h = row - p.hq - (key ? 0 : p.hkv);
          uint2 o0 = w0, o1 = w1;
          if (key && turns) {
            uint32_t y[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const double2* cd = p.rope_dd + static_cast<size_t>(token.x) * kHalfDim + j0 + e;
              uint32_t y0, y1;
              if (!rotated_bf16_quick(a[e], b[e], cs[e].x, cs[e].z, y0)) y0 = rotated_bf16_slow(a[e], b[e], cs[e], cd);
              if (!rotated_bf16_quick(b[e], -a[e], cs[e].x, cs[e].z, y1)) y1 = rotated_bf16_slow(b[e], -a[e], cs[e], cd);
              y[kInterleaved ? 2 * e : e] = y0;
              y[kInterleaved ? 2 * e + 1 : 4 + e] = y1;
            }
            o0 = make_uint2(y[0] | y[1] << 16, y[2] | y[3] << 16);
            o1 = make_uint2(y[4] | y[5] << 16, y[6] | y[7] << 16);
          }
          uint16_t* dst = page + (h * 2 + (key ? 0 : 1)) * (kHalfBytes / 2);
          *reinterpret_cast<uint2*>(dst + d0) = o0;
          *reinterpret_cast<uint2*>(dst + d1) = o1;
        }
      }
      __syncwarp();  // this warp has read the stage
      if (lane == 0) mbar_arrive(smem_addr(&empty[st]));
    }
  }
  if (failed && lane == 0) atomicOr(p.err, PKV_ERR_TIMEOUT);
}

}  // namespace
}  // namespace pkv

extern "C" int paged_rope_append(pkv_pool_t* pool, const void* q, long long q_stride, const void* k,
                                 long long k_stride, const void* v, long long v_stride, float* q_rot,
                                 const int32_t* slot_map, const int32_t* positions, int tokens,
                                 int num_q_heads, const void* rope_table, int rope_positions, int rot_dim,
                                 int interleaved, void* stream) {
  using namespace pkv;
  if (!pool || tokens < 0 || num_q_heads < 1 || num_q_heads % pool->num_kv_heads || rope_positions < 1 ||
      rope_positions >= (1 << 24) || rot_dim < 8 || rot_dim > kHeadDim || rot_dim % 8)
    return -EINVAL;
  const long long q_row = static_cast<long long>(num_q_heads) * kHeadDim;
  const long long kv_row = static_cast<long long>(pool->num_kv_heads) * kHeadDim;
  if (num_q_heads > kMaxKvHeads * PKV_MAX_GROUP || q_stride < q_row || k_stride < kv_row || v_stride < kv_row ||
      q_stride % 8 || k_stride % 8 || v_stride % 8)
    return -EINVAL;
  if (tokens == 0) return 0;
  if (!q || !k || !v || !q_rot || !slot_map || !positions || !rope_table) return -EINVAL;
  for (const void* x : {q, k, v, static_cast<const void*>(q_rot), rope_table})
    if (reinterpret_cast<uintptr_t>(x) & 15u) return -EINVAL;
  if (const int rc = check_pool_device(pool)) return rc;
  RopeAppendParams p;
  p.pool = static_cast<uint16_t*>(pool->storage);
  p.num_pages = pool->num_pages;
  p.hkv = pool->num_kv_heads;
  p.hq = num_q_heads;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_rot = q_rot;
  p.slot_map = slot_map;
  p.positions = positions;
  p.rope_ff = static_cast<const float4*>(rope_table);
  p.rope_dd = reinterpret_cast<const double2*>(p.rope_ff + static_cast<size_t>(rope_positions) * kHalfDim);
  p.rope_positions = rope_positions;
  p.rot_dim = rot_dim;
  p.err = pool->d_err;
  // Units of a token: as few as hold its rows, of even size.
  const int rows = num_q_heads + 2 * pool->num_kv_heads;
  p.tokens = tokens;
  p.units = (rows + kUnitRows - 1) / kUnitRows;
  p.unit_rows = (rows + p.units - 1) / p.units;
  p.units = (rows + p.unit_rows - 1) / p.unit_rows;
  const int sms = device_sm_count(pool->device);
  if (sms < 1) return -EIO;
  const long long all = static_cast<long long>(tokens) * p.units;
  const long long most = static_cast<long long>(kRopeCtas) * sms;
  const unsigned grid = static_cast<unsigned>(all < most ? all : most);
  auto kernel = interleaved ? rope_append_kernel<true> : rope_append_kernel<false>;
  kernel<<<grid, kRopeThreads, kRopeStages * kStageBytes, static_cast<cudaStream_t>(stream)>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return -EIO;
  }
  return 0;
}
