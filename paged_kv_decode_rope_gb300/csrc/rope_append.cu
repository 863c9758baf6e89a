// rope_append.cu -- RoPE of a step's q and k in either pairing, of all or part
// of the head, with the append of k and v into the pool by slot.
//
// Pair j < r/2 of a head is dims (j, j + r/2), or (2j, 2j + 1) when
// interleaved; with c, s the cos and sin of the token's row of the RoPE table,
//     y0 = x0 c - x1 s,   y1 = x1 c + x0 s,
// dims from r on unchanged. q is rotated in fp32 and kept in fp32; k is rounded
// to bf16 once, exactly as the fp64 rotation rounds it (rotated_bf16_fast
// certifies the rounding in fp32 double words, rotate_key_dim does it in fp64
// where it cannot), as every other append of this library; v is copied.
//
// The kernel moves (Hq + 2 Hkv) * 128 bytes in and Hq * 256 + Hkv * 256 out a
// token and computes next to nothing, so memory bounds it. One CTA a token:
// 16 threads hold a head's row, 4 dims (8 bytes of bf16, 16 of fp32) each, so
// that every access is a full row in one go; a thread keeps the same 4 dims of
// every row it takes and therefore reads its cos and sin once. The rotated
// partner of a dim is in the same thread (interleaved) or in another of the
// same 16 (half pairs: rot_dim is a multiple of 8, so partners come in whole
// 4-dim pieces), reached by a shuffle. kRows rows a thread are loaded before
// the first is used, ahead of the position -> table row chain.
#include <cerrno>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kHalfDim = kHeadDim / 2;
constexpr int kPieces = kHeadDim / 4;  // threads a row
constexpr int kRopeThreads = 256;
constexpr int kRows = 4;               // rows a thread loads at once

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
  int* err;
};

// One dim of the rotated key in fp64: bf16 of x c - xp s, every operation
// rounded once.
__device__ __noinline__ uint16_t rotate_key_dim(float x, float xp, const double2* cs) {
  const double2 c = *cs;
  return double_to_bf16_rne(__dsub_rn(__dmul_rn(static_cast<double>(x), c.x),
                                      __dmul_rn(static_cast<double>(xp), c.y)));
}

template <bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeAppendParams p) {
  const int tkn = blockIdx.x, tid = threadIdx.x;
  const int piece = tid % kPieces;                     // this thread's dims: 4 piece .. + 3
  const int step = blockDim.x / kPieces;               // rows a pass of the CTA
  const int rows = p.hq + 2 * p.hkv;                   // q heads, then k heads, then v heads
  const int half = p.rot_dim / 2;
  const bool turns = 4 * piece < p.rot_dim;
  // half pairs: the piece that holds this one's partners, on which side this one is
  const bool upper = !kInterleaved && 4 * piece >= half;
  const int partner = !turns ? piece : upper ? piece - half / 4 : piece + half / 4;

  auto load = [&](int row) {
    if (row >= rows) return make_uint2(0u, 0u);
    const uint16_t* src = row < p.hq ? p.q + tkn * p.q_stride + row * kHeadDim
                          : row < p.hq + p.hkv ? p.k + tkn * p.k_stride + (row - p.hq) * kHeadDim
                                               : p.v + tkn * p.v_stride + (row - p.hq - p.hkv) * kHeadDim;
    return __ldg(reinterpret_cast<const uint2*>(src + 4 * piece));
  };
  uint2 x[kRows];
  int row0 = tid / kPieces;
#pragma unroll
  for (int i = 0; i < kRows; ++i) x[i] = load(row0 + i * step);

  const int pos = p.positions[tkn];
  const int slot = p.slot_map[tkn];
  const bool in_table = pos >= 0 && pos < p.rope_positions;
  bool stores = in_table && slot >= 0;
  if (stores && slot / kPage >= p.num_pages) {
    stores = false;
    if (tid == 0) atomicOr(p.err, PKV_ERR_PAGE_ID);
  }
  if (!in_table && tid == 0) atomicOr(p.err, PKV_ERR_POSITION);
  // cos and sin of the thread's dims: entry j of dim e (hi and lo of each)
  float4 cs[4];
  const int j0 = kInterleaved ? 2 * piece : upper ? 4 * piece - half : 4 * piece;
  const size_t at = static_cast<size_t>(in_table ? pos : 0) * kHalfDim + j0;
#pragma unroll
  for (int e = 0; e < 4; ++e) cs[e] = make_float4(1.f, 0.f, 0.f, 0.f);
  if (turns) {
#pragma unroll
    for (int e = 0; e < 4; ++e) cs[e] = __ldg(p.rope_ff + at + (kInterleaved ? e / 2 : e));
  }
  uint16_t* page_base = p.pool + (stores ? static_cast<size_t>(slot / kPage) : 0) * p.hkv * (kHeadPageBytes / 2) +
                        (slot & (kPage - 1)) * kHeadDim + 4 * piece;
  const int lane0 = (tid & 31) & ~(kPieces - 1);

  for (; row0 - tid / kPieces < rows; row0 += kRows * step) {  // the same trip count in all threads
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int row = row0 + i * step;
      const uint2 w = x[i];
      x[i] = load(row + kRows * step);
      float2 a = bf16x2_to_float2(w.x), b = bf16x2_to_float2(w.y);
      const float own[4] = {a.x, a.y, b.x, b.y};
      float other[4];  // what each dim's sin multiplies, with its sign: y = own cos - other sin
      if (kInterleaved) {
        other[0] = own[1];
        other[1] = -own[0];
        other[2] = own[3];
        other[3] = -own[2];
      } else {
        a = bf16x2_to_float2(__shfl_sync(kFull, w.x, lane0 + partner));
        b = bf16x2_to_float2(__shfl_sync(kFull, w.y, lane0 + partner));
        other[0] = upper ? -a.x : a.x;
        other[1] = upper ? -a.y : a.y;
        other[2] = upper ? -b.x : b.x;
        other[3] = upper ? -b.y : b.y;
      }
      if (row >= rows) continue;
      if (row < p.hq) {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[e] = turns ? own[e] * cs[e].x - other[e] * cs[e].z : own[e];
          if (!in_table) y[e] = 0.f;
        }
        *reinterpret_cast<float4*>(p.q_rot + (static_cast<size_t>(tkn) * p.hq + row) * kHeadDim + 4 * piece) =
            make_float4(y[0], y[1], y[2], y[3]);
      } else if (stores) {
        const bool key = row < p.hq + p.hkv;
        const int h = row - p.hq - (key ? 0 : p.hkv);
        uint2 out = w;
        if (key && turns) {
          uint16_t y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!rotated_bf16_fast(own[e], other[e], cs[e].x, cs[e].y, cs[e].z, cs[e].w, y[e]))
              y[e] = rotate_key_dim(own[e], other[e], p.rope_dd + at + (kInterleaved ? e / 2 : e));
          out = make_uint2(y[0] | static_cast<uint32_t>(y[1]) << 16, y[2] | static_cast<uint32_t>(y[3]) << 16);
        }
        *reinterpret_cast<uint2*>(page_base + (h * 2 + (key ? 0 : 1)) * (kHalfBytes / 2)) = out;
      }
    }
  }
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
      q_stride % 4 || k_stride % 4 || v_stride % 4)
    return -EINVAL;
  if (tokens == 0) return 0;
  if (!q || !k || !v || !q_rot || !slot_map || !positions || !rope_table) return -EINVAL;
  auto aligned = [](const void* x, uintptr_t n) { return reinterpret_cast<uintptr_t>(x) % n == 0; };
  if (!aligned(q, 8) || !aligned(k, 8) || !aligned(v, 8) || !aligned(q_rot, 16) || !aligned(rope_table, 16))
    return -EINVAL;
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
  auto kernel = interleaved ? rope_append_kernel<true> : rope_append_kernel<false>;
  kernel<<<tokens, kRopeThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    record_cuda_error(e);
    return -EIO;
  }
  return 0;
}
