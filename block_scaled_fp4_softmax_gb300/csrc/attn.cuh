// Shared parts of the attention operators: the paged cache on the device, the
// packed sequences, and the host checks of both.
#pragma once

#include "attn.h"
#include "common.cuh"

namespace attn {

constexpr int kMaxSlots = 0x7FFFFFFF - 2048;

struct Half {  // FP16
  using T = __half;
  using T2 = __half2;
  static __device__ __forceinline__ float2 up(uint32_t v) { return __half22float2(*reinterpret_cast<T2*>(&v)); }
  static __device__ __forceinline__ uint32_t down(float lo, float hi) {
    const T2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
struct Brain {  // BF16
  using T = __nv_bfloat16;
  using T2 = __nv_bfloat162;
  static __device__ __forceinline__ float2 up(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t down(float lo, float hi) {
    const T2 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

// 8 elements of FP32 -> 16 bits
template <class E>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(E::down(f[0], f[1]), E::down(f[2], f[3]), E::down(f[4], f[5]), E::down(f[6], f[7]));
}

// Sequence b of the batch: its committed slots and its tokens in flight.
struct Seq {
  int len, first, n;
  bool ok;
};

// `cap`: slots a sequence may have in all.
__device__ __forceinline__ Seq sequence(const int32_t* __restrict__ cu, const int32_t* __restrict__ lens, int b,
                                        int tokens, long long cap) {
  Seq s;
  s.len = __ldg(lens + b);
  s.first = __ldg(cu + b);
  const int end = __ldg(cu + b + 1);
  s.ok = s.first >= 0 && end >= s.first && end <= tokens && s.len >= 0;
  s.n = s.ok ? end - s.first : 0;
  s.ok = s.ok && (long long)s.len + s.n <= cap;
  return s;
}

// The sequence that token t belongs to: the last b with cu[b] <= t (for
// ascending cu; any cu gives an index in range, which `sequence` then checks
// together with first <= t < first + n).
__device__ __forceinline__ int sequence_of(const int32_t* __restrict__ cu, int batch, int t) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Elements from the cache's base to row `slot` of head h of sequence b, or -1
// where the page table holds no page.
__device__ __forceinline__ long long slot_offset(const attn_cache& c, int b, int slot, int h) {
  const int p = slot / c.page_size;
  const int page = __ldg(c.page_table + (size_t)b * c.max_pages + p);
  if ((unsigned)page >= (unsigned)c.pages) return -1;
  return page * c.page_stride + h * c.head_stride + (long long)(slot - p * c.page_size) * c.row_stride;
}

// Bits j0 .. j0 + 31 of a draft's ancestor row (bit i: it sees draft j0 + i);
// row < 0 is impossible, j0 may be negative (bits below draft 0 are 0).
__device__ __forceinline__ uint32_t tree_bits(const uint64_t* __restrict__ words, int count, int j0) {
  uint32_t r = 0;
#pragma unroll
  for (int part = 0; part < 2; ++part) {  // the two 32-bit halves that j0 straddles
    const int w32 = (j0 >> 5) + part;
    if (w32 < 0 || w32 >= 2 * count) continue;
    const uint64_t w = __ldg(words + (w32 >> 1));
    const uint32_t v = (uint32_t)(w >> (32 * (w32 & 1)));
    const int s = j0 & 31;
    if (part == 0) r |= v >> s;
    else if (s) r |= v << (32 - s);
  }
  return r;
}

// Bits j0 .. j0 + 31 of the chain's row i: drafts 0 .. i.
__device__ __forceinline__ uint32_t chain_bits(int i, int j0) {
  const int n = i + 1 - j0;  // how many of the 32, from the lowest
  uint32_t r = n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
  if (j0 < 0) r &= j0 <= -32 ? 0u : 0xFFFFFFFFu << -j0;
  return r;
}

// ---------------------------------------------------------------------------
// Host checks
// ---------------------------------------------------------------------------

// Strides of axes of one element play no part; they are set to something sane.
inline int check_cache(const attn_cache* in, attn_cache& c) {
  if (!in) return MOE_ERR_INVALID_ARG;
  c = *in;
  if (!c.k || !c.v || !c.page_table || c.batch <= 0 || c.max_pages <= 0 || c.pages <= 0 || c.kv_heads <= 0)
    return MOE_ERR_INVALID_ARG;
  if (c.dtype != ATTN_BF16 && c.dtype != ATTN_FP16) return MOE_ERR_UNSUPPORTED;
  if (c.head_dim < 16 || c.head_dim > 256 || c.head_dim % 8 != 0) return MOE_ERR_UNSUPPORTED;
  if (c.page_size < 8 || c.page_size > (1 << 20) || c.page_size % 8 != 0) return MOE_ERR_UNSUPPORTED;
  if ((long long)c.max_pages * c.page_size > kMaxSlots || c.kv_heads > 65535 || c.batch > (1 << 20))
    return MOE_ERR_UNSUPPORTED;
  if (c.pages == 1) c.page_stride = c.head_dim;
  if (c.kv_heads == 1) c.head_stride = c.head_dim;
  const long long st[3] = {c.page_stride, c.head_stride, c.row_stride};
  for (long long s : st)
    if (s < c.head_dim || s % 8 != 0 || s >= (1ll << 38)) return MOE_ERR_UNSUPPORTED;
  if (!moe::aligned16(c.k) || !moe::aligned16(c.v)) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

inline int check_queries(const attn_cache& c, const void* q, long long q_stride, const int32_t* cu,
                         const int32_t* lens, int tokens, int q_heads, const uint64_t* tree, int tree_words) {
  if ((!q && tokens > 0) || !cu || !lens || tokens < 0 || q_heads <= 0) return MOE_ERR_INVALID_ARG;
  // (words of no array would be taken for a chain)
  if (tree ? tree_words <= 0 : tree_words != 0) return MOE_ERR_INVALID_ARG;
  if (q_heads % c.kv_heads != 0 || q_heads > 65535) return MOE_ERR_UNSUPPORTED;
  if (tree && tree_words > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  if (tokens > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  if (q_stride < (long long)q_heads * c.head_dim || q_stride % 8 != 0) return MOE_ERR_UNSUPPORTED;
  if (!moe::aligned16(q)) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

// The rows (token x query head) of a sequence and KV head are counted in an int.
inline bool rows_fit(const attn_cache& c, int tokens, int q_heads) {
  return (long long)tokens * (q_heads / c.kv_heads) <= kMaxSlots;
}

}  // namespace attn
