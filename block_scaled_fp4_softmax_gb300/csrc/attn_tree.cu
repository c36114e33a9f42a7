// Attention of the tokens in flight over a paged cache: one block per token
// and query head, a running maximum and sum over the keys.
#include "attn.cuh"

namespace {

constexpr int kWarps = 4;

struct TreeArgs {
  const void* q;
  long long q_stride;
  const int32_t *cu, *lens;
  int tokens, q_heads;
  const uint64_t* tree;
  int tree_words;
  float scale;
  attn_cache c;
  void* out;
  float* lse;
  int32_t* st;
};

template <class E>
__global__ void __launch_bounds__(kWarps * 32) tree_kernel(const __grid_constant__ TreeArgs a) {
  using T = typename E::T;
  __shared__ float s_o[kWarps][256];
  __shared__ float s_m[kWarps], s_l[kWarps];
  const int t = blockIdx.x, hq = blockIdx.y, D = a.c.head_dim;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d0 = lane * 8;
  const int b = attn::sequence_of(a.cu, a.c.batch, t);
  const attn::Seq s = attn::sequence(a.cu, a.lens, b, a.tokens, (long long)a.c.max_pages * a.c.page_size);
  const bool ok = s.ok && t >= s.first && t < s.first + s.n;
  const int h = hq / (a.q_heads / a.c.kv_heads);
  float q[8] = {}, o[8] = {};
  float m = -INFINITY, l = 0.f;
  if (d0 < D) {
    attn::unpack8<E>(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + t * a.q_stride + (long long)hq * D + d0), q);
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] *= a.scale;
  }
  bool bad = !ok;
  for (int j = warp; j < (ok ? s.len + s.n : 0); j += kWarps) {
    if (j >= s.len) {
      const int d = j - s.len;
      const uint32_t w = a.tree ? attn::tree_bits(a.tree + (long long)t * a.tree_words, a.tree_words, d) : attn::chain_bits(t - s.first, d);
      if (!(w & 1u)) continue;
    }
    const long long off = attn::slot_offset(a.c, b, j, h);
    if (off < 0) {
      bad = true;
      moe::status_or(a.st, ATTN_DEV_BAD_PAGE);
      continue;
    }
    float k[8] = {}, v[8] = {};
    if (d0 < D) {
      attn::unpack8<E>(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.c.k) + off + d0), k);
      attn::unpack8<E>(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.c.v) + off + d0), v);
    }
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) x = fmaf(q[i], k[i], x);
    x = moe::warp_sum(x);
    const float top = fmaxf(m, x);
    const float f = __expf(m - top), p = __expf(x - top);
    l = l * f + p;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = o[i] * f + p * v[i];
    m = top;
  }
  if (!ok && threadIdx.x == 0) moe::status_or(a.st, ATTN_DEV_BAD_LENGTH);
  if (bad) l = __uint_as_float(0x7FC00000u), m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s_o[warp][d0 + i] = o[i];
  if (lane == 0) s_m[warp] = m, s_l[warp] = l;
  __syncthreads();
  if (warp != 0) return;
  float top = -INFINITY;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
  float sum = 0.f, y[8] = {};
  for (int w = 0; w < kWarps; ++w) {
    const float f = s_m[w] == -INFINITY ? 0.f : __expf(s_m[w] - top);
    sum += s_l[w] * f;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] += s_o[w][d0 + i] * f;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] *= inv;
  if (d0 < D)
    *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + ((long long)t * a.q_heads + hq) * D + d0) = attn::pack8<E>(y);
  if (lane == 0 && a.lse) a.lse[(long long)t * a.q_heads + hq] = sum == 0.f ? -INFINITY : top + logf(sum);
}

}  // namespace

extern "C" {

size_t attn_tree_decode_workspace(const attn_cache* cache) {
  attn_cache c;
  if (attn::check_cache(cache, c)) return 0;
  return 16;
}

int attn_tree_decode(const void* q, long long q_stride, const int32_t* cu, const int32_t* lens, int tokens,
                     int q_heads, const uint64_t* tree, int tree_words, double scale, const attn_cache* cache,
                     void* out, float* lse, void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream) {
  TreeArgs a;
  if (const int rc = attn::check_cache(cache, a.c)) return rc;
  if (const int rc = attn::check_queries(a.c, q, q_stride, cu, lens, tokens, q_heads, tree, tree_words)) return rc;
  if ((!out && tokens > 0) || !workspace) return MOE_ERR_INVALID_ARG;
  if (!moe::aligned16(out) || !moe::aligned16(workspace)) return MOE_ERR_ALIGNMENT;
  if (ws_bytes < attn_tree_decode_workspace(cache)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (tokens == 0) return MOE_OK;
  a.q = q, a.q_stride = q_stride, a.cu = cu, a.lens = lens, a.tokens = tokens, a.q_heads = q_heads;
  a.tree = tree, a.tree_words = tree_words, a.scale = (float)scale, a.out = out, a.lse = lse, a.st = dev_status;
  const cudaStream_t st = (cudaStream_t)stream;
  const dim3 grid(tokens, q_heads);
  if (a.c.dtype == ATTN_BF16) tree_kernel<attn::Brain><<<grid, kWarps * 32, 0, st>>>(a);
  else tree_kernel<attn::Half><<<grid, kWarps * 32, 0, st>>>(a);
  return moe::launch_status();
}

}  // extern "C"
