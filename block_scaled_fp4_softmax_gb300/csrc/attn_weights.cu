// The softmax weight each cached slot received: one warp per slot and KV
// head, a loop over the rows that see it.
#include "attn.cuh"

namespace {

constexpr int kWarps = 8;

struct WeightArgs {
  const void* q;
  long long q_stride;
  const float* lse;
  const int32_t *cu, *lens;
  int tokens, q_heads;
  const uint64_t* tree;
  int tree_words;
  float scale;
  attn_cache c;
  const float* acc;
  float decay;
  float* acc_out;
  int slot_cap;
  int32_t* st;
};

template <class E>
__global__ void __launch_bounds__(kWarps * 32) weights_kernel(const __grid_constant__ WeightArgs a) {
  using T = typename E::T;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, D = a.c.head_dim, d0 = lane * 8;
  const int h = blockIdx.y, b = blockIdx.z;
  const long long most = (long long)a.c.max_pages * a.c.page_size;
  const attn::Seq s = attn::sequence(a.cu, a.lens, b, a.tokens, most < a.slot_cap ? most : a.slot_cap);
  const int G = a.q_heads / a.c.kv_heads;
  const long long base = ((long long)b * a.c.kv_heads + h) * a.slot_cap;
  if (!s.ok) {
    if (threadIdx.x == 0) moe::status_or(a.st, ATTN_DEV_BAD_LENGTH);
    for (long long j = blockIdx.x * kWarps * 32 + threadIdx.x; j < a.slot_cap; j += (long long)gridDim.x * kWarps * 32)
      a.acc_out[base + j] = __uint_as_float(0x7FC00000u);
    return;
  }
  for (int j = blockIdx.x * kWarps + warp; j < s.len + s.n; j += gridDim.x * kWarps) {
    float sum = j < s.len ? a.decay * a.acc[base + j] : 0.f;
    const long long off = attn::slot_offset(a.c, b, j, h);
    float k[8] = {};
    if (off < 0) {
      sum = __uint_as_float(0x7FC00000u);
      moe::status_or(a.st, ATTN_DEV_BAD_PAGE);
    } else if (d0 < D) {
      attn::unpack8<E>(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.c.k) + off + d0), k);
    }
    for (int i = 0; i < s.n; ++i) {
      const int t = s.first + i;
      if (j >= s.len) {
        const uint32_t w = a.tree ? attn::tree_bits(a.tree + (long long)t * a.tree_words, a.tree_words, j - s.len) : attn::chain_bits(i, j - s.len);
        if (!(w & 1u)) continue;
      }
      for (int g = 0; g < G; ++g) {
        const int hq = h * G + g;
        float q[8] = {};
        if (d0 < D) attn::unpack8<E>(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + t * a.q_stride + (long long)hq * D + d0), q);
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) x = fmaf(q[e], k[e], x);
        x = moe::warp_sum(x);
        const float lse = a.lse[(long long)t * a.q_heads + hq];
        if (lse != -INFINITY) sum += expf(x * a.scale - lse);
      }
    }
    if (lane == 0) a.acc_out[base + j] = sum;
  }
}

}  // namespace

extern "C" int attn_cache_weights(const void* q, long long q_stride, const float* lse, const int32_t* cu,
                                  const int32_t* lens, int tokens, int q_heads, const uint64_t* tree, int tree_words,
                                  double scale, const attn_cache* cache, const float* acc, double decay,
                                  float* acc_out, int slot_cap, int32_t* dev_status, void* stream) {
  WeightArgs a;
  if (const int rc = attn::check_cache(cache, a.c)) return rc;
  if (const int rc = attn::check_queries(a.c, q, q_stride, cu, lens, tokens, q_heads, tree, tree_words)) return rc;
  if ((!lse && tokens > 0) || !acc || !acc_out || slot_cap <= 0) return MOE_ERR_INVALID_ARG;
  a.q = q, a.q_stride = q_stride, a.lse = lse, a.cu = cu, a.lens = lens, a.tokens = tokens, a.q_heads = q_heads;
  a.tree = tree, a.tree_words = tree_words, a.scale = (float)scale, a.acc = acc, a.decay = (float)decay;
  a.acc_out = acc_out, a.slot_cap = slot_cap, a.st = dev_status;
  const cudaStream_t st = (cudaStream_t)stream;
  if (a.c.batch > 65535) return MOE_ERR_UNSUPPORTED;
  const dim3 grid(64, a.c.kv_heads, a.c.batch);
  if (a.c.dtype == ATTN_BF16) weights_kernel<attn::Brain><<<grid, kWarps * 32, 0, st>>>(a);
  else weights_kernel<attn::Half><<<grid, kWarps * 32, 0, st>>>(a);
  return moe::launch_status();
}
