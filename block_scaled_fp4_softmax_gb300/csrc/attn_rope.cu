// Head norm, position rotation and cache append in one pass over q, k and v.
//
// Every head row is read once and written once; the arithmetic is about ten
// flops an element, so the pass is HBM bound.  A row of D elements belongs to
// a group of 4, 8, 16 or 32 lanes, 8 elements (16 bytes) a lane: loads and
// stores are whole rows, the mean square is a shuffle sum inside the group.
// A block takes a few tokens at a time; its threads compute their sines and
// cosines once into shared memory for all of their heads.
//
// Angles.  pos * inv_freq loses whole turns' worth of bits in FP32 at far
// positions.  inv_freq / 2 pi is turned into a 64-bit fixed-point fraction F
// of a turn once per block; pos * F modulo 2^64 is then the angle modulo one
// turn, exactly: an integer multiply does the reduction.  Its top 32 bits as a
// signed fraction go to sincospif.
#include "attn.cuh"

namespace {

constexpr int kThreads = 256;

struct RopeArgs {
  const void *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  const int32_t *pos, *cu, *lens;
  int tokens, q_heads;
  const void *q_weight, *k_weight;
  float eps;
  const double* inv_freq;
  int rot, interleaved;
  float magnitude;
  void* q_out;
  int32_t* slot_pos;
  int slot_cap;
  attn_cache c;
  int32_t* st;
  int tokens_per_block;
};

// LANES per row, so that LANES * 8 >= D.  PAIRED: the half-split partner of a
// lane's 8 channels is another lane's 8 channels (rot / 2 a multiple of 8), a
// shuffle; otherwise it goes through shared memory.  Interleaved pairs never
// leave the lane.  A block takes kRound rows of each group at a time with all
// of their loads in flight; the rows of up to kTokens tokens make up the list.
constexpr int kRound = 4;
constexpr int kTokens = 4;

template <class E, int LANES, bool PAIRED>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kGroups = kThreads / LANES;
  using T = typename E::T;
  __shared__ float2 s_cs[kTokens][128];  // magnitude * (cos, sin) of the tokens' pairs
  __shared__ int s_pos[kTokens], s_seq[kTokens], s_slot[kTokens];  // slot -1: out of range
  __shared__ float s_row[PAIRED ? 1 : kGroups][PAIRED ? 1 : LANES * 8 + 4];
  const int D = a.c.head_dim, half = a.rot / 2;
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const int d0 = lane * 8;
  const bool mine = d0 < D;
  const int heads = a.q_heads + 2 * a.c.kv_heads;
  const bool norm = a.q_weight != nullptr;
  // the weights and frequencies are parameters of the model: read before the wait
  // on the kernel that makes q, k and v
  unsigned long long turn = 0;  // inv_freq / 2 pi as a fraction of 2^64
  if (threadIdx.x % 128 < half) {
    const double t = a.inv_freq[threadIdx.x % 128] * 0.15915494309189533577;
    const double f = t - floor(t);
    turn = f < 1.0 ? (unsigned long long)(f * 18446744073709551616.0) : 0ull;
  }
  uint4 wq = make_uint4(0u, 0u, 0u, 0u), wk = wq;
  if (norm && mine) {
    wq = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.q_weight) + d0));
    wk = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.k_weight) + d0));
  }
  moe::pdl_wait();
  moe::pdl_launch_dependents();

  for (int t0 = blockIdx.x * a.tokens_per_block; t0 < a.tokens; t0 += gridDim.x * a.tokens_per_block) {
    const int n_tok = min(a.tokens_per_block, a.tokens - t0);
    __syncthreads();  // the tokens before are done with the shared arrays
    if (threadIdx.x < n_tok) {
      const int t = t0 + threadIdx.x;
      const int b = attn::sequence_of(a.cu, a.c.batch, t);
      const attn::Seq s = attn::sequence(a.cu, a.lens, b, a.tokens, (long long)a.c.max_pages * a.c.page_size);
      const bool ok = s.ok && t >= s.first && t < s.first + s.n;
      const int slot = s.len + (t - s.first);
      s_pos[threadIdx.x] = __ldg(a.pos + t);
      s_seq[threadIdx.x] = b;
      s_slot[threadIdx.x] = ok ? slot : -1;
      if (!ok || (a.slot_pos && slot >= a.slot_cap)) moe::status_or(a.st, ATTN_DEV_BAD_LENGTH);
    }
    for (int i = threadIdx.x / 128; i < n_tok; i += kThreads / 128) {
      if (threadIdx.x % 128 < half) {
        const unsigned long long u = turn * (unsigned long long)(long long)__ldg(a.pos + t0 + i);
        float sn, cs;
        sincospif((float)(int32_t)(u >> 32) * 0x1p-31f, &sn, &cs);
        s_cs[i][threadIdx.x % 128] = make_float2(cs * a.magnitude, sn * a.magnitude);
      }
    }
    __syncthreads();
    const int rows = n_tok * heads;
    for (int r0 = 0; r0 < rows; r0 += kRound * kGroups) {  // uniform over the block: the shuffles need whole warps
      uint4 raw[kRound];
      int tok[kRound], head[kRound];  // head counted over q, k, v
#pragma unroll
      for (int i = 0; i < kRound; ++i) {
        const int r = r0 + i * kGroups + group;
        tok[i] = r / heads;
        head[i] = r - tok[i] * heads;
        raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (mine && r < rows) {
          const long long t = t0 + tok[i];
          const T* src = head[i] < a.q_heads
                             ? static_cast<const T*>(a.q) + t * a.q_stride + (long long)head[i] * D
                         : head[i] < a.q_heads + a.c.kv_heads
                             ? static_cast<const T*>(a.k) + t * a.k_stride + (long long)(head[i] - a.q_heads) * D
                             : static_cast<const T*>(a.v) + t * a.v_stride +
                                   (long long)(head[i] - a.q_heads - a.c.kv_heads) * D;
          raw[i] = *reinterpret_cast<const uint4*>(src + d0);
        }
      }
#pragma unroll
      for (int i = 0; i < kRound; ++i) {
        const bool live = mine && r0 + i * kGroups + group < rows;
        const int kind = head[i] < a.q_heads ? 0 : head[i] < a.q_heads + a.c.kv_heads ? 1 : 2;  // q, k, v
        const float2* cs_of = s_cs[live ? tok[i] : 0];
        float x[8];
        attn::unpack8<E>(raw[i], x);
        if (norm) {
          float ss = 0.f, wt[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
          for (int m = LANES / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
          const float r = rsqrtf(ss / (float)D + a.eps);
          attn::unpack8<E>(kind == 0 ? wq : wk, wt);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= r * wt[e];
        }
        float y[8];
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const int j = (d0 + e) / 2;
            if (j < half) {
              const float2 cs = cs_of[j];
              y[e] = x[e] * cs.x - x[e + 1] * cs.y;
              y[e + 1] = x[e] * cs.y + x[e + 1] * cs.x;
            } else {
              y[e] = x[e];
              y[e + 1] = x[e + 1];
            }
          }
        } else {
          float p[8];  // the other channel of each pair
          if (PAIRED) {
            const int other = d0 < half ? lane + half / 8 : lane - half / 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = __shfl_sync(0xffffffffu, x[e], other, LANES);
          } else {
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 8; ++e) s_row[group][d0 + e] = x[e];
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int d = d0 + e;
              p[e] = d < a.rot ? s_row[group][d < half ? d + half : d - half] : 0.f;
            }
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int d = d0 + e;
            if (d < half) {
              const float2 cs = cs_of[d];
              y[e] = x[e] * cs.x - p[e] * cs.y;
            } else if (d < a.rot) {
              const float2 cs = cs_of[d - half];
              y[e] = p[e] * cs.y + x[e] * cs.x;
            } else {
              y[e] = x[e];
            }
          }
        }
        if (!live) continue;
        const int slot = s_slot[tok[i]], b = s_seq[tok[i]];
        if (kind == 0) {
          if (slot < 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(0x7FC00000u);
          }
          *reinterpret_cast<uint4*>(static_cast<T*>(a.q_out) + ((long long)(t0 + tok[i]) * a.q_heads + head[i]) * D + d0) =
              attn::pack8<E>(y);
        } else if (slot >= 0) {
          const int hk = head[i] - a.q_heads - (kind == 2 ? a.c.kv_heads : 0);
          const long long off = attn::slot_offset(a.c, b, slot, hk);
          if (off < 0) {
            moe::status_or(a.st, ATTN_DEV_BAD_PAGE);
          } else {
            T* dst = static_cast<T*>(kind == 1 ? a.c.k : a.c.v) + off + d0;
            *reinterpret_cast<uint4*>(dst) = kind == 1 ? attn::pack8<E>(y) : raw[i];
            if (kind == 1 && lane == 0 && a.slot_pos && slot < a.slot_cap)
              a.slot_pos[((long long)b * a.c.kv_heads + hk) * a.slot_cap + slot] = s_pos[tok[i]];
          }
        }
      }
    }
  }
}

template <class E, int LANES>
int launch(RopeArgs& a, cudaStream_t st) {
  const bool paired = a.interleaved || (a.rot / 2) % 8 == 0;
  const int sms = moe::device_info().sms;
  if (sms <= 0) return MOE_ERR_CUDA;
  // several tokens a block share its set-up, once there are enough to fill the GPU
  a.tokens_per_block = a.tokens >= 16 * sms ? kTokens : 1;
  const int blocks = (a.tokens + a.tokens_per_block - 1) / a.tokens_per_block;
  const int grid = blocks < 8 * sms ? blocks : 8 * sms;
  return paired ? moe::launch_pdl(qk_norm_rope_kernel<E, LANES, true>, dim3(grid), dim3(kThreads), 0, st, a)
                : moe::launch_pdl(qk_norm_rope_kernel<E, LANES, false>, dim3(grid), dim3(kThreads), 0, st, a);
}

template <class E>
int launch(RopeArgs& a, cudaStream_t st) {
  if (a.c.head_dim <= 32) return launch<E, 4>(a, st);
  if (a.c.head_dim <= 64) return launch<E, 8>(a, st);
  if (a.c.head_dim <= 128) return launch<E, 16>(a, st);
  return launch<E, 32>(a, st);
}

}  // namespace

extern "C" int attn_qk_norm_rope(const void* q, const void* k, const void* v, long long q_stride, long long k_stride,
                                 long long v_stride, const int32_t* pos, const int32_t* cu, const int32_t* lens,
                                 int tokens, int q_heads, const void* q_weight, const void* k_weight, double eps,
                                 const double* inv_freq, int rot, int interleaved, double magnitude, void* q_out,
                                 int32_t* slot_pos, int slot_cap, const attn_cache* cache, int32_t* dev_status,
                                 void* stream) {
  RopeArgs a;
  if (const int rc = attn::check_cache(cache, a.c)) return rc;
  if (const int rc = attn::check_queries(a.c, q, q_stride, cu, lens, tokens, q_heads, nullptr, 0)) return rc;
  if ((tokens > 0 && (!k || !v || !pos || !q_out)) || (rot > 0 && !inv_freq) || rot < 0 || (q_weight == nullptr) != (k_weight == nullptr) ||
      (slot_pos && slot_cap <= 0) || !(eps >= 0.0))
    return MOE_ERR_INVALID_ARG;
  if (rot % 2 != 0 || rot > a.c.head_dim) return MOE_ERR_UNSUPPORTED;
  const long long kv = (long long)a.c.kv_heads * a.c.head_dim;
  if (k_stride < kv || k_stride % 8 != 0 || v_stride < kv || v_stride % 8 != 0) return MOE_ERR_UNSUPPORTED;
  if (tokens > 0 && q_out == q && q_stride != (long long)q_heads * a.c.head_dim) return MOE_ERR_INVALID_ARG;
  if (!moe::aligned16(k) || !moe::aligned16(v) || !moe::aligned16(q_out) || !moe::aligned16(q_weight) ||
      !moe::aligned16(k_weight))
    return MOE_ERR_ALIGNMENT;
  if (tokens == 0) return MOE_OK;
  a.q = q, a.k = k, a.v = v;
  a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
  a.pos = pos, a.cu = cu, a.lens = lens, a.tokens = tokens, a.q_heads = q_heads;
  a.q_weight = q_weight, a.k_weight = k_weight, a.eps = (float)eps;
  a.inv_freq = inv_freq, a.rot = rot, a.interleaved = interleaved, a.magnitude = (float)magnitude;
  a.q_out = q_out, a.slot_pos = slot_pos, a.slot_cap = slot_cap, a.st = dev_status;
  const cudaStream_t st = (cudaStream_t)stream;
  return a.c.dtype == ATTN_BF16 ? launch<attn::Brain>(a, st) : launch<attn::Half>(a, st);
}
