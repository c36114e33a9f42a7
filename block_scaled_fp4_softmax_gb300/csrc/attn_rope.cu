// Head norm, position rotation and cache append in one pass over q, k and v.
//
// Every head row is read once and written once; the arithmetic is about ten
// flops an element, so the pass is HBM bound.  A row of D elements belongs to
// a group of 4, 8, 16 or 32 lanes, 8 elements (16 bytes) a lane: loads and
// stores are whole rows, the mean square is a shuffle sum inside the group.
// A block takes one token after another; the first rot / 2 threads compute
// the token's sines and cosines once into shared memory for all of its heads.
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
};

// LANES per row, so that LANES * 8 >= D.  PAIRED: the half-split partner of a
// lane's 8 channels is another lane's 8 channels (rot / 2 a multiple of 8), a
// shuffle; otherwise it goes through shared memory.  Interleaved pairs never
// leave the lane.
template <class E, int LANES, bool PAIRED>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kGroups = kThreads / LANES;
  __shared__ float2 s_cs[128];  // magnitude * (cos, sin) of the token's pairs
  __shared__ float s_row[PAIRED ? 1 : kGroups][PAIRED ? 1 : LANES * 8 + 4];
  const int D = a.c.head_dim, half = a.rot / 2;
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const int d0 = lane * 8;
  const bool mine = d0 < D;
  const int heads = a.q_heads + 2 * a.c.kv_heads;
  using T = typename E::T;

  unsigned long long turn = 0;  // inv_freq / 2 pi as a fraction of 2^64
  if (threadIdx.x < half) {
    const double t = a.inv_freq[threadIdx.x] * 0.15915494309189533577;
    const double f = t - floor(t);
    turn = f < 1.0 ? (unsigned long long)(f * 18446744073709551616.0) : 0ull;
  }
  float wq[8], wk[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) wq[i] = wk[i] = 1.f;
  const bool norm = a.q_weight != nullptr;
  if (norm && mine) {
    attn::unpack8<E>(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.q_weight) + d0)), wq);
    attn::unpack8<E>(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.k_weight) + d0)), wk);
  }

  for (int t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    const int pos = __ldg(a.pos + t);
    const int b = attn::sequence_of(a.cu, a.c.batch, t);
    const attn::Seq s = attn::sequence(a.cu, a.lens, b, a.tokens, (long long)a.c.max_pages * a.c.page_size);
    const bool ok = s.ok && t >= s.first && t < s.first + s.n;
    const int slot = s.len + (t - s.first);
    const bool pos_ok = a.slot_pos == nullptr || slot < a.slot_cap;
    __syncthreads();  // the token before is done with s_cs
    if (threadIdx.x < half) {
      const unsigned long long u = turn * (unsigned long long)(long long)pos;
      float sn, cs;
      sincospif((float)(int32_t)(u >> 32) * 0x1p-31f, &sn, &cs);
      s_cs[threadIdx.x] = make_float2(cs * a.magnitude, sn * a.magnitude);
    }
    if (threadIdx.x == 0 && (!ok || !pos_ok)) moe::status_or(a.st, ATTN_DEV_BAD_LENGTH);
    __syncthreads();
    for (int h0 = 0; h0 < heads; h0 += kGroups) {  // uniform over the block: the shuffles below need whole warps
      const int h = h0 + group;
      const bool live = mine && h < heads;
      const int kind = h < a.q_heads ? 0 : h < a.q_heads + a.c.kv_heads ? 1 : 2;  // q, k, v
      const int hk = kind == 0 ? h : kind == 1 ? h - a.q_heads : h - a.q_heads - a.c.kv_heads;
      uint4 raw = make_uint4(0u, 0u, 0u, 0u);
      if (live) {
        const T* src = kind == 0   ? static_cast<const T*>(a.q) + t * a.q_stride
                       : kind == 1 ? static_cast<const T*>(a.k) + t * a.k_stride
                                   : static_cast<const T*>(a.v) + t * a.v_stride;
        raw = *reinterpret_cast<const uint4*>(src + (long long)hk * D + d0);
      }
      float x[8];
      attn::unpack8<E>(raw, x);
      if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int m = LANES / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        const float r = rsqrtf(ss / (float)D + a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= r * (kind == 0 ? wq[i] : wk[i]);
      }
      float y[8];
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const int j = (d0 + i) / 2;
          if (j < half) {
            const float2 cs = s_cs[j];
            y[i] = x[i] * cs.x - x[i + 1] * cs.y;
            y[i + 1] = x[i] * cs.y + x[i + 1] * cs.x;
          } else {
            y[i] = x[i];
            y[i + 1] = x[i + 1];
          }
        }
      } else {
        float p[8];  // the other channel of each pair
        if (PAIRED) {
          const int other = d0 < half ? lane + half / 8 : lane - half / 8;
#pragma unroll
          for (int i = 0; i < 8; ++i) p[i] = __shfl_sync(0xffffffffu, x[i], other, LANES);
        } else {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) s_row[group][d0 + i] = x[i];
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int d = d0 + i;
            p[i] = d < a.rot ? s_row[group][d < half ? d + half : d - half] : 0.f;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int d = d0 + i;
          if (d < half) {
            const float2 cs = s_cs[d];
            y[i] = x[i] * cs.x - p[i] * cs.y;
          } else if (d < a.rot) {
            const float2 cs = s_cs[d - half];
            y[i] = p[i] * cs.y + x[i] * cs.x;
          } else {
            y[i] = x[i];
          }
        }
      }
      if (!live) continue;
      if (kind == 0) {
        if (!ok) {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = __uint_as_float(0x7FC00000u);
        }
        *reinterpret_cast<uint4*>(static_cast<T*>(a.q_out) + ((long long)t * a.q_heads + hk) * D + d0) =
            attn::pack8<E>(y);
      } else if (ok) {
        const long long off = attn::slot_offset(a.c, b, slot, hk);
        if (off < 0) {
          moe::status_or(a.st, ATTN_DEV_BAD_PAGE);
        } else {
          T* dst = static_cast<T*>(kind == 1 ? a.c.k : a.c.v) + off + d0;
          *reinterpret_cast<uint4*>(dst) = kind == 1 ? attn::pack8<E>(y) : raw;
          if (kind == 1 && lane == 0 && a.slot_pos && pos_ok)
            a.slot_pos[((long long)b * a.c.kv_heads + hk) * a.slot_cap + slot] = pos;
        }
      }
    }
  }
}

template <class E, int LANES>
int launch(const RopeArgs& a, cudaStream_t st) {
  const bool paired = a.interleaved || (a.rot / 2) % 8 == 0;
  const int sms = moe::device_info().sms;
  if (sms <= 0) return MOE_ERR_CUDA;
  const int grid = a.tokens < 8 * sms ? a.tokens : 8 * sms;
  if (paired) qk_norm_rope_kernel<E, LANES, true><<<grid, kThreads, 0, st>>>(a);
  else qk_norm_rope_kernel<E, LANES, false><<<grid, kThreads, 0, st>>>(a);
  return moe::launch_status();
}

template <class E>
int launch(const RopeArgs& a, cudaStream_t st) {
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
