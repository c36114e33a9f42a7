// Head norm, position rotation and cache append in one pass over q, k and v.
//
// Every head row is read once and written once.  HBM bounds the pass for many
// tokens, but only if a row costs few instructions: at 48 rows of 256 bytes a
// token, some 200 instructions a row and warp already take as long as the bytes.
// Measured: 12255 tokens of 32 + 2 x 8 heads of 128, BF16: 65 us, 4.6 TB/s (69% of
// the copy bandwidth); one token: 3 us.  No unit is full: 166 instructions a pair of
// rows use 65% of the issue slots, with 44% of the warps that an SM can hold (64
// registers); loads that leave earlier cost 4 us, arithmetic by twos gained 4.
// A row of D elements belongs to a group of 4, 8, 16 or 32 lanes, 8 elements a
// lane in two blocks of 4: for the half-split rotation the blocks are a block
// of the first half and the one it is paired with, so no lane needs another's
// channels; otherwise they lie side by side.  The mean square is a shuffle sum
// inside the group.  A block takes a few tokens at a time: its threads compute
// their sines, cosines and cache slots once into shared memory for all of their
// heads.
//
// Angles.  pos * inv_freq loses whole turns' worth of bits in FP32 at far
// positions.  inv_freq / 2 pi is turned into a 64-bit fixed-point fraction F
// of a turn once per block (FP64: off by up to inv_freq * 2^-54 turns, and 2^-64);
// pos * F modulo 2^64 is then the angle modulo one turn without any further
// error: an integer multiply does the reduction.  Its top 32 bits as a signed
// fraction, rounded to FP32, go to sincospif.
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

constexpr int kRound = 2;   // rows of q of a group whose loads are in flight together, beside one of k or v
constexpr int kTokens = 8;  // tokens whose sines and slots are held

// How a row's channels pair up, and where a lane's two blocks of 4 lie.
enum Pairing {
  kBlocks,    // half-split, rot % 8 == 0: blocks 4 l and rot / 2 + 4 l; behind rot side by side
  kInside,    // interleaved: side by side, pairs inside a block
  kScattered  // half-split, any other rot: side by side, partners by shared memory
};

// Two products or multiply-adds at a time: the pass is short of issue slots.
__device__ __forceinline__ float2 mul2(const float2& a, const float2& b) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(r))
      : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)));
  return r;
}

// Eight channels of a row: a lane's two blocks of 4.
struct Channels {
  float2 x[2], z[2];
};
template <class E>
__device__ __forceinline__ Channels up8(const uint2 (&v)[2]) {
  return {{E::up(v[0].x), E::up(v[0].y)}, {E::up(v[1].x), E::up(v[1].y)}};
}

// LANES per row, so that LANES * 8 >= D.
template <class E, int LANES, Pairing P>
__global__ void __launch_bounds__(kThreads, 4) qk_norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kGroups = kThreads / LANES;
  using T = typename E::T;
  // pairs 2 j and 2 j + 1 of a token at [j % 2][j / 2]: magnitude * (cos, cos', sin, sin')
  __shared__ float4 s_cs[kTokens][2][33];
  __shared__ int s_pos[kTokens], s_seq[kTokens], s_slot[kTokens];  // slot -1: out of range
  __shared__ long long s_off[kTokens];                             // of the slot in head 0, -1: nothing is appended
  alignas(16) __shared__ float s_row[P == kScattered ? kGroups : 1][P == kScattered ? LANES * 8 + 4 : 4];
  const int D = a.c.head_dim, half = a.rot / 2;
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  // the lane's blocks start at channels c0 and c1
  int c0 = lane * 8, c1 = c0 + 4;
  bool turns = false;  // kBlocks: the two blocks are each other's partners
  if (P == kBlocks) {
    turns = lane * 4 < half;
    if (turns) c0 = lane * 4, c1 = half + c0;
  }
  const bool mine = lane * 8 < D;
  const bool norm = a.q_weight != nullptr;
  const float inv_d = 1.f / (float)D;
  moe::pdl_wait();
  moe::pdl_launch_dependents();
  unsigned long long turn = 0;  // inv_freq / 2 pi as a fraction of 2^64
  if (threadIdx.x % 128 < half) {
    const double t = a.inv_freq[threadIdx.x % 128] * 0.15915494309189533577;
    const double f = t - floor(t);
    turn = f < 1.0 ? (unsigned long long)(f * 18446744073709551616.0) : 0ull;
  }
  uint2 wt[2][2] = {};  // [q, k][block]
  if (norm && mine) {
    const T* w[2] = {static_cast<const T*>(a.q_weight), static_cast<const T*>(a.k_weight)};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      wt[i][0] = __ldg(reinterpret_cast<const uint2*>(w[i] + c0));
      wt[i][1] = __ldg(reinterpret_cast<const uint2*>(w[i] + c1));
    }
  }

  for (int t0 = blockIdx.x * a.tokens_per_block; t0 < a.tokens; t0 += gridDim.x * a.tokens_per_block) {
    const int n_tok = min(a.tokens_per_block, a.tokens - t0);
    // The first rows' loads leave before the tokens' set-up.
    auto load = [&](const T* src, bool there, uint2 (&raw)[2]) {
      raw[0] = raw[1] = make_uint2(0u, 0u);
      if (there) {
        raw[0] = *reinterpret_cast<const uint2*>(src + c0);
        raw[1] = *reinterpret_cast<const uint2*>(src + c1);
      }
    };
    // row `h` of the 2 kv_heads rows of k and v
    auto load_kv = [&](long long t, int h, uint2 (&raw)[2]) {
      const bool is_k = h < a.c.kv_heads;
      load(is_k ? static_cast<const T*>(a.k) + t * a.k_stride + h * D
                : static_cast<const T*>(a.v) + t * a.v_stride + (h - a.c.kv_heads) * D,
           mine && h < 2 * a.c.kv_heads, raw);
    };
    auto load_q = [&](long long t, int h, uint2 (&raw)[kRound][2]) {
#pragma unroll
      for (int k = 0; k < kRound; ++k)
        load(static_cast<const T*>(a.q) + t * a.q_stride + (h + k * kGroups) * D, mine && h + k * kGroups < a.q_heads, raw[k]);
    };
    uint2 raw_q[kRound][2], raw_kv[2];
    load_q(t0, group, raw_q);
    load_kv(t0, group, raw_kv);
    __syncthreads();  // the tokens before are done with the shared arrays
    if (threadIdx.x < n_tok) {
      const int tt = t0 + threadIdx.x;
      const int b = attn::sequence_of(a.cu, a.c.batch, tt);
      const attn::Seq s = attn::sequence(a.cu, a.lens, b, a.tokens, (long long)a.c.max_pages * a.c.page_size);
      const bool ok = s.ok && tt >= s.first && tt < s.first + s.n;
      const int slot = s.len + (tt - s.first);
      s_pos[threadIdx.x] = __ldg(a.pos + tt);
      s_seq[threadIdx.x] = b;
      s_slot[threadIdx.x] = ok ? slot : -1;
      // a slot without a position would be lost on attn_cache_evict: it is not filled either
      const bool fits = ok && (!a.slot_pos || slot < a.slot_cap);
      s_off[threadIdx.x] = fits ? attn::slot_offset(a.c, b, slot, 0) : -1;
      if (!fits) moe::status_or(a.st, ATTN_DEV_BAD_LENGTH);
      else if (s_off[threadIdx.x] < 0) moe::status_or(a.st, ATTN_DEV_BAD_PAGE);
    }
    for (int m = threadIdx.x / 128; m < n_tok; m += kThreads / 128) {
      const int j = threadIdx.x % 128;
      if (j < half) {
        const unsigned long long u = turn * (unsigned long long)(long long)__ldg(a.pos + t0 + m);
        float sn, cs;
        sincospif((float)(int32_t)(u >> 32) * 0x1p-31f, &sn, &cs);
        float* to = &s_cs[m][(j >> 1) & 1][j >> 2].x + (j & 1);
        to[0] = cs * a.magnitude, to[2] = sn * a.magnitude;
      }
    }
    __syncthreads();
    for (int i = 0; i < n_tok; ++i) {
      const long long t = t0 + i;
      const int slot = s_slot[i];
      // a lane's four pairs are the same in every head
      float2 cs[2], sn[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int j = lane * 4 + 2 * q;
        float4 e = P != kScattered && j < half ? s_cs[i][q][lane] : make_float4(1.f, 1.f, 0.f, 0.f);
        if (j + 1 >= half) e.y = 1.f, e.w = 0.f;
        cs[q] = make_float2(e.x, e.y), sn[q] = make_float2(e.z, e.w);
      }
      // norm and rotation of one row; w: its weights.  Whole warps come here.
      auto turned = [&](const uint2 (&raw)[2], const uint2 (&w)[2], uint2 (&out)[2]) {
        Channels y = up8<E>(raw);
        if (norm) {
          float2 s2 = mul2(y.x[0], y.x[0]);
          s2 = moe::ffma2(y.x[1], y.x[1], s2);
          s2 = moe::ffma2(y.z[0], y.z[0], s2);
          s2 = moe::ffma2(y.z[1], y.z[1], s2);
          float ss = s2.x + s2.y;
#pragma unroll
          for (int m = LANES / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
          const float r = rsqrtf(ss * inv_d + a.eps);
          const float2 rr = make_float2(r, r);
          const Channels g = up8<E>(w);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            y.x[q] = mul2(y.x[q], mul2(rr, g.x[q]));
            y.z[q] = mul2(y.z[q], mul2(rr, g.z[q]));
          }
        }
        if (P == kBlocks) {
          if (turns) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float2 p = y.x[q], v = y.z[q], down = make_float2(-sn[q].x, -sn[q].y);
              y.x[q] = moe::ffma2(v, down, mul2(p, cs[q]));
              y.z[q] = moe::ffma2(p, sn[q], mul2(v, cs[q]));
            }
          }
        } else if (P == kInside) {  // behind rot the angle is 0
          auto turn2 = [](float2& u, float c, float s) { u = make_float2(u.x * c - u.y * s, u.x * s + u.y * c); };
          const int j = lane * 4;
          if (j < half) turn2(y.x[0], cs[0].x, sn[0].x);
          if (j + 1 < half) turn2(y.x[1], cs[0].y, sn[0].y);
          if (j + 2 < half) turn2(y.z[0], cs[1].x, sn[1].x);
          if (j + 3 < half) turn2(y.z[1], cs[1].y, sn[1].y);
        } else {
          float* row = s_row[group];
          __syncwarp();
          *reinterpret_cast<float4*>(row + c0) = make_float4(y.x[0].x, y.x[0].y, y.x[1].x, y.x[1].y);
          *reinterpret_cast<float4*>(row + c1) = make_float4(y.z[0].x, y.z[0].y, y.z[1].x, y.z[1].y);
          __syncwarp();
          auto turn1 = [&](float u, int d) {
            if (d >= a.rot) return u;
            const bool low = d < half;
            const int j = low ? d : d - half;
            const float* c = &s_cs[i][(j >> 1) & 1][j >> 2].x + (j & 1);
            const float p = row[low ? d + half : j];
            return low ? u * c[0] - p * c[2] : p * c[2] + u * c[0];
          };
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            y.x[q] = make_float2(turn1(y.x[q].x, c0 + 2 * q), turn1(y.x[q].y, c0 + 2 * q + 1));
            y.z[q] = make_float2(turn1(y.z[q].x, c1 + 2 * q), turn1(y.z[q].y, c1 + 2 * q + 1));
          }
        }
        out[0] = make_uint2(E::down(y.x[0].x, y.x[0].y), E::down(y.x[1].x, y.x[1].y));
        out[1] = make_uint2(E::down(y.z[0].x, y.z[0].y), E::down(y.z[1].x, y.z[1].y));
      };
      if (i > 0) {
        load_q(t, group, raw_q);
        load_kv(t, group, raw_kv);
      }
      for (int h0 = 0; h0 < a.q_heads; h0 += kRound * kGroups) {  // uniform over the block
        if (h0 > 0) load_q(t, h0 + group, raw_q);
#pragma unroll
        for (int k = 0; k < kRound; ++k) {
          if (h0 + k * kGroups >= a.q_heads) break;  // uniform
          const int h = h0 + k * kGroups + group;
          uint2 out[2];
          turned(raw_q[k], wt[0], out);
          if (!mine || h >= a.q_heads) continue;
          if (slot < 0) out[0].x = out[0].y = out[1].x = out[1].y = E::down(__uint_as_float(0x7FC00000u), __uint_as_float(0x7FC00000u));
          T* dst = static_cast<T*>(a.q_out) + (t * a.q_heads + h) * D;
          *reinterpret_cast<uint2*>(dst + c0) = out[0];
          *reinterpret_cast<uint2*>(dst + c1) = out[1];
        }
      }
      const long long off = s_off[i];
      for (int h0 = 0; h0 < 2 * a.c.kv_heads; h0 += kGroups) {
        const int h = h0 + group;
        if (h0 > 0) load_kv(t, h, raw_kv);
        const bool is_k = h < a.c.kv_heads;
        uint2 out[2] = {raw_kv[0], raw_kv[1]};
        if (h0 < a.c.kv_heads) {  // uniform: rows of k among them
          uint2 of_k[2];
          turned(raw_kv, wt[1], of_k);
          if (is_k) out[0] = of_k[0], out[1] = of_k[1];
        }
        if (!mine || h >= 2 * a.c.kv_heads || off < 0) continue;
        const int hk = is_k ? h : h - a.c.kv_heads;
        T* dst = static_cast<T*>(is_k ? a.c.k : a.c.v) + off + hk * a.c.head_stride;
        *reinterpret_cast<uint2*>(dst + c0) = out[0];
        *reinterpret_cast<uint2*>(dst + c1) = out[1];
        if (is_k && lane == 0 && a.slot_pos)
          a.slot_pos[((long long)s_seq[i] * a.c.kv_heads + hk) * a.slot_cap + slot] = s_pos[i];
      }
    }
  }
}

template <class E, int LANES>
int launch(RopeArgs& a, cudaStream_t st) {
  const int sms = moe::device_info().sms;
  if (sms <= 0) return MOE_ERR_CUDA;
  // tokens share a block's set-up as far as every SM still gets its four blocks twice
  const int share = a.tokens / (8 * sms);
  a.tokens_per_block = share < 1 ? 1 : share < kTokens ? share : kTokens;
  // and so that the blocks, four to an SM, make whole waves (12255 tokens of 48 rows x 128: 70.7 us, 69.4 so)
  const int waves = (a.tokens + 4 * sms * a.tokens_per_block - 1) / (4 * sms * a.tokens_per_block);
  a.tokens_per_block = (a.tokens + 4 * sms * waves - 1) / (4 * sms * waves);
  const int grid = (a.tokens + a.tokens_per_block - 1) / a.tokens_per_block;
  const auto kernel = a.interleaved      ? qk_norm_rope_kernel<E, LANES, kInside>
                      : a.rot % 8 == 0 ? qk_norm_rope_kernel<E, LANES, kBlocks>
                                       : qk_norm_rope_kernel<E, LANES, kScattered>;
  return moe::launch_pdl(kernel, dim3(grid), dim3(kThreads), 0, st, a);
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
