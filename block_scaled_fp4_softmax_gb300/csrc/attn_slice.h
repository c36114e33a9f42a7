// How attn_cache_evict divides the slots of one (sequence, head) among the warps
// of its cluster, for host and device.  A warp has `slice_slots` consecutive slots,
// a multiple of 128, and the last ones have fewer or none.  Up to 2^31 - 2049 slots
// with 2^16 of rounding pass 31 bits: the ends are formed in 32 bits without a sign,
// and what a warp adds to a slot inside its slice stays below 2^31.
#pragma once

#ifdef __CUDACC__
#define ATTN_HD __host__ __device__ __forceinline__
#else
#define ATTN_HD inline
#endif

namespace attn {

ATTN_HD int slice_slots(int n, int warps) {
  return (int)((((unsigned)n + (unsigned)warps - 1u) / (unsigned)warps + 127u) & ~127u);
}
// First slot of warp `w` of a cluster, and so the end of warp w - 1.
ATTN_HD int slice_begin(int n, int slots, int w) {
  const unsigned at = (unsigned)w * (unsigned)slots;
  return at < (unsigned)n ? (int)at : n;
}

}  // namespace attn
