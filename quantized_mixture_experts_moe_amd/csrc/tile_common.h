// Building blocks of the tiled matrix products: copies from memory straight
// to LDS with their waits, and the row tiles of the experts (not installed).
#pragma once
#include "block_common.h"

namespace qmoe {
namespace bk {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr unsigned kNowhere = 0xC0000000u;  // an offset behind every buffer of gathered rows

// Buffer descriptor of `bytes` bytes at p (raw, no swizzle); reads behind the
// end give zeros.
typedef __amdgpu_buffer_rsrc_t Rsrc;
__device__ inline Rsrc rsrc(const void* p, size_t bytes) {
  const unsigned n = bytes < 0xfffffff0u ? (unsigned)bytes : 0xfffffff0u;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)n, 0x00027000);
}
// 16 bytes per lane from voff (per lane) + soff (the wave's) to LDS, in lane
// order.
__device__ inline void copy16(Rsrc r, unsigned voff, unsigned soff, uint8_t* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16,
                                           (int)voff, (int)soff, 0, 0);
}
__device__ inline void copy4(Rsrc r, unsigned voff, float* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 4,
                                           (int)voff, 0, 0, 0);
}
// Waits until at most N of the wave's memory operations are under way (they
// end in order; a barrier alone does not wait for copies to LDS).
template <int N>
__device__ inline void wait_memory() {
  static_assert(N < 64, "six bits");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4 << 14));
}

// Barrier of the block that leaves copies to LDS under way (the fence of
// __syncthreads waits for every one): the wave's own LDS reads and writes are
// done, and none of the compiler's is moved across.
__device__ inline void block_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// The row tiles of the experts, found by every wave from expert_offsets: a
// lane holds the tiles of E / 64 consecutive experts, a prefix sum over the
// lanes places them.
template <int BM>
struct Spans {
  int first, mine, per;  // tiles before this lane's experts, its own, experts per lane
  template <class G>
  __device__ inline int tiles(const G& g, int e) const {
    return (g.expert_offsets[e + 1] - g.expert_offsets[e] + BM - 1) / BM;
  }
  template <class G>
  __device__ inline int count(const G& g) {
    const int lane = threadIdx.x & 63;
    per = (g.E + 63) / 64;
    mine = 0;
    for (int i = 0; i < per; i++)
      if (lane * per + i < g.E) mine += tiles(g, lane * per + i);
    int sum = mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int v = __shfl_up(sum, off, 64);
      if (lane >= off) sum += v;
    }
    first = sum - mine;
    return __builtin_amdgcn_readlane(sum, 63);
  }
  // Expert and rows [*m0, *mend) of row tile t (below count).
  template <class G>
  __device__ inline int find(const G& g, int t, int* m0, int* mend) const {
    const unsigned long long at = __ballot(first <= t && t < first + mine);
    const int lane = (int)__ffsll(at) - 1;
    int left = t - __builtin_amdgcn_readlane(first, lane);
    const int per_lane = __builtin_amdgcn_readfirstlane(per);
    int e = lane * per_lane;
    for (int i = 0; i + 1 < per_lane && left >= tiles(g, e); i++) left -= tiles(g, e++);
    *m0 = g.expert_offsets[e] + left * BM;
    *mend = min(*m0 + BM, g.expert_offsets[e + 1]);
    return e;
  }
};

template <int V>
struct Int {
  static constexpr int value = V;
};

}  // namespace bk
}  // namespace qmoe
