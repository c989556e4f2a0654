// Quantization to OCP e4m3 with one fp32 scale per 128 values (along the row
// and/or along the column) or per 128 x 128 block.
//
//   a = max |v| over the group, s = a / 448, code = e4m3(v / s)
//
// (group_scale in block_common.h states the corners).  With act, v is
// SiLU(gate) * up of a row [gate | up].  The bound is HBM: every value is
// read once and every code written once.
#include "block_common.h"

namespace qmoe {
namespace {
using namespace bk;

// Eight values of row m from column c, zeros outside the row (ACT: v the
// gate's, u the up projection's).
template <bool F32, bool ACT>
__device__ inline void load_vals(const void* x, size_t m, int c, int K, bool vec, float v[8],
                                 float u[8]) {
  const size_t row = m * (size_t)(ACT ? 2 * (size_t)K : (size_t)K);
  if (vec && c + 8 <= K) {
    load8<F32>(x, row + c, v);
    if constexpr (ACT) load8<F32>(x, row + K + c, u);
  } else {
#pragma unroll
    for (int j = 0; j < 8; j++) {
      v[j] = u[j] = 0.f;
      if (c + j < K) {
        v[j] = load1<F32>(x, row + c + j);
        if constexpr (ACT) u[j] = load1<F32>(x, row + K + c + j);
      }
    }
  }
}

__device__ inline uint32_t amax8(const float v[8]) {
  uint32_t a = abs_bits(v[0]);
#pragma unroll
  for (int j = 1; j < 8; j++) a = max(a, abs_bits(v[j]));
  return a;
}

// Row form.  A block covers 16 rows and kspan K blocks: 16 lanes hold one
// group of 128 (8 values each), so a pass of 256 threads quantizes one K
// block of 16 rows and writes its 16 scales side by side.  The next K block is
// loaded before this one is worked on.  K is split until 2048 blocks are there.
// SiLU(gate) * up of 16384 x 768 in bf16: 13.4 us, 4.7 TB/s of the 5.1 that a
// large copy reaches.
template <bool F32, bool ACT>
__global__ __launch_bounds__(256) void fp8_quant_rows_kernel(const void* __restrict__ x, int M,
                                                             int K, int KB, int kspan, bool vec,
                                                             uint8_t* __restrict__ codes,
                                                             float* __restrict__ scale) {
  const int m = blockIdx.x * 16 + (threadIdx.x >> 4);
  const int l = threadIdx.x & 15;
  const int kb0 = blockIdx.y * kspan, kb1 = min(KB, kb0 + kspan);
  if (m >= M) return;  // whole 16-lane rows leave together
  float v[8], nv[8], nu[8];
  load_vals<F32, ACT>(x, m, kb0 * 128 + l * 8, K, vec, nv, nu);
  for (int kb = kb0; kb < kb1; kb++) {
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = ACT ? silu_mul(nv[j], nu[j]) : nv[j];
    if (kb + 1 < kb1) load_vals<F32, ACT>(x, m, kb * 128 + 128 + l * 8, K, vec, nv, nu);
    const Quant q(row16_max(amax8(v)), 448.0f);
    const u32x2 c = {q.e4m3x4(v[0], v[1], v[2], v[3]), q.e4m3x4(v[4], v[5], v[6], v[7])};
    *reinterpret_cast<u32x2*>(codes + (size_t)m * KB * 128 + kb * 128 + l * 8) = c;
    if (l == 0) scale[(size_t)kb * M + m] = q.s;
  }
}

// Maximum over aligned groups of 8 lanes.
__device__ inline uint32_t lanes8_max(uint32_t x) {
  x = max(x, dpp<0xB1>(x));
  x = max(x, dpp<0x4E>(x));
  return max(x, dpp<0x141>(x));  // row_half_mirror: the other quad of the eight
}

// Column form, both forms, or 128 x 128 blocks.  A block of 512 threads holds
// a 128 x 128 tile in registers (16 lanes per row, 4 rows per thread); the
// columns pass through LDS 64 at a time (33 KiB: four blocks per CU, against
// two with the whole tile there, 22 us instead of 15.5), where eight lanes take
// a column, 16 rows each, so that they write 128 consecutive bytes.  Both forms
// of 4111 x 2048 in fp32: 15.5 us, 3.3 TB/s; the 528 blocks are on the chip at
// once and read together, then write together.
constexpr int kTileThreads = 512, kPitch = 65;
template <bool F32, bool ACT, bool BLOCK>
__global__ __launch_bounds__(kTileThreads) void fp8_quant_tile_kernel(
    const void* __restrict__ x, int M, int K, int KB, int MB, bool vec,
    uint8_t* __restrict__ codes, float* __restrict__ scale, uint8_t* __restrict__ codes_t,
    float* __restrict__ scale_t) {
  __shared__ float tile[128 * kPitch];
  __shared__ uint32_t part[kTileThreads / 64];
  const int kb = blockIdx.x, mb = blockIdx.y;
  const size_t b = blockIdx.z;  // matrix of a stack (blocks only)
  x = reinterpret_cast<const typename El<F32>::T*>(x) + b * M * (size_t)(ACT ? 2 * K : K);
  if (codes) codes += b * M * (size_t)KB * 128;
  if (codes_t) codes_t += b * K * (size_t)MB * 128;
  const int l = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  float v[4][8], u[4][8];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int m = mb * 128 + r0 + 32 * i;
    if (m < M) {
      load_vals<F32, ACT>(x, m, kb * 128 + l * 8, K, vec, v[i], u[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++) v[i][j] = u[i][j] = 0.f;
    }
  }
  if constexpr (ACT) {
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int j = 0; j < 8; j++) v[i][j] = silu_mul(v[i][j], u[i][j]);
  }
  uint32_t whole = 0;  // BLOCK: the tile's maximum
  if constexpr (BLOCK) {
#pragma unroll
    for (int i = 0; i < 4; i++) whole = max(whole, amax8(v[i]));
    whole = wave_max(whole);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = whole;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kTileThreads / 64; w++) whole = max(whole, part[w]);
    if (threadIdx.x == 0) {
      const Quant q(whole, 448.0f);
      if (codes) scale[(b * MB + mb) * KB + kb] = q.s;
      if (codes_t) scale_t[(b * KB + kb) * MB + mb] = q.s;
    }
  }
  if (codes) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int m = mb * 128 + r0 + 32 * i;
      const Quant q(BLOCK ? whole : row16_max(amax8(v[i])), 448.0f);
      if (m < M) {
        const u32x2 c = {q.e4m3x4(v[i][0], v[i][1], v[i][2], v[i][3]),
                         q.e4m3x4(v[i][4], v[i][5], v[i][6], v[i][7])};
        *reinterpret_cast<u32x2*>(codes + (size_t)m * KB * 128 + kb * 128 + l * 8) = c;
        if (!BLOCK && l == 0) scale[(size_t)kb * M + m] = q.s;
      }
    }
  }
  if (!codes_t) return;
  const int c = threadIdx.x >> 3, chunk = threadIdx.x & 7;
#pragma unroll
  for (int half = 0; half < 2; half++) {
    __syncthreads();
    if (l >> 3 == half) {
#pragma unroll
      for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 8; j++) tile[(r0 + 32 * i) * kPitch + (l & 7) * 8 + j] = v[i][j];
    }
    __syncthreads();
    float t[16];
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 16; i++) {
      t[i] = tile[(chunk * 16 + i) * kPitch + c];
      a = max(a, abs_bits(t[i]));
    }
    const Quant q(BLOCK ? whole : lanes8_max(a), 448.0f);
    const int col = kb * 128 + half * 64 + c;
    if (col < K) {
      u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; i++)
        w[i] = q.e4m3x4(t[4 * i], t[4 * i + 1], t[4 * i + 2], t[4 * i + 3]);
      *reinterpret_cast<u32x4*>(codes_t + (size_t)col * MB * 128 + mb * 128 + chunk * 16) = w;
      if (!BLOCK && chunk == 0) scale_t[(size_t)mb * K + col] = q.s;
    }
  }
}

template <bool F32, bool ACT>
hipError_t launch(const Fp8QuantArgs& a, hipStream_t s) {
  const int KB = (a.K + 127) / 128, MB = (a.M + 127) / 128;
  const size_t align = F32 ? 4 : 8;  // elements per 16 bytes
  const bool vec = a.K % align == 0 && a.K % 8 == 0 && (uintptr_t)a.x % 16 == 0;
  if (a.block) {
    if constexpr (!ACT) {
      hipLaunchKernelGGL((fp8_quant_tile_kernel<F32, false, true>), dim3(KB, MB, a.B),
                         dim3(kTileThreads), 0, s, a.x, a.M, a.K, KB, MB, vec, a.codes, a.scale,
                         a.codes_t, a.scale_t);
      return hipGetLastError();
    }
    return hipErrorInvalidValue;
  }
  if (a.codes_t) {
    hipLaunchKernelGGL((fp8_quant_tile_kernel<F32, ACT, false>), dim3(KB, MB, 1),
                       dim3(kTileThreads), 0, s, a.x, a.M, a.K, KB, MB, vec, a.codes, a.scale,
                       a.codes_t, a.scale_t);
    return hipGetLastError();
  }
  const int mb = (a.M + 15) / 16;
  int kspan = KB;
  while (kspan > 1 && (long long)mb * ((KB + kspan - 1) / kspan) < 2048) kspan = (kspan + 1) / 2;
  hipLaunchKernelGGL((fp8_quant_rows_kernel<F32, ACT>), dim3(mb, (KB + kspan - 1) / kspan),
                     dim3(256), 0, s, a.x, a.M, a.K, KB, kspan, vec, a.codes, a.scale);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_quant(const Fp8QuantArgs& a, hipStream_t s) {
  if (a.f32) return a.act ? launch<true, true>(a, s) : launch<true, false>(a, s);
  return a.act ? launch<false, true>(a, s) : launch<false, false>(a, s);
}

}  // namespace qmoe
