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

// Value (m, c) of the source, zero outside it.
template <bool F32, bool ACT>
__device__ inline void load_vals(const void* x, size_t m, int c, int K, bool vec, float v[8]) {
  const size_t row = m * (size_t)(ACT ? 2 * (size_t)K : (size_t)K);
  if (vec && c + 8 <= K) {
    load8<F32>(x, row + c, v);
    if constexpr (ACT) {
      float u[8];
      load8<F32>(x, row + K + c, u);
#pragma unroll
      for (int j = 0; j < 8; j++) v[j] = silu_mul(v[j], u[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; j++) {
      v[j] = 0.f;
      if (c + j < K) {
        v[j] = load1<F32>(x, row + c + j);
        if constexpr (ACT) v[j] = silu_mul(v[j], load1<F32>(x, row + K + c + j));
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
// block of 16 rows and writes its 16 scales side by side.
template <bool F32, bool ACT>
__global__ __launch_bounds__(256) void fp8_quant_rows_kernel(const void* __restrict__ x, int M,
                                                             int K, int KB, int kspan, bool vec,
                                                             uint8_t* __restrict__ codes,
                                                             float* __restrict__ scale) {
  const int m = blockIdx.x * 16 + (threadIdx.x >> 4);
  const int l = threadIdx.x & 15;
  const int kb1 = min(KB, (int)(blockIdx.y + 1) * kspan);
  if (m >= M) return;  // whole 16-lane rows leave together
  for (int kb = blockIdx.y * kspan; kb < kb1; kb++) {
    float v[8];
    load_vals<F32, ACT>(x, m, kb * 128 + l * 8, K, vec, v);
    const Quant q(row16_max(amax8(v)), 448.0f);
    const u32x2 c = {q.e4m3x4(v[0], v[1], v[2], v[3]), q.e4m3x4(v[4], v[5], v[6], v[7])};
    *reinterpret_cast<u32x2*>(codes + (size_t)m * KB * 128 + kb * 128 + l * 8) = c;
    if (l == 0) scale[(size_t)kb * M + m] = q.s;
  }
}

// Column form, both forms, or 128 x 128 blocks: a block of 256 threads holds
// a 128 x 128 tile of values in LDS (fp32, pitch 129 words: a wave walks 64
// columns of one row, or one column, without bank conflicts).
constexpr int kPitch = 129;
template <bool F32, bool ACT, bool BLOCK>
__global__ __launch_bounds__(256) void fp8_quant_tile_kernel(
    const void* __restrict__ x, int M, int K, int KB, int MB, bool vec,
    uint8_t* __restrict__ codes, float* __restrict__ scale, uint8_t* __restrict__ codes_t,
    float* __restrict__ scale_t) {
  __shared__ float tile[128 * kPitch];
  __shared__ uint32_t part[4];
  const int kb = blockIdx.x, mb = blockIdx.y;
  const size_t b = blockIdx.z;  // matrix of a stack (blocks only)
  x = reinterpret_cast<const typename El<F32>::T*>(x) + b * M * (size_t)(ACT ? 2 * K : K);
  if (codes) codes += b * M * (size_t)KB * 128;
  if (codes_t) codes_t += b * K * (size_t)MB * 128;
  const int l = threadIdx.x & 15;
  uint32_t whole = 0;
  for (int r = threadIdx.x >> 4; r < 128; r += 16) {
    const int m = mb * 128 + r;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (m < M) load_vals<F32, ACT>(x, m, kb * 128 + l * 8, K, vec, v);
#pragma unroll
    for (int j = 0; j < 8; j++) tile[r * kPitch + l * 8 + j] = v[j];
    const uint32_t a = amax8(v);
    if constexpr (BLOCK) {
      whole = max(whole, a);
    } else if (codes) {
      const Quant q(row16_max(a), 448.0f);
      if (m < M) {
        const u32x2 c = {q.e4m3x4(v[0], v[1], v[2], v[3]), q.e4m3x4(v[4], v[5], v[6], v[7])};
        *reinterpret_cast<u32x2*>(codes + (size_t)m * KB * 128 + kb * 128 + l * 8) = c;
        if (l == 0) scale[(size_t)kb * M + m] = q.s;
      }
    }
  }
  if constexpr (BLOCK) {
    whole = wave_max(whole);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = whole;
  }
  __syncthreads();
  if constexpr (BLOCK) {
    const Quant q(max(max(part[0], part[1]), max(part[2], part[3])), 448.0f);
    if (threadIdx.x == 0) {
      if (codes) scale[(b * MB + mb) * KB + kb] = q.s;
      if (codes_t) scale_t[(b * KB + kb) * MB + mb] = q.s;
    }
    if (codes) {
      for (int r = threadIdx.x >> 4; r < 128; r += 16) {
        const int m = mb * 128 + r;
        const float* v = tile + r * kPitch + l * 8;
        if (m < M) {
          const u32x2 c = {q.e4m3x4(v[0], v[1], v[2], v[3]), q.e4m3x4(v[4], v[5], v[6], v[7])};
          *reinterpret_cast<u32x2*>(codes + (size_t)m * KB * 128 + kb * 128 + l * 8) = c;
        }
      }
    }
  }
  if (!codes_t) return;
  // Columns: two threads per column, 64 rows each.
  const int c = threadIdx.x & 127, half = threadIdx.x >> 7;
  const int col = kb * 128 + c;
  __shared__ uint32_t cmax[2][128];
  uint32_t a = 0;
  if constexpr (!BLOCK) {
    for (int r = 0; r < 64; r++) a = max(a, abs_bits(tile[(half * 64 + r) * kPitch + c]));
    cmax[half][c] = a;
    __syncthreads();
    a = max(cmax[0][c], cmax[1][c]);
  } else {
    a = max(max(part[0], part[1]), max(part[2], part[3]));
  }
  if (col >= K) return;
  const Quant q(a, 448.0f);
  if (!BLOCK && half == 0) scale_t[(size_t)mb * K + col] = q.s;
  uint8_t* dst = codes_t + (size_t)col * MB * 128 + mb * 128 + half * 64;
#pragma unroll
  for (int g = 0; g < 4; g++) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float* v = tile + (half * 64 + g * 16 + i * 4) * kPitch + c;
      w[i] = q.e4m3x4(v[0], v[kPitch], v[2 * kPitch], v[3 * kPitch]);
    }
    *reinterpret_cast<u32x4*>(dst + g * 16) = w;
  }
}

template <bool F32, bool ACT>
hipError_t launch(const Fp8QuantArgs& a, hipStream_t s) {
  const int KB = (a.K + 127) / 128, MB = (a.M + 127) / 128;
  const size_t align = F32 ? 4 : 8;  // elements per 16 bytes
  const bool vec = a.K % align == 0 && a.K % 8 == 0 && (uintptr_t)a.x % 16 == 0;
  if (a.block) {
    if constexpr (!ACT) {
      hipLaunchKernelGGL((fp8_quant_tile_kernel<F32, false, true>), dim3(KB, MB, a.B), dim3(256),
                         0, s, a.x, a.M, a.K, KB, MB, vec, a.codes, a.scale, a.codes_t,
                         a.scale_t);
      return hipGetLastError();
    }
    return hipErrorInvalidValue;
  }
  if (a.codes_t) {
    hipLaunchKernelGGL((fp8_quant_tile_kernel<F32, ACT, false>), dim3(KB, MB, 1), dim3(256), 0, s,
                       a.x, a.M, a.K, KB, MB, vec, a.codes, a.scale, a.codes_t, a.scale_t);
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
