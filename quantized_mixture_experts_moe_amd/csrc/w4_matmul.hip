// Dense products with 4-bit weights and a scale per group of G values along K:
//
//   out[m,n] = sum_g s[n,g] * sum_{i<G} x[m, G g + i] q[n, G g + i]
//
// x bf16; q int4 (two's complement) with fp16 scales, G = 32, 64 or 128, or
// e2m1 with e8m0 scales, G = 32.  The inner sum runs on the matrix cores in
// fp32 over exact values of q, the scale multiplies it once, in fp32: no weight
// is rounded.
//
// int4 as bf16: with u = q ^ 8 = q + 8 in the four highest mantissa bits of 1.0,
// the pattern 0x3f80 | u << 3 is 1.5 + q / 16, two per word by one shift and one
// bit operation; the accumulator starts from -1.5 sum_i x (a matrix product with
// a constant, shared by the sub-tiles of columns), so that it ends as the sum of
// x q / 16.
#include "block_common.h"
#include "qmoe_internal.h"

namespace qmoe {
namespace {
using namespace bk;
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

enum { kInt4G32, kInt4G64, kInt4G128, kMxfp4 };

// Eight codes (element i in bits 4 i .. 4 i + 3) as bf16: 1.5 + q / 16 of an
// int4, the value of an e2m1.
template <int FMT>
__device__ inline bf16x8 widen8(uint32_t v) {
  if constexpr (FMT == kMxfp4) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 3);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  } else {
    const uint32_t u = v ^ 0x88888888u;
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; j++)
      // byte j times (2^3 + 2^15): its low nibble at bit 3, its high one at 19
      w[j] = (((u >> (8 * j)) & 0xffu) * 0x8008u & 0x00780078u) | 0x3f803f80u;
    return __builtin_bit_cast(bf16x8, w);
  }
}

// The scales of a step of 128 values of K, as loaded.
struct RawScale {
  uint32_t lo, hi;
};
// The scale of block i (32 values) of the step.
template <int FMT>
__device__ inline float scale_of(const RawScale& r, int i) {
  if constexpr (FMT == kMxfp4) {
    const uint32_t e = r.lo >> (8 * i) & 0xffu;
    // 2^(e - 127): 2^-127 is subnormal, 255 is no number
    return __uint_as_float(e == 0xffu ? 0x7fc00000u : e == 0u ? 0x00400000u : e << 23);
  } else {
    const int j = FMT == kInt4G32 ? i : FMT == kInt4G64 ? i / 2 : 0;
    const uint32_t w = j < 2 ? r.lo : r.hi;
    return (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> (16 * (j & 1))));
  }
}
constexpr int scales_per_step(int fmt) { return fmt == kInt4G64 ? 2 : fmt == kInt4G128 ? 1 : 4; }

// ---------------------------------------------------------------------------
// Few rows: the work is reading the codes once.  A block computes 16 MS rows x
// 16 NS columns, its KS waves taking every KS-th step of 128 values of K; the
// waves' sums are added in wave order through LDS.  A lane reads 16 bytes, the
// block of 32 codes q of its column's step (64 consecutive bytes of a column
// per four lanes); a 4 x 4 turn over the four lane groups then gives every lane
// its eight codes of each block, so that a matrix instruction sums one block.
// With act the two sub-tiles are gate and up columns.
template <int KS, int MS, int NS, int RING, int FMT>
__global__ __launch_bounds__(64 * KS) void w4_rows_kernel(W4Args g) {
  __shared__ f32x4 part[KS][MS * NS][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int l = lane & 15, q = lane >> 4;
  const int cols = g.act ? g.N / 2 : g.N;
  const int n0 = blockIdx.x * (g.act ? 16 : 16 * NS), m0 = blockIdx.y * 16 * MS;
  const int KB = (g.K + 127) / 128;
  const bool whole = g.K % 128 == 0;
  constexpr int SPS = scales_per_step(FMT), SB = FMT == kMxfp4 ? 1 : 2;  // scales, their bytes
  const int srow = g.K / (128 / SPS);  // scales per column
  const uint8_t* cp[NS];
  const uint8_t* sp[NS];
#pragma unroll
  for (int s = 0; s < NS; s++) {
    const int n = g.act ? s * cols + min(n0 + l, cols - 1) : min(n0 + 16 * s + l, cols - 1);
    cp[s] = g.codes + (size_t)n * (g.K / 2) + 16 * q;
    sp[s] = reinterpret_cast<const uint8_t*>(g.scale) + (size_t)n * srow * SB;
  }
  const uint16_t* xp[MS];
#pragma unroll
  for (int m = 0; m < MS; m++)
    xp[m] = g.x + (size_t)min(m0 + 16 * m + l, g.M - 1) * g.K + 8 * q;

  struct Step {
    u32x4 c[NS], x[MS][4];
    RawScale s[NS];
  };
  Step ring[RING];
  const u32x4 none = {0u, 0u, 0u, 0u};
  auto load = [&](Step& st, int kb) {
    const int at = kb * 128;
#pragma unroll
    for (int s = 0; s < NS; s++) {
      st.c[s] = at + 32 * q < g.K ? *reinterpret_cast<const u32x4*>(cp[s] + at / 2) : none;
      const uint8_t* p = sp[s] + (size_t)kb * SPS * SB;
      st.s[s] = RawScale{0u, 0u};
      if (whole) {  // (aligned: a step's scales are SPS * SB bytes)
        if constexpr (SPS * SB == 8) {
          const u32x2 v = *reinterpret_cast<const u32x2*>(p);
          st.s[s] = RawScale{v[0], v[1]};
        } else if constexpr (SPS * SB == 4) {
          st.s[s].lo = *reinterpret_cast<const uint32_t*>(p);
        } else {
          st.s[s].lo = *reinterpret_cast<const uint16_t*>(p);
        }
      } else {
#pragma unroll
        for (int j = 0; j < SPS; j++) {
          if (kb * SPS + j >= srow) continue;
          const uint32_t v = SB == 1 ? p[j] : reinterpret_cast<const uint16_t*>(p)[j];
          if (SB * j < 4)
            st.s[s].lo |= v << (8 * SB * j);
          else
            st.s[s].hi |= v << (8 * (SB * j - 4));
        }
      }
    }
#pragma unroll
    for (int m = 0; m < MS; m++)
#pragma unroll
      for (int i = 0; i < 4; i++)
        st.x[m][i] =
            at + 32 * i < g.K ? *reinterpret_cast<const u32x4*>(xp[m] + at + 32 * i) : none;
  };
  f32x4 acc[MS][NS];
#pragma unroll
  for (int m = 0; m < MS; m++)
#pragma unroll
    for (int s = 0; s < NS; s++) acc[m][s] = f32x4{0.f, 0.f, 0.f, 0.f};
  const __bf16 mb = __builtin_bit_cast(__bf16, (uint16_t)0xbfc0);  // -1.5
  const bf16x8 minus = {mb, mb, mb, mb, mb, mb, mb, mb};
  auto compute = [&](const Step& st) {
    u32x4 c[NS];
#pragma unroll
    for (int s = 0; s < NS; s++) {
      // (swaps of lane groups: 2, 3 of one register with 0, 1 of another, then
      // 1, 3 with 0, 2)
      const auto a = __builtin_amdgcn_permlane32_swap(st.c[s][0], st.c[s][2], false, false);
      const auto b = __builtin_amdgcn_permlane32_swap(st.c[s][1], st.c[s][3], false, false);
      const auto u = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
      const auto v = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
      c[s] = u32x4{(uint32_t)u[0], (uint32_t)u[1], (uint32_t)v[0], (uint32_t)v[1]};
    }
    constexpr int BPG = FMT == kInt4G64 ? 2 : FMT == kInt4G128 ? 4 : 1;  // blocks per group
#pragma unroll
    for (int i0 = 0; i0 < 4; i0 += BPG) {
      f32x4 z[MS];
#pragma unroll
      for (int m = 0; m < MS; m++) {
        z[m] = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (FMT != kMxfp4) {
#pragma unroll
          for (int i = i0; i < i0 + BPG; i++)
            z[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8, st.x[m][i]), minus, z[m], 0, 0, 0);
        }
      }
#pragma unroll
      for (int s = 0; s < NS; s++) {
        const float sc = scale_of<FMT>(st.s[s], i0);
        f32x4 t[MS];
#pragma unroll
        for (int m = 0; m < MS; m++) t[m] = z[m];
#pragma unroll
        for (int i = i0; i < i0 + BPG; i++) {
          const bf16x8 w = widen8<FMT>(c[s][i]);
#pragma unroll
          for (int m = 0; m < MS; m++)
            t[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                __builtin_bit_cast(bf16x8, st.x[m][i]), w, t[m], 0, 0, 0);
        }
#pragma unroll
        for (int m = 0; m < MS; m++)
#pragma unroll
          for (int r = 0; r < 4; r++) acc[m][s][r] = __builtin_fmaf(t[m][r], sc, acc[m][s][r]);
      }
    }
  };
#pragma unroll
  for (int u = 0; u < RING; u++)
    if (wave + u * KS < KB) load(ring[u], wave + u * KS);
  for (int k0 = wave; k0 < KB; k0 += RING * KS) {
#pragma unroll
    for (int u = 0; u < RING; u++) {
      const int kb = k0 + u * KS, next = kb + RING * KS;
      if (kb < KB) {
        compute(ring[u]);
        if (next < KB) load(ring[u], next);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MS; m++)
#pragma unroll
    for (int s = 0; s < NS; s++) part[wave][m * NS + s][lane] = acc[m][s];
  __syncthreads();
  auto total = [&](int j) {
    f32x4 v = part[0][j][lane];
#pragma unroll
    for (int w = 1; w < KS; w++) {
      const f32x4 y = part[w][j][lane];
#pragma unroll
      for (int r = 0; r < 4; r++) v[r] += y[r];
    }
    if constexpr (FMT != kMxfp4) {
#pragma unroll
      for (int r = 0; r < 4; r++) v[r] *= 16.f;
    }
    return v;
  };
  auto put = [&](int m, int n, const f32x4& v) {
    if (n >= cols) return;
#pragma unroll
    for (int r = 0; r < 4; r++) {
      const int row = m0 + 16 * m + 4 * q + r;
      if (row >= g.M) continue;
      const size_t o = (size_t)row * cols + n;
      if (g.out_f32)
        store1<true>(g.out, o, g.add ? load1<true>(g.add, o) + v[r] : v[r]);
      else
        store1<false>(g.out, o, g.add ? load1<false>(g.add, o) + v[r] : v[r]);
    }
  };
  if (g.act) {
    if constexpr (NS == 2) {
      for (int m = wave; m < MS; m += KS) {
        const f32x4 gate = total(2 * m), up = total(2 * m + 1);
        f32x4 v;
#pragma unroll
        for (int r = 0; r < 4; r++) v[r] = silu_mul(gate[r], up[r]);
        put(m, n0 + l, v);
      }
    }
  } else {
    for (int j = wave; j < MS * NS; j += KS) put(j / NS, n0 + 16 * (j % NS) + l, total(j));
  }
}

template <int KS, int MS, int NS, int RING, int FMT>
hipError_t launch_rows(const W4Args& g, hipStream_t s) {
  const int cols = g.act ? g.N / 2 : g.N, step = g.act ? 16 : 16 * NS;
  const int mt = (g.M + 16 * MS - 1) / (16 * MS);
  if (mt > 65535) return hipErrorInvalidValue;
  hipLaunchKernelGGL((w4_rows_kernel<KS, MS, NS, RING, FMT>), dim3((cols + step - 1) / step, mt),
                     dim3(64 * KS), 0, s, g);
  return hipGetLastError();
}

template <int FMT>
hipError_t launch(const W4Args& g, hipStream_t s) {
  if (g.M <= 16) return launch_rows<8, 1, 2, 2, FMT>(g, s);
  return launch_rows<8, 2, 2, 2, FMT>(g, s);
}

}  // namespace

size_t w4_matmul_parts_bytes(int, int, int) { return 0; }

hipError_t launch_w4_matmul(const W4Args& g, hipStream_t s) {
  if (g.mxfp4) return launch<kMxfp4>(g, s);
  return g.group == 32 ? launch<kInt4G32>(g, s)
                       : g.group == 64 ? launch<kInt4G64>(g, s) : launch<kInt4G128>(g, s);
}

}  // namespace qmoe
