// Dense products with 4-bit weights and a scale per group of G values along K:
//
//   out[m,n] = sum_g s[n,g] * sum_{i<G} x[m, G g + i] q[n, G g + i]
//
// x bf16; q int4 (two's complement) with fp16 scales, G = 32, 64 or 128, or
// e2m1 with e8m0 scales, G = 32.  The inner sum runs on the matrix cores in
// fp32 over exact values of q, the scale multiplies it once, in fp32: no weight
// is rounded.
//
// An int4 code enters as q / 16, exact in bf16: a code of 0 adds nothing, whatever x
// holds there, and a sum's error is a fraction of sum |x q|.  (The pattern 0x3f80 | (q +
// 8) << 3 of 1.5 + q / 16 takes 9 instead of 13 instructions for eight codes, but its
// 1.5 comes off by a product of x with a constant, after both are rounded: an error of 24
// sum |x| half steps, also where all codes are 0.)
//
// Measured (int4 in groups of 32 unless said): 1 x 4096 x 4096 5.1 us, 9.4 MB at 1.8
// TB/s, bound by the launch, a trip to memory and the joining of the waves; 1 x 65536
// x 4096, groups of 128, fp32 out, 32-36 us, 139 MB at 3.9-4.3 TB/s; 1500 x 4096 x 2048
// with add 48-55 us, 0.46-0.52 PFLOP/s.
#include "block_common.h"
#include "qmoe_internal.h"
#include "tile_common.h"

namespace qmoe {
namespace {
using namespace bk;
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

enum { kInt4G32, kInt4G64, kInt4G128, kMxfp4 };

// Eight codes (element i in bits 4 i .. 4 i + 3) as bf16: q / 16 of an int4, the value
// of an e2m1.
template <int FMT>
__device__ inline bf16x8 widen8(uint32_t v) {
  if constexpr (FMT == kMxfp4) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.0f, 3);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  } else {
    // The conversion takes the low four bits of a byte as q, and gives q / 16 in fp32,
    // whose lower half is 0.
    uint32_t o = v >> 4;
    asm("" : "+v"(o));  // (one shift: the bytes are the conversion's operands)
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const float even = __builtin_amdgcn_cvt_off_f32_i4((int)(v >> (8 * j) & 0xffu));
      const float odd = __builtin_amdgcn_cvt_off_f32_i4((int)(o >> (8 * j) & 0xffu));
      w[j] = __builtin_amdgcn_perm(__float_as_uint(odd), __float_as_uint(even), 0x07060302u);
    }
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
// The scales of step kb of a column whose `count` scales begin at p; whole: K is a
// multiple of 128, so that a step's are aligned together.
template <int FMT>
__device__ inline RawScale load_scale(const uint8_t* p, int kb, int count, bool whole) {
  constexpr int SPS = scales_per_step(FMT), SB = FMT == kMxfp4 ? 1 : 2;
  RawScale r = {0u, 0u};
  p += (size_t)kb * SPS * SB;
  if (whole) {
    if constexpr (SPS * SB == 8) {
      const u32x2 v = *reinterpret_cast<const u32x2*>(p);
      r = RawScale{v[0], v[1]};
    } else if constexpr (SPS * SB == 4) {
      r.lo = *reinterpret_cast<const uint32_t*>(p);
    } else {
      r.lo = *reinterpret_cast<const uint16_t*>(p);
    }
  } else {
#pragma unroll
    for (int j = 0; j < SPS; j++) {
      if (kb * SPS + j >= count) continue;
      const uint32_t v = SB == 1 ? p[j] : reinterpret_cast<const uint16_t*>(p)[j];
      if (SB * j < 4)
        r.lo |= v << (8 * SB * j);
      else
        r.hi |= v << (8 * (SB * j - 4));
    }
  }
  return r;
}

// N values of out at o[r] (those with in[r]); add's are loaded before the first store
// (add may be out).
template <int N>
__device__ inline void put(const W4Args& g, const size_t (&o)[N], const bool (&in)[N],
                           float (&v)[N]) {
  if (g.add != nullptr) {
    float a[N];
#pragma unroll
    for (int r = 0; r < N; r++)
      a[r] = !in[r] ? 0.f : g.out_f32 ? load1<true>(g.add, o[r]) : load1<false>(g.add, o[r]);
#pragma unroll
    for (int r = 0; r < N; r++) v[r] += a[r];
  }
#pragma unroll
  for (int r = 0; r < N; r++) {
    if (!in[r]) continue;
    if (g.out_f32)
      store1<true>(g.out, o[r], v[r]);
    else
      store1<false>(g.out, o[r], v[r]);
  }
}

// ---------------------------------------------------------------------------
// Few rows: the work is reading the codes once.  A block computes 16 MS rows x
// 16 NS columns, each of its KS waves a run of K's steps of 128 values; the waves'
// sums are added in wave order through LDS.  A lane reads 16 bytes, the block of
// 32 codes q of its column's step (64 consecutive bytes of a column per four
// lanes); a 4 x 4 turn over the four lane groups then gives every lane its eight
// codes of each block, so that a matrix instruction sums one block.  With act the
// two sub-tiles are gate and up columns.
//
// What bounds it beside the bytes is the number of loads: 16 lanes of a scale's or
// x's load look up 16 lines.  So the scales of kGroup steps come in one load, and
// up to four rows of x (FOUR) in one load per step: lanes 4 i .. 4 i + 3 of a row of
// 16 read block i, which moves down to lanes 0 .. 3 in front of its product (the
// rows behind hold other blocks' values, and are not stored).  One token, 65536
// columns of 4096 values, group 128: 43 us with a load per step each, 31 without the
// scales', 35 without x's.
template <int FMT>
constexpr int group_steps() {
  return FMT == kInt4G32 ? 2 : 4;
}

template <int KS, int MS, int NS, int RING, bool FOUR, int FMT>
__global__ __launch_bounds__(64 * KS) void w4_rows_kernel(W4Args g) {
  static_assert(!FOUR || MS == 1, "four rows");
  constexpr int SV = group_steps<FMT>();
  static_assert(SV % RING == 0, "a step's slot is known");
  __shared__ f32x4 part[KS][MS * NS][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int l = lane & 15, q = lane >> 4;
  const int cols = g.act ? g.N / 2 : g.N;
  const int n0 = blockIdx.x * (g.act ? 16 : 16 * NS), m0 = blockIdx.y * 16 * MS;
  const int KB = (g.K + 127) / 128;
  constexpr int SPS = scales_per_step(FMT), SB = FMT == kMxfp4 ? 1 : 2;  // scales, their bytes
  constexpr int BYTES = SPS * SB * SV;  // of a group's scales: 16, or 8
  const int srow = g.K / (128 / SPS);  // scales per column
  const bool whole = g.K % 128 == 0, wide = srow * SB % BYTES == 0;
  // The wave's steps, a whole number of groups.
  const int per = (KB + KS * SV - 1) / (KS * SV) * SV;
  const int first = wave * per, end = min(KB, first + per);
  const uint8_t* cp[NS];
  const uint8_t* sp[NS];
#pragma unroll
  for (int s = 0; s < NS; s++) {
    const int n = g.act ? s * cols + min(n0 + l, cols - 1) : min(n0 + 16 * s + l, cols - 1);
    cp[s] = g.codes + (size_t)n * (g.K / 2) + 16 * q;
    sp[s] = reinterpret_cast<const uint8_t*>(g.scale) + (size_t)n * srow * SB;
  }
  const uint16_t* xp[MS];
  bool there[MS];  // (rows that are not there are not read)
#pragma unroll
  for (int m = 0; m < MS; m++) {
    const int row = m0 + (FOUR ? l & 3 : 16 * m + l);
    there[m] = row < g.M;
    xp[m] = g.x + (size_t)min(row, g.M - 1) * g.K + 8 * q;
  }

  struct Step {
    u32x4 c[NS], x[MS][FOUR ? 1 : 4];
  };
  Step ring[RING];
  const u32x4 none = {0u, 0u, 0u, 0u};
  auto load = [&](Step& st, int kb) {
    const int at = kb * 128;
#pragma unroll
    for (int s = 0; s < NS; s++)
      st.c[s] = at + 32 * q < g.K ? *reinterpret_cast<const u32x4*>(cp[s] + at / 2) : none;
#pragma unroll
    for (int m = 0; m < MS; m++) {
      if constexpr (FOUR) {
        const int i = l >> 2;
        st.x[m][0] = there[m] && at + 32 * i < g.K
                         ? *reinterpret_cast<const u32x4*>(xp[m] + at + 32 * i)
                         : none;
      } else {
#pragma unroll
        for (int i = 0; i < 4; i++)
          st.x[m][i] = there[m] && at + 32 * i < g.K
                           ? *reinterpret_cast<const u32x4*>(xp[m] + at + 32 * i)
                           : none;
      }
    }
  };
  typedef RawScale Scales[SV][NS];
  auto load_scales = [&](Scales& r, int kb) {
#pragma unroll
    for (int s = 0; s < NS; s++) {
      if (wide) {  // (whole groups of a column's scales, aligned)
        uint32_t w[4];
        if constexpr (BYTES == 16) {
          const u32x4 v = *reinterpret_cast<const u32x4*>(sp[s] + (size_t)kb * SPS * SB);
#pragma unroll
          for (int j = 0; j < 4; j++) w[j] = v[j];
        } else {
          const u32x2 v = *reinterpret_cast<const u32x2*>(sp[s] + (size_t)kb * SPS * SB);
          w[0] = v[0];
          w[1] = v[1];
        }
#pragma unroll
        for (int u = 0; u < SV; u++) {
          if constexpr (SPS * SB == 8)
            r[u][s] = RawScale{w[2 * u], w[2 * u + 1]};
          else if constexpr (SPS * SB == 4)
            r[u][s] = RawScale{w[u], 0u};
          else
            r[u][s] = RawScale{w[u / 2] >> (16 * (u & 1)), 0u};
        }
      } else {
#pragma unroll
        for (int u = 0; u < SV; u++)
          r[u][s] = kb + u < KB ? load_scale<FMT>(sp[s], kb + u, srow, whole) : RawScale{0u, 0u};
      }
    }
  };
  f32x4 acc[MS][NS];
#pragma unroll
  for (int m = 0; m < MS; m++)
#pragma unroll
    for (int s = 0; s < NS; s++) acc[m][s] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const Step& st, const RawScale (&sc)[NS]) {
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
    bf16x8 x[MS][4];
#pragma unroll
    for (int m = 0; m < MS; m++) {
      if constexpr (FOUR) {
        const u32x4 v = st.x[m][0];
        u32x4 d;
        x[m][0] = __builtin_bit_cast(bf16x8, v);
#pragma unroll
        for (int j = 0; j < 4; j++) d[j] = dpp<0x104>(v[j]);  // row_shl 4
        x[m][1] = __builtin_bit_cast(bf16x8, d);
#pragma unroll
        for (int j = 0; j < 4; j++) d[j] = dpp<0x108>(v[j]);  // row_shl 8
        x[m][2] = __builtin_bit_cast(bf16x8, d);
#pragma unroll
        for (int j = 0; j < 4; j++) d[j] = dpp<0x10C>(v[j]);  // row_shl 12
        x[m][3] = __builtin_bit_cast(bf16x8, d);
      } else {
#pragma unroll
        for (int i = 0; i < 4; i++) x[m][i] = __builtin_bit_cast(bf16x8, st.x[m][i]);
      }
    }
    constexpr int BPG = FMT == kInt4G64 ? 2 : FMT == kInt4G128 ? 4 : 1;  // blocks per group
#pragma unroll
    for (int i0 = 0; i0 < 4; i0 += BPG) {
#pragma unroll
      for (int s = 0; s < NS; s++) {
        const float f = scale_of<FMT>(sc[s], i0);
        f32x4 t[MS];
#pragma unroll
        for (int m = 0; m < MS; m++) t[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = i0; i < i0 + BPG; i++) {
          const bf16x8 w = widen8<FMT>(c[s][i]);
#pragma unroll
          for (int m = 0; m < MS; m++)
            t[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[m][i], w, t[m], 0, 0, 0);
        }
#pragma unroll
        for (int m = 0; m < MS; m++)
#pragma unroll
          for (int r = 0; r < 4; r++) acc[m][s][r] = __builtin_fmaf(t[m][r], f, acc[m][s][r]);
      }
    }
  };
  Scales sc, next;
  if (first < end) {
    load_scales(sc, first);
#pragma unroll
    for (int u = 0; u < RING; u++)
      if (first + u < end) load(ring[u], first + u);
  }
  for (int k0 = first; k0 < end; k0 += SV) {
    if (k0 + SV < end) load_scales(next, k0 + SV);
#pragma unroll
    for (int u = 0; u < SV; u++) {
      if (k0 + u < end) {
        compute(ring[u % RING], sc[u]);
        if (k0 + u + RING < end) load(ring[u % RING], k0 + u + RING);
      }
    }
#pragma unroll
    for (int u = 0; u < SV; u++)
#pragma unroll
      for (int s = 0; s < NS; s++) sc[u][s] = next[u][s];
  }
#pragma unroll
  for (int m = 0; m < MS; m++)
#pragma unroll
    for (int s = 0; s < NS; s++) part[wave][m * NS + s][lane] = acc[m][s];
  __syncthreads();
  auto total = [&](int j) {
    f32x4 v = part[0][j][lane];
#pragma unroll 4
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
  auto store = [&](int m, int n, const f32x4& v) {
    size_t o[4];
    bool in[4];
    float w[4];
#pragma unroll
    for (int r = 0; r < 4; r++) {
      const int row = m0 + 16 * m + 4 * q + r;
      o[r] = (size_t)row * cols + n;
      in[r] = n < cols && row < g.M;
      w[r] = v[r];
    }
    put<4>(g, o, in, w);
  };
  if (g.act) {
    if constexpr (NS == 2) {
      for (int m = wave; m < MS; m += KS) {
        const f32x4 gate = total(2 * m), up = total(2 * m + 1);
        f32x4 v;
#pragma unroll
        for (int r = 0; r < 4; r++) v[r] = silu_mul(gate[r], up[r]);
        store(m, n0 + l, v);
      }
    }
  } else {
    for (int j = wave; j < MS * NS; j += KS) store(j / NS, n0 + 16 * (j % NS) + l, total(j));
  }
}

template <int KS, int MS, int NS, int RING, bool FOUR, int FMT>
hipError_t launch_rows(const W4Args& g, hipStream_t s) {
  const int cols = g.act ? g.N / 2 : g.N, step = g.act ? 16 : 16 * NS;
  const int mt = (g.M + 16 * MS - 1) / (16 * MS);
  if (mt > 65535 || (g.act && NS != 2)) return hipErrorInvalidValue;
  hipLaunchKernelGGL((w4_rows_kernel<KS, MS, NS, RING, FOUR, FMT>),
                     dim3((cols + step - 1) / step, mt), dim3(64 * KS), 0, s, g);
  return hipGetLastError();
}

// KS waves x NS sub-tiles, 16 rows (32 where there are more than 16).  One sub-tile
// gives the most blocks, two or four share x's loads; us (rows x columns x K, int4 in
// groups of 32):
//                        8x1    8x2    4x4
//   1 x 4096 x 4096       5.1    7.0   12.4
//   4 x 12288 x 2048      6.8    7.3    8.2
//   1 x 32768 x 4096     21.4   20.7   23.2
//   16 x 4096 x 4096      7.7    9.4   13.5
//   8 x 8192 x 4096      10.3    8.6   14.2
//   12 x 12288 x 2048     9.9   10.2    8.5
//   16 x 32768 x 4096    42.8   34.4   25.8
template <int FMT>
hipError_t rows(const W4Args& g, hipStream_t s) {
  const int cols = g.act ? g.N / 2 : g.N, cus = device_cu_count();
  if (g.M > 16) return launch_rows<8, 2, 2, 1, false, FMT>(g, s);
  if (g.M <= 4) {
    if (g.act || cols >= 48 * cus) return launch_rows<8, 1, 2, 2, true, FMT>(g, s);
    return launch_rows<8, 1, 1, 2, true, FMT>(g, s);
  }
  if (g.act || (cols >= 24 * cus && cols < 40 * cus))
    return launch_rows<8, 1, 2, 2, false, FMT>(g, s);
  return cols < 24 * cus ? launch_rows<8, 1, 1, 2, false, FMT>(g, s)
                         : launch_rows<4, 1, 4, 1, false, FMT>(g, s);
}

// ---------------------------------------------------------------------------
// Many rows: a block of WM x WN waves computes BM rows x BN columns, a wave SM x SN
// sub-tiles of 32 x 32, in K blocks of 128 values that go from memory straight into
// LDS, two stages: x as two halves of 64 values (128 bytes per row, 16-byte chunks in
// the order c ^ (row / 2 % 8)), the codes as they are (64 bytes per column, 16-byte
// units in the order u ^ (column / 4 % 4)); the scales go to registers.  x is the
// matrix core's row operand and the weights its column operand, so that a lane's
// results share a column and its scale.  Of a block of 32 values lane half h holds
// values 16 h .. 16 h + 15, eight per instruction.
//
// Bound: every 32 values of K a lane scales 16 sums per sub-tile and widens 16 codes
// per column, 491 vector instructions beside 32 matrix ones per K block (int4, groups
// of 32).  At 2048 x 4096 x 4096 (105 us, 0.65 PFLOP/s) the matrix cores are busy 29%
// of the time, the vector units 62%: they hardly run at once, whatever the order
// of the two.  MXFP4's codes take a third of the instructions to widen: 91 us, 34% and
// 58%; groups of 128 a quarter of the scalings: 83 us.
template <int BM_, int BN_, int WM_, int WN_>
struct W4Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int SM = BM / WM / 32, SN = BN / WN / 32;
  static constexpr int XC = BM / 4 / WAVES, CC = BN / 16 / WAVES;  // copies per wave, K block
  static constexpr int C_AT = BM * 256, STAGE = C_AT + BN * 64;
  static_assert(SM * WM * 32 == BM && SN * WN * 32 == BN && SN % 2 == 0, "whole sub-tiles");
  static_assert(XC * WAVES * 4 == BM && CC * WAVES * 16 == BN, "whole copies");
  static_assert(2 * STAGE <= 80 * 1024, "two blocks on a CU");
};

template <class C, int FMT>
__global__ __launch_bounds__(C::THREADS, 2) void w4_tile_kernel(W4Args g) {
  constexpr int SM = C::SM, SN = C::SN;
  constexpr int SPS = scales_per_step(FMT), SB = FMT == kMxfp4 ? 1 : 2;
  __shared__ __align__(1024) uint8_t lds[2 * C::STAGE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave % C::WM, wn = wave / C::WM;
  const int r32 = lane & 31, h = lane >> 5;
  // With act the sub-tiles are gate and up columns in turn.
  const int cols = g.act ? g.N / 2 : g.N, tn = g.act ? C::BN / 2 : C::BN;
  const int ntn = (cols + tn - 1) / tn, ntm = (g.M + C::BM - 1) / C::BM;
  // Each XCD takes a contiguous run of tiles, column-tile by column-tile inside
  // bands of kBand row tiles.
  constexpr int kBand = 8;
  const int total = ntn * ntm, per = (total + 7) / 8;
  const int id = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8);
  if (id >= total || (int)(blockIdx.x / 8) >= per) return;
  const int band = id / (kBand * ntn), in = id - band * kBand * ntn;
  const int rows = min(kBand, ntm - band * kBand);
  const int m0 = (band * kBand + in % rows) * C::BM, n0 = in / rows * tn;
  const int kb0 = blockIdx.y * g.split_kb, kb1 = min((g.K + 127) / 128, kb0 + g.split_kb);
  const bool whole = g.K % 128 == 0;
  // Weight row of the tile's column c (behind the last one: none).
  auto weight_row = [&](int c) {
    return g.act ? (c / 32 & 1) * cols + n0 + c / 64 * 32 + c % 32 : n0 + c;
  };
  const unsigned xrow = 2u * (unsigned)g.K, crow = (unsigned)g.K / 2;
  const Rsrc rx = rsrc(g.x + (size_t)m0 * g.K, (size_t)min(g.M - m0, C::BM) * xrow);
  const unsigned swz[2] = {16u * ((lane & 7) ^ ((lane >> 4) & 7)),
                           16u * ((lane & 7) ^ ((4 + (lane >> 4)) & 7))};
  auto copy = [&](uint8_t* st, int kb, int c) {
    const unsigned any = kb < kb1 ? 1 : 0;
    if (c < C::XC) {
      // 8 lanes per row: rows 8 t .. 8 t + 7 of half `half`
      const int u = wave * C::XC + c, half = u / (C::BM / 8), t = u % (C::BM / 8);
      const unsigned from = any * (kb * 256 + half * 128), left = xrow > from ? xrow - from : 0;
      const unsigned ch = t & 1 ? swz[1] : swz[0];
      const unsigned v = (unsigned)(t * 8 + (lane >> 3)) * xrow + ch;
      copy16(rx, any && ch < left ? v : kNowhere, from, st + half * C::BM * 128 + t * 1024);
    } else {
      // 4 lanes per column: columns 16 t .. 16 t + 15
      const int t = wave * C::CC + (c - C::XC), col = t * 16 + (lane >> 2);
      const unsigned from = any * kb * 64, left = crow - from;
      const unsigned ch = 16u * ((lane & 3) ^ ((col >> 2) & 3));
      const int first = weight_row(t * 16);  // (its 16 columns are consecutive rows)
      const Rsrc rc =
          rsrc(g.codes + (size_t)first * crow, (size_t)(min(max(g.N - first, 0), 16) * any) * crow);
      copy16(rc, ch < left ? (unsigned)(lane >> 2) * crow + ch : kNowhere, from,
             st + C::C_AT + t * 1024);
    }
  };
  // The scales of the lane's columns (in every half), one K block ahead.
  const int srow = g.K / (128 / SPS);
  const uint8_t* sp[SN];
#pragma unroll
  for (int i = 0; i < SN; i++)
    sp[i] = reinterpret_cast<const uint8_t*>(g.scale) +
            (size_t)min(weight_row((wn * SN + i) * 32 + r32), g.N - 1) * srow * SB;
  auto load_scales = [&](RawScale (&r)[SN], int kb) {
#pragma unroll
    for (int i = 0; i < SN; i++)
      r[i] = load_scale<FMT>(sp[i], kb < kb1 ? kb : kb1 - 1, srow, whole);
  };
  int off[2][2];  // x: (block of 32 in its half, instruction)
#pragma unroll
  for (int b = 0; b < 2; b++)
#pragma unroll
    for (int s = 0; s < 2; s++)
      off[b][s] = r32 * 128 + 16 * ((4 * b + 2 * h + s) ^ ((r32 >> 1) & 7));
  f32x16 acc[SM][SN];
#pragma unroll
  for (int j = 0; j < SM; j++)
#pragma unroll
    for (int i = 0; i < SN; i++)
#pragma unroll
      for (int r = 0; r < 16; r++) acc[j][i][r] = 0.f;
  auto block = [&](const uint8_t* __restrict__ st, uint8_t* __restrict__ nx, int kb,
                   const RawScale (&sc)[SN]) {
#pragma unroll
    for (int c = 0; c < C::XC + C::CC; c++) copy(nx, kb + 1, c);
    // Blocks per group that are summed before the scale (64 values: two have one scale).
    constexpr int BPG = FMT == kInt4G128 ? 4 : 1;
    constexpr int AHEAD = BPG == 1 ? 2 : 1;  // blocks in registers
    bf16x8 x[AHEAD][SM][2], w[AHEAD][SN][2];
    u32x2 c[SN];
    auto read = [&](int b) {
#pragma unroll
      for (int j = 0; j < SM; j++)
#pragma unroll
        for (int s = 0; s < 2; s++)
          x[b % AHEAD][j][s] = __builtin_bit_cast(
              bf16x8, *reinterpret_cast<const u32x4*>(st + (b / 2) * C::BM * 128 +
                                                      (j * C::WM + wm) * 4096 + off[b & 1][s]));
#pragma unroll
      for (int i = 0; i < SN; i++)
        c[i] = *reinterpret_cast<const u32x2*>(
            st + C::C_AT + ((wn * SN + i) * 32 + r32) * 64 + 16 * (b ^ ((r32 >> 2) & 3)) + 8 * h);
    };
    auto widen = [&](int b) {
#pragma unroll
      for (int i = 0; i < SN; i++)
#pragma unroll
        for (int s = 0; s < 2; s++) w[b % AHEAD][i][s] = widen8<FMT>(c[i][s]);
    };
    f32x16 zero;
#pragma unroll
    for (int r = 0; r < 16; r++) zero[r] = 0.f;
    read(0);
    widen(0);
    if constexpr (BPG == 1) {
      // Row q % SM of sub-tiles in block q / SM.  Between its matrix instructions run
      // the scaling of the row before and the widening of the next block's codes, which
      // are as long.
      f32x16 t[2][SN];
      float f[2][SN];
      auto scaled = [&](int q) {
#pragma unroll
        for (int i = 0; i < SN; i++)
#pragma unroll
          for (int r = 0; r < 16; r++)
            acc[q % SM][i][r] =
                __builtin_fmaf(t[q & 1][i][r], f[q / SM & 1][i], acc[q % SM][i][r]);
      };
#pragma unroll
      for (int q = 0; q < 4 * SM; q++) {
        const int b = q / SM, j = q % SM;
        if (j == 0) {
#pragma unroll
          for (int i = 0; i < SN; i++) f[b & 1][i] = scale_of<FMT>(sc[i], b);
          if (b < 3) read(b + 1);
        }
#pragma unroll
        for (int s = 0; s < 2; s++)
#pragma unroll
          for (int i = 0; i < SN; i++)
            t[q & 1][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                x[b % AHEAD][j][s], w[b % AHEAD][i][s], s == 0 ? zero : t[q & 1][i], 0, 0, 0);
        if (q > 0) scaled(q - 1);
        if (j == SM - 1 && b < 3) widen(b + 1);
#pragma unroll
        for (int m = 0; m < 2 * SN; m++) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // a matrix instruction
          __builtin_amdgcn_sched_group_barrier(0x002, 10, 0);  // vector instructions
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      scaled(4 * SM - 1);
    } else {
      f32x16 t[SM][SN];
#pragma unroll
      for (int b = 0; b < 4; b++) {
        if (b > 0) {
          read(b);
          widen(b);
        }
#pragma unroll
        for (int j = 0; j < SM; j++) {
#pragma unroll
          for (int s = 0; s < 2; s++) {
#pragma unroll
            for (int i = 0; i < SN; i++)
              t[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                  x[b % AHEAD][j][s], w[b % AHEAD][i][s], b == 0 && s == 0 ? zero : t[j][i], 0, 0,
                  0);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int j = 0; j < SM; j++)
#pragma unroll
        for (int i = 0; i < SN; i++) {
          const float s = scale_of<FMT>(sc[i], 0);
#pragma unroll
          for (int r = 0; r < 16; r++)
            acc[j][i][r] = __builtin_fmaf(t[j][i][r], s, acc[j][i][r]);
        }
    }
  };
  RawScale sc[SN], next[SN];
#pragma unroll
  for (int c = 0; c < C::XC + C::CC; c++) copy(lds, kb0, c);
  load_scales(sc, kb0);
  uint8_t *st = lds, *nx = lds + C::STAGE;
  for (int kb = kb0; kb < kb1; kb++) {
    wait_memory<0>();
    block_barrier();
    load_scales(next, kb + 1);
    block(st, nx, kb, sc);
#pragma unroll
    for (int i = 0; i < SN; i++) sc[i] = next[i];
    uint8_t* const t = nx;
    nx = st;
    st = t;
  }
  wait_memory<0>();  // no copy is under way when the block ends
  constexpr float UNIT = FMT == kMxfp4 ? 1.f : 16.f;
  // A lane holds rows 8 (r / 4) + 4 h + r % 4 of its column.
  float* const parts = g.parts + (size_t)blockIdx.y * g.M * g.N;
  const bool vec = cols % 8 == 0 && ((uintptr_t)g.out | (uintptr_t)g.add) % 16 == 0;
  __syncthreads();  // the last K block has been read
#pragma unroll
  for (int j = 0; j < SM; j++) {
    const int mrow = m0 + (j * C::WM + wm) * 32 + 4 * h;
    if (g.splits > 1) {
#pragma unroll
      for (int i = 0; i < SN; i++) {
        const int c = (wn * SN + i) * 32 + r32, n = weight_row(c);
        const bool in = (g.act ? n - (c / 32 & 1) * cols : n) < cols;
#pragma unroll
        for (int r = 0; r < 16; r++) {
          const int m = mrow + 8 * (r >> 2) + (r & 3);
          if (in && m < g.M) parts[(size_t)m * g.N + n] = acc[j][i][r] * UNIT;
        }
      }
      continue;
    }
#pragma unroll
    for (int i = 0; i < SN; i++) {
      if (g.act && (i & 1)) continue;
      const int n = g.act ? n0 + (wn * SN + i) / 2 * 32 + r32 : n0 + (wn * SN + i) * 32 + r32;
      float v[16];
#pragma unroll
      for (int r = 0; r < 16; r++) {
        v[r] = acc[j][i][r] * UNIT;
        if (g.act) v[r] = silu_mul(v[r], acc[j][i + 1 < SN ? i + 1 : i][r] * UNIT);
      }
      if (vec) {
        // Turned over in LDS, so that a lane stores eight consecutive columns (two-byte
        // stores and loads of add: 69 us for 1500 x 4096 x 2048 with add).
        float* const mine = reinterpret_cast<float*>(lds) + wave * 1024;
#pragma unroll
        for (int r = 0; r < 16; r++)
          mine[(8 * (r >> 2) + 4 * h + (r & 3)) * 32 + (r32 ^ (h << 4))] = v[r];
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int u = 0; u < 2; u++) {
          const int row = u * 16 + lane / 4, m = m0 + (j * C::WM + wm) * 32 + row;
          const int c = n - r32 + lane % 4 * 8;
          float w[8], a[8];
          const float* from = mine + row * 32 + ((lane % 4 * 8) ^ ((row & 4) << 2));
          load8<true>(from, 0, w);
          if (m >= g.M || c >= cols) continue;
          const size_t o = (size_t)m * cols + c;
          if (g.add != nullptr) {
            if (g.out_f32)
              load8<true>(g.add, o, a);
            else
              load8<false>(g.add, o, a);
#pragma unroll
            for (int r = 0; r < 8; r++) w[r] += a[r];
          }
          if (g.out_f32)
            store8<true>(g.out, o, w);
          else
            store8<false>(g.out, o, w);
        }
        __builtin_amdgcn_wave_barrier();
        continue;
      }
      size_t o[16];
      bool in[16];
#pragma unroll
      for (int r = 0; r < 16; r++) {
        const int m = mrow + 8 * (r >> 2) + (r & 3);
        o[r] = (size_t)m * cols + n;
        in[r] = n < cols && m < g.M;
      }
      put<16>(g, o, in, v);
    }
  }
}

// out of the parts of a K split, added in order.
__global__ __launch_bounds__(256) void w4_sum_kernel(W4Args g) {
  const int cols = g.act ? g.N / 2 : g.N;
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x, count = (size_t)g.M * g.N;
  if (i >= (size_t)g.M * cols) return;
  const size_t m = i / cols, at = m * g.N + (i - m * cols);
  float v = g.parts[at], u = g.act ? g.parts[at + cols] : 0.f;
  for (int p = 1; p < g.splits; p++) {
    v += g.parts[p * count + at];
    if (g.act) u += g.parts[p * count + at + cols];
  }
  const size_t o[1] = {i};
  const bool in[1] = {true};
  float w[1] = {g.act ? silu_mul(v, u) : v};
  put<1>(g, o, in, w);
}

// The rows kernel reads the codes again for every 32 rows, from the L2; it is the
// faster one up to 32 rows, and up to 64 where there are few columns.  A product whose
// tiles leave CUs without work is split along K in up to 8 parts of 4 K blocks or more.
// us (int4 in groups of 32):
//                        rows   Half in 1     2     4     8 parts   Wide
//   32 x 4096 x 4096     13.0        38.8  23.9  16.2  13.9
//   64 x 4096 x 4096     13.5        38.9  24.5  17.5  16.5
//   64 x 16384 x 2048    26.3        22.6  21.0  22.6  28.5
//   128 x 4096 x 4096    24.5        39.1  25.9  20.6  23.6
//   300 x 4096 x 2048                22.7  27.7                       31.1
//   2048 x 4096 x 4096              132                              107
typedef W4Tile<128, 128, 2, 2> Wide;
typedef W4Tile<64, 128, 2, 2> Half;
enum { kRows, kHalf, kWide };
struct Plan {
  int kernel, splits;
};
Plan plan(int M, int N, int K) {
  const int KB = (K + 127) / 128, cus = device_cu_count();
  if (M <= 32 || (M <= 64 && N <= 24 * cus)) return {kRows, 1};
  auto tiles = [&](int bm) { return (long long)((M + bm - 1) / bm) * ((N + 127) / 128); };
  const int kernel = M > 64 && tiles(128) >= cus ? kWide : kHalf;
  const long long t = tiles(kernel == kWide ? 128 : 64);
  int s = 8;
  while (s > 1 && (t * s > cus || KB / s < 4)) s /= 2;
  const int per = (KB + s - 1) / s;
  return {kernel, (KB + per - 1) / per};  // no part without a K block
}

template <class C, int FMT>
hipError_t launch_tile(W4Args g, int splits, hipStream_t s) {
  const int cols = g.act ? g.N / 2 : g.N, tn = g.act ? C::BN / 2 : C::BN;
  const long long total = (long long)((cols + tn - 1) / tn) * ((g.M + C::BM - 1) / C::BM);
  if (total >= (1ll << 24)) return hipErrorInvalidValue;  // (2^32 threads; out has 256 GiB)
  const int KB = (g.K + 127) / 128;
  g.splits = splits;
  g.split_kb = (KB + splits - 1) / splits;
  hipLaunchKernelGGL((w4_tile_kernel<C, FMT>), dim3((unsigned)((total + 7) / 8 * 8), splits),
                     dim3(C::THREADS), 0, s, g);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  const dim3 grid((unsigned)(((size_t)g.M * cols + 255) / 256));
  hipLaunchKernelGGL(w4_sum_kernel, grid, dim3(256), 0, s, g);
  return hipGetLastError();
}

template <int FMT>
hipError_t launch(const W4Args& g, hipStream_t s) {
  const Plan p = plan(g.M, g.N, g.K);
  if (p.kernel == kWide) return launch_tile<Wide, FMT>(g, p.splits, s);
  if (p.kernel == kHalf) return launch_tile<Half, FMT>(g, p.splits, s);
  return rows<FMT>(g, s);
}

}  // namespace

size_t w4_matmul_parts_bytes(int M, int N, int K) {
  const Plan p = plan(M, N, K);
  return p.splits > 1 ? (size_t)p.splits * M * N * 4 : 0;
}

hipError_t launch_w4_matmul(const W4Args& g, hipStream_t s) {
  if (g.mxfp4) return launch<kMxfp4>(g, s);
  return g.group == 32 ? launch<kInt4G32>(g, s)
                       : g.group == 64 ? launch<kInt4G64>(g, s) : launch<kInt4G128>(g, s);
}

}  // namespace qmoe
