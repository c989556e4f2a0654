// Matrix products of OCP e4m3 operands with one fp32 scale per 128 values
// along K (both operands) or per 128 x 128 block (b):
//
//   out[m,n] = sum_j sa[j,m] * sb(j,n) * sum_{i<128} a[m,128j+i] * b[n,128j+i]
//
// dense, or for every expert of an MoE layer over the row tiles of
// qmoe_align.  The inner sum of a K block is one matrix-core product in fp32
// from a zero accumulator; the scales multiply it once, in fp32, on the way
// into the running sum.
//
// The fp8 matrix instruction lines up eight products at a time with their
// largest and drops what lies 13 or more bits below it: on normal data a K
// block's sum is then 1.4e-5 off (2-norm, either shape of the instruction),
// which a bf16 output's rounding (2e-3) covers and an fp32 output's does not.
// fp32 outputs therefore widen the codes to bf16 (exact) and take the bf16
// instruction, which sums in fp32 (7e-9 off on the same data) at half the
// rate.
//
// b feeds the matrix core's row operand and a its
// column operand, so a lane's results share one row of a (one scale) and are
// consecutive columns of out.
#include "block_common.h"

namespace qmoe {
namespace {
using namespace bk;
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kUnit = 127;  // e8m0 of 1: the instruction's own scales are not used

__device__ inline i32x8 join(u32x4 lo, u32x4 hi) {
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
               (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// Eight codes (two words) as bf16, exactly.
__device__ inline bf16x8 widen8(uint32_t lo, uint32_t hi) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A K block of a 16 x 16 tile: row operand x, column operand y, 32 codes per
// lane each (the same 32 positions of K in every lane of a row or column).
template <bool EXACT>
__device__ inline f32x4 kblock16(const i32x8& x, const i32x8& y) {
  f32x4 z = {0.f, 0.f, 0.f, 0.f};
  if constexpr (EXACT) {
#pragma unroll
    for (int j = 0; j < 4; j++)
      z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8(x[2 * j], x[2 * j + 1]),
                                                  widen8(y[2 * j], y[2 * j + 1]), z, 0, 0, 0);
    return z;
  } else {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, z, 0, 0, 0, kUnit, 0, kUnit);
  }
}

// Where a tile's rows of a and out are.  Dense: row i of the tile is row
// m0 + i.  Grouped: it is the pair in slot m0 + i of the expert-sorted list,
// out's row is the pair, a's row the pair or its token.
template <bool GROUPED>
struct Rows {
  __device__ static inline int out_row(const Fp8MatmulArgs& g, int slot) {
    if constexpr (GROUPED) {
      const int p = g.sorted[slot];
      return p < g.P ? p : -1;
    } else {
      return slot < g.M ? slot : -1;
    }
  }
  __device__ static inline int a_row(const Fp8MatmulArgs& g, int out_row) {
    if (out_row < 0) return 0;
    if constexpr (GROUPED) return g.pair_rows ? out_row : out_row / g.k;
    return out_row;
  }
};

// 16 rows x 64 columns per wave, operands straight from memory.
template <bool GROUPED, bool BBLOCK, bool F32>
__global__ __launch_bounds__(256) void fp8_matmul_rows16_kernel(Fp8MatmulArgs g) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l = lane & 15, q = lane >> 4;
  const int n0 = (blockIdx.x * 4 + wave) * 64;
  const int m0 = blockIdx.y * 16;
  if (n0 >= g.N) return;
  const uint8_t* b = g.b;
  const float* bs = g.b_scale;
  if constexpr (GROUPED) {
    if (m0 >= *g.num_padded) return;
    const int e = g.tile_expert[m0 / g.block_m];
    if (e < 0) return;
    b += (size_t)e * g.N * g.K;
    bs += (size_t)e * ((g.N + 127) / 128) * g.KB;
  }
  const int orow = Rows<GROUPED>::out_row(g, m0 + l);
  const int arow = Rows<GROUPED>::a_row(g, orow);
  const uint8_t* ap = g.a + (size_t)arow * g.K + 16 * q;
  const uint8_t* bp[4];
#pragma unroll
  for (int s = 0; s < 4; s++)
    bp[s] = b + (size_t)min(n0 + 16 * s + l, g.N - 1) * g.K + 16 * q;
  f32x4 acc[4];
#pragma unroll
  for (int s = 0; s < 4; s++) acc[s] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int kb = 0; kb < g.KB; kb++) {
    const i32x8 av = join(*reinterpret_cast<const u32x4*>(ap + kb * 128),
                          *reinterpret_cast<const u32x4*>(ap + kb * 128 + 64));
    const float sa = g.a_scale[(size_t)kb * g.Ma + arow];
#pragma unroll
    for (int s = 0; s < 4; s++) {
      const i32x8 bv = join(*reinterpret_cast<const u32x4*>(bp[s] + kb * 128),
                            *reinterpret_cast<const u32x4*>(bp[s] + kb * 128 + 64));
      const f32x4 t = kblock16<F32>(bv, av);
      if constexpr (BBLOCK) {
        const int nb = min(n0 + 16 * s, g.N - 1) / 128;
        const float sc = sa * bs[(size_t)nb * g.KB + kb];
#pragma unroll
        for (int r = 0; r < 4; r++) acc[s][r] = __builtin_fmaf(t[r], sc, acc[s][r]);
      } else {
#pragma unroll
        for (int r = 0; r < 4; r++) {
          const int n = min(n0 + 16 * s + 4 * q + r, g.N - 1);
          acc[s][r] = __builtin_fmaf(t[r] * bs[(size_t)kb * g.N + n], sa, acc[s][r]);
        }
      }
    }
  }
  if (orow < 0) return;
#pragma unroll
  for (int s = 0; s < 4; s++)
#pragma unroll
    for (int r = 0; r < 4; r++) {
      const int n = n0 + 16 * s + 4 * q + r;
      if (n < g.N) store1<F32>(g.out, (size_t)orow * g.N + n, acc[s][r]);
    }
}

// ---------------------------------------------------------------------------
// Tiled kernel: a block of WM x WN waves computes BM rows x BN columns, a
// wave SM x SN sub-tiles of 32 x 32.  Both operands' K blocks (128 bytes per
// row) go from memory straight into LDS, two stages; a row's eight 16-byte
// chunks are stored in the order c ^ (row / 2 % 8), so that the 16 rows that
// are read together lie in different banks (the permutation is applied to the
// memory addresses: the copy writes LDS in lane order).
typedef float f32x16 __attribute__((ext_vector_type(16)));

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
__device__ inline float load_f32(Rsrc r, unsigned voff) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, (int)voff, 0, 0));
}

// Waits for the wave's copies (vmcnt 0; the barrier alone does not wait for
// copies to LDS), then for the other waves'.
__device__ inline void wait_copies() { __builtin_amdgcn_s_waitcnt(0x0F70); }
__device__ inline void landed() {
  wait_copies();
  __syncthreads();
}

template <int BM_, int BN_, int WM_, int WN_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int SM = BM / WM / 32, SN = BN / WN / 32;
  static constexpr int AC = BM / 8 / WAVES, BC = BN / 8 / WAVES;  // copies per wave and K block
  static_assert(SM * WM * 32 == BM && SN * WN * 32 == BN, "whole sub-tiles");
  static_assert(AC * WAVES * 8 == BM && BC * WAVES * 8 == BN, "whole copies");
};

template <class C, bool GROUPED, bool BBLOCK, bool F32>
__global__ __launch_bounds__(C::THREADS, 2) void fp8_matmul_tile_kernel(Fp8MatmulArgs g) {
  constexpr int SM = C::SM, SN = C::SN;
  __shared__ float c0[BBLOCK ? 1 : C::BN], c1[BBLOCK ? 1 : C::BN];  // b's row scales
  __shared__ __align__(1024) uint8_t lds[2 * (C::BM + C::BN) * 128];
  uint8_t* const a0 = lds;
  uint8_t* const b0 = a0 + C::BM * 128;
  uint8_t* const a1 = b0 + C::BN * 128;
  uint8_t* const b1 = a1 + C::BM * 128;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave % C::WM, wn = wave / C::WM;
  const int ntn = (g.N + C::BN - 1) / C::BN;
  const int ntm = ((GROUPED ? *g.num_padded : g.M) + C::BM - 1) / C::BM;
  // The launch order deals blocks to the XCDs in turn: give each XCD a
  // contiguous run of tiles, column-tile by column-tile inside bands of
  // kBand row tiles, so that its L2 sees the same rows again.
  constexpr int kBand = 8;
  const int total = ntn * ntm, per = (total + 7) / 8;
  const int id = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8);
  if (id >= total || (int)(blockIdx.x / 8) >= per) return;  // also past the tiles in use
  const int band = id / (kBand * ntn), in = id - band * kBand * ntn;
  const int rows = min(kBand, ntm - band * kBand);
  const int m0 = (band * kBand + in % rows) * C::BM, n0 = in / rows * C::BN;
  const uint8_t* b = g.b;
  const float* bs = g.b_scale;
  if constexpr (GROUPED) {
    const int e = g.tile_expert[m0 / g.block_m];
    if (e < 0) return;
    b += (size_t)e * g.N * g.K;
    bs += (size_t)e * ((g.N + 127) / 128) * g.KB;
  }
  // Copies: 8 lanes per row, the rows of a wave's copy t being 8 t .. 8 t + 7.
  // The chunk order alternates with t, hence two lane offsets where the rows
  // are consecutive; gathered rows have one per copy.
  const size_t K = g.K;
  auto swz = [&](int t) { return 16u * ((lane & 7) ^ ((4 * t + (lane >> 4)) & 7)); };
  const uint8_t* abase = GROUPED ? g.a : g.a + (size_t)m0 * K;
  const uint8_t* bbase = b + (size_t)n0 * K;
  const size_t abytes = (GROUPED ? (size_t)g.Ma : (size_t)(g.M - m0)) * K;
  const size_t bbytes = (size_t)(g.N - n0) * K;
  unsigned av[GROUPED ? C::AC : 2];
  const unsigned bv[2] = {(lane >> 3) * (unsigned)g.K + swz(0), (lane >> 3) * (unsigned)g.K + swz(1)};
  if constexpr (GROUPED) {
#pragma unroll
    for (int i = 0; i < C::AC; i++) {
      const int t = wave * C::AC + i;
      const int row = Rows<true>::a_row(g, Rows<true>::out_row(g, m0 + t * 8 + (lane >> 3)));
      av[i] = (unsigned)row * (unsigned)g.K + swz(t);
    }
  } else {
    av[0] = bv[0];
    av[1] = bv[1];
  }
  // Scales of the lane's rows, one K block ahead.
  const int r32 = lane & 31, h = lane >> 5;
  int orow[SM];
  unsigned so[SM];
#pragma unroll
  for (int s = 0; s < SM; s++) {
    orow[s] = Rows<GROUPED>::out_row(g, m0 + (wm * SM + s) * 32 + r32);
    so[s] = 4u * (unsigned)Rows<GROUPED>::a_row(g, orow[s]);
  }
  const int nw = n0 + wn * SN * 32;  // the wave's first column
  const float* sbp = bs + (BBLOCK ? (size_t)(min(nw, g.N - 1) / 128) * g.KB : 0);
  float sa[SM], nsa[SM], nsb = 1.0f;  // of this K block, of the next one
  auto take = [&]() {
#pragma unroll
    for (int s = 0; s < SM; s++) sa[s] = nsa[s] * nsb;
  };
  // (K blocks behind the last one are copies of nothing: empty buffers.)
  auto load_scales = [&](float* lc, int kb) {
    const bool any = kb < g.KB;
    const Rsrc rs = rsrc(g.a_scale + (size_t)kb * g.Ma, any ? (size_t)g.Ma * 4 : 0);
#pragma unroll
    for (int s = 0; s < SM; s++) nsa[s] = load_f32(rs, so[s]);
    if constexpr (BBLOCK) {
      nsb = load_f32(rsrc(sbp + kb, any ? 4 : 0), 0);
    } else if (wave < C::BN / 64) {
      const Rsrc rc = rsrc(bs + (size_t)kb * g.N + n0, any ? (size_t)(g.N - n0) * 4 : 0);
      copy4(rc, wave * 256 + lane * 4, lc + wave * 64);
    }
  };
  // Copy c of the wave's AC + BC ones of a K block.
  auto load = [&](uint8_t* la, uint8_t* lb, int kb, int c) {
    const bool any = kb < g.KB;
    if (c < C::AC) {
      const int t = wave * C::AC + c;
      const Rsrc ra = rsrc(abase, any ? abytes : 0);
      if constexpr (GROUPED)
        copy16(ra, av[c], kb * 128, la + t * 1024);
      else
        copy16(ra, (C::AC % 2 == 0 ? c : t) % 2 ? av[1] : av[0], t * 8 * g.K + kb * 128,
               la + t * 1024);
    } else {
      const int i = c - C::AC, t = wave * C::BC + i;
      const Rsrc rb = rsrc(bbase, any ? bbytes : 0);
      copy16(rb, (C::BC % 2 == 0 ? i : t) % 2 ? bv[1] : bv[0], t * 8 * g.K + kb * 128,
             lb + t * 1024);
    }
  };
  // Reads: lane's row in a sub-tile and its half of each 64 positions of K.
  int off[2][2];
#pragma unroll
  for (int j = 0; j < 2; j++)
#pragma unroll
    for (int e = 0; e < 2; e++)
      off[j][e] = r32 * 128 + 16 * ((4 * j + 2 * h + e) ^ ((r32 >> 1) & 7));
  f32x16 acc[SN][SM];
#pragma unroll
  for (int i = 0; i < SN; i++)
#pragma unroll
    for (int s = 0; s < SM; s++)
#pragma unroll
      for (int r = 0; r < 16; r++) acc[i][s][r] = 0.f;

  auto frag = [&](const uint8_t* t, int sub, int j) {
    return join(*reinterpret_cast<const u32x4*>(t + sub * 4096 + off[j][0]),
                *reinterpret_cast<const u32x4*>(t + sub * 4096 + off[j][1]));
  };
  f32x4 sbn[BBLOCK ? 1 : SN][4];  // b's scales of the lane's 16 columns per sub-tile
  auto row_scales = [&](const float* lc) {
    if constexpr (!BBLOCK) {
#pragma unroll
      for (int i = 0; i < SN; i++)
#pragma unroll
        for (int q = 0; q < 4; q++)
          sbn[i][q] =
              *reinterpret_cast<const f32x4*>(lc + (wn * SN + i) * 32 + 8 * q + 4 * h);
    }
  };
  auto scaled = [&](const f32x16& t, int i, int s) {
#pragma unroll
    for (int r = 0; r < 16; r++) {
      if constexpr (BBLOCK)
        acc[i][s][r] = __builtin_fmaf(t[r], sa[s], acc[i][s][r]);
      else
        acc[i][s][r] = __builtin_fmaf(t[r] * sbn[i][r >> 2][r & 3], sa[s], acc[i][s][r]);
    }
  };
  // One K block from LDS; the next one's copies (to na, nb) are issued between
  // the matrix instructions, so that no wave waits in front of them for the
  // memory pipe to take its copies.
  auto compute = [&](const uint8_t* la, const uint8_t* lb, const float* lc, uint8_t* na, uint8_t* nb,
                     float* nc, int kb) {
    row_scales(lc);
    load_scales(nc, kb + 1);
    if constexpr (F32) {
      // The codes widened to bf16, 16 positions of K per instruction: a lane's
      // chunk of 16 codes feeds two.
      f32x16 t[SN][SM];
#pragma unroll
      for (int i = 0; i < SN; i++)
#pragma unroll
        for (int s = 0; s < SM; s++)
#pragma unroll
          for (int r = 0; r < 16; r++) t[i][s][r] = 0.f;
#pragma unroll
      for (int c = 0; c < 4; c++) {
        const int o = r32 * 128 + 16 * ((2 * c + h) ^ ((r32 >> 1) & 7));
        u32x4 x[SM], y[SN];
#pragma unroll
        for (int i = 0; i < SN; i++)
          y[i] = *reinterpret_cast<const u32x4*>(lb + (wn * SN + i) * 4096 + o);
#pragma unroll
        for (int s = 0; s < SM; s++)
          x[s] = *reinterpret_cast<const u32x4*>(la + (wm * SM + s) * 4096 + o);
#pragma unroll
        for (int u = c * (C::AC + C::BC) / 4; u < (c + 1) * (C::AC + C::BC) / 4; u++)
          load(na, nb, kb + 1, u);
#pragma unroll
        for (int j = 0; j < 2; j++) {
          bf16x8 xs[SM];
#pragma unroll
          for (int s = 0; s < SM; s++) xs[s] = widen8(x[s][2 * j], x[s][2 * j + 1]);
#pragma unroll
          for (int i = 0; i < SN; i++) {
            const bf16x8 ys = widen8(y[i][2 * j], y[i][2 * j + 1]);
#pragma unroll
            for (int s = 0; s < SM; s++)
              t[i][s] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ys, xs[s], t[i][s], 0, 0, 0);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < SN; i++)
#pragma unroll
        for (int s = 0; s < SM; s++) scaled(t[i][s], i, s);
    } else {
      i32x8 bf[SN][2];
#pragma unroll
      for (int i = 0; i < SN; i++)
#pragma unroll
        for (int j = 0; j < 2; j++) bf[i][j] = frag(lb, wn * SN + i, j);
      f32x16 t[2];
#pragma unroll
      for (int s = 0; s < SM; s++) {
        const i32x8 x0 = frag(la, wm * SM + s, 0), x1 = frag(la, wm * SM + s, 1);
#pragma unroll
        for (int i = 0; i < SN; i++) {
          const int q = s * SN + i;
          f32x16 z;
#pragma unroll
          for (int r = 0; r < 16; r++) z[r] = 0.f;
          z = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(bf[i][0], x0, z, 0, 0, 0, kUnit, 0,
                                                              kUnit);
          z = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(bf[i][1], x1, z, 0, 0, 0, kUnit, 0,
                                                              kUnit);
          t[q & 1] = z;
          constexpr int kParts = (SM * SN + 1) / 2;  // all copies by the middle of the step
#pragma unroll
          for (int u = 0; u < C::AC + C::BC; u++)
            if (u * kParts / (C::AC + C::BC) == q) load(na, nb, kb + 1, u);
          // The scaling of the sub-tile before runs while the matrix core works.
          if (q > 0) scaled(t[(q - 1) & 1], (q - 1) % SN, (q - 1) / SN);
        }
      }
      scaled(t[(SM * SN - 1) & 1], SN - 1, SM - 1);
    }
  };
  load_scales(c0, 0);
#pragma unroll
  for (int u = 0; u < C::AC + C::BC; u++) load(a0, b0, 0, u);
  for (int kb = 0; kb < g.KB; kb += 2) {
    landed();  // stage 0 is there, stage 1 is free
    take();
    compute(a0, b0, c0, a1, b1, c1, kb);
    if (kb + 1 >= g.KB) break;
    landed();
    take();
    compute(a1, b1, c1, a0, b0, c0, kb + 1);
  }
  wait_copies();  // no copy outlives the block's LDS
  // A lane holds four times four consecutive columns of its row per sub-tile.
  // Where rows can be stored in 16-byte pieces, each wave turns its tile over
  // in LDS, 32 rows at a time, so that consecutive lanes store consecutive
  // bytes (the pieces of a row in the order p ^ row % 8, against bank
  // conflicts).
  constexpr int EB = F32 ? 4 : 2;             // bytes per value
  constexpr int RB = SN * 32 * EB;            // bytes per row of the wave's tile
  constexpr int PIECES = RB / 16, RPI = 64 / PIECES;  // pieces per row, rows per store
  static_assert(C::WAVES * 32 * RB <= (int)sizeof(lds), "every wave has room for 32 rows");
  if (g.N % (16 / EB) == 0 && (uintptr_t)g.out % 16 == 0) {
    __syncthreads();  // the last K block has been read
    uint8_t* const mine = lds + wave * 32 * RB;
#pragma unroll
    for (int s = 0; s < SM; s++) {
#pragma unroll
      for (int i = 0; i < SN; i++)
#pragma unroll
        for (int q = 0; q < 4; q++) {
          const int byte = (i * 32 + 8 * q + 4 * h) * EB;
          uint8_t* d = mine + r32 * RB + ((byte / 16) ^ (r32 % 8 % PIECES)) * 16 + byte % 16;
          const float v[4] = {acc[i][s][4 * q], acc[i][s][4 * q + 1], acc[i][s][4 * q + 2],
                              acc[i][s][4 * q + 3]};
          store4<F32>(d, 0, v);
        }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int u = 0; u < 32 / RPI; u++) {
        const int row = u * RPI + lane / PIECES, piece = lane % PIECES;
        const int n = nw + piece * (16 / EB);
        const int orw = Rows<GROUPED>::out_row(g, m0 + (wm * SM + s) * 32 + row);
        const u32x4 v =
            *reinterpret_cast<const u32x4*>(mine + row * RB + (piece ^ (row % 8 % PIECES)) * 16);
        if (orw >= 0 && n < g.N)
          *reinterpret_cast<u32x4*>(reinterpret_cast<uint8_t*>(g.out) +
                                    ((size_t)orw * g.N + n) * EB) = v;
      }
      __builtin_amdgcn_wave_barrier();
    }
    return;
  }
#pragma unroll
  for (int s = 0; s < SM; s++) {
    if (orow[s] < 0) continue;
    const size_t o = (size_t)orow[s] * g.N;
#pragma unroll
    for (int i = 0; i < SN; i++)
#pragma unroll
      for (int r = 0; r < 16; r++) {
        const int n = nw + i * 32 + 8 * (r >> 2) + 4 * h + (r & 3);
        if (n < g.N) store1<F32>(g.out, o + n, acc[i][s][r]);
      }
  }
}

template <class C, bool GROUPED, bool BBLOCK, bool F32>
hipError_t launch_tile(const Fp8MatmulArgs& g, hipStream_t s) {
  const long long total =
      (long long)((g.N + C::BN - 1) / C::BN) * ((g.M + C::BM - 1) / C::BM);
  if (total > (1ll << 30)) return hipErrorInvalidValue;
  hipLaunchKernelGGL((fp8_matmul_tile_kernel<C, GROUPED, BBLOCK, F32>),
                     dim3((unsigned)((total + 7) / 8 * 8)), dim3(C::THREADS), 0, s, g);
  return hipGetLastError();
}

}  // namespace

size_t fp8_matmul_parts_bytes(int, int, int) { return 0; }

// Rows up to which the untiled kernel is taken.
constexpr int kFewRows = 32;

hipError_t launch_fp8_matmul(const Fp8MatmulArgs& g, hipStream_t s) {
  typedef Tile<128, 128, 2, 2> Mid;
  typedef Tile<256, 256, 2, 4> Big;
  if (g.M >= kFewRows) {
    if (g.out_f32)
      return g.b_block ? launch_tile<Mid, false, true, true>(g, s)
                       : launch_tile<Mid, false, false, true>(g, s);
    if (!g.b_block) return launch_tile<Mid, false, false, false>(g, s);
    const long long big = (long long)((g.M + 255) / 256) * ((g.N + 255) / 256);
    return big >= 200 ? launch_tile<Big, false, true, false>(g, s)
                      : launch_tile<Mid, false, true, false>(g, s);
  }
  const dim3 grid((g.N + 255) / 256, (g.M + 15) / 16), block(256);
#define QMOE_CALL(BB, F32) \
  hipLaunchKernelGGL((fp8_matmul_rows16_kernel<false, BB, F32>), grid, block, 0, s, g)
  if (g.b_block && g.out_f32)
    QMOE_CALL(true, true);
  else if (g.b_block)
    QMOE_CALL(true, false);
  else if (g.out_f32)
    QMOE_CALL(false, true);
  else
    QMOE_CALL(false, false);
#undef QMOE_CALL
  return hipGetLastError();
}

namespace {
template <bool F32>
hipError_t grouped(const Fp8MatmulArgs& g, hipStream_t s) {
  if (g.block_m == 128) return launch_tile<Tile<128, 128, 2, 2>, true, true, F32>(g, s);
  if (g.block_m == 64) return launch_tile<Tile<64, 128, 1, 4>, true, true, F32>(g, s);
  if (g.block_m == 32) return launch_tile<Tile<32, 128, 1, 4>, true, true, F32>(g, s);
  const dim3 grid((g.N + 255) / 256, (g.M + 15) / 16), block(256);
  hipLaunchKernelGGL((fp8_matmul_rows16_kernel<true, true, F32>), grid, block, 0, s, g);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_fp8_grouped_matmul(const Fp8MatmulArgs& g, hipStream_t s) {
  return g.out_f32 ? grouped<true>(g, s) : grouped<false>(g, s);
}

}  // namespace qmoe
