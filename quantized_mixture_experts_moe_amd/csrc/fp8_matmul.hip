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
// b feeds the matrix core's row operand and a its column operand, so a lane's
// results share one row of a (one scale) and are consecutive columns of out.
//
// Measured: 4096 x 4096 x 4096 in bf16 63-73 us (1.9-2.2 PFLOP/s, by the power
// that the values draw), fp32 outputs of 1500 x 2048 x 4224 39 us (0.67), 2048
// tokens on 128 experts of 1536 x 2048 123 us (3.7 TB/s), 4 tokens 17-19 us (4.8
// TB/s), one row of 2048 x 2048 3.5 us (1.2 TB/s).
#include "block_common.h"
#include "qmoe_internal.h"

namespace qmoe {
namespace {
using namespace bk;
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr unsigned kNowhere = 0xC0000000u;  // an offset behind every buffer of gathered rows
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

// ---------------------------------------------------------------------------
// Few rows: the work is reading b once.  A block computes 16 MS rows x 16 NS
// columns, its KS waves taking every KS-th K block, so that together they read
// KS * 128 consecutive bytes of each of b's rows; operands go straight from
// memory to registers, RING K blocks ahead, and the waves' sums are added in
// wave order through LDS.
template <int KS, int MS, int NS, int RING, bool GROUPED, bool BBLOCK, bool F32>
__global__ __launch_bounds__(64 * KS) void fp8_matmul_rows_kernel(Fp8MatmulArgs g) {
  __shared__ f32x4 part[KS][MS * NS][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int l = lane & 15, q = lane >> 4;
  const int n0 = blockIdx.x * 16 * NS;
  const int m0 = blockIdx.y * 16 * MS;
  const uint8_t* b = g.b;
  const float* bs = g.b_scale;
  if constexpr (GROUPED) {
    if (m0 >= *g.num_padded) return;
    const int e = g.tile_expert[m0 / g.block_m];
    b += (size_t)e * g.N * g.K;
    bs += (size_t)e * ((g.N + 127) / 128) * g.KB;
  }
  int arow[MS];
  const uint8_t* ap[MS];
#pragma unroll
  for (int m = 0; m < MS; m++) {
    arow[m] = Rows<GROUPED>::a_row(g, Rows<GROUPED>::out_row(g, m0 + 16 * m + l));
    ap[m] = g.a + (size_t)arow[m] * g.K + 16 * q;
  }
  const uint8_t* bp[NS];
#pragma unroll
  for (int s = 0; s < NS; s++)
    bp[s] = b + (size_t)min(n0 + 16 * s + l, g.N - 1) * g.K + 16 * q;
  const float* sbp = bs + (BBLOCK ? (size_t)(n0 / 128) * g.KB : 0);  // 16 NS divides 128

  struct Step {
    u32x4 a[MS][2], b[NS][2];
    float sa[MS], sb;
  };
  Step ring[RING];
  auto load = [&](Step& st, int kb) {
    const size_t at = (size_t)kb * 128;
#pragma unroll
    for (int s = 0; s < NS; s++) {
      st.b[s][0] = *reinterpret_cast<const u32x4*>(bp[s] + at);
      st.b[s][1] = *reinterpret_cast<const u32x4*>(bp[s] + at + 64);
    }
#pragma unroll
    for (int m = 0; m < MS; m++) {
      st.a[m][0] = *reinterpret_cast<const u32x4*>(ap[m] + at);
      st.a[m][1] = *reinterpret_cast<const u32x4*>(ap[m] + at + 64);
      st.sa[m] = g.a_scale[(size_t)kb * g.Ma + arow[m]];
    }
    st.sb = BBLOCK ? sbp[kb] : 1.0f;
  };
  f32x4 acc[MS][NS];
#pragma unroll
  for (int m = 0; m < MS; m++)
#pragma unroll
    for (int s = 0; s < NS; s++) acc[m][s] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const Step& st, int kb) {
#pragma unroll
    for (int s = 0; s < NS; s++) {
      const i32x8 bv = join(st.b[s][0], st.b[s][1]);
      f32x4 sn = {st.sb, st.sb, st.sb, st.sb};
      if constexpr (!BBLOCK) {
#pragma unroll
        for (int r = 0; r < 4; r++)
          sn[r] = bs[(size_t)kb * g.N + min(n0 + 16 * s + 4 * q + r, g.N - 1)];
      }
#pragma unroll
      for (int m = 0; m < MS; m++) {
        const f32x4 t = kblock16<F32>(bv, join(st.a[m][0], st.a[m][1]));
#pragma unroll
        for (int r = 0; r < 4; r++)
          acc[m][s][r] = __builtin_fmaf(t[r], st.sa[m] * sn[r], acc[m][s][r]);
      }
    }
  };
#pragma unroll
  for (int u = 0; u < RING; u++)
    if (wave + u * KS < g.KB) load(ring[u], wave + u * KS);
  for (int k0 = wave; k0 < g.KB; k0 += RING * KS) {
#pragma unroll
    for (int u = 0; u < RING; u++) {
      const int kb = k0 + u * KS, next = kb + RING * KS;
      if (kb < g.KB) {
        compute(ring[u], kb);
        if (next < g.KB) load(ring[u], next);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MS; m++)
#pragma unroll
    for (int s = 0; s < NS; s++) part[wave][m * NS + s][lane] = acc[m][s];
  __syncthreads();
#pragma unroll
  for (int j = wave; j < MS * NS; j += KS) {
    f32x4 v = part[0][j][lane];
#pragma unroll
    for (int w = 1; w < KS; w++) {
      const f32x4 x = part[w][j][lane];
#pragma unroll
      for (int r = 0; r < 4; r++) v[r] += x[r];
    }
    const int orow = Rows<GROUPED>::out_row(g, m0 + 16 * (j / NS) + l);
    const int n = n0 + 16 * (j % NS) + 4 * q;
    if (orow < 0) continue;
    const size_t o = (size_t)orow * g.N + n;
    if (g.N % 4 == 0 && (uintptr_t)g.out % 16 == 0) {
      const float w[4] = {v[0], v[1], v[2], v[3]};
      if (n < g.N) store4<F32>(g.out, o, w);
    } else {
#pragma unroll
      for (int r = 0; r < 4; r++)
        if (n + r < g.N) store1<F32>(g.out, o + r, v[r]);
    }
  }
}

template <int MS, bool GROUPED, bool BBLOCK, bool F32>
hipError_t launch_rows(const Fp8MatmulArgs& g, hipStream_t s) {
  const int mt = (g.M + 16 * MS - 1) / (16 * MS);
  if (mt > 65535) return hipErrorInvalidValue;
  // KS waves share K, NS sub-tiles share a block's rows of a.  Many waves read
  // one column's K at once, which is what counts for a few blocks; few waves with
  // two sub-tiles hold the most bytes under way where blocks fill the chip twice;
  // two sub-tiles also halve how often a is read.  In us (K, rows x columns; the
  // grouped ones: tokens of 8 picks on 128 experts):
  //   KS x NS             4x2   16x2  16x1  8x1   4x1
  //   2048, 64 t. x 1536   68    82   110    96    78   4x2: chip full
  //   1024, 16 x 16384    5.6   5.7   7.6   6.3   6.4
  //   4096, 16 x 8192    11.1   9.3  10.6  10.7  10.5   16x2: many columns, rows
  //   4096, 32 x 4096    11.2  10.1   8.2   8.7   9.3   16x1: long K
  //   8192, 1 x 1024     11.0  10.5   6.9   6.9   8.1
  //   2048, 16 x 2048     5.7   5.3   4.3   4.3   4.7   8x1: half as long
  //   512, 1 x 2048       2.6   2.8   2.5   2.4   2.3   4x1: four K blocks
  const long long blocks2 = (long long)mt * ((g.N + 31) / 32);
  const int cus = device_cu_count();
#define QMOE_CALL(KS, NS, RING)                                                                \
  hipLaunchKernelGGL((fp8_matmul_rows_kernel<KS, MS, NS, RING, GROUPED, BBLOCK, F32>),         \
                     dim3((g.N + 16 * NS - 1) / (16 * NS), mt), dim3(64 * KS), 0, s, g)
  if (blocks2 >= 2 * cus && (GROUPED || g.KB < 32))
    QMOE_CALL(4, 2, 2);
  else if (g.KB >= 32 && blocks2 >= cus && g.M > 8)
    QMOE_CALL(16, 2, 1);
  else if (g.KB >= 32)
    QMOE_CALL(16, 1, 1);
  else if (g.KB >= 8)
    QMOE_CALL(8, 1, 2);
  else
    QMOE_CALL(4, 1, 2);
#undef QMOE_CALL
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Tiled kernel: a block of WM x WN waves computes BM rows x BN columns, a
// wave SM x SN sub-tiles of 32 x 32.  Both operands' K blocks (128 bytes per
// row) go from memory straight into LDS, two stages; a row's eight 16-byte
// chunks are stored in the order c ^ (row / 2 % 8), so that the 16 rows that
// are read together lie in different banks (the permutation is applied to the
// memory addresses: the copy writes LDS in lane order).
//
// Bound: a K block of the 256 x 256 tile takes 1.74 us on random codes (4096 x
// 4096 by K), 2048 of its clocks in the matrix core, at 2.17 GHz 54%; with
// prologue, stores and the launch (10 us in all) the 4096^3 product keeps it
// busy 45% of its time.  On zeros, which draw less power, the K block takes
// 1.30 us: 1.10 without the repeated reads of a's fragments, 1.17 without the
// scaling, 0.92 without both.  fp32 outputs: one 64 x 128 tile on a CU takes 0.69
// us per K block, two take 1.00, the matrix core busy 30% and 42% of that.  On
// the 128 x 128 tile (0.98 us) copies, widening and scaling are about 0.1 each,
// and without all three it takes 0.71; the widening instruction issues at the
// full rate and hides behind the matrix core, so no form of the codes in LDS
// would save it.
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

template <int BM_, int BN_, int WM_, int WN_, int STAGES_, int EU_ = 2>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, STAGES = STAGES_;
  static constexpr int EU = EU_;  // waves per SIMD that the registers allow for
  static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int SM = BM / WM / 32, SN = BN / WN / 32;
  static constexpr int AC = BM / 8 / WAVES, BC = BN / 8 / WAVES;  // copies per wave and K block
  static constexpr int COPIES = AC + BC + 1;                      // with the scales' one
  static constexpr int AS = (BM + 63) / 64;                       // waves that copy a's scales
  // LDS of a stage: a, b, 64 scales per wave.
  static constexpr int B_AT = BM * 128, S_AT = B_AT + BN * 128, STAGE = S_AT + WAVES * 256;
  static_assert(SM * WM * 32 == BM && SN * WN * 32 == BN, "whole sub-tiles");
  static_assert(AC * WAVES * 8 == BM && BC * WAVES * 8 == BN, "whole copies");
  static_assert(STAGES * STAGE <= 160 * 1024, "LDS");
};

// The row tiles of the experts, found by every wave from expert_offsets: a
// lane holds the tiles of E / 64 consecutive experts, a prefix sum over the
// lanes places them.
template <int BM>
struct Spans {
  int first, mine, per;  // tiles before this lane's experts, its own, experts per lane
  __device__ inline int tiles(const Fp8MatmulArgs& g, int e) const {
    return (g.expert_offsets[e + 1] - g.expert_offsets[e] + BM - 1) / BM;
  }
  __device__ inline int count(const Fp8MatmulArgs& g) {
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
  __device__ inline int find(const Fp8MatmulArgs& g, int t, int* m0, int* mend) const {
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

// OUT32: out is fp32 (the sums of a K split, and fp32 outputs); EXACT: the
// codes are widened to bf16.  blockIdx.y is the part of a K split.
template <class C, bool GROUPED, bool BBLOCK, bool EXACT, bool OUT32>
__global__ __launch_bounds__(C::THREADS, C::EU) void fp8_matmul_tile_kernel(Fp8MatmulArgs g) {
  constexpr int SM = C::SM, SN = C::SN;
  static_assert(C::AS + (BBLOCK ? 1 : (C::BN + 63) / 64) <= C::WAVES, "one scale copy per wave");
  __shared__ __align__(1024) uint8_t lds[C::STAGES * C::STAGE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave % C::WM, wn = wave / C::WM;
  const int ntn = (g.N + C::BN - 1) / C::BN;
  // Grouped: a row tile is up to BM rows of one expert, however many of
  // qmoe_align's tiles they are, so that the expert's matrix is read as seldom
  // as BM allows.
  Spans<C::BM> spans;
  int ntm = (g.M + C::BM - 1) / C::BM;
  if constexpr (GROUPED) ntm = spans.count(g);
  // The launch order deals blocks to the XCDs in turn: give each XCD a
  // contiguous run of tiles, column-tile by column-tile inside bands of
  // kBand row tiles, so that its L2 sees the same rows again.
  constexpr int kBand = 8;
  const int total = ntn * ntm, per = (total + 7) / 8;
  const int id = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8);
  if (id >= total || (int)(blockIdx.x / 8) >= per) return;  // also past the tiles in use
  const int band = id / (kBand * ntn), in = id - band * kBand * ntn;
  const int rows = min(kBand, ntm - band * kBand);
  const int mt = band * kBand + in % rows, n0 = in / rows * C::BN;
  int m0 = mt * C::BM, mend = g.M;
  const int kb0 = blockIdx.y * g.split_kb, kb1 = min(g.KB, kb0 + g.split_kb);
  const int NB = (g.N + 127) / 128;
  const uint8_t* b = g.b;
  const float* bs = g.b_scale;
  if constexpr (GROUPED) {
    const int e = spans.find(g, mt, &m0, &mend);
    b += (size_t)e * g.N * g.K;
    bs += (size_t)e * NB * g.KB;
  }
  auto out_row = [&](int slot) {
    return GROUPED && slot >= mend ? -1 : Rows<GROUPED>::out_row(g, slot);
  };
  // The wave's sub-tiles of rows are wm, wm + WM, ...; those behind the last
  // one with a row (an expert's rows stand in front of its padding) are left
  // out.
  int live = SM;
  if constexpr (GROUPED) {
    live = 0;
#pragma unroll
    for (int s = 0; s < SM; s++)
      if (__ballot(out_row(m0 + (s * C::WM + wm) * 32 + (lane & 31)) >= 0) != 0) live = s + 1;
    live = __builtin_amdgcn_readfirstlane(live);
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
  const unsigned bv[2] = {(lane >> 3) * (unsigned)g.K + swz(0),
                          (lane >> 3) * (unsigned)g.K + swz(1)};
  if constexpr (GROUPED) {
#pragma unroll
    for (int i = 0; i < C::AC; i++) {
      const int t = wave * C::AC + i;
      const int o = out_row(m0 + t * 8 + (lane >> 3));
      // no row: behind every buffer, so nothing is read
      av[i] = o < 0 ? kNowhere : (unsigned)Rows<true>::a_row(g, o) * (unsigned)g.K + swz(t);
    }
  } else {
    av[0] = bv[0];
    av[1] = bv[1];
  }
  // The wave's scale copy: 64 rows of a, 64 rows of b, or (lanes 0 and 1) the
  // tile's two blocks of b; a wave without one copies nothing, so that every
  // wave has the same number under way.
  const uint8_t* sbase = reinterpret_cast<const uint8_t*>(bs);
  size_t sstep = BBLOCK ? 4 : (size_t)g.N * 4, sbytes = 0;
  unsigned sv = 0;
  if (wave < C::AS) {
    sbase = reinterpret_cast<const uint8_t*>(g.a_scale);
    sstep = sbytes = (size_t)g.Ma * 4;
    const int o = wave * 64 + lane < C::BM ? out_row(m0 + wave * 64 + lane) : -1;
    sv = 4u * (unsigned)Rows<GROUPED>::a_row(g, o);
  } else if constexpr (BBLOCK) {
    if (wave == C::AS) {
      sbytes = (size_t)NB * g.KB * 4;
      sv = 4u * (unsigned)(n0 / 128 + (lane & 1)) * (unsigned)g.KB;
    }
  } else if (wave < C::AS + (C::BN + 63) / 64) {
    sbytes = (size_t)g.N * 4;
    sv = 4u * (unsigned)(n0 + (wave - C::AS) * 64 + lane);
  }
  // Copy c of the wave's COPIES of K block kb, to stage st.  (K blocks behind
  // the last one are copies of nothing, from empty buffers.)  The row is in the
  // lane's offset, which alone is behind the buffer for a row behind its last
  // one; the wave's is the place in the row.
  auto load = [&](uint8_t* st, int kb, int c) {
    const bool any = kb < kb1;
    const unsigned at = any ? kb * 128 : 0;
    if (c < C::AC) {
      const int t = wave * C::AC + c;
      const Rsrc ra = rsrc(abase, any ? abytes : 0);
      if constexpr (GROUPED)
        copy16(ra, av[c], at, st + t * 1024);
      else
        copy16(ra, ((C::AC % 2 == 0 ? c : t) % 2 ? av[1] : av[0]) + t * 8 * (unsigned)g.K, at,
               st + t * 1024);
    } else if (c < C::AC + C::BC) {
      const int i = c - C::AC, t = wave * C::BC + i;
      const Rsrc rb = rsrc(bbase, any ? bbytes : 0);
      copy16(rb, ((C::BC % 2 == 0 ? i : t) % 2 ? bv[1] : bv[0]) + t * 8 * (unsigned)g.K, at,
             st + C::B_AT + t * 1024);
    } else {
      const Rsrc rs = rsrc(sbase + (any ? (size_t)kb * sstep : 0), any ? sbytes : 0);
      copy4(rs, sv, reinterpret_cast<float*>(st + C::S_AT + wave * 256));
    }
  };
  // Reads: lane's row in a sub-tile and its half of each 64 positions of K.
  const int r32 = lane & 31, h = lane >> 5;
  int off[2][2];
#pragma unroll
  for (int j = 0; j < 2; j++)
#pragma unroll
    for (int e = 0; e < 2; e++)
      off[j][e] = r32 * 128 + 16 * ((4 * j + 2 * h + e) ^ ((r32 >> 1) & 7));
  const int nw = n0 + wn * SN * 32;  // the wave's first column
  const int nblk = wn * SN * 32 / 128;
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
  // One K block from stage st; the copies of K block kb + STAGES - 1 (to nx)
  // are issued between the matrix instructions, so that no wave waits in front
  // of them for the memory pipe to take its copies.
  auto compute = [&](auto live_, const uint8_t* st, uint8_t* nx, int kb) {
    constexpr int LIVE = decltype(live_)::value;  // sub-tile rows to compute
    const uint8_t* la = st;
    const uint8_t* lb = st + C::B_AT;
    const float* ls = reinterpret_cast<const float*>(st + C::S_AT);
    const int next = kb + C::STAGES - 1;
    float sa[SM];
    const float sb = BBLOCK ? ls[C::AS * 64 + nblk] : 1.0f;
#pragma unroll
    for (int s = 0; s < SM; s++) sa[s] = ls[(s * C::WM + wm) * 32 + r32] * sb;
    f32x4 sbn[BBLOCK ? 1 : SN][4];  // b's scales of the lane's 16 columns per sub-tile
    if constexpr (!BBLOCK) {
#pragma unroll
      for (int i = 0; i < SN; i++)
#pragma unroll
        for (int q = 0; q < 4; q++)
          sbn[i][q] = *reinterpret_cast<const f32x4*>(ls + C::AS * 64 + (wn * SN + i) * 32 +
                                                      8 * q + 4 * h);
    }
    auto scaled = [&](const f32x16& t, int i, int s) {
#pragma unroll
      for (int r = 0; r < 16; r++) {
        if constexpr (BBLOCK)
          acc[i][s][r] = __builtin_fmaf(t[r], sa[s], acc[i][s][r]);
        else
          acc[i][s][r] = __builtin_fmaf(t[r] * sbn[i][r >> 2][r & 3], sa[s], acc[i][s][r]);
      }
    };
    if constexpr (LIVE == 0) {
#pragma unroll
      for (int u = 0; u < C::COPIES; u++) load(nx, next, u);
    } else if constexpr (EXACT) {
      // The codes widened to bf16, 16 positions of K per instruction: a lane's
      // chunk of 16 codes feeds two.
      f32x16 t[SN][SM];
#pragma unroll
      for (int i = 0; i < SN; i++)
#pragma unroll
        for (int s = 0; s < LIVE; s++)
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
        for (int s = 0; s < LIVE; s++)
          x[s] = *reinterpret_cast<const u32x4*>(la + (s * C::WM + wm) * 4096 + o);
#pragma unroll
        for (int u = c * C::COPIES / 4; u < (c + 1) * C::COPIES / 4; u++) load(nx, next, u);
#pragma unroll
        for (int j = 0; j < 2; j++) {
          bf16x8 xs[SM];
#pragma unroll
          for (int s = 0; s < LIVE; s++) xs[s] = widen8(x[s][2 * j], x[s][2 * j + 1]);
#pragma unroll
          for (int i = 0; i < SN; i++) {
            const bf16x8 ys = widen8(y[i][2 * j], y[i][2 * j + 1]);
#pragma unroll
            for (int s = 0; s < LIVE; s++)
              t[i][s] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ys, xs[s], t[i][s], 0, 0, 0);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < SN; i++)
#pragma unroll
        for (int s = 0; s < LIVE; s++) scaled(t[i][s], i, s);
    } else {
      i32x8 bf[SN][2];
#pragma unroll
      for (int i = 0; i < SN; i++)
#pragma unroll
        for (int j = 0; j < 2; j++) bf[i][j] = frag(lb, wn * SN + i, j);
      f32x16 t[2];
#pragma unroll
      for (int s = 0; s < LIVE; s++) {
        const i32x8 x0 = frag(la, s * C::WM + wm, 0), x1 = frag(la, s * C::WM + wm, 1);
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
          constexpr int kParts = (LIVE * SN + 1) / 2;  // all copies by the middle of the step
#pragma unroll
          for (int u = 0; u < C::COPIES; u++)
            if (u * kParts / C::COPIES == q) load(nx, next, u);
          // The scaling of the sub-tile before runs while the matrix core works.
          if (q > 0) scaled(t[(q - 1) & 1], (q - 1) % SN, (q - 1) / SN);
        }
      }
      scaled(t[(LIVE * SN - 1) & 1], SN - 1, LIVE - 1);
    }
  };
#pragma unroll
  for (int s = 0; s < C::STAGES - 1; s++)
#pragma unroll
    for (int u = 0; u < C::COPIES; u++) load(lds + s * C::STAGE, kb0 + s, u);
  auto k_loop = [&](auto live_) {
    for (int kb = kb0;;) {
      bool done = false;
#pragma unroll
      for (int s = 0; s < C::STAGES; s++) {
        if (done) continue;
        // Stage s has landed (the stages behind it may be under way), in every
        // wave; and every wave is done with the stage before, which is free now.
        wait_memory<(C::STAGES - 2) * C::COPIES>();
        block_barrier();
        compute(live_, lds + s * C::STAGE, lds + (s + C::STAGES - 1) % C::STAGES * C::STAGE, kb);
        done = ++kb >= kb1;
      }
      if (done) break;
    }
  };
  if constexpr (GROUPED) {  // (the same number of barriers in every one)
    switch (live) {
      case 0: k_loop(Int<0>{}); break;
      case 1: k_loop(Int<1>{}); break;
      case 2: if constexpr (SM >= 2) k_loop(Int<2>{}); break;
      case 3: if constexpr (SM >= 3) k_loop(Int<3>{}); break;
      default: if constexpr (SM >= 4) k_loop(Int<4>{}); break;
    }
  } else {
    k_loop(Int<SM>{});
  }
  wait_memory<0>();  // no copy is under way when LDS is used again, or ends

  // A lane holds four times four consecutive columns of its row per sub-tile.
  // Where rows can be stored in 16-byte pieces, each wave turns its tile over
  // in LDS, 32 rows at a time, so that consecutive lanes store consecutive
  // bytes (the pieces of a row in the order p ^ row % 8, against bank
  // conflicts).
  uint8_t* const out = reinterpret_cast<uint8_t*>(g.out) + (size_t)blockIdx.y * g.M * g.N * 4;
  constexpr int EB = OUT32 ? 4 : 2;           // bytes per value
  constexpr int RB = SN * 32 * EB;            // bytes per row of the wave's tile
  constexpr int PIECES = RB / 16, RPI = 64 / PIECES;  // pieces per row, rows per store
  static_assert(C::WAVES * 32 * RB <= (int)sizeof(lds), "every wave has room for 32 rows");
  if (g.N % (16 / EB) == 0 && (uintptr_t)out % 16 == 0) {
    int orow[SM][32 / RPI];  // before the stores: a load behind them would wait for them
#pragma unroll
    for (int s = 0; s < SM; s++)
#pragma unroll
      for (int u = 0; u < 32 / RPI; u++)
        orow[s][u] = out_row(m0 + (s * C::WM + wm) * 32 + u * RPI + lane / PIECES);
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
          store4<OUT32>(d, 0, v);
        }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int u = 0; u < 32 / RPI; u++) {
        const int row = u * RPI + lane / PIECES, piece = lane % PIECES;
        const int n = nw + piece * (16 / EB);
        const u32x4 v =
            *reinterpret_cast<const u32x4*>(mine + row * RB + (piece ^ (row % 8 % PIECES)) * 16);
        if (orow[s][u] >= 0 && n < g.N)
          *reinterpret_cast<u32x4*>(out + ((size_t)orow[s][u] * g.N + n) * EB) = v;
      }
      __builtin_amdgcn_wave_barrier();
    }
    return;
  }
#pragma unroll
  for (int s = 0; s < SM; s++) {
    const int orow = out_row(m0 + (s * C::WM + wm) * 32 + r32);
    if (orow < 0) continue;
    const size_t o = (size_t)orow * g.N;
#pragma unroll
    for (int i = 0; i < SN; i++)
#pragma unroll
      for (int r = 0; r < 16; r++) {
        const int n = nw + i * 32 + 8 * (r >> 2) + 4 * h + (r & 3);
        if (n < g.N) store1<OUT32>(out, o + n, acc[i][s][r]);
      }
  }
}

// out = the sum of the parts of a K split, in order.
template <bool F32>
__global__ __launch_bounds__(256) void fp8_matmul_sum_kernel(const float* __restrict__ parts,
                                                             int splits, size_t count, void* out,
                                                             bool wide) {
  const size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= count) return;
  if (wide) {  // count is a multiple of 4, out is aligned for 4 values
    f32x4 v = *reinterpret_cast<const f32x4*>(parts + i);
    for (int p = 1; p < splits; p++) {
      const f32x4 x = *reinterpret_cast<const f32x4*>(parts + p * count + i);
#pragma unroll
      for (int r = 0; r < 4; r++) v[r] += x[r];
    }
    const float w[4] = {v[0], v[1], v[2], v[3]};
    store4<F32>(out, i, w);
  } else {
    for (size_t j = i; j < i + 4 && j < count; j++) {
      float v = parts[j];
      for (int p = 1; p < splits; p++) v += parts[p * count + j];
      store1<F32>(out, j, v);
    }
  }
}

// Tiles of a product; `splits` parts of K with fp32 outputs (OUT32).
template <class C, bool GROUPED, bool BBLOCK, bool EXACT, bool OUT32 = EXACT>
hipError_t launch_tile(Fp8MatmulArgs g, hipStream_t s, int splits = 1) {
  // Grouped: at most one row tile per BM rows and one more per expert.
  const long long ntm = GROUPED ? g.M / C::BM + (g.E < g.P ? g.E : g.P) : (g.M + C::BM - 1) / C::BM;
  const long long total = (long long)((g.N + C::BN - 1) / C::BN) * ntm;
  if (total > (1ll << 30)) return hipErrorInvalidValue;
  g.split_kb = (g.KB + splits - 1) / splits;  // (a part of `splits` has one K block at least)
  hipLaunchKernelGGL((fp8_matmul_tile_kernel<C, GROUPED, BBLOCK, EXACT, OUT32>),
                     dim3((unsigned)((total + 7) / 8 * 8), splits), dim3(C::THREADS), 0, s, g);
  return hipGetLastError();
}

// A product whose K is split: the parts' sums in g.parts, then their total.
template <class C, bool BBLOCK, bool EXACT>
hipError_t launch_split(Fp8MatmulArgs g, int splits, hipStream_t s) {
  if (splits == 1) return launch_tile<C, false, BBLOCK, EXACT>(g, s);
  void* out = g.out;
  g.out = g.parts;
  const hipError_t e = launch_tile<C, false, BBLOCK, EXACT, true>(g, s, splits);
  if (e != hipSuccess) return e;
  const size_t count = (size_t)g.M * g.N;
  const bool wide = count % 4 == 0 && (uintptr_t)out % 16 == 0;
  const dim3 grid((unsigned)((count + 1023) / 1024));
  if (g.out_f32)
    hipLaunchKernelGGL(fp8_matmul_sum_kernel<true>, grid, dim3(256), 0, s, g.parts, splits, count,
                       out, wide);
  else
    hipLaunchKernelGGL(fp8_matmul_sum_kernel<false>, grid, dim3(256), 0, s, g.parts, splits, count,
                       out, wide);
  return hipGetLastError();
}

// The tiles, from the sharpest reuse of what a CU copies (64 KiB of operands
// feed 32 matrix instructions per SIMD in Big, 16 KiB 2 in Small) to the
// most blocks and the shortest latency.
typedef Tile<256, 256, 2, 4, 2> Big;
typedef Tile<128, 256, 2, 4, 3> Wide;
typedef Tile<128, 128, 2, 2, 2> Mid;
typedef Tile<64, 128, 2, 2, 3> Half;
typedef Tile<64, 64, 2, 2, 4> Small;
typedef Tile<32, 128, 1, 4, 2> Low;
typedef Tile<32, 128, 1, 4, 3> LowFew;
enum { kRows, kSmall, kHalf, kMid, kBig };

// Kernel and parts of K of a dense product: the largest tile that still gives
// every CU its blocks (two per CU, one of Big's), measured (us) as
//   rows x columns x K      Small  Half   Mid    Big
//   512 x 2048 x 2048         8.4   9.6   14.5
//   2048 x 2048 x 2048       18.9  14.7   16.0   29.0
//   2048 x 4096 x 4096       63.3  47.2   37.7   53.3
//   4096 x 4096 x 1024       39.9  28.1   23.5   22.5
// Mid's rounds over the chip cost 1 where Big's cost 1.9.  Where Small's tiles
// leave CUs without work, K is split in up to 8 parts of 6 K blocks or more
// (33 x 4096 x 4096: 9.3 us in four parts, 12 in one), which a second launch
// adds.
struct Plan {
  int kernel, splits;
};
Plan plan(int M, int N, int K, bool big) {
  if (M <= 32) return {kRows, 1};
  const int KB = K / 128, cus = device_cu_count();
  auto tiles = [&](int bm, int bn) {
    return (long long)((M + bm - 1) / bm) * ((N + bn - 1) / bn);
  };
  if (tiles(64, 64) <= 2 * cus) {
    int s = 8;
    while (s > 1 && (tiles(64, 64) * s > cus || KB / s < 6)) s /= 2;
    const int per = (KB + s - 1) / s;
    return {kSmall, (KB + per - 1) / per};  // no part without a K block
  }
  if (tiles(64, 128) <= 2 * cus) return {kHalf, 1};
  const long long mid = (tiles(128, 128) + 2 * cus - 1) / (2 * cus);
  const long long wide = (tiles(256, 256) + cus - 1) / cus;
  return {big && 1.9 * wide <= mid ? kBig : kMid, 1};
}

}  // namespace

size_t fp8_matmul_parts_bytes(int M, int N, int K) {
  const int a = plan(M, N, K, true).splits, b = plan(M, N, K, false).splits;
  const int most = a > b ? a : b;
  return most > 1 ? (size_t)most * M * N * 4 : 0;
}

namespace {
template <bool BBLOCK, bool EXACT>
hipError_t dense(const Fp8MatmulArgs& g, hipStream_t s) {
  // (Big is built for the products that reach its size: weights, bf16.)
  const Plan p = plan(g.M, g.N, g.K, BBLOCK && !EXACT);
  if constexpr (BBLOCK && !EXACT) {
    if (p.kernel == kBig) return launch_tile<Big, false, true, false>(g, s);
  }
  switch (p.kernel) {
    case kRows:
      return g.M <= 16 ? launch_rows<1, false, BBLOCK, EXACT>(g, s)
                       : launch_rows<2, false, BBLOCK, EXACT>(g, s);
    case kSmall: return launch_split<Small, BBLOCK, EXACT>(g, p.splits, s);
    case kHalf: return launch_tile<Half, false, BBLOCK, EXACT>(g, s);
    default: return launch_tile<Mid, false, BBLOCK, EXACT>(g, s);
  }
}

// By the mean rows per expert: the tile that holds most experts' rows at once,
// so that a matrix is read once (128 experts of 1536 x 2048, top-8, us):
//   tokens (mean)   rows16   Low   Half  Wide  Mid   Big
//   64 (4)            68      74    77
//   256 (16)         104      77    80          108
//   512 (32)                  90    84    86     92   102
//   1024 (64)                131   108    96    101   109
//   2048 (128)                            130   142   124
// and a smaller one where that leaves CUs without a block.  Low's two stages let
// more blocks share a CU, LowFew's three serve a block that has one to itself
// (us, Low / LowFew: 256 tokens of 8 on 128 experts of 2048 x 768 36.7 / 40.7;
// 128 of 2 on 8 of 1536 x 2048 12.6 / 9.2).  The rules go by the mean, which is
// known on the host: a router that sends most rows to few experts gets the tiles
// of an even one.
template <bool EXACT>
hipError_t grouped(const Fp8MatmulArgs& g, hipStream_t s) {
  const double mean = (double)g.P / g.E;
  const int cus = device_cu_count();
  if (g.block_m == 16 && mean <= 6) return launch_rows<1, true, true, EXACT>(g, s);
  auto blocks = [&](int bm, int bn) {  // experts that have rows, and full tiles
    return ((double)g.P / bm + (g.E < g.P ? g.E : g.P) * 0.5) * ((g.N + bn - 1) / bn);
  };
  if constexpr (EXACT) {  // (its sums of a K block need the registers of a smaller tile)
    if (mean > 48 && blocks(128, 128) >= 2 * cus) return launch_tile<Mid, true, true, true>(g, s);
  } else {
    if (mean > 96 && blocks(256, 256) >= 2 * cus) return launch_tile<Big, true, true, false>(g, s);
    if (mean > 48 && blocks(128, 256) >= 2 * cus) return launch_tile<Wide, true, true, false>(g, s);
  }
  if (mean > 20 && blocks(64, 128) >= cus) return launch_tile<Half, true, true, EXACT>(g, s);
  return blocks(32, 128) >= 2 * cus ? launch_tile<Low, true, true, EXACT>(g, s)
                                    : launch_tile<LowFew, true, true, EXACT>(g, s);
}
}  // namespace

hipError_t launch_fp8_matmul(const Fp8MatmulArgs& g, hipStream_t s) {
  if (g.b_block) return g.out_f32 ? dense<true, true>(g, s) : dense<true, false>(g, s);
  return g.out_f32 ? dense<false, true>(g, s) : dense<false, false>(g, s);
}

hipError_t launch_fp8_grouped_matmul(const Fp8MatmulArgs& g, hipStream_t s) {
  return g.out_f32 ? grouped<true>(g, s) : grouped<false>(g, s);
}

}  // namespace qmoe
