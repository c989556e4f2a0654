// Matrix products of every expert over its routed rows in bf16, the types the
// experts are trained in:
//
//   out[p] = a[row(p)] . b[e(p)]^T      b [E,N,K]   (projections)
//   out[p] = a[row(p)] . b[e(p)]        b [E,K,N]   (gradients of the rows)
//   dw[e]  = sum over e's pairs p of dy[p]^T x[row(p)]
//
// over qmoe_align's list, sums in fp32 on the matrix cores; SiLU * mul, or its
// gradient, is applied to the sums on their way out.
#include "block_common.h"
#include "qmoe_internal.h"
#include "tile_common.h"

namespace qmoe {
namespace {
using namespace bk;
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

enum { kPlain, kSilu, kSiluGrad };

template <class T>
__device__ inline bf16x8 as_bf16(T v) {
  static_assert(sizeof(T) == 16, "eight values");
  return __builtin_bit_cast(bf16x8, v);
}

// The pair in slot `slot` of the expert-sorted list, -1 for padding.
__device__ inline int pair_of(const GroupedArgs& g, int slot) {
  const int p = g.sorted[slot];
  return (unsigned)p < (unsigned)g.P ? p : -1;
}
__device__ inline int a_row(const GroupedArgs& g, int p) { return g.pair_rows ? p : p / g.k; }

// SiLU(g) u's gradients for the gradient d of the product.  With t = exp(-|g|)
// neither the sigmoid nor 1 minus it is a difference.
__device__ inline void silu_mul_grad(float d, float g, float u, float* dg, float* du) {
  const float t = expf(-fabsf(g)), r = 1.0f / (1.0f + t);
  const float s = g >= 0.f ? r : t * r, o = g >= 0.f ? t * r : r;  // (NaN: t is NaN)
  *dg = d * u * (s * (1.0f + g * o));
  *du = d * (g * s);
}

// ---------------------------------------------------------------------------
// Few rows: the work is reading b once.  A block computes 16 rows x 16 NS
// columns, its KS waves taking every KS-th K block of 64 values; operands go
// from memory to registers, RING K blocks ahead, and the waves' sums are added
// in wave order through LDS.  With SiLU * mul the two sub-tiles are a gate one
// and the up one of the same columns.
template <int KS, int NS, int RING, int ACT, bool F32>
__global__ __launch_bounds__(64 * KS) void grouped_rows_kernel(GroupedArgs g) {
  static_assert(ACT != kSilu || NS == 2, "gate and up");
  __shared__ f32x4 part[KS][NS][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int l = lane & 15, q = lane >> 4;
  const int cols = ACT == kSilu ? g.N / 2 : g.N;
  const int n0 = blockIdx.x * (ACT == kSilu ? 16 : 16 * NS);
  const int m0 = blockIdx.y * 16;
  if (m0 >= *g.num_padded) return;
  const int p = pair_of(g, m0 + l);
  if (__ballot(p >= 0) == 0) return;  // (padding alone)
  const uint16_t* b = g.b + (size_t)g.tile_expert[m0 / g.block_m] * g.N * g.K;
  const uint16_t* ap = g.a + (size_t)(p < 0 ? 0 : a_row(g, p)) * g.K + 8 * q;
  const uint16_t* bp[NS];
#pragma unroll
  for (int s = 0; s < NS; s++) {
    const int n = ACT == kSilu ? s * cols + min(n0 + l, cols - 1) : min(n0 + 16 * s + l, cols - 1);
    bp[s] = b + (size_t)n * g.K + 8 * q;
  }
  const int KB = (g.K + 63) / 64;
  struct Step {
    u32x4 a[2], b[NS][2];
  };
  Step ring[RING];
  const u32x4 none = {0u, 0u, 0u, 0u};
  // K block kb: the lane's values 8 q .. 8 q + 7 of each half of 32 (zeros
  // behind the row's end, which only the last block can reach).
  auto load = [&](Step& st, int kb) {
    const int at = kb * 64;
    const bool in0 = at + 8 * q < g.K, in1 = at + 32 + 8 * q < g.K;
#pragma unroll
    for (int s = 0; s < NS; s++) {
      st.b[s][0] = in0 ? *reinterpret_cast<const u32x4*>(bp[s] + at) : none;
      st.b[s][1] = in1 ? *reinterpret_cast<const u32x4*>(bp[s] + at + 32) : none;
    }
    st.a[0] = in0 ? *reinterpret_cast<const u32x4*>(ap + at) : none;
    st.a[1] = in1 ? *reinterpret_cast<const u32x4*>(ap + at + 32) : none;
  };
  f32x4 acc[NS];
#pragma unroll
  for (int s = 0; s < NS; s++) acc[s] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const Step& st) {
#pragma unroll
    for (int s = 0; s < NS; s++)
#pragma unroll
      for (int j = 0; j < 2; j++)
        acc[s] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16(st.b[s][j]), as_bf16(st.a[j]),
                                                         acc[s], 0, 0, 0);
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
  for (int s = 0; s < NS; s++) part[wave][s][lane] = acc[s];
  __syncthreads();
  auto total = [&](int s) {
    f32x4 v = part[0][s][lane];
#pragma unroll
    for (int w = 1; w < KS; w++) {
      const f32x4 x = part[w][s][lane];
#pragma unroll
      for (int r = 0; r < 4; r++) v[r] += x[r];
    }
    return v;
  };
  if (p < 0) return;
  if constexpr (ACT == kSilu) {
    const int n = n0 + 4 * q;
    if (wave != 0 || n >= cols) return;
    const f32x4 gate = total(0), up = total(1);
    float h[4];
#pragma unroll
    for (int r = 0; r < 4; r++) h[r] = silu_mul(gate[r], up[r]);
    store4<F32>(g.out, (size_t)p * cols + n, h);
    if (g.gu != nullptr) {
      const float a4[4] = {gate[0], gate[1], gate[2], gate[3]};
      const float b4[4] = {up[0], up[1], up[2], up[3]};
      store4<false>(g.gu, (size_t)p * g.N + n, a4);
      store4<false>(g.gu, (size_t)p * g.N + cols + n, b4);
    }
  } else {
#pragma unroll
    for (int s = wave; s < NS; s += KS) {
      const int n = n0 + 16 * s + 4 * q;
      if (n >= cols) continue;
      const f32x4 v = total(s);
      const float w[4] = {v[0], v[1], v[2], v[3]};
      store4<F32>(g.out, (size_t)p * g.N + n, w);
    }
  }
}

// ---------------------------------------------------------------------------
// Tiled kernels: a block of WM x WN waves computes BM rows x BN columns, a wave
// SM x SN sub-tiles of 32 x 32, in K blocks of 64 values that go from memory
// straight into LDS, STAGES of them.
//
// An operand whose rows hold consecutive values of K ("straight") has 128 bytes
// per row and K block, eight 16-byte chunks in the order c ^ (row / 2 % 8), so
// that the 16 rows that are read together lie in different banks.  One whose
// rows are the values of K ("turned": b of a row gradient, both operands of a
// weight gradient) lies in LDS as it does in memory, 64 rows of the tile's
// width, and is turned on the way to registers by LDS's transposing read (four
// rows x 16 columns per 16 lanes); the 32-byte units of a row are stored in the
// order u ^ 2 (row % 4), so that the four rows lie in different banks.
template <int BM_, int BN_, int WM_, int WN_, int STAGES_, int EU_ = 2>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, STAGES = STAGES_;
  static constexpr int EU = EU_;  // waves per SIMD that the registers allow for
  static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int SM = BM / WM / 32, SN = BN / WN / 32;
  static constexpr int AC = BM / 8 / WAVES, BC = BN / 8 / WAVES;  // copies per wave and K block
  static constexpr int COPIES = AC + BC;
  static constexpr int B_AT = BM * 128, STAGE = B_AT + BN * 128;
  static_assert(SM * WM * 32 == BM && SN * WN * 32 == BN, "whole sub-tiles");
  static_assert(AC * WAVES * 8 == BM && BC * WAVES * 8 == BN, "whole copies");
  static_assert(STAGES * STAGE <= 160 * 1024, "LDS");
};

// A turned operand of W columns in LDS: what the lane copies, and where it
// reads.
template <int W>
struct Turned {
  static constexpr int CPR = W / 8;        // 16-byte chunks per row
  static constexpr int RPC = 64 / CPR;     // rows per copy of a wave
  __device__ static inline int row(int t, int lane) { return t * RPC + lane / CPR; }
  // Column (in values) that the lane's chunk of copy t holds.
  __device__ static inline int col(int t, int lane) {
    return 8 * ((lane % CPR) ^ (4 * (row(t, lane) & 3) & (CPR - 1)));
  }
  // Byte offset of the lane's first four values of K in sub-tile `sub`, K 0.
  __device__ static inline int off(int sub, int lane) {
    const int i = lane & 15, g = lane >> 4;
    const int unit = (2 * sub + (g & 1)) ^ (2 * (i >> 2) & (W / 16 - 1));
    return (8 * (g >> 1) + (i >> 2)) * 2 * W + unit * 32 + (i & 3) * 8;
  }
  // Values 16 s + 8 h .. + 7 of K (h the lane's half) at the offset.
  __device__ static inline bf16x8 frag(const uint8_t* t, int off, int s) {
    typedef __attribute__((address_space(3))) s16x4* P;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(t + off + (16 * s) * 2 * W));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(t + off + (16 * s + 4) * 2 * W));
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    return as_bf16(s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
  }
};

template <int V>
struct Int {
  static constexpr int value = V;
};

// The K loop: STAGES - 1 K blocks under way, copy(stage, kb, c) one of a K
// block's COPIES copies of this wave (of nothing behind the last block),
// compute(stage, next stage, kb) a K block, with the next one's copies in it.
template <class C, class Copy, class Compute>
__device__ inline void k_loop(uint8_t* lds, int KB, const Copy& copy, const Compute& compute) {
#pragma unroll
  for (int s = 0; s < C::STAGES - 1; s++)
#pragma unroll
    for (int u = 0; u < C::COPIES; u++) copy(lds + s * C::STAGE, s, u);
  for (int kb = 0; kb < KB;) {
#pragma unroll
    for (int s = 0; s < C::STAGES; s++) {
      if (kb >= KB) continue;
      // Stage s has landed (the stages behind it may be under way), in every
      // wave; and every wave is done with the stage before, which is free now.
      wait_memory<(C::STAGES - 2) * C::COPIES>();
      block_barrier();
      compute(lds + s * C::STAGE, lds + (s + C::STAGES - 1) % C::STAGES * C::STAGE, kb);
      kb++;
    }
  }
  wait_memory<0>();  // no copy is under way when LDS is used again, or ends
}

// A wave's 32 rows x SN 32 columns of sums, turned over in LDS so that
// consecutive lanes hold consecutive bytes of a row (the 16-byte pieces of a
// row in the order p ^ row % 8, against bank conflicts).  value(i, r): the
// lane's sum r of sub-tile i; then piece(row, byte, address) for 16 bytes each.
template <int SN, bool F32, class Value, class Piece>
__device__ inline void turn_over(uint8_t* mine, const Value& value, const Piece& piece) {
  constexpr int EB = F32 ? 4 : 2, RB = SN * 32 * EB, PIECES = RB / 16, RPI = 64 / PIECES;
  const int lane = threadIdx.x & 63, r32 = lane & 31, h = lane >> 5;
#pragma unroll
  for (int i = 0; i < SN; i++)
#pragma unroll
    for (int q = 0; q < 4; q++) {
      const int byte = (i * 32 + 8 * q + 4 * h) * EB;
      uint8_t* d = mine + r32 * RB + ((byte / 16) ^ (r32 % 8 % PIECES)) * 16 + byte % 16;
      const float v[4] = {value(i, 4 * q), value(i, 4 * q + 1), value(i, 4 * q + 2),
                          value(i, 4 * q + 3)};
      store4<F32>(d, 0, v);
    }
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int u = 0; u < 32 / RPI; u++) {
    const int row = u * RPI + lane / PIECES, at = lane % PIECES;
    piece(u, row, at * 16, mine + row * RB + (at ^ (row % 8 % PIECES)) * 16);
  }
  __builtin_amdgcn_wave_barrier();
}

// out of every expert.  TRANS: b is [E,K,N] (turned).
template <class C, bool TRANS, int ACT, bool F32>
__global__ __launch_bounds__(C::THREADS, C::EU) void grouped_tile_kernel(GroupedArgs g) {
  constexpr int SM = C::SM, SN = C::SN;
  static_assert(ACT != kSilu || (SN % 2 == 0 && !TRANS), "gate and up sub-tiles");
  static_assert(ACT != kSiluGrad || TRANS, "the gradient's way back");
  __shared__ __align__(1024) uint8_t lds[C::STAGES * C::STAGE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave % C::WM, wn = wave / C::WM;
  // With SiLU * mul a tile is BN / 2 gate rows of b and the BN / 2 up rows of
  // the same columns, in alternating sub-tiles of 32.
  constexpr int TN = ACT == kSilu ? C::BN / 2 : C::BN;
  const int cols = ACT == kSilu ? g.N / 2 : g.N;
  const int ntn = (cols + TN - 1) / TN;
  Spans<C::BM> spans;
  const int ntm = spans.count(g);
  // The launch order deals blocks to the XCDs in turn: give each XCD a
  // contiguous run of tiles, column-tile by column-tile inside bands of kBand
  // row tiles, so that its L2 sees the same rows again.
  constexpr int kBand = 8;
  const int total = ntn * ntm, per = (total + 7) / 8;
  const int id = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8);
  if (id >= total || (int)(blockIdx.x / 8) >= per) return;  // also past the tiles in use
  const int band = id / (kBand * ntn), in = id - band * kBand * ntn;
  const int rows = min(kBand, ntm - band * kBand);
  const int mt = band * kBand + in % rows, n0 = in / rows * TN;
  int m0, mend;
  const int e = spans.find(g, mt, &m0, &mend);
  const uint16_t* b = g.b + (size_t)e * g.N * g.K;
  const int KB = (g.K + 63) / 64;
  auto out_row = [&](int slot) { return slot < mend ? pair_of(g, slot) : -1; };
  // The wave's sub-tiles of rows are wm, wm + WM, ...; those behind the last
  // one with a row (an expert's rows stand in front of its padding) are left
  // out.
  int live = 0;
#pragma unroll
  for (int s = 0; s < SM; s++)
    if (__ballot(out_row(m0 + (s * C::WM + wm) * 32 + (lane & 31)) >= 0) != 0) live = s + 1;
  live = __builtin_amdgcn_readfirstlane(live);

  // Copies of a straight operand: 8 lanes per row, the rows of a wave's copy t
  // being 8 t .. 8 t + 7; the chunk order alternates with t.
  const unsigned rowb = 2u * (unsigned)g.K;  // bytes per straight row
  const unsigned swz[2] = {16u * ((lane & 7) ^ ((lane >> 4) & 7)),
                           16u * ((lane & 7) ^ ((4 + (lane >> 4)) & 7))};
  const size_t abytes = (size_t)g.Ma * rowb;
  unsigned av[C::AC];
#pragma unroll
  for (int i = 0; i < C::AC; i++) {
    const int p = out_row(m0 + (wave * C::AC + i) * 8 + (lane >> 3));
    // no row: behind every buffer, so nothing is read
    av[i] = p < 0 ? kNowhere : (unsigned)a_row(g, p) * rowb;
  }
  auto copy = [&](uint8_t* st, int kb, int c) {
    const bool any = kb < KB;
    const unsigned at = any ? kb * 128 : 0, left = rowb - at;  // bytes of the row from here
    if (c < C::AC) {
      const int t = wave * C::AC + c;
      const unsigned ch = swz[(C::AC % 2 == 0 ? c : t) & 1];
      // chunks behind the row's end are zeros
      const unsigned v = ch < left && av[c] != kNowhere ? av[c] + ch : kNowhere;
      copy16(rsrc(g.a, any ? abytes : 0), v, at, st + t * 1024);
    } else if constexpr (TRANS) {
      typedef Turned<C::BN> Tn;
      const int t = wave * C::BC + (c - C::AC);
      const uint16_t* base = b + (any ? (size_t)kb * 64 * g.N : 0) + n0;
      const size_t bytes = any ? ((size_t)(g.K - kb * 64) * g.N - n0) * 2 : 0;
      copy16(rsrc(base, bytes),
             2u * ((unsigned)Tn::row(t, lane) * (unsigned)g.N + (unsigned)Tn::col(t, lane)), 0,
             st + C::B_AT + t * 1024);
    } else {
      const int i = c - C::AC, t = wave * C::BC + i;
      const unsigned ch = swz[(C::BC % 2 == 0 ? i : t) & 1];
      int row = t * 8, first = n0;
      if constexpr (ACT == kSilu) {
        row = t / 8 * 32 + t % 4 * 8;
        first += (t / 4 & 1) * cols;
      }
      const Rsrc rb = rsrc(b + (size_t)first * g.K,
                           any && first < g.N ? (size_t)(g.N - first) * rowb : 0);
      const unsigned v = (unsigned)(row + (lane >> 3)) * rowb + ch;
      copy16(rb, ch < left ? v : kNowhere, at, st + C::B_AT + t * 1024);
    }
  };
  // Reads: lane's row in a sub-tile and its half of each 16 values of K.
  const int r32 = lane & 31, h = lane >> 5;
  int off[4], offb[TRANS ? SN : 1];
#pragma unroll
  for (int s = 0; s < 4; s++) off[s] = r32 * 128 + 16 * ((2 * s + h) ^ ((r32 >> 1) & 7));
  if constexpr (TRANS) {
#pragma unroll
    for (int i = 0; i < SN; i++) offb[i] = Turned<C::BN>::off(wn * SN + i, lane);
  }
  auto straight = [&](const uint8_t* t, int sub, int s) {
    return as_bf16(*reinterpret_cast<const u32x4*>(t + sub * 4096 + off[s]));
  };
  f32x16 acc[SN][SM];
#pragma unroll
  for (int i = 0; i < SN; i++)
#pragma unroll
    for (int s = 0; s < SM; s++)
#pragma unroll
      for (int r = 0; r < 16; r++) acc[i][s][r] = 0.f;
  auto run = [&](auto live_) {
    constexpr int LIVE = decltype(live_)::value;  // sub-tile rows to compute
    k_loop<C>(lds, KB, copy, [&](const uint8_t* st, uint8_t* nx, int kb) {
      const int next = kb + C::STAGES - 1;
#pragma unroll
      for (int s = 0; s < 4; s++) {
        bf16x8 bf[SN], af[SM];
        if constexpr (LIVE > 0) {
#pragma unroll
          for (int i = 0; i < SN; i++) {
            if constexpr (TRANS)
              bf[i] = Turned<C::BN>::frag(st + C::B_AT, offb[i], s);
            else
              bf[i] = straight(st + C::B_AT, wn * SN + i, s);
          }
#pragma unroll
          for (int j = 0; j < LIVE; j++) af[j] = straight(st, j * C::WM + wm, s);
        }
#pragma unroll
        for (int u = s * C::COPIES / 4; u < (s + 1) * C::COPIES / 4; u++) copy(nx, next, u);
        if constexpr (LIVE > 0) {
#pragma unroll
          for (int j = 0; j < LIVE; j++)
#pragma unroll
            for (int i = 0; i < SN; i++)
              acc[i][j] =
                  __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf[i], af[j], acc[i][j], 0, 0, 0);
        }
      }
    });
  };
  switch (live) {  // (the same number of barriers in every one)
    case 0: run(Int<0>{}); break;
    case 1: run(Int<1>{}); break;
    case 2: if constexpr (SM >= 2) run(Int<2>{}); break;
    case 3: if constexpr (SM >= 3) run(Int<3>{}); break;
    default: if constexpr (SM >= 4) run(Int<4>{}); break;
  }

  // A lane holds four times four consecutive columns of its row per sub-tile.
  constexpr bool WIDE = F32 || ACT == kSiluGrad;  // turned over in fp32
  constexpr int EB = F32 ? 4 : 2, RB = SN * 32 * (WIDE ? 4 : 2);
  constexpr int RPI = 64 / (RB / 16);
  static_assert(C::WAVES * 32 * RB <= (int)sizeof(lds), "every wave has room for 32 rows");
  uint8_t* const out = reinterpret_cast<uint8_t*>(g.out);
  __syncthreads();  // the last K block has been read
  uint8_t* const mine = lds + wave * 32 * RB;
  // Global column of byte `byte` of a turned row of values of W bytes, whose
  // sub-tiles lie `step` columns apart.
#pragma unroll
  for (int s = 0; s < SM; s++) {
    if (s >= live) break;
    const int base = m0 + (s * C::WM + wm) * 32;
    int orow[32 / RPI];
#pragma unroll
    for (int u = 0; u < 32 / RPI; u++) orow[u] = out_row(base + u * RPI + lane / (RB / 16));
    if constexpr (ACT == kPlain) {
      turn_over<SN, F32>(
          mine, [&](int i, int r) { return acc[i][s][r]; },
          [&](int u, int, int byte, const uint8_t* v) {
            const int n = n0 + wn * SN * 32 + byte / EB;
            if (orow[u] >= 0 && n < cols)
              *reinterpret_cast<u32x4*>(out + ((size_t)orow[u] * cols + n) * EB) =
                  *reinterpret_cast<const u32x4*>(v);
          });
    } else if constexpr (ACT == kSilu) {
      if (g.gu != nullptr) {
        constexpr int RPG = 64 / (SN * 4);  // rows per store of bf16 pieces
        int grow[32 / RPG];
#pragma unroll
        for (int u = 0; u < 32 / RPG; u++) grow[u] = out_row(base + u * RPG + lane / (SN * 4));
        turn_over<SN, false>(
            mine, [&](int i, int r) { return acc[i][s][r]; },
            [&](int u, int, int byte, const uint8_t* v) {
              const int i = byte / 64, n = n0 + (wn * SN + i) / 2 * 32 + byte % 64 / 2;
              if (grow[u] >= 0 && n < cols)
                *reinterpret_cast<u32x4*>(g.gu + (size_t)grow[u] * g.N + (i & 1) * cols + n) =
                    *reinterpret_cast<const u32x4*>(v);
            });
      }
      constexpr int PH = SN / 2 * 32 * EB / 16, RPH = 64 / PH;
      int hrow[32 / RPH];
#pragma unroll
      for (int u = 0; u < 32 / RPH; u++) hrow[u] = out_row(base + u * RPH + lane / PH);
      turn_over<SN / 2, F32>(
          mine, [&](int i, int r) { return silu_mul(acc[2 * i][s][r], acc[2 * i + 1][s][r]); },
          [&](int u, int, int byte, const uint8_t* v) {
            const int n = n0 + wn * SN * 16 + byte / EB;
            if (hrow[u] >= 0 && n < cols)
              *reinterpret_cast<u32x4*>(out + ((size_t)hrow[u] * cols + n) * EB) =
                  *reinterpret_cast<const u32x4*>(v);
          });
    } else {
      turn_over<SN, true>(
          mine, [&](int i, int r) { return acc[i][s][r]; },
          [&](int u, int, int byte, const uint8_t* v) {
            const int n = n0 + wn * SN * 32 + byte / 4;
            if (orow[u] < 0 || n >= cols) return;
            const f32x4 d = *reinterpret_cast<const f32x4*>(v);
            const uint16_t* gu = g.gu + (size_t)orow[u] * 2 * cols + n;
            const u32x2 gt = *reinterpret_cast<const u32x2*>(gu);
            const u32x2 up = *reinterpret_cast<const u32x2*>(gu + cols);
            float dg[4], du[4];
#pragma unroll
            for (int r = 0; r < 4; r++)
              silu_mul_grad(d[r], bf16_f32((uint16_t)(gt[r / 2] >> (16 * (r & 1)))),
                            bf16_f32((uint16_t)(up[r / 2] >> (16 * (r & 1)))), &dg[r], &du[r]);
            store4<F32>(g.out, (size_t)orow[u] * 2 * cols + n, dg);
            store4<F32>(g.out, (size_t)orow[u] * 2 * cols + cols + n, du);
          });
    }
  }
}

// dw of every expert: BM rows (of dw: columns of dy) x BN columns (of x), both
// operands turned, K the expert's pairs.  A tile of an expert without pairs is
// zeros.
template <class C, bool F32>
__global__ __launch_bounds__(C::THREADS, C::EU) void grouped_wgrad_kernel(WgradArgs g) {
  constexpr int SM = C::SM, SN = C::SN;
  typedef Turned<C::BM> Ta;
  typedef Turned<C::BN> Tb;
  __shared__ __align__(1024) uint8_t lds[C::STAGES * C::STAGE];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave % C::WM, wn = wave / C::WM;
  const int ntn = (g.K + C::BN - 1) / C::BN, ntm = (g.N + C::BM - 1) / C::BM;
  // Each XCD takes a contiguous run of tiles, an expert's one after another,
  // so that its L2 holds the expert's rows.
  const int total = ntn * ntm * g.E, per = (total + 7) / 8;
  const int id = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8);
  if (id >= total || (int)(blockIdx.x / 8) >= per) return;
  const int e = id / (ntn * ntm), in = id - e * ntn * ntm;
  const int n0 = in % ntm * C::BM, k0 = in / ntm * C::BN;
  const int first = g.expert_offsets[e], end = g.expert_offsets[e + 1];
  const int KB = (end - first + 63) / 64;
  const size_t dbytes = (size_t)g.P * g.N * 2, xbytes = (size_t)g.Mx * g.K * 2;
  // The copies' rows are pairs of the list, looked up one K block before they
  // are copied.
  int pa[C::AC], pb[C::BC];
  auto look = [&](int kb) {
#pragma unroll
    for (int i = 0; i < C::AC; i++) {
      const int slot = first + kb * 64 + Ta::row(wave * C::AC + i, lane);
      pa[i] = slot < end ? g.sorted[slot] : g.P;
    }
#pragma unroll
    for (int i = 0; i < C::BC; i++) {
      const int slot = first + kb * 64 + Tb::row(wave * C::BC + i, lane);
      pb[i] = slot < end ? g.sorted[slot] : g.P;
    }
  };
  auto copy = [&](uint8_t* st, int kb, int c) {
    if (c == 0) look(kb);
    if (c < C::AC) {
      const int t = wave * C::AC + c, col = n0 + Ta::col(t, lane);
      const unsigned v = (unsigned)pa[c] < (unsigned)g.P && col < g.N
                             ? 2u * ((unsigned)pa[c] * (unsigned)g.N + (unsigned)col)
                             : kNowhere;
      copy16(rsrc(g.dy, dbytes), v, 0, st + t * 1024);
    } else {
      const int i = c - C::AC, t = wave * C::BC + i, col = k0 + Tb::col(t, lane);
      const int row = g.pair_rows ? pb[i] : pb[i] / g.k;
      const unsigned v = (unsigned)pb[i] < (unsigned)g.P && col < g.K
                             ? 2u * ((unsigned)row * (unsigned)g.K + (unsigned)col)
                             : kNowhere;
      copy16(rsrc(g.x, xbytes), v, 0, st + C::B_AT + t * 1024);
    }
  };
  int offa[SM], offb[SN];
#pragma unroll
  for (int j = 0; j < SM; j++) offa[j] = Ta::off(j * C::WM + wm, lane);
#pragma unroll
  for (int i = 0; i < SN; i++) offb[i] = Tb::off(wn * SN + i, lane);
  f32x16 acc[SN][SM];
#pragma unroll
  for (int i = 0; i < SN; i++)
#pragma unroll
    for (int s = 0; s < SM; s++)
#pragma unroll
      for (int r = 0; r < 16; r++) acc[i][s][r] = 0.f;
  k_loop<C>(lds, KB, copy, [&](const uint8_t* st, uint8_t* nx, int kb) {
    const int next = kb + C::STAGES - 1;
#pragma unroll
    for (int s = 0; s < 4; s++) {
      bf16x8 bf[SN], af[SM];
#pragma unroll
      for (int i = 0; i < SN; i++) bf[i] = Tb::frag(st + C::B_AT, offb[i], s);
#pragma unroll
      for (int j = 0; j < SM; j++) af[j] = Ta::frag(st, offa[j], s);
#pragma unroll
      for (int u = s * C::COPIES / 4; u < (s + 1) * C::COPIES / 4; u++) copy(nx, next, u);
#pragma unroll
      for (int j = 0; j < SM; j++)
#pragma unroll
        for (int i = 0; i < SN; i++)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf[i], af[j], acc[i][j], 0, 0, 0);
    }
  });
  constexpr int EB = F32 ? 4 : 2, RB = SN * 32 * EB;
  static_assert(C::WAVES * 32 * RB <= (int)sizeof(lds), "every wave has room for 32 rows");
  __syncthreads();  // the last K block has been read
  uint8_t* const mine = lds + wave * 32 * RB;
  uint8_t* const out = reinterpret_cast<uint8_t*>(g.out) + (size_t)e * g.N * g.K * EB;
#pragma unroll
  for (int s = 0; s < SM; s++)
    turn_over<SN, F32>(
        mine, [&](int i, int r) { return acc[i][s][r]; },
        [&](int, int row, int byte, const uint8_t* v) {
          const int n = n0 + (s * C::WM + wm) * 32 + row, k = k0 + wn * SN * 32 + byte / EB;
          if (n >= g.N || k >= g.K) return;
          u32x4* o = reinterpret_cast<u32x4*>(out + ((size_t)n * g.K + k) * EB);
          u32x4 w = *reinterpret_cast<const u32x4*>(v);
          if (g.accumulate) {  // (fp32 only)
            const u32x4 was = *o;
#pragma unroll
            for (int r = 0; r < 4; r++)
              w[r] = __float_as_uint(__uint_as_float(was[r]) + __uint_as_float(w[r]));
          }
          *o = w;
        });
}

typedef Tile<256, 256, 2, 4, 2> Big;
typedef Tile<128, 128, 2, 2, 2> Mid;
typedef Tile<32, 256, 1, 4, 2> Low;

template <class C, bool TRANS, int ACT, bool F32>
hipError_t launch_tile(const GroupedArgs& g, hipStream_t s) {
  constexpr int TN = ACT == kSilu ? C::BN / 2 : C::BN;
  const int cols = ACT == kSilu ? g.N / 2 : g.N;
  // At most one row tile per BM rows and one more per expert.
  const long long ntm = g.M / C::BM + (g.E < g.P ? g.E : g.P);
  const long long total = (long long)((cols + TN - 1) / TN) * ntm;
  if (total > (1ll << 30)) return hipErrorInvalidValue;
  hipLaunchKernelGGL((grouped_tile_kernel<C, TRANS, ACT, F32>),
                     dim3((unsigned)((total + 7) / 8 * 8)), dim3(C::THREADS), 0, s, g);
  return hipGetLastError();
}

template <int ACT, bool F32>
hipError_t launch_rows(const GroupedArgs& g, hipStream_t s) {
  const int cols = ACT == kSilu ? g.N / 2 : g.N, step = ACT == kSilu ? 16 : 32;
  const int mt = g.M / 16;
  if (mt > 65535) return hipErrorInvalidValue;
  hipLaunchKernelGGL((grouped_rows_kernel<4, 2, 2, ACT, F32>), dim3((cols + step - 1) / step, mt),
                     dim3(256), 0, s, g);
  return hipGetLastError();
}

template <bool TRANS, int ACT, bool F32>
hipError_t launch(const GroupedArgs& g, hipStream_t s) {
  const double mean = (double)g.P / g.E;
  if constexpr (!TRANS) {
    if (mean <= 6) return launch_rows<ACT, F32>(g, s);
  }
  if (mean > 128) return launch_tile<Big, TRANS, ACT, F32>(g, s);
  if (mean > 24) return launch_tile<Mid, TRANS, ACT, F32>(g, s);
  return launch_tile<Low, TRANS, ACT, F32>(g, s);
}

template <class C>
hipError_t launch_wgrad(const WgradArgs& g, hipStream_t s) {
  const long long total =
      (long long)((g.K + C::BN - 1) / C::BN) * ((g.N + C::BM - 1) / C::BM) * g.E;
  if (total > (1ll << 30)) return hipErrorInvalidValue;
  const dim3 grid((unsigned)((total + 7) / 8 * 8));
  if (g.out_f32)
    hipLaunchKernelGGL((grouped_wgrad_kernel<C, true>), grid, dim3(C::THREADS), 0, s, g);
  else
    hipLaunchKernelGGL((grouped_wgrad_kernel<C, false>), grid, dim3(C::THREADS), 0, s, g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_matmul(const GroupedArgs& g, hipStream_t s) {
  const int which = g.act == QMOE_ACT_SILU_MUL ? 2 : g.act == QMOE_ACT_SILU_MUL_BACKWARD ? 3
                    : g.trans                  ? 1
                                               : 0;
  switch (which) {
    case 0: return g.out_f32 ? launch<false, kPlain, true>(g, s) : launch<false, kPlain, false>(g, s);
    case 1: return g.out_f32 ? launch<true, kPlain, true>(g, s) : launch<true, kPlain, false>(g, s);
    case 2: return g.out_f32 ? launch<false, kSilu, true>(g, s) : launch<false, kSilu, false>(g, s);
    default:
      return g.out_f32 ? launch<true, kSiluGrad, true>(g, s) : launch<true, kSiluGrad, false>(g, s);
  }
}

hipError_t launch_grouped_wgrad(const WgradArgs& g, hipStream_t s) {
  return launch_wgrad<Mid>(g, s);
}

}  // namespace qmoe
