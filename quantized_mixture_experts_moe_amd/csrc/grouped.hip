// Matrix products of every expert over its routed rows in bf16, the types the
// experts are trained in:
//
//   out[p] = a[row(p)] . b[e(p)]^T      b [E,N,K]   (projections)
//   out[p] = a[row(p)] . b[e(p)]        b [E,K,N]   (gradients of the rows)
//   dw[e]  = sum over e's pairs p of dy[p]^T x[row(p)]
//
// over qmoe_align's list, sums in fp32 on the matrix cores; SiLU * mul, or its
// gradient, is applied to the sums on their way out, so that each is rounded once.
//
// Bounds and measured (the rates of a large copy 5.1, of reads alone 6.2, of a fill
// 6.9 TB/s, of a large dense bf16 product 1.45 PFLOP/s): 4 tokens on 128 experts of
// 1536 x 2048 (top-8) 38 us, 183 MB of weights at 4.8 TB/s; 2048 tokens there with
// SiLU * mul and the gate/up kept 192-225 us, 0.89 GB at 4.0-4.6 TB/s; their way back
// through the down projection 125-133 us, 0.57 GB at 4.3-4.6 TB/s; 4111 tokens on 8 experts
// of 4096 x 4096 (top-2) 282 us, 0.98 PFLOP/s; weight gradients of 128 experts in fp32
// 276-310 us, 1.67 GB at 5.4-6.0 TB/s, of 8 experts of 2048 x 1536 60-68 us, 0.76-0.86
// PFLOP/s.  (The first figure is for calls on changing inputs; the second for the same call
// again and again, back to back.)
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

// Four values past the L2, which is left to the operands.
template <bool F32>
__device__ inline void store4_past(void* p, size_t i, const float v[4]) {
  if constexpr (F32)
    __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]},
                                reinterpret_cast<f32x4*>(reinterpret_cast<float*>(p) + i));
  else
    __builtin_nontemporal_store(u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])},
                                reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(p) + i));
}

// SiLU(g) u's gradients for the gradient d of the product.  With t = exp(-|g|)
// neither the sigmoid nor 1 minus it is a difference; t and the quotient are formed as
// silu_mul does.  The slope, at most 1.1, goes to the larger of d and u first: d u
// alone can leave fp32's range where the result does not, and the slope times the
// smaller one can fall below it.
__device__ inline void silu_mul_grad(float d, float g, float u, float* dg, float* du) {
  const float x = fminf(fabsf(g), 1000.0f);  // (a NaN of g is in g's own products below)
  const float hi = x * -1.44269502162933349609375f;
  const float lo = __builtin_fmaf(x, -1.44269502162933349609375f, -hi) - x * 1.925963033500e-8f;
  float t = __builtin_amdgcn_exp2f(hi);
  t = __builtin_fmaf(t, lo * 0.693147180559945f, t);
  const float v = 1.0f + t;
  float r = __builtin_amdgcn_rcpf(v);
  r = __builtin_fmaf(__builtin_fmaf(-v, r, 1.0f), r, r);
  const float s = g >= 0.f ? r : t * r, o = g >= 0.f ? t * r : r;
  const bool more = fabsf(d) > fabsf(u);
  *dg = (s * (1.0f + g * o)) * (more ? d : u) * (more ? u : d);
  *du = d * (g * s);
}

// ---------------------------------------------------------------------------
// Few rows: the work is reading b once.  A block computes 16 rows x 16 NS
// columns, its KS waves taking every KS-th K block of 64 values; operands go
// from memory to registers, RING K blocks ahead (no other wave needs them), and
// the waves' sums are added in wave order through LDS.  With SiLU * mul the two
// sub-tiles are a gate one and the up one of the same columns.  b in 16-row
// fragments: four lanes read 64 consecutive bytes of a row; 32-row ones, 32 bytes a
// row, look up twice the lines per load, and the wide tiles fed that way from
// registers took 266 us where LDS takes 232 (2048 tokens, 128 experts).
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
template <int BM_, int BN_, int WM_, int WN_, int STAGES_, int EU_ = 2,
          int SPREAD_ = 2, int STEPS_ = 4>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, STAGES = STAGES_;
  static constexpr int EU = EU_;  // waves per SIMD that the registers allow for
  static constexpr int SPREAD = SPREAD_;  // steps of a K block that issue the next one's copies
  static constexpr int STEPS = STEPS_;    // steps of 16 values of K per K block
  static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int SM = BM / WM / 32, SN = BN / WN / 32;
  // copies of 1 KiB per wave and K block
  static constexpr int AC = BM * STEPS / 32 / WAVES, BC = BN * STEPS / 32 / WAVES;
  static constexpr int COPIES = AC + BC;
  static constexpr int B_AT = BM * STEPS * 32, STAGE = B_AT + BN * STEPS * 32;
  static constexpr int FIT = 160 * 1024 / (STAGES * STAGE + WAVES * 4096 + 2 * BM * 4 + 1028 * 4);
  static constexpr int PER_CU = FIT > 0 ? FIT : 1;  // blocks
  static_assert(SM * WM * 32 == BM && SN * WN * 32 == BN, "whole sub-tiles");
  static_assert(AC * WAVES * 32 == BM * STEPS && BC * WAVES * 32 == BN * STEPS, "whole copies");
  static_assert(STAGES * STAGE <= 160 * 1024, "LDS");
};

// A turned operand of W columns in LDS: what the lane copies, and where it
// reads.
template <int W>
struct Turned {
  static constexpr int CPR = W / 8;  // 16-byte chunks per row
  static_assert(W % 128 == 0, "rows start in the same bank");
  __device__ static inline int row(int t, int lane) { return (t * 64 + lane) / CPR; }
  // Column (in values) that the lane's chunk of copy t holds.
  __device__ static inline int col(int t, int lane) {
    return 8 * ((t * 64 + lane) % CPR ^ 4 * (row(t, lane) & 3));
  }
  // Byte offset of the lane's first four values of K in sub-tile `sub`, K 0.
  __device__ static inline int off(int sub, int lane) {
    const int i = lane & 15, g = lane >> 4;
    const int unit = (2 * sub + (g & 1)) ^ 2 * (i >> 2);
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

// The largest divisor of n that is at most b.
constexpr int part_of(int n, int b) { return n <= b ? n : n % b == 0 ? b : part_of(n, b - 1); }

template <int N>
constexpr int largest(const int (&v)[N]) {
  int m = v[0];
  for (int i = 1; i < N; i++) m = v[i] > m ? v[i] : m;
  return m;
}

// The time of a K block in stage st: the wave issues the matrix instructions of
// the step before (the last one's of the block before at first; FIRST: there is
// none), between them the reads of the next step and copies to stage nx, in the
// order written here (the compiler would gather the reads of a step in front of it
// and the copies behind).  copy(nx, c) issues one of the wave's COPIES copies;
// read(st, s, r) one of the NR fragments of step s, to the half s % 2 of the
// wave's; mul(s, m) one of the NM matrix instructions on them.  The last step's
// are left to the next K block, or to the end.  The stages are __restrict__: the
// compiler cannot tell them apart otherwise and waits for every copy under way in
// front of each transposing read.  (A 4096^3 product: 122 us with a step's reads in
// front of it, 111 so; its turned form 141 with those waits, 120 without, 112 so.)
template <class C, int NR, int NM, bool FIRST, class Copy, class Read, class Mul>
__device__ inline void k_block(const uint8_t* __restrict__ st, uint8_t* __restrict__ nx,
                               const Copy& copy, const Read& read, const Mul& mul) {
  constexpr int PER = (C::COPIES + C::SPREAD - 1) / C::SPREAD;  // copies per step
#pragma unroll
  for (int s = 0; s < C::STEPS; s++) {
#pragma unroll
    for (int m = 0; m < NM; m++) {
      if (!FIRST || s > 0) mul((s + C::STEPS - 1) % C::STEPS, m);
#pragma unroll
      for (int r = 0; r < NR; r++)
        if (r * NM / NR == m) read(st, s, r);
#pragma unroll
      for (int c = 0; c < PER; c++)
        if (c * NM / PER == m && s * PER + c < C::COPIES) copy(nx, s * PER + c);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// The K loop of a block with one tile, STAGES - 1 K blocks under way: copy(stage,
// kb, c) is of nothing behind the last block.
template <class C, int NR, int NM, class Copy, class Read, class Mul>
__device__ inline void k_loop(uint8_t* lds, int KB, const Copy& copy, const Read& read,
                              const Mul& mul) {
#pragma unroll
  for (int s = 0; s < C::STAGES - 1; s++)
#pragma unroll
    for (int u = 0; u < C::COPIES; u++) copy(lds + s * C::STAGE, s, u);
  if (KB > 0) {
    // The block's stage has landed (those behind it may be under way), in every
    // wave; and every wave is done with the stage before, which is free now.
    auto step = [&](auto first, uint8_t* st, uint8_t* nx, int kb) {
      wait_memory<(C::STAGES - 2) * C::COPIES>();
      block_barrier();
      k_block<C, NR, NM, decltype(first)::value != 0>(
          st, nx, [&](uint8_t* to, int c) { copy(to, kb + C::STAGES - 1, c); }, read, mul);
    };
    step(Int<1>{}, lds, lds + (C::STAGES - 1) * C::STAGE, 0);
    uint8_t *nx = lds, *st = lds + C::STAGE;
    for (int kb = 1; kb < KB; kb++) {
      step(Int<0>{}, st, nx, kb);
      nx = st;
      st = st == lds + (C::STAGES - 1) * C::STAGE ? lds : st + C::STAGE;
    }
#pragma unroll
    for (int m = 0; m < NM; m++) mul(C::STEPS - 1, m);
  }
  wait_memory<0>();  // no copy is under way when LDS is used again, or ends
}

// 32 rows x 8 NQ columns of a wave's sums (NQ at most ROW bytes of them), turned
// over in LDS, ROWS rows at a time, so that consecutive lanes hold consecutive bytes
// of a row.  The 16-byte pieces of a row lie in an order that changes from row to row
// (every row where 128 bytes or more make a row, every fourth of 64 bytes), against
// bank conflicts.  value(q, r): the lane's value of column 8 q + 4 h + r, h its half;
// then piece(u, byte, address) for 16 bytes of row u * 64 / (ROW / 16) + lane / (ROW
// / 16).
template <int NQ, bool F32, int ROW, int ROWS, class Value, class Piece>
__device__ inline void turn_over(uint8_t* mine, const Value& value, const Piece& piece) {
  constexpr int EB = F32 ? 4 : 2, PIECES = ROW / 16, RPI = 64 / PIECES;
  static_assert(NQ * 8 * EB <= ROW, "a row's bytes");
  const int lane = threadIdx.x & 63, r32 = lane & 31, h = lane >> 5;
  static_assert(ROW >= 64 && ROWS % RPI == 0, "four pieces, whole turns");
  auto order = [](int row) { return (ROW >= 128 ? row : row >> 2) & 7 & (PIECES - 1); };
  float v[NQ][4];
#pragma unroll
  for (int q = 0; q < NQ; q++)
#pragma unroll
    for (int r = 0; r < 4; r++) v[q][r] = value(q, r);
#pragma unroll
  for (int part = 0; part < 32 / ROWS; part++) {
    if (ROWS == 32 || r32 / ROWS == part) {
#pragma unroll
      for (int q = 0; q < NQ; q++) {
        const int byte = (8 * q + 4 * h) * EB;
        uint8_t* d = mine + r32 % ROWS * ROW + ((byte / 16) ^ order(r32)) * 16 + byte % 16;
        store4<F32>(d, 0, v[q]);
      }
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int u = part * ROWS / RPI; u < (part + 1) * ROWS / RPI; u++) {
      const int row = u * RPI + lane / PIECES, at = lane % PIECES;
      if (at * 16 < NQ * 8 * EB)
        piece(u, at * 16, mine + row % ROWS * ROW + (at ^ order(row)) * 16);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// LDS of a tile: the stages, room where each wave turns its sums over, ROWS rows x ROW
// bytes at a time, and the pairs of two tiles; kOffsets more for expert_offsets.
constexpr int kOffsets = 1028;
template <class C, int ACT, bool F32>
struct Room {
  static constexpr bool WIDE = F32 || ACT == kSiluGrad;  // in fp32 (the gradient: rounded behind)
  static constexpr int PAIRS = 2 * C::BM * 4;
  static constexpr int LEFT =
      (160 * 1024 - C::STAGES * C::STAGE - PAIRS - kOffsets * 4) / C::WAVES;
  static constexpr int ROWS = LEFT < 2048 ? 8 : 32;
  static constexpr int ROW =
      ROWS == 32 && (LEFT < 4096 || (ACT == kSilu && !F32 && C::SN < 4)) ? 64 : 128;
  static constexpr int BYTES = C::STAGES * C::STAGE + C::WAVES * ROWS * ROW + PAIRS;
  static_assert(ROWS * ROW <= LEFT, "LDS");
};

// expert_offsets in LDS (a look-up in memory would wait behind the stores of a tile).
struct List {
  const int32_t* expert_offsets;
  int E;
};

// Column tiles (with SiLU * mul, N is gate and up together, and so is BN).
template <class C>
__host__ __device__ inline int columns(int N) {
  return (N + C::BN - 1) / C::BN;
}

// out of every expert.  TRANS: b is [E,K,N] (turned).
//
// A block takes one tile after another.  While it works on a tile's last K block
// the next tile's first one is on its way, and the finished sums go to memory
// under the next tile's second one, so that neither a tile's start nor its end
// leaves the memory idle (128 experts, 2048 tokens, us with a block per tile and so:
// 1536 x 512 69 and 64, 2048 x 768 114 and 107, 1536 x 2048 235 and 232).  Stores
// go past the L2, which the operands' rows need (that product 212 us so).
//
// Of several tiles (MORE) the block takes the one whose rounds over the chip cost least
// for the rows that each expert has: a router that spreads its rows unevenly fills other
// tiles than one that does not, and the host does not know.
//
// Bound (that product with 192 x 256 tiles, back to back, us; all of it 214-225): the
// copies alone 161, with the stores 184, everything but the stores 188; the matrix cores
// are busy a quarter of the time.  Its way back (192 x 384; 130-133): copies 93, with the
// gradient's reads and stores 130, everything but those 94.  At 4096^3 the matrix cores
// are busy 63% of the time, at the 1.8 GHz that the power leaves.
template <class C, bool TRANS, int ACT, bool F32>
__device__ inline void grouped_tiles(const GroupedArgs& g, const List& list, uint8_t* lds) {
  constexpr int SM = C::SM, SN = C::SN;
  static_assert(C::STAGES == 2 && C::STEPS == 4, "two stages of 64 values");
  static_assert(ACT != kSilu || !TRANS, "a projection");
  static_assert(ACT != kSiluGrad || TRANS, "the gradient's way back");
  static_assert(C::BM <= C::THREADS, "a thread per row");
  typedef Room<C, ACT, F32> Rm;
  constexpr bool WIDE = Rm::WIDE;
  constexpr int ROWS = Rm::ROWS, ROW = Rm::ROW, ROOM = ROWS * ROW;
  uint8_t* const turn = lds + C::STAGES * C::STAGE;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave % C::WM, wn = wave / C::WM;
  uint8_t* const mine = turn + wave * ROOM;
  // The tile's pairs, and the next one's.
  int32_t* pairs = reinterpret_cast<int32_t*>(turn + C::WAVES * ROOM);
  int32_t* next_pairs = pairs + C::BM;
  // With SiLU * mul a tile is BN / 2 gate rows of b and the BN / 2 up rows of
  // the same columns, eight of each in turn, so that a lane holds both sums.
  constexpr int TN = ACT == kSilu ? C::BN / 2 : C::BN;
  const int cols = ACT == kSilu ? g.N / 2 : g.N;
  const int ntn = columns<C>(g.N), KB = (g.K + 63) / 64;
  Spans<C::BM> spans;
  const int ntm = spans.count(list);
  // The launch order deals blocks to the XCDs in turn: each XCD's blocks take a
  // contiguous run of tiles, column-tile by column-tile inside bands of kBand
  // row tiles, so that its L2 sees the same rows again.
  constexpr int kBand = 8;
  const int total = ntn * ntm, per = (total + 7) / 8, stride = gridDim.x / 8;
  const int last = min(total, ((int)(blockIdx.x % 8) + 1) * per);
  int id = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8) + g.first;
  if (id >= last) return;  // also past the tiles in use

  // A tile: expert e, rows from slot m0 to mend, columns from n0.
  struct Where {
    int e, m0, mend, n0;
  };
  auto find = [&](int at) {
    Where w;
    const int band = at / (kBand * ntn), in = at - band * kBand * ntn;
    const int rows = min(kBand, ntm - band * kBand);
    w.n0 = in / rows * TN;
    w.e = spans.find(list, band * kBand + in % rows, &w.m0, &w.mend);
    return w;
  };
  auto my_pair = [&](const Where& w) {
    const int slot = w.m0 + (int)threadIdx.x;
    return threadIdx.x < C::BM && slot < w.mend ? pair_of(g, slot) : -1;
  };
  // What the block copies: rows of a (byte offsets, behind every buffer where
  // there is none), and b from the tile's first row or column.
  const unsigned rowb = 2u * (unsigned)g.K;  // bytes per straight row
  const size_t abytes = (size_t)g.Ma * rowb;
  unsigned av[C::AC];
  Where at;
  auto set_rows = [&](const int32_t* of) {
#pragma unroll
    for (int i = 0; i < C::AC; i++) {
      const int p = of[(wave * C::AC + i) * 8 + (lane >> 3)];
      av[i] = p < 0 ? kNowhere : (unsigned)a_row(g, p) * rowb;
    }
  };
  // Copies of a straight operand: 8 lanes per row, the rows of a wave's copy t
  // being 8 t .. 8 t + 7; the chunk order alternates with t.
  const unsigned swz[2] = {16u * ((lane & 7) ^ ((lane >> 4) & 7)),
                           16u * ((lane & 7) ^ ((4 + (lane >> 4)) & 7))};
  // Copy c of K block kb of the tile `at`, of nothing behind the last block.
  auto copy = [&](uint8_t* st, int kb, int c) {
    const unsigned any = kb < KB ? 1 : 0;
    const unsigned from = any * kb * 128, left = rowb - from;  // bytes of the row from here
    const uint16_t* const b = g.b + (size_t)at.e * g.N * g.K;
    if (c < C::AC) {
      const int t = wave * C::AC + c;
      const unsigned ch = swz[(C::AC % 2 == 0 ? c : t) & 1];
      // chunks behind the row's end are zeros
      const unsigned v = ch < left && av[c] != kNowhere ? av[c] + ch : kNowhere;
      copy16(rsrc(g.a, abytes * any), v, from, st + t * 1024);
    } else if constexpr (TRANS) {
      typedef Turned<C::BN> Tn;
      const int t = wave * C::BC + (c - C::AC);
      const int k0 = any * kb * 64;
      copy16(rsrc(b + (size_t)k0 * g.N + at.n0, ((size_t)(g.K - k0) * g.N - at.n0) * 2 * any),
             2u * ((unsigned)Tn::row(t, lane) * (unsigned)g.N + (unsigned)Tn::col(t, lane)), 0,
             st + C::B_AT + t * 1024);
    } else {
      const int i = c - C::AC, t = wave * C::BC + i;
      const unsigned ch = swz[(C::BC % 2 == 0 ? i : t) & 1];
      int row = t * 8, first = at.n0;
      if constexpr (ACT == kSilu) {
        row = t / 2 * 8;
        first += (t & 1) * cols;
      }
      const unsigned v = (unsigned)(row + (lane >> 3)) * rowb + ch;
      copy16(rsrc(b + (size_t)first * g.K, (size_t)(max(g.N - first, 0) * any) * rowb),
             ch < left ? v : kNowhere, from, st + C::B_AT + t * 1024);
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

  constexpr int PIECES = ROW / 16, RPI = 64 / PIECES;
  // A lane holds four times four consecutive columns of its row per sub-tile; 32
  // rows x ROW bytes of them are turned over in LDS at a time, so that consecutive
  // lanes store consecutive bytes.
  auto write_out = [&](f32x16 (&acc)[SN][SM], int live, int n0) {
    constexpr int EB = F32 ? 4 : 2, NQ = ROW / (WIDE ? 32 : 16);  // eights of columns per turn
    uint8_t* const out = reinterpret_cast<uint8_t*>(g.out);
#pragma unroll
    for (int s = 0; s < SM; s++) {
      if (s >= live) break;
      int row[32 / RPI];
#pragma unroll
      for (int u = 0; u < 32 / RPI; u++)
        row[u] = pairs[(s * C::WM + wm) * 32 + u * RPI + lane / PIECES];
      // The lane's sums of sub-tile row s: columns 8 q + 4 h + r of the wave's.
      auto sum = [&](int q, int r) { return acc[q / 4][s][4 * (q % 4) + r]; };
      auto put = [&](uint8_t* to, int width, int u, int n, const uint8_t* v) {
        const int p = row[u];
        if (p >= 0 && n < cols)
          __builtin_nontemporal_store(*reinterpret_cast<const u32x4*>(v),
                                      reinterpret_cast<u32x4*>(to + (size_t)p * width));
      };
      if constexpr (ACT == kPlain) {
        constexpr int Q = part_of(4 * SN, NQ);
#pragma unroll
        for (int q0 = 0; q0 < 4 * SN; q0 += Q)
          turn_over<Q, F32, ROW, ROWS>(
              mine, [&](int q, int r) { return sum(q0 + q, r); },
              [&](int u, int byte, const uint8_t* v) {
                const int n = n0 + wn * SN * 32 + q0 * 8 + byte / EB;
                put(out + (size_t)n * EB, cols * EB, u, n, v);
              });
      } else if constexpr (ACT == kSilu) {
        const int nw = n0 + wn * SN * 16;  // the wave's first column of out
        if (g.gu != nullptr) {
          constexpr int Q = part_of(2 * SN, ROW / 16);
#pragma unroll
          for (int up = 0; up < 2; up++)
#pragma unroll
            for (int q0 = 0; q0 < 2 * SN; q0 += Q)
              turn_over<Q, false, ROW, ROWS>(
                  mine, [&](int q, int r) { return sum(2 * (q0 + q) + up, r); },
                  [&](int u, int byte, const uint8_t* v) {
                    const int n = nw + q0 * 8 + byte / 2;
                    put(reinterpret_cast<uint8_t*>(g.gu + up * cols + n), g.N * 2, u, n, v);
                  });
        }
        constexpr int Q = part_of(2 * SN, NQ);
#pragma unroll
        for (int q0 = 0; q0 < 2 * SN; q0 += Q)
          turn_over<Q, F32, ROW, ROWS>(
              mine,
              [&](int q, int r) {
                return silu_mul(sum(2 * (q0 + q), r), sum(2 * (q0 + q) + 1, r));
              },
              [&](int u, int byte, const uint8_t* v) {
                const int n = nw + q0 * 8 + byte / EB;
                put(out + (size_t)n * EB, cols * EB, u, n, v);
              });
      } else {
#pragma unroll
        for (int q0 = 0; q0 < 4 * SN; q0 += NQ)
          turn_over<NQ, true, ROW, ROWS>(
              mine, [&](int q, int r) { return sum(q0 + q, r); },
              [&](int u, int byte, const uint8_t* v) {
                const int n = n0 + wn * SN * 32 + q0 * 8 + byte / 4, p = row[u];
                if (p < 0 || n >= cols) return;
                const f32x4 d = *reinterpret_cast<const f32x4*>(v);
                const size_t o2 = (size_t)p * 2 * cols + n;
                const u32x2 gt = *reinterpret_cast<const u32x2*>(g.gu + o2);
                const u32x2 up = *reinterpret_cast<const u32x2*>(g.gu + o2 + cols);
                float dg[4], du[4];
#pragma unroll
                for (int r = 0; r < 4; r++)
                  silu_mul_grad(d[r], bf16_f32((uint16_t)(gt[r / 2] >> (16 * (r & 1)))),
                                bf16_f32((uint16_t)(up[r / 2] >> (16 * (r & 1)))), &dg[r], &du[r]);
                store4_past<F32>(g.out, o2, dg);
                store4_past<F32>(g.out, o2 + cols, du);
              });
      }
    }
  };

  // The first tile's pairs, and its first K block.
  at = find(id);
  {
    const int p = my_pair(at);
    if (threadIdx.x < C::BM) pairs[threadIdx.x] = p;
  }
  __syncthreads();
  set_rows(pairs);
  uint8_t *st = lds, *nx = lds + C::STAGE;
#pragma unroll
  for (int u = 0; u < C::COPIES; u++) copy(st, 0, u);
  // Block 0 has landed, in every wave, and the stage of the block before it is free:
  // block 1 is copied there.
  auto second = [&] {
    wait_memory<0>();
    block_barrier();
    if (KB > 1) {
#pragma unroll
      for (int u = 0; u < C::COPIES; u++) copy(nx, 1, u);
    }
  };
  second();
  for (;;) {
    const bool more = KB > 1 && id + stride < last;  // (one block has no second one for it)
    const Where next = more ? find(id + stride) : at;
    const int p = more ? my_pair(next) : -1, n0 = at.n0;
    // The wave's sub-tiles of rows are wm, wm + WM, ...; those behind the last one
    // with a row (an expert's rows stand in front of its padding) are left out.
    int live = 0;
#pragma unroll
    for (int s = 0; s < SM; s++)
      if (__ballot(pairs[(s * C::WM + wm) * 32 + r32] >= 0) != 0) live = s + 1;
    live = __builtin_amdgcn_readfirstlane(live);
    auto run = [&](auto live_) {
      constexpr int LIVE = decltype(live_)::value;  // sub-tile rows to compute
      f32x16 acc[SN][SM];
#pragma unroll
      for (int i = 0; i < SN; i++)
#pragma unroll
        for (int s = 0; s < SM; s++)
#pragma unroll
          for (int r = 0; r < 16; r++) acc[i][s][r] = 0.f;
      bf16x8 bf[2][SN], af[2][LIVE];
      auto read = [&](const uint8_t* t, int s, int r) {
        if (r >= SN)
          af[s & 1][r - SN] = straight(t, (r - SN) * C::WM + wm, s);
        else if constexpr (TRANS)
          bf[s & 1][r] = Turned<C::BN>::frag(t + C::B_AT, offb[r], s);
        else
          bf[s & 1][r] = straight(t + C::B_AT, wn * SN + r, s);
      };
      auto mul = [&](int s, int m) {
        const int j = m / SN, i = m % SN;
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf[s & 1][i], af[s & 1][j], acc[i][j],
                                                            0, 0, 0);
      };
      constexpr int NR = SN + LIVE, NM = SN * LIVE;
      k_block<C, NR, NM, true>(st, nx, [](uint8_t*, int) {}, read, mul);
      int from = 1;
      for (int kb = 1; kb < KB; kb++) {
        wait_memory<0>();
        block_barrier();
        uint8_t* const t = nx;
        nx = st;
        st = t;
        if (kb == 1 && more && threadIdx.x < C::BM) next_pairs[threadIdx.x] = p;
        from = kb + 1;
        if (from == KB && more) {  // the next tile's first block
          if (KB == 2) __syncthreads();
          at = next;
          set_rows(next_pairs);
          from = 0;
        }
        k_block<C, NR, NM, false>(
            st, nx, [&](uint8_t* to, int c) { copy(to, from, c); }, read, mul);
      }
#pragma unroll
      for (int m = 0; m < NM; m++) mul(3, m);
      uint8_t* const t = nx;
      nx = st;
      st = t;
      if (more) second();
      write_out(acc, live, n0);
    };
    switch (live) {  // (the same number of barriers in every one)
      case 0:
      case 1: run(Int<1>{}); break;
      case 2: run(Int<SM < 2 ? SM : 2>{}); break;
      case 3: run(Int<SM < 3 ? SM : 3>{}); break;
      default: run(Int<SM < 4 ? SM : 4>{}); break;
    }
    if (!more) break;
    int32_t* const t = pairs;
    pairs = next_pairs;
    next_pairs = t;
    id += stride;
  }
}

// Row tiles of the lane's experts, and what the rounds of `tiles` of them cost.
template <class C>
__device__ inline int lanes_tiles(const List& list) {
  int n = 0;
  for (int e = threadIdx.x & 63; e < list.E; e += 64)
    n += (list.expert_offsets[e + 1] - list.expert_offsets[e] + C::BM - 1) / C::BM;
  return n;
}
template <class C>
__device__ inline long long cost(const GroupedArgs& g, int tiles) {
  const int per_xcd = (tiles * columns<C>(g.N) + 7) / 8, slots = max(g.slots / 8, 1);
  return (long long)((per_xcd + slots - 1) / slots) * C::ROUND;
}

template <bool TRANS, int ACT, bool F32, class C, class... MORE>
__global__ __launch_bounds__(C::THREADS, C::EU) void grouped_tile_kernel(GroupedArgs g) {
  constexpr int sizes[] = {Room<C, ACT, F32>::BYTES, Room<MORE, ACT, F32>::BYTES...};
  constexpr int BYTES = largest(sizes);
  __shared__ __align__(1024) uint8_t lds[BYTES];
  __shared__ int32_t offsets[kOffsets];
  for (int e = threadIdx.x; e <= g.E; e += C::THREADS) offsets[e] = g.expert_offsets[e];
  __syncthreads();
  const List list = {offsets, g.E};
  if constexpr (sizeof...(MORE) == 0) {
    grouped_tiles<C, TRANS, ACT, F32>(g, list, lds);
  } else {
    static_assert(((MORE::THREADS == C::THREADS && MORE::EU == C::EU) && ...), "one launch");
    int tiles[] = {lanes_tiles<C>(list), lanes_tiles<MORE>(list)...};
#pragma unroll
    for (int off = 1; off < 64; off <<= 1)
#pragma unroll
      for (int& n : tiles) n += __shfl_xor(n, off, 64);
#pragma unroll
    for (int& n : tiles) n = __builtin_amdgcn_readfirstlane(n);
    int i = 0, best = 0;
    long long least = cost<C>(g, tiles[0]);
    auto look = [&](long long c) {
      i++;
      if (c < least) least = c, best = i;
    };
    (look(cost<MORE>(g, tiles[i + 1])), ...);
    if (best == 0) return grouped_tiles<C, TRANS, ACT, F32>(g, list, lds);
    i = 0;
    ((best == ++i ? grouped_tiles<MORE, TRANS, ACT, F32>(g, list, lds) : void()), ...);
  }
}

// dw of every expert: BM rows (of dw: columns of dy) x BN columns (of x), both
// operands turned, K the expert's pairs.  A tile of an expert without pairs is
// zeros.  Bound: dw's bytes where the experts have few rows (128 experts of 1536 x
// 2048 in fp32, kernel durations: the stores alone 254-261 us, all of it 251-280; through
// the L2 an earlier form of 256 x 256 tiles took 455 instead of 375).  Of 8 experts of 2048
// x 1536 with 1028 rows the waves wait for half of their cycles, for K blocks of 32 rows
// that are copied one ahead: the matrix cores are busy 38% and LDS 24% of the time.
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
  constexpr int KROWS = 16 * C::STEPS;  // pairs per K block
  const int KB = (end - first + KROWS - 1) / KROWS;
  const size_t dbytes = (size_t)g.P * g.N * 2, xbytes = (size_t)g.Mx * g.K * 2;
  // The copies' rows are pairs of the list, looked up one K block before they
  // are copied.
  int pa[C::AC], pb[C::BC];
  unsigned va[C::AC], vb[C::BC];
  auto look = [&](int kb) {
#pragma unroll
    for (int i = 0; i < C::AC; i++) {
      const int slot = first + kb * KROWS + Ta::row(wave * C::AC + i, lane);
      pa[i] = slot < end ? g.sorted[slot] : g.P;
    }
#pragma unroll
    for (int i = 0; i < C::BC; i++) {
      const int slot = first + kb * KROWS + Tb::row(wave * C::BC + i, lane);
      pb[i] = slot < end ? g.sorted[slot] : g.P;
    }
  };
  // (Called for K blocks in order, copy 0 first; the look-up of the next block's
  // rows is under way before the copies.)
  look(0);
  auto copy = [&](uint8_t* st, int kb, int c) {
    if (c == 0) {
#pragma unroll
      for (int i = 0; i < C::AC; i++) {
        const int col = n0 + Ta::col(wave * C::AC + i, lane);
        va[i] = (unsigned)pa[i] < (unsigned)g.P && col < g.N
                    ? 2u * ((unsigned)pa[i] * (unsigned)g.N + (unsigned)col)
                    : kNowhere;
      }
#pragma unroll
      for (int i = 0; i < C::BC; i++) {
        const int col = k0 + Tb::col(wave * C::BC + i, lane);
        const int row = g.pair_rows ? pb[i] : pb[i] / g.k;
        vb[i] = (unsigned)pb[i] < (unsigned)g.P && col < g.K
                    ? 2u * ((unsigned)row * (unsigned)g.K + (unsigned)col)
                    : kNowhere;
      }
      look(kb + 1);
    }
    if (c < C::AC)
      copy16(rsrc(g.dy, dbytes), va[c], 0, st + (wave * C::AC + c) * 1024);
    else
      copy16(rsrc(g.x, xbytes), vb[c - C::AC], 0,
             st + C::B_AT + (wave * C::BC + c - C::AC) * 1024);
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
  bf16x8 bf[2][SN], af[2][SM];
  k_loop<C, SN + SM, SN * SM>(
      lds, KB, copy,
      [&](const uint8_t* st, int s, int r) {
        if (r < SN)
          bf[s & 1][r] = Tb::frag(st + C::B_AT, offb[r], s);
        else
          af[s & 1][r - SN] = Ta::frag(st, offa[r - SN], s);
      },
      [&](int s, int m) {
        const int j = m / SN, i = m % SN;
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf[s & 1][i], af[s & 1][j], acc[i][j],
                                                            0, 0, 0);
      });
  constexpr int EB = F32 ? 4 : 2, ROW = SN * 32 * EB, RPI = 64 / (ROW / 16);
  static_assert(C::WAVES * 32 * ROW <= (int)sizeof(lds), "every wave has room for 32 rows");
  __syncthreads();  // the last K block has been read
  uint8_t* const mine = lds + wave * 32 * ROW;
  uint8_t* const out = reinterpret_cast<uint8_t*>(g.out) + (size_t)e * g.N * g.K * EB;
#pragma unroll
  for (int s = 0; s < SM; s++)
    turn_over<4 * SN, F32, ROW, 32>(
        mine, [&](int q, int r) { return acc[q / 4][s][4 * (q % 4) + r]; },
        [&](int u, int byte, const uint8_t* v) {
          const int n = n0 + (s * C::WM + wm) * 32 + u * RPI + lane / (ROW / 16);
          const int k = k0 + wn * SN * 32 + byte / EB;
          if (n >= g.N || k >= g.K) return;
          u32x4* o = reinterpret_cast<u32x4*>(out + ((size_t)n * g.K + k) * EB);
          u32x4 w = *reinterpret_cast<const u32x4*>(v);
          if (g.accumulate) {  // (fp32 only)
            const u32x4 was = *o;
#pragma unroll
            for (int r = 0; r < 4; r++)
              w[r] = __float_as_uint(__uint_as_float(was[r]) + __uint_as_float(w[r]));
          }
          // (past the L2, which holds the rows that the next tiles read)
          __builtin_nontemporal_store(w, o);
        });
}

// ROUND: the cost of a round over the chip (one tile per CU), of 320 for Wide's.
struct Big : Tile<256, 256, 2, 4, 2> {
  static constexpr int ROUND = 384;
};
struct Broad : Tile<192, 384, 2, 4, 2> {
  static constexpr int ROUND = 490;
};
struct Wide : Tile<192, 256, 2, 4, 2> {
  static constexpr int ROUND = 320;
};
struct Mid : Tile<128, 256, 2, 4, 2> {
  static constexpr int ROUND = 250;
};
typedef Tile<64, 128, 2, 2, 2> Half;
typedef Tile<32, 128, 1, 2, 2> Low;

constexpr int kBlocks = 1 << 21;  // of a launch

// At most one row tile per BM rows and one more per expert.
template <class C>
long long most_tiles(const GroupedArgs& g) {
  return columns<C>(g.N) * (long long)(g.M / C::BM + (g.E < g.P ? g.E : g.P));
}

template <bool TRANS, int ACT, bool F32, class C, class... MORE>
hipError_t launch_tile(GroupedArgs g, hipStream_t s) {
  long long total = most_tiles<C>(g);
  ((total = most_tiles<MORE>(g) > total ? most_tiles<MORE>(g) : total), ...);
  if (total > (1ll << 30)) return hipErrorInvalidValue;
  // As many blocks as run at once, each with every so-many'th tile of its XCD (a K
  // of one block has no second one to look the next tile up under: a block each).
  g.slots = device_cu_count() * C::PER_CU;
  const long long grid = g.K > 64 && total > g.slots ? g.slots : total;
  // A grid holds fewer than 2^32 threads.
  for (long long at = 0; at < grid; at += kBlocks) {
    const long long n = grid - at < kBlocks ? grid - at : kBlocks;
    g.first = (int)(at / 8);
    hipLaunchKernelGGL((grouped_tile_kernel<TRANS, ACT, F32, C, MORE...>),
                       dim3((unsigned)((n + 7) / 8 * 8)), dim3(C::THREADS), 0, s, g);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
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

// The tile.  By the mean rows per expert, one that holds most experts' rows at once, so
// that a matrix is read once, in us (128 experts, top-8; the row gradient's tiles with
// SiLU * mul's gradient; "up" 1536 x 2048, "down" 2048 x 768):
//   tokens (mean)     Low    Half   Mid    Wide   Big
//   up    256 (16)    169    172    173    174    178
//         512 (32)    212    171    174    177    176
//         1024 (64)   240    223    184    182    186
//         2048 (128)  359    307    272    209    204
//         4000 (250)  626    481    375    340    308
//   down  256 (16)     84     83     92     94     96
//         1024 (64)   120    105     98    100    105
//         2048 (128)  184    148    133    115    123
//   back  256 (16)     84     94    111    114    122
//         1024 (64)   141    137    128    131    144
//         4000 (250)  349    291    265    252    302
// Where the four widest leave half of the CUs without a tile, Half (8 experts of 1536 x
// 2048, top-2, 1024 tokens: 32 against 39, 42 and 53 us); among them the kernel takes the
// one whose rounds over the chip cost least.  Rounds and us, Mid / Wide / Big / Broad:
//   back, 768 columns   1024 (64)   2 123  2 127  2 140  1 100
//                       2048 (128)  3 194  2 151  2 183  1 127
//                       the same, uneven (some experts above 192 rows)
//                                   3 192  2 160         2 208
//                       3000 (188)  3 198  3 227  2 234  2 223
//   up                  2048 (128)  5 269  3 203  3 197  2 201
//   down                2500 (156)  8 162  4 119  4 135  3 150
//   32 experts, 1536 x 2048, top-4, 2500 (312)  3 94  2 79  2 92  1 70
// Projections of few rows per expert go to the rows kernel ("up": 16 tokens (mean 1) 96
// us, 128 (8) 168; Low 140 and 172).
template <bool TRANS, int ACT, bool F32>
hipError_t launch(const GroupedArgs& g, hipStream_t s) {
  const double mean = (double)g.P / g.E;
  if constexpr (!TRANS) {
    if (mean <= 8) return launch_rows<ACT, F32>(g, s);
  }
  if (mean <= 20) return launch_tile<TRANS, ACT, F32, Low>(g, s);
  const double of_one = g.E == 1 ? ceil(mean / Mid::BM) : fmax(mean / Mid::BM + 0.5, 1.0);
  const double mids = of_one * g.E * columns<Mid>(g.N);  // expected
  if (mean <= 44 || mids < device_cu_count() / 2) return launch_tile<TRANS, ACT, F32, Half>(g, s);
  return launch_tile<TRANS, ACT, F32, Big, Broad, Wide, Mid>(g, s);
}

// Weight gradients.  Short: three blocks on a CU, one storing while others add; Long:
// the most values of K per byte copied.
typedef Tile<128, 128, 2, 2, 2, 3, 2, 2> Short;
typedef Tile<256, 256, 4, 4, 2, 4, 2> Long;

template <class C>
long long wgrad_tiles(const WgradArgs& g) {
  return (long long)((g.K + C::BN - 1) / C::BN) * ((g.N + C::BM - 1) / C::BM) * g.E;
}
template <class C>
hipError_t launch_wgrad(const WgradArgs& all, hipStream_t s) {
  // As many experts per launch as a grid holds (one always: its matrix would not fit the
  // memory).
  const long long each = wgrad_tiles<C>(all) / all.E;
  if (each * C::THREADS > 0x7fffffffll * 2) return hipErrorInvalidValue;
  const int most = each < kBlocks ? (int)(kBlocks / each) : 1;
  const size_t bytes = (size_t)all.N * all.K * (all.out_f32 ? 4 : 2);
  for (int e0 = 0; e0 < all.E; e0 += most) {
    WgradArgs g = all;
    g.E = all.E - e0 < most ? all.E - e0 : most;
    g.expert_offsets += e0;
    g.out = reinterpret_cast<uint8_t*>(g.out) + e0 * bytes;
    const dim3 grid((unsigned)((each * g.E + 7) / 8 * 8));
    if (g.out_f32)
      hipLaunchKernelGGL((grouped_wgrad_kernel<C, true>), grid, dim3(C::THREADS), 0, s, g);
    else
      hipLaunchKernelGGL((grouped_wgrad_kernel<C, false>), grid, dim3(C::THREADS), 0, s, g);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_grouped_matmul(const GroupedArgs& g, hipStream_t s) {
  const int which = g.act == QMOE_ACT_SILU_MUL ? 2 : g.act == QMOE_ACT_SILU_MUL_BACKWARD ? 3
                    : g.trans                  ? 1
                                               : 0;
  switch (which) {
    case 0:
      return g.out_f32 ? launch<false, kPlain, true>(g, s) : launch<false, kPlain, false>(g, s);
    case 1: return g.out_f32 ? launch<true, kPlain, true>(g, s) : launch<true, kPlain, false>(g, s);
    case 2: return g.out_f32 ? launch<false, kSilu, true>(g, s) : launch<false, kSilu, false>(g, s);
    default:
      return g.out_f32 ? launch<true, kSiluGrad, true>(g, s) : launch<true, kSiluGrad, false>(g, s);
  }
}

hipError_t launch_grouped_wgrad(const WgradArgs& g, hipStream_t s) {
  // Long where the experts have many rows and its rounds over the chip, each 1.12 of
  // Short's, are the fewer (us, Short / Long: 128 experts of 1536 x 2048 in fp32, 128
  // rows each 296 / 341, 250 rows 404 / 415; 8 experts, 1028 rows, 2048 x 1536 63 / 67;
  // 1024 rows, 4096 x 4096 356 / 308; one, 4096 rows 163 / 134).
  const double cus = device_cu_count(), shorts = wgrad_tiles<Short>(g) / (3 * cus);
  if ((double)g.P / g.E > 320 && 1.12 * ceil(wgrad_tiles<Long>(g) / cus) < shorts)
    return launch_wgrad<Long>(g, s);
  return launch_wgrad<Short>(g, s);
}

}  // namespace qmoe
