// RMS norms before and after a block, with the block's gate and the residual
// scale, and their gradients.
//
//   before:  n = x * r * w,  r = 1 / sqrt(mean(x^2) + eps), stored as bf16,
//            fp32, or quantized: int8 or e4m3 with one fp32 scale per token
//            (what the grouped FFN takes), e4m3 with one per 128 columns
//   after:   out = alpha * x + g * (y * r * w), g a gate per column, per
//            token, per value, or 1; optionally also n = norm(out) * w2 of the
//            stored out, the next block's input
//   gradients, with h = v * r of the normed v (x before, y after):
//            before: dx = dres + r * (dh - h * mean(dh * h)), dh = dn * w,
//                    dw = sum_t dn * h
//            after:  du = dout * g, dh = du * w, dy as dx above without dres,
//                    dres = alpha * dout, dw = sum_t du * h,
//                    dg = dout * h * w summed over the axes g is broadcast on
//
// The bound is HBM: a row is read once into registers (TPR threads per row,
// NV groups of eight values per thread), reduced, and written once.  The
// gradients need two sums of the row, sum(v^2) and sum(dh * v), which one
// reduction takes together (sum(dh * h) = r * sum(dh * v)), so nothing of
// the forward pass is kept.  The column sums dw and dg run over the rows of a
// block in registers, then over the blocks in a second launch, in a fixed
// order: the same bits on every run.
//
// In bf16: after with the next block's codes at 4096 x 4096 28 us (4.2 TB/s),
// its gradients with a gate per value at 4111 x 2048 25 + 4 us (4.0 TB/s in the
// first launch); before at one row of 4096 3.0 us, which is latency.
#include "block_common.h"
#include "grid_common.h"

namespace qmoe {

int norm_max_columns() { return 16384; }
int norm_max_scalar_columns() { return 8192; }
bool norm_vec_ok(int H, std::initializer_list<const void*> ps) {
  if (H % 8 != 0) return false;
  for (const void* p : ps)
    if ((uintptr_t)p % 16 != 0) return false;
  return true;
}

namespace {
using namespace bk;

// Threads per row, vectors of eight per thread, and whether a thread's eight
// values are consecutive (16-byte loads) or TPR apart (any H and alignment).
template <int TPR_, int NV_, bool VEC_>
struct Shape {
  static constexpr int TPR = TPR_, NV = NV_;
  static constexpr bool VEC = VEC_;
  static constexpr int BLOCK = TPR < 256 ? 256 : TPR;
  static constexpr int RPB = BLOCK / TPR;  // rows per block
  static constexpr int WAVES = TPR / 64;   // waves per row
};

template <class S>
__device__ inline int col(int v, int j, int tr) {
  return S::VEC ? (v * S::TPR + tr) * 8 + j : (v * 8 + j) * S::TPR + tr;
}

template <class S, bool F32>
__device__ inline void load_row(const void* p, size_t row, int H, int tr, float x[S::NV][8]) {
#pragma unroll
  for (int v = 0; v < S::NV; v++) {
    if constexpr (S::VEC) {
      if (col<S>(v, 0, tr) < H) {
        load8<F32>(p, row * H + col<S>(v, 0, tr), x[v]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++) x[v][j] = 0.f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++)
        x[v][j] = col<S>(v, j, tr) < H ? load1<F32>(p, row * H + col<S>(v, j, tr)) : 0.f;
    }
  }
}

template <class S, bool F32>
__device__ inline void store_row(void* p, size_t row, int H, int tr, const float x[S::NV][8]) {
#pragma unroll
  for (int v = 0; v < S::NV; v++) {
    if constexpr (S::VEC) {
      if (col<S>(v, 0, tr) < H) store8<F32>(p, row * H + col<S>(v, 0, tr), x[v]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++)
        if (col<S>(v, j, tr) < H) store1<F32>(p, row * H + col<S>(v, j, tr), x[v][j]);
    }
  }
}

// Sums over the threads of a row; `red` holds BLOCK / 64 x 2 floats.  Every
// thread of the block calls it.
template <class S>
__device__ inline void row_sum2(float& a, float& b, float* red) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (S::WAVES > 1) {
    const int w = threadIdx.x >> 6;
    __syncthreads();  // the last use of `red`
    if ((threadIdx.x & 63) == 0) {
      red[2 * w] = a;
      red[2 * w + 1] = b;
    }
    __syncthreads();
    a = red[0];
    b = red[1];
#pragma unroll
    for (int i = 1; i < S::WAVES; i++) {
      a += red[2 * i];
      b += red[2 * i + 1];
    }
  }
}
template <class S>
__device__ inline float row_sum(float a, float* red) {
  float b = 0.f;
  row_sum2<S>(a, b, red);
  return a;
}
template <class S>
__device__ inline uint32_t row_max(uint32_t a, float* red) {
  a = wave_max(a);
  if constexpr (S::WAVES > 1) {
    const int w = threadIdx.x >> 6;
    uint32_t* r = reinterpret_cast<uint32_t*>(red);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) r[w] = a;
    __syncthreads();
    a = r[0];
#pragma unroll
    for (int i = 1; i < S::WAVES; i++) a = max(a, r[i]);
  }
  return a;
}

template <class S>
__device__ inline float sum_sq(const float x[S::NV][8]) {
  float s = 0.f;
#pragma unroll
  for (int v = 0; v < S::NV; v++)
#pragma unroll
    for (int j = 0; j < 8; j++) s = __builtin_fmaf(x[v][j], x[v][j], s);
  return s;
}

__device__ inline float rms_inv(float sumsq, int H, float eps) {
  return 1.0f / sqrtf(sumsq / (float)H + eps);
}

// Rows of the gradients whose sum of squares is near the end of fp32's range are
// taken times kShrink instead: h is the same, and the norm's gradient is kShrink
// times that of the smaller row.
constexpr float kLarge = 0x1p120f, kShrink = 0x1p-72f;
// (The row's gradient d is hidden from the compiler, so that it keeps no product
// of it in registers for this rare second pass.)
template <class S>
__device__ inline void shrink(float v[S::NV][8], float d[S::NV][8]) {
#pragma unroll
  for (int i = 0; i < S::NV; i++)
#pragma unroll
    for (int j = 0; j < 8; j++) {
      v[i][j] *= kShrink;
      asm("" : "+v"(d[i][j]));
    }
}

// The forward norms' r in fp64, from a sum of squares in fp64: it does not
// depend on how a row is spread over threads, and rows whose squares are beyond
// fp32 keep it.
template <class S>
__device__ inline double row_rms_inv(const float x[S::NV][8], int H, float eps, double* red) {
  double s = 0.0;
#pragma unroll
  for (int v = 0; v < S::NV; v++)
#pragma unroll
    for (int j = 0; j < 8; j++) s += (double)x[v][j] * (double)x[v][j];
  s = wave_sum64(s);
  if constexpr (S::WAVES > 1) {
    const int w = threadIdx.x >> 6;
    __syncthreads();  // the last use of `red`
    if ((threadIdx.x & 63) == 0) red[w] = s;
    __syncthreads();
    s = red[0];
#pragma unroll
    for (int i = 1; i < S::WAVES; i++) s += red[i];
  }
  return rsqrt(s / H + (double)eps);
}

// v in fp64, converted here: a conversion that the compiler shared with the sum
// of squares would stay in registers in between.
__device__ inline double wide_here(float v) {
  asm("" : "+v"(v));
  return (double)v;
}

// Writes a row of normed values in the form asked for.  `grp` (LDS, 128
// words) serves the column groups of rows that are not taken by vectors.
template <class S>
__device__ inline void write_form(const NormForm& f, size_t row, bool live, int T, int H, int tr,
                                  const float n[S::NV][8], float* red, uint32_t* grp) {
  if (f.form == QMOE_FORM_BF16 || f.form == QMOE_FORM_F32) {
    if (!live) return;
    if (f.form == QMOE_FORM_BF16)
      store_row<S, false>(f.n, row, H, tr, n);
    else
      store_row<S, true>(f.n, row, H, tr, n);
    return;
  }
  uint8_t* out = reinterpret_cast<uint8_t*>(f.n);
  const float qmax = f.form == QMOE_FORM_INT8 ? 127.0f : 448.0f;
  if (f.form != QMOE_FORM_E4M3_B128) {
    uint32_t a = 0;
#pragma unroll
    for (int v = 0; v < S::NV; v++)
#pragma unroll
      for (int j = 0; j < 8; j++) a = max(a, abs_bits(n[v][j]));
    const Quant q(row_max<S>(a, red), qmax);
    if (!live) return;
    if (tr == 0) f.scale[row] = q.s;
#pragma unroll
    for (int v = 0; v < S::NV; v++) {
      u32x2 c;
      if (f.form == QMOE_FORM_INT8)
        c = u32x2{q.i8x4(n[v][0], n[v][1], n[v][2], n[v][3]),
                  q.i8x4(n[v][4], n[v][5], n[v][6], n[v][7])};
      else
        c = u32x2{q.e4m3x4(n[v][0], n[v][1], n[v][2], n[v][3]),
                  q.e4m3x4(n[v][4], n[v][5], n[v][6], n[v][7])};
      if constexpr (S::VEC) {
        if (col<S>(v, 0, tr) < H)
          *reinterpret_cast<u32x2*>(out + row * H + col<S>(v, 0, tr)) = c;
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++)
          if (col<S>(v, j, tr) < H)
            out[row * H + col<S>(v, j, tr)] = (uint8_t)(c[j >> 2] >> (8 * (j & 3)));
      }
    }
    return;
  }
  // One scale per 128 columns, rows padded with zeros to a multiple of 128.
  const int HB = (H + 127) / 128;
  const size_t pitch = (size_t)HB * 128;
  if constexpr (S::VEC) {
#pragma unroll
    for (int v = 0; v < S::NV; v++) {  // 16 lanes hold one group
      uint32_t a = 0;
#pragma unroll
      for (int j = 0; j < 8; j++) a = max(a, abs_bits(n[v][j]));
      const Quant q(row16_max(a), qmax);
      const int c0 = col<S>(v, 0, tr);
      if (live && c0 < HB * 128) {
        *reinterpret_cast<u32x2*>(out + row * pitch + c0) =
            u32x2{q.e4m3x4(n[v][0], n[v][1], n[v][2], n[v][3]),
                  q.e4m3x4(n[v][4], n[v][5], n[v][6], n[v][7])};
        if ((tr & 15) == 0) f.scale[(size_t)(c0 / 128) * T + row] = q.s;
      }
    }
  } else {  // one row per block
    __syncthreads();
    for (int i = tr; i < 128; i += S::TPR) grp[i] = 0;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < S::NV; v++)
#pragma unroll
      for (int j = 0; j < 8; j++)
        if (col<S>(v, j, tr) < H) atomicMax(&grp[col<S>(v, j, tr) / 128], abs_bits(n[v][j]));
    __syncthreads();
    if (!live) return;
#pragma unroll
    for (int v = 0; v < S::NV; v++)
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const int c = col<S>(v, j, tr);
        if (c < HB * 128) {
          const Quant q(grp[c / 128], qmax);
          out[row * pitch + c] = (uint8_t)q.e4m3x4(n[v][j], 0.f, 0.f, 0.f);
          if (c % 128 == 0) f.scale[(size_t)(c / 128) * T + row] = q.s;
        }
      }
  }
}

template <class S>
struct Lds {
  union {
    float red[2 * (S::BLOCK / 64)];
    double red64[S::BLOCK / 64];
  };
  uint32_t grp[128];
};

template <class S, bool F32>
__global__ __launch_bounds__(S::BLOCK) void pre_norm_kernel(const void* __restrict__ x,
                                                            const float* __restrict__ w, float eps,
                                                            int T, int H, NormForm f) {
  __shared__ Lds<S> lds;
  const int tr = threadIdx.x % S::TPR;
  const size_t row = block_of_grid() * S::RPB + threadIdx.x / S::TPR;
  const bool live = row < (size_t)T;
  float v[S::NV][8], wt[S::NV][8];
  load_row<S, F32>(x, live ? row : (size_t)T - 1, H, tr, v);
  load_row<S, true>(w, 0, H, tr, wt);
  const float r = (float)row_rms_inv<S>(v, H, eps, lds.red64);
#pragma unroll
  for (int i = 0; i < S::NV; i++)
#pragma unroll
    for (int j = 0; j < 8; j++) v[i][j] = v[i][j] * r * wt[i][j];
  write_form<S>(f, row, live, T, H, tr, v, lds.red, lds.grp);
}

// The gate's values of a row: G is QMOE_GATE_COLUMN or QMOE_GATE_FULL, or
// QMOE_GATE_TOKEN for one value per row (1 where there is no gate).
template <class S, bool F32, int G>
__device__ inline void load_gate(const void* gate, size_t row, int H, int tr,
                                 float g[S::NV][8]) {
  if constexpr (G == QMOE_GATE_COLUMN) {
    load_row<S, true>(gate, 0, H, tr, g);
  } else if constexpr (G == QMOE_GATE_FULL) {
    load_row<S, F32>(gate, row, H, tr, g);
  } else {
    const float s = gate ? reinterpret_cast<const float*>(gate)[row] : 1.0f;
#pragma unroll
    for (int v = 0; v < S::NV; v++)
#pragma unroll
      for (int j = 0; j < 8; j++) g[v][j] = s;
  }
}

// `out` may be `x`: a value is read before the same thread writes it.
// The next norm reads a bf16 out as stored, so a value that fp32 steps had left
// on the other side of a bf16 border (3 of 10^5) would put a whole bf16 step
// into an fp32 n or scale.  A sum that lies nearer to a border than the steps
// may be off (five half steps of its terms, with the one that the exact sum is
// off in fp32 less than 2^-21 of them: about one sum of 2000) is therefore formed
// again in fp64 and rounded to fp32 once; that is what bf16 rounds.  With that
// check 4096 x 4096 with the next norm takes 32.2 us, without it 29.6.
template <class S, bool F32, int G>
__global__ __launch_bounds__(S::BLOCK) void post_norm_kernel(
    const void* __restrict__ y, const void* x, const float* __restrict__ w,
    const void* __restrict__ gate, float alpha, float eps, int T, int H, void* out,
    const float* __restrict__ w2, NormForm f) {
  __shared__ Lds<S> lds;
  const int tr = threadIdx.x % S::TPR;
  const size_t row = block_of_grid() * S::RPB + threadIdx.x / S::TPR;
  const bool live = row < (size_t)T;
  const size_t rd = live ? row : (size_t)T - 1;
  float v[S::NV][8], g[S::NV][8], t[S::NV][8], res[S::NV][8];
  load_row<S, F32>(y, rd, H, tr, v);
  load_row<S, F32>(x, rd, H, tr, res);
  load_gate<S, F32, G>(gate, rd, H, tr, g);
  load_row<S, true>(w, 0, H, tr, t);
  const double r = row_rms_inv<S>(v, H, eps, lds.red64);
#pragma unroll
  for (int i = 0; i < S::NV; i++)
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const float p = alpha * res[i][j], q = g[i][j] * (v[i][j] * (float)r * t[i][j]);
      float o = p + q;
      if constexpr (!F32) {  // as stored
        const float tie = __uint_as_float((__float_as_uint(o) & 0xffff0000u) | 0x8000u);
        const float err = __builtin_fmaf(0x1p-21f, fabsf(p) + fabsf(q), 0x1p-140f);
        if (!(fabsf(o - tie) > err))
          o = (float)fma((double)alpha, (double)res[i][j],
                         wide_here(v[i][j]) * t[i][j] * r * g[i][j]);
        o = bf16_f32(f32_bf16(o));
      }
      v[i][j] = o;
    }
  if (live) store_row<S, F32>(out, row, H, tr, v);
  if (w2 == nullptr) return;
  load_row<S, true>(w2, 0, H, tr, t);
  const float r2 = (float)row_rms_inv<S>(v, H, eps, lds.red64);
#pragma unroll
  for (int i = 0; i < S::NV; i++)
#pragma unroll
    for (int j = 0; j < 8; j++) v[i][j] = v[i][j] * r2 * t[i][j];
  write_form<S>(f, row, live, T, H, tr, v, lds.red, lds.grp);
}

// Adds the RPB rows' column sums of a block and writes part[block][H].
template <class S>
__device__ inline void write_partial(float* part, int H, int tr, float a[S::NV][8], float* buf) {
  if constexpr (S::RPB > 1) {
    const int slot = threadIdx.x / S::TPR;
    __syncthreads();
#pragma unroll
    for (int s = S::RPB - 1; s >= 1; s--) {
      if (slot == s) {
#pragma unroll
        for (int v = 0; v < S::NV; v++)
#pragma unroll
          for (int j = 0; j < 8; j++) buf[(v * 8 + j) * S::TPR + tr] = a[v][j];
      }
      __syncthreads();
      if (slot == 0) {
#pragma unroll
        for (int v = 0; v < S::NV; v++)
#pragma unroll
          for (int j = 0; j < 8; j++) a[v][j] += buf[(v * 8 + j) * S::TPR + tr];
      }
      __syncthreads();
    }
    if (slot != 0) return;
  }
  store_row<S, true>(part, blockIdx.x, H, tr, a);
}

// `dx` may be `dres`.
template <class S, bool F32>
__global__ __launch_bounds__(S::BLOCK) void pre_norm_backward_kernel(
    const void* __restrict__ dn, const void* __restrict__ x, const float* __restrict__ w,
    const void* dres, float eps, int T, int H, void* dx, float* __restrict__ part) {
  __shared__ Lds<S> lds;
  __shared__ float buf[S::RPB > 1 ? S::TPR * S::NV * 8 : 1];
  const int tr = threadIdx.x % S::TPR;
  float wt[S::NV][8], dw[S::NV][8];
  load_row<S, true>(w, 0, H, tr, wt);
#pragma unroll
  for (int i = 0; i < S::NV; i++)
#pragma unroll
    for (int j = 0; j < 8; j++) dw[i][j] = 0.f;
  for (size_t r0 = (size_t)blockIdx.x * S::RPB; r0 < (size_t)T;
       r0 += (size_t)gridDim.x * S::RPB) {
    const size_t row = r0 + threadIdx.x / S::TPR;
    const bool live = row < (size_t)T;
    const size_t rd = live ? row : (size_t)T - 1;
    float v[S::NV][8], d[S::NV][8];
    load_row<S, F32>(x, rd, H, tr, v);
    load_row<S, F32>(dn, rd, H, tr, d);
    float ss, sd, scale = 1.f;
    auto sums = [&]() {
      ss = sum_sq<S>(v), sd = 0.f;
#pragma unroll
      for (int i = 0; i < S::NV; i++)
#pragma unroll
        for (int j = 0; j < 8; j++) sd = __builtin_fmaf(d[i][j] * wt[i][j], v[i][j], sd);
      row_sum2<S>(ss, sd, lds.red);
    };
    sums();
    if (ss > kLarge) {  // the same for the whole row
      scale = kShrink;
      shrink<S>(v, d);
      sums();
    }
    const float r = rms_inv(ss, H, eps * scale * scale), rs = r * scale;
    const float c = sd * r * rs / (float)H;  // mean(dh * h) * r
    if (!live) continue;  // no barrier below this point of the loop
#pragma unroll
    for (int i = 0; i < S::NV; i++)
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float h = v[i][j] * r;
        dw[i][j] = __builtin_fmaf(d[i][j], h, dw[i][j]);
        v[i][j] = rs * (d[i][j] * wt[i][j]) - h * c;
      }
    if (dres != nullptr) {
      load_row<S, F32>(dres, row, H, tr, d);
#pragma unroll
      for (int i = 0; i < S::NV; i++)
#pragma unroll
        for (int j = 0; j < 8; j++) v[i][j] += d[i][j];
    }
    store_row<S, F32>(dx, row, H, tr, v);
  }
  write_partial<S>(part, H, tr, dw, buf);
}

template <class S, bool F32, int G>
__global__ __launch_bounds__(S::BLOCK) void post_norm_backward_kernel(
    const void* dout, const void* __restrict__ y, const float* __restrict__ w,
    const void* __restrict__ gate, float alpha, float eps, int T, int H, void* dy,
    void* dres, void* dgate, float* __restrict__ part, float* __restrict__ gpart) {
  __shared__ Lds<S> lds;
  __shared__ float buf[S::RPB > 1 ? S::TPR * S::NV * 8 : 1];
  const int tr = threadIdx.x % S::TPR;
  float wt[S::NV][8], dw[S::NV][8], dg[S::NV][8];
  load_row<S, true>(w, 0, H, tr, wt);
#pragma unroll
  for (int i = 0; i < S::NV; i++)
#pragma unroll
    for (int j = 0; j < 8; j++) dw[i][j] = dg[i][j] = 0.f;
  for (size_t r0 = (size_t)blockIdx.x * S::RPB; r0 < (size_t)T;
       r0 += (size_t)gridDim.x * S::RPB) {
    const size_t row = r0 + threadIdx.x / S::TPR;
    const bool live = row < (size_t)T;
    const size_t rd = live ? row : (size_t)T - 1;
    float v[S::NV][8], d[S::NV][8], g[S::NV][8];
    load_row<S, F32>(y, rd, H, tr, v);
    load_row<S, F32>(dout, rd, H, tr, d);
    load_gate<S, F32, G>(gate, rd, H, tr, g);
    // ss = sum v^2, sd = sum dh * v, st = sum dout * w * v (the token gate's).
    float ss, sd, st, scale = 1.f;
    auto sums = [&]() {
      ss = sum_sq<S>(v), sd = 0.f, st = 0.f;
#pragma unroll
      for (int i = 0; i < S::NV; i++)
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const float p = d[i][j] * wt[i][j] * v[i][j];
          st += p;
          sd = __builtin_fmaf(p, g[i][j], sd);
        }
      row_sum2<S>(ss, sd, lds.red);
    };
    sums();
    if (ss > kLarge) {  // the same for the whole row
      scale = kShrink;
      shrink<S>(v, d);
      sums();
    }
    if constexpr (G == QMOE_GATE_TOKEN)
      if (dgate) st = row_sum<S>(st, lds.red);
    const float r = rms_inv(ss, H, eps * scale * scale), rs = r * scale;
    const float c = sd * r * rs / (float)H;
    if (!live) continue;  // no barrier below this point of the loop
    if (G == QMOE_GATE_TOKEN && dgate && tr == 0) reinterpret_cast<float*>(dgate)[row] = st * r;
    float o[S::NV][8];
#pragma unroll
    for (int i = 0; i < S::NV; i++)
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float h = v[i][j] * r, du = d[i][j] * g[i][j];
        dw[i][j] = __builtin_fmaf(du, h, dw[i][j]);
        o[i][j] = rs * (du * wt[i][j]) - h * c;
        v[i][j] = d[i][j] * h * wt[i][j];  // the gate's gradient
        d[i][j] *= alpha;
      }
    store_row<S, F32>(dy, row, H, tr, o);
    store_row<S, F32>(dres, row, H, tr, d);
    if constexpr (G == QMOE_GATE_FULL) store_row<S, F32>(dgate, row, H, tr, v);
    if constexpr (G == QMOE_GATE_COLUMN) {
#pragma unroll
      for (int i = 0; i < S::NV; i++)
#pragma unroll
        for (int j = 0; j < 8; j++) dg[i][j] += v[i][j];
    }
  }
  write_partial<S>(part, H, tr, dw, buf);
  if constexpr (G == QMOE_GATE_COLUMN) write_partial<S>(gpart, H, tr, dg, buf);
}

// out[c] = sum over the nb rows of part[nb][H], in fp64: a block sums 64
// columns, each of its 16 waves every 16th row.
__global__ __launch_bounds__(1024) void norm_colsum_kernel(const float* __restrict__ part0,
                                                           float* __restrict__ out0,
                                                           const float* __restrict__ part1,
                                                           float* __restrict__ out1, int nb,
                                                           int H) {
  __shared__ double s[16][64];
  const float* part = blockIdx.y == 0 ? part0 : part1;
  float* out = blockIdx.y == 0 ? out0 : out1;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  double a = 0.0;
  if (c < H) {
#pragma unroll 8
    for (int b = wave; b < nb; b += 16) a += (double)part[(size_t)b * H + c];
  }
  s[wave][lane] = a;
  __syncthreads();
  if (wave != 0 || c >= H) return;
#pragma unroll
  for (int w = 1; w < 16; w++) a += s[w][lane];
  out[c] = (float)a;
}

// Picks the shape for H: 64 threads per row up to 2048 columns, then 256 and
// 512, two or four vectors of eight per thread (1024 threads would halve the
// registers a thread may hold, which the gradients then spill); rows that are
// not 16-byte aligned take the scalar shapes, up to 8192 columns.
#define QMOE_NORM_SHAPES(VECOK, H, CALL)          \
  {                                               \
  if (!(VECOK) && (H) > norm_max_scalar_columns()) return hipErrorInvalidValue; \
  if (VECOK) {                                    \
    if (H <= 512) CALL((Shape<64, 1, true>))      \
    else if (H <= 1024) CALL((Shape<64, 2, true>)) \
    else if (H <= 2048) CALL((Shape<64, 4, true>)) \
    else if (H <= 4096) CALL((Shape<256, 2, true>)) \
    else if (H <= 8192) CALL((Shape<512, 2, true>)) \
    else CALL((Shape<512, 4, true>))             \
  } else {                                        \
    if (H <= 4096) CALL((Shape<256, 2, false>))   \
    else CALL((Shape<512, 2, false>))            \
  }                                               \
  }

#define QMOE_UNPAREN(...) __VA_ARGS__

int rows_per_block(int H, bool vec) { return vec && H <= 2048 ? 4 : 1; }
int backward_blocks(int T, int H, bool vec) {
  const int rpb = rows_per_block(H, vec);
  const int need = (T + rpb - 1) / rpb;
  return need < norm_partial_rows() ? need : norm_partial_rows();
}

template <bool F32>
hipError_t pre(const void* x, const float* w, float eps, int T, int H, const NormForm& f,
               hipStream_t s) {
  const bool vec = norm_vec_ok(H, {x, w, f.n});
#define QMOE_CALL(SH)                                                                        \
  {                                                                                          \
    typedef QMOE_UNPAREN SH S;                                                               \
    const dim3 grid = grid_of(((long long)T + S::RPB - 1) / S::RPB);                         \
    hipLaunchKernelGGL((pre_norm_kernel<S, F32>), grid, dim3(S::BLOCK), 0, s, x, w, eps, T,  \
                       H, f);                                                                \
  }
  QMOE_NORM_SHAPES(vec, H, QMOE_CALL)
#undef QMOE_CALL
  return hipGetLastError();
}

template <bool F32, int G>
hipError_t post(const PostNormArgs& a, hipStream_t s) {
  const void* gate = a.gate_kind == QMOE_GATE_NONE ? nullptr : a.gate;
  const bool vec = norm_vec_ok(a.H, {a.y, a.x, a.w, a.out}) &&
                   (G == QMOE_GATE_TOKEN || norm_vec_ok(a.H, {gate})) &&
                   (a.w2 == nullptr || norm_vec_ok(a.H, {a.w2, a.f.n}));
#define QMOE_CALL(SH)                                                                        \
  {                                                                                          \
    typedef QMOE_UNPAREN SH S;                                                               \
    const dim3 grid = grid_of(((long long)a.T + S::RPB - 1) / S::RPB);                       \
    hipLaunchKernelGGL((post_norm_kernel<S, F32, G>), grid, dim3(S::BLOCK), 0, s, a.y, a.x,  \
                       a.w, gate, a.alpha, a.eps, a.T, a.H, a.out, a.w2, a.f);               \
  }
  QMOE_NORM_SHAPES(vec, a.H, QMOE_CALL)
#undef QMOE_CALL
  return hipGetLastError();
}

hipError_t colsum(const float* p0, float* o0, const float* p1, float* o1, int nb, int H,
                  hipStream_t s) {
  hipLaunchKernelGGL(norm_colsum_kernel, dim3((H + 63) / 64, p1 ? 2 : 1), dim3(1024), 0, s, p0, o0,
                     p1, o1, nb, H);
  return hipGetLastError();
}

template <bool F32>
hipError_t pre_bwd(const PreNormBwdArgs& a, hipStream_t s) {
  const bool vec = norm_vec_ok(a.H, {a.dn, a.x, a.w, a.dres, a.dx});
  const int nb = backward_blocks(a.T, a.H, vec);
#define QMOE_CALL(SH)                                                                         \
  {                                                                                           \
    typedef QMOE_UNPAREN SH S;                                                                \
    hipLaunchKernelGGL((pre_norm_backward_kernel<S, F32>), dim3(nb), dim3(S::BLOCK), 0, s,    \
                       a.dn, a.x, a.w, a.dres, a.eps, a.T, a.H, a.dx, a.part);                \
  }
  if (nb > 0) QMOE_NORM_SHAPES(vec, a.H, QMOE_CALL)
#undef QMOE_CALL
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return colsum(a.part, a.dw, nullptr, nullptr, nb, a.H, s);
}

template <bool F32, int G>
hipError_t post_bwd(const PostNormBwdArgs& a, hipStream_t s) {
  const bool colg = G == QMOE_GATE_COLUMN;
  const void* gate = a.gate_kind == QMOE_GATE_NONE ? nullptr : a.gate;
  void* dgate = a.gate_kind == QMOE_GATE_NONE ? nullptr : a.dgate;
  const bool vec = norm_vec_ok(a.H, {a.dout, a.y, a.w, a.dy, a.dres}) &&
                   (G == QMOE_GATE_TOKEN || norm_vec_ok(a.H, {gate})) &&
                   (G != QMOE_GATE_FULL || norm_vec_ok(a.H, {dgate}));
  const int nb = backward_blocks(a.T, a.H, vec);
  float* gpart = a.part + (size_t)norm_partial_rows() * a.H;
#define QMOE_CALL(SH)                                                                          \
  {                                                                                            \
    typedef QMOE_UNPAREN SH S;                                                                 \
    hipLaunchKernelGGL((post_norm_backward_kernel<S, F32, G>), dim3(nb), dim3(S::BLOCK), 0, s, \
                       a.dout, a.y, a.w, gate, a.alpha, a.eps, a.T, a.H, a.dy, a.dres, dgate,  \
                       a.part, gpart);                                                         \
  }
  if (nb > 0) QMOE_NORM_SHAPES(vec, a.H, QMOE_CALL)
#undef QMOE_CALL
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return colsum(a.part, a.dw, colg ? gpart : nullptr, reinterpret_cast<float*>(a.dgate), nb, a.H,
                s);
}

}  // namespace

int norm_partial_rows() { return 512; }

hipError_t launch_pre_norm(const void* x, bool f32, const float* w, float eps, int T, int H,
                           const NormForm& f, hipStream_t s) {
  return f32 ? pre<true>(x, w, eps, T, H, f, s) : pre<false>(x, w, eps, T, H, f, s);
}
#define QMOE_BY_GATE(FN, A)                                                        \
  switch ((A).gate_kind) {                                                         \
    case QMOE_GATE_COLUMN:                                                         \
      return (A).f32 ? FN<true, QMOE_GATE_COLUMN>(A, s) : FN<false, QMOE_GATE_COLUMN>(A, s); \
    case QMOE_GATE_FULL:                                                           \
      return (A).f32 ? FN<true, QMOE_GATE_FULL>(A, s) : FN<false, QMOE_GATE_FULL>(A, s);     \
    default:                                                                       \
      return (A).f32 ? FN<true, QMOE_GATE_TOKEN>(A, s) : FN<false, QMOE_GATE_TOKEN>(A, s);   \
  }

hipError_t launch_post_norm(const PostNormArgs& a, hipStream_t s) { QMOE_BY_GATE(post, a) }
hipError_t launch_pre_norm_backward(const PreNormBwdArgs& a, hipStream_t s) {
  return a.f32 ? pre_bwd<true>(a, s) : pre_bwd<false>(a, s);
}
hipError_t launch_post_norm_backward(const PostNormBwdArgs& a, hipStream_t s) {
  QMOE_BY_GATE(post_bwd, a)
}

}  // namespace qmoe
