// Gradient of the routed sum out[t] = sum_j w[t,j] y[t k + j] and of the
// weights' softmax over the picked logits:
//   dy[t k + j] = w[t,j] dout[t],   dw[t,j] = <dout[t], y[t k + j]>,
//   dlogits[t, ids[t,j]] += w[t,j] (dw[t,j] - sum_i w[t,i] dw[t,i]).
// Bound: y is read once and dy written once.  WPT waves take a token: a lane
// holds eight columns of dout at a time and passes over the token's rows of y,
// whose products it keeps for the rows of a group of kGroup (dout is read once per
// group).  All of a group's rows are loaded before the first is used, past the caches,
// as dy is stored: 4111 tokens, top-8, 2048 columns in bf16 50-53 us, 291 MB at 5.5-5.8
// TB/s, a large copy's rate and more (88 us with a row's load behind its id and through the
// caches; 58 with the weights loaded again at the end).  A small batch is one trip
// to memory behind the other: 64 tokens, top-2, 256 columns 5.2 us.
#include "block_common.h"
#include "qmoe_internal.h"

namespace qmoe {
namespace {
using namespace bk;
constexpr int kGroup = 8, kMaxK = 16;

// Eight values as loaded, and eight stored, that no other wave reads.
template <bool F32>
struct Raw8 {
  u32x4 q[F32 ? 2 : 1];
};
template <bool F32>
__device__ inline Raw8<F32> load_once(const void* p, size_t i) {
  Raw8<F32> r;
  const u32x4* q = reinterpret_cast<const u32x4*>(reinterpret_cast<const uint8_t*>(p) +
                                                  i * (F32 ? 4 : 2));
  r.q[0] = __builtin_nontemporal_load(q);
  if constexpr (F32) r.q[1] = __builtin_nontemporal_load(q + 1);
  return r;
}
template <bool F32>
__device__ inline void unpack(const Raw8<F32>& r, float v[8]) {
#pragma unroll
  for (int i = 0; i < 8; i++) {
    if constexpr (F32)
      v[i] = __uint_as_float(r.q[i / 4][i % 4]);
    else
      v[i] = __uint_as_float(i & 1 ? r.q[0][i / 2] & 0xffff0000u : r.q[0][i / 2] << 16);
  }
}
template <bool F32>
__device__ inline void store_past(void* p, size_t i, const float v[8]) {
  u32x4* q = reinterpret_cast<u32x4*>(reinterpret_cast<uint8_t*>(p) + i * (F32 ? 4 : 2));
  if constexpr (F32) {
#pragma unroll
    for (int h = 0; h < 2; h++)
      __builtin_nontemporal_store(
          u32x4{__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]),
                __float_as_uint(v[4 * h + 2]), __float_as_uint(v[4 * h + 3])},
          q + h);
  } else {
    __builtin_nontemporal_store(u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                      pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])},
                                q);
  }
}

template <int WPT, bool F32>
__global__ __launch_bounds__(256) void combine_backward_kernel(CombineBwdArgs g) {
  constexpr int TPB = 4 / WPT;  // tokens per block
  __shared__ float sums[4][kMaxK], weights[4][kMaxK];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int t = blockIdx.x * TPB + wave / WPT;
  const bool on = t < g.T;
  const int k = g.k, H = g.H;
  const size_t p0 = (size_t)t * k;
  const int c0 = ((wave % WPT) * 64 + lane) * 8, step = WPT * 512;
  if (on) {
    for (int j0 = 0; j0 < k; j0 += kGroup) {
      float w[kGroup], dot[kGroup];
      bool in[kGroup];  // the pair's id is an expert's
#pragma unroll
      for (int u = 0; u < kGroup; u++) {
        dot[u] = 0.f;
        const int j = min(j0 + u, k - 1);
        in[u] = j0 + u < k && (unsigned)g.ids[p0 + j] < (unsigned)g.E;
        w[u] = g.w[p0 + j];
      }
      for (int c = c0; c < H; c += step) {
        float d[8];
        Raw8<F32> y[kGroup];  // (all loads before the first is used)
        load8<F32>(g.dout, (size_t)t * H + c, d);
#pragma unroll
        for (int u = 0; u < kGroup; u++)
          if (j0 + u < k) y[u] = load_once<F32>(g.y, (p0 + j0 + u) * H + c);
#pragma unroll
        for (int u = 0; u < kGroup; u++) {
          if (j0 + u >= k) continue;
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; i++) v[i] = in[u] ? w[u] * d[i] : 0.f;
          if (in[u]) {
            float f[8];
            unpack<F32>(y[u], f);
#pragma unroll
            for (int i = 0; i < 8; i++) dot[u] = __builtin_fmaf(d[i], f[i], dot[u]);
          }
          store_past<F32>(g.dy, (p0 + j0 + u) * H + c, v);
        }
      }
#pragma unroll
      for (int u = 0; u < kGroup; u++) {
        if (j0 + u >= k) continue;
        const float s = wave_sum(dot[u]);
        if (lane == 0) {
          sums[wave][j0 + u] = s;
          weights[wave][j0 + u] = in[u] ? w[u] : 0.f;  // a dropped pair's counts nothing
        }
      }
    }
  }
  __syncthreads();
  if (!on) return;
  float dw[kMaxK], mean = 0.f;
  const int first = wave / WPT * WPT;
#pragma unroll
  for (int j = 0; j < kMaxK; j++) {
    dw[j] = 0.f;
    if (j < k) {
#pragma unroll
      for (int v = 0; v < WPT; v++) dw[j] += sums[first + v][j];
      mean = __builtin_fmaf(weights[wave][j], dw[j], mean);
    }
  }
  const int at = (wave % WPT) * 64 + lane;
  if (g.dw != nullptr) {
#pragma unroll
    for (int j = 0; j < kMaxK; j++)
      if (j < k && at == j) g.dw[p0 + j] = dw[j];
  }
  if (g.dlogits != nullptr) {
    float dz[kMaxK];
    int id[kMaxK];
#pragma unroll
    for (int j = 0; j < kMaxK; j++) {
      dz[j] = 0.f;
      id[j] = -1;
      if (j < k) {
        dz[j] = weights[wave][j] * (dw[j] - mean);
        id[j] = g.ids[p0 + j];
      }
    }
    const size_t row = (size_t)t * g.E;
    for (int e = at; e < g.E; e += WPT * 64) {
      float v = g.add != nullptr ? g.add[row + e] : 0.f;
#pragma unroll
      for (int j = 0; j < kMaxK; j++)
        if (j < k && id[j] == e) v += dz[j];
      g.dlogits[row + e] = v;
    }
  }
}

}  // namespace

hipError_t launch_combine_backward(const CombineBwdArgs& all, hipStream_t s) {
  // A wave's pass covers 512 columns: one wave per token up to there.
#define QMOE_CALL(WPT, F32)                                                                \
  hipLaunchKernelGGL((combine_backward_kernel<WPT, F32>),                                  \
                     dim3((unsigned)((g.T + 4 / WPT - 1) / (4 / WPT))), dim3(256), 0, s, g)
  // A grid holds fewer than 2^32 threads (one with more runs only what is left of their
  // number behind 32 bits, without an error).
  constexpr int kTokens = 1 << 22;
  const size_t row = (size_t)all.H * (all.f32 ? 4 : 2);
  for (int t0 = 0; t0 < all.T; t0 += kTokens) {
    CombineBwdArgs g = all;
    const size_t pairs = (size_t)t0 * g.k, logits = (size_t)t0 * g.E;
    g.T = all.T - t0 < kTokens ? all.T - t0 : kTokens;
    g.dout = reinterpret_cast<const uint8_t*>(g.dout) + t0 * row;
    g.y = reinterpret_cast<const uint8_t*>(g.y) + pairs * row;
    g.dy = reinterpret_cast<uint8_t*>(g.dy) + pairs * row;
    g.ids += pairs;
    g.w += pairs;
    if (g.dw != nullptr) g.dw += pairs;
    if (g.dlogits != nullptr) g.dlogits += logits;
    if (g.add != nullptr) g.add += logits;
    if (g.H <= 512) {
      if (g.f32)
        QMOE_CALL(1, true);
      else
        QMOE_CALL(1, false);
    } else {
      if (g.f32)
        QMOE_CALL(4, true);
      else
        QMOE_CALL(4, false);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
#undef QMOE_CALL
  return hipSuccess;
}

}  // namespace qmoe
