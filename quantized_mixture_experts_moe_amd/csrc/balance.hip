// Balance loss of the router with per-expert counts, and its gradient.
//
//   p[t] = softmax(logits[t]) over the E experts, for the n kept tokens
//   f_e  = count_e / (k n),  P_e = sum_t p[t,e] / n
//   loss = coef * E * sum_e f_e P_e
//   dlogits[t,e] = dloss * coef * E / n * p[t,e] * (f_e - sum_j f_j p[t,j])
//
// The counts carry no gradient (they are whole numbers).  One wave holds a
// token's logits in registers, EPL per lane, as in the routing kernel.  The
// sums run in a fixed order (per wave over its tokens and over a block's waves
// in fp32, which for terms that are not negative is a half step of the sum per
// addition at most, then over the blocks in fp64), the counts are integer atomics, whose order
// does not matter: results are the same bits on every run.  What bounds the
// calls is latency: 8192 x 512 takes 7.4 us for the partial sums (2.3 TB/s),
// 6.1 to join them, 10.8 for the gradient (3.1 TB/s); 64 x 8 takes 4.5 and 3.4.
// 16-byte loads (four experts per lane) made the first and last 0.4 us slower.
#include "block_common.h"

namespace qmoe {
namespace {
using namespace bk;

// Softmax of one row held as z[EPL] (expert e = lane + 64 i; missing experts
// hold -inf): p in place.  A row of -inf alone (every expert masked) has no
// softmax and gives zeros; a NaN or +inf gives NaN.  The difference to the
// maximum comes first (logits down to the lowest finite number are masks too),
// then its product with log2 e: two roundings of z - max in the exponent, which
// are small where p is not.
template <int EPL>
__device__ inline void softmax_row(float z[EPL]) {
  constexpr float kLog2e = 1.44269502162933349609375f;
  float mx = z[0];
#pragma unroll
  for (int i = 1; i < EPL; i++) mx = fmaxf(mx, z[i]);
  mx = wave_fmax(mx);
  const float m0 = mx == -INFINITY ? 0.f : mx;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < EPL; i++) {
    z[i] = __builtin_amdgcn_exp2f((z[i] - m0) * kLog2e);
    sum += z[i];
  }
  sum = wave_sum(sum);
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
  for (int i = 0; i < EPL; i++) z[i] *= inv;
}

template <int EPL>
__device__ inline void load_row(const float* row, int E, float z[EPL]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < EPL; i++) z[i] = lane + 64 * i < E ? row[lane + 64 * i] : -INFINITY;
}

// A wave loads the logits of kAhead tokens before it works on them: the loads'
// latency is what a short batch consists of.
constexpr int kAhead = 4;

// A block's share of the tokens (WAVES waves, a token per wave at a time): the
// waves' probability sums in ps, the counts in hist, the kept tokens returned.
template <int EPL, int WAVES>
struct Share {
  float ps[WAVES][64 * EPL];
  int hist[64 * EPL];
  int kept[WAVES];

  __device__ inline int run(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                            const uint8_t* __restrict__ mask, int T, int E, int k) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    for (int e = threadIdx.x; e < 64 * EPL; e += 64 * WAVES) hist[e] = 0;
    __syncthreads();
    float acc[EPL], z[kAhead][EPL];
#pragma unroll
    for (int i = 0; i < EPL; i++) acc[i] = 0.f;
    int n = 0;
    const int step = gridDim.x * WAVES;
    for (int t0 = blockIdx.x * WAVES + wave; t0 < T; t0 += step * kAhead) {
      int pick[kAhead];
      bool keep[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; a++) {
        const int t = t0 + a * step;
        keep[a] = t < T && (!mask || mask[t] != 0);  // the same for the whole wave
        pick[a] = -1;
        if (t < T) {
          load_row<EPL>(logits + (size_t)t * E, E, z[a]);
          if (lane < k) pick[a] = ids[(size_t)t * k + lane];
        }
      }
#pragma unroll
      for (int a = 0; a < kAhead; a++) {
        if (!keep[a]) continue;
        n++;
        if (pick[a] >= 0 && pick[a] < E) atomicAdd(&hist[pick[a]], 1);
        softmax_row<EPL>(z[a]);
#pragma unroll
        for (int i = 0; i < EPL; i++) acc[i] += z[a][i];
      }
    }
#pragma unroll
    for (int i = 0; i < EPL; i++) ps[wave][lane + 64 * i] = acc[i];
    if (lane == 0) kept[wave] = n;
    __syncthreads();
    n = 0;
#pragma unroll
    for (int w = 0; w < WAVES; w++) n += kept[w];
    return n;
  }
};

// Sum over the waves of a block, in every thread; `s` holds WAVES doubles.
template <int WAVES>
__device__ inline double block_sum64(double x, double* s) {
  x = wave_sum64(x);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = x;
  __syncthreads();
  x = 0.0;
#pragma unroll
  for (int w = 0; w < WAVES; w++) x += s[w];
  return x;
}

constexpr int kWaves = 8;  // of a partial block

template <int EPL>
__global__ __launch_bounds__(64 * kWaves) void balance_partial_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids,
    const uint8_t* __restrict__ mask, int T, int E, int k, BalanceParts w) {
  __shared__ Share<EPL, kWaves> share;
  const int n = share.run(logits, ids, mask, T, E, k);
  for (int e = threadIdx.x; e < E; e += 64 * kWaves) {
    float s = share.ps[0][e];
#pragma unroll
    for (int v = 1; v < kWaves; v++) s += share.ps[v][e];
    w.psum[(size_t)blockIdx.x * E + e] = s;
    w.csum[(size_t)blockIdx.x * E + e] = share.hist[e];
  }
  if (threadIdx.x == 0) {
    w.nsum[blockIdx.x] = n;
    if (blockIdx.x == 0) *w.arrived = 0;
  }
}

// Adds the partials of nb blocks: a block sums 32 experts, 32 threads each
// over every 32nd partial; the last block to arrive forms the loss from the
// blocks' terms, in order.
constexpr int kFinish = 32;
__global__ __launch_bounds__(1024) void balance_finish_kernel(BalanceParts w, int nb, int E, int k,
                                                              float coef, float* __restrict__ loss,
                                                              int32_t* __restrict__ counts,
                                                              float* __restrict__ probs,
                                                              int32_t* __restrict__ tokens) {
  __shared__ double ps[32][kFinish], sums[16];
  __shared__ int cs[32][kFinish];
  const int col = threadIdx.x % kFinish, group = threadIdx.x / kFinish;
  const int e = blockIdx.x * kFinish + col;
  double p = 0.0;
  int c = 0;
  if (e < E) {
#pragma unroll 8
    for (int b = group; b < nb; b += 32) {
      p += (double)w.psum[(size_t)b * E + e];
      c += w.csum[(size_t)b * E + e];
    }
  }
  ps[group][col] = p;
  cs[group][col] = c;
  const double kept = (int)threadIdx.x < nb ? (double)w.nsum[threadIdx.x] : 0.0;
  const int n = (int)block_sum64<16>(kept, sums);  // with barriers before the reads below
  if (threadIdx.x >= 64) return;
  double term = 0.0;
  if (group == 0) {
#pragma unroll
    for (int v = 1; v < 32; v++) {
      p += ps[v][col];
      c += cs[v][col];
    }
    p = n > 0 ? p / n : 0.0;
    if (e < E) {
      counts[e] = c;
      probs[e] = (float)p;
      if (n > 0) term = (double)c / ((double)k * n) * p;
    }
  }
  term = wave_sum64(term);
  if (threadIdx.x != 0) return;
  w.terms[blockIdx.x] = term;
  __threadfence();
  if (atomicAdd(w.arrived, 1) != (int)gridDim.x - 1) return;
  __threadfence();
  double s = 0.0;
  for (int b = 0; b < (int)gridDim.x; b++)
    s += __hip_atomic_load(&w.terms[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  *loss = (float)((double)coef * E * s);
  *tokens = n;
}

// Small batches in one launch of one block.
constexpr int kSmallWaves = 16;
template <int EPL>
__global__ __launch_bounds__(64 * kSmallWaves) void balance_small_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids,
    const uint8_t* __restrict__ mask, int T, int E, int k, float coef, float* __restrict__ loss,
    int32_t* __restrict__ counts, float* __restrict__ probs, int32_t* __restrict__ tokens) {
  __shared__ Share<EPL, kSmallWaves> share;
  __shared__ double sums[kSmallWaves];
  const int n = share.run(logits, ids, mask, T, E, k);
  double term = 0.0;
  const int e = threadIdx.x;  // E <= 1024
  if (e < E) {
    double p = 0.0;
#pragma unroll
    for (int v = 0; v < kSmallWaves; v++) p += (double)share.ps[v][e];
    p = n > 0 ? p / n : 0.0;
    counts[e] = share.hist[e];
    probs[e] = (float)p;
    if (n > 0) term = (double)share.hist[e] / ((double)k * n) * p;
  }
  term = block_sum64<kSmallWaves>(term, sums);
  if (threadIdx.x == 0) {
    *loss = (float)((double)coef * E * term);
    *tokens = n;
  }
}

// `dlogits` may be `logits`: a wave reads its row before it writes it.
template <int EPL>
__global__ __launch_bounds__(256) void balance_backward_kernel(
    const float* logits, const uint8_t* __restrict__ mask,
    const int32_t* __restrict__ counts, const int32_t* __restrict__ tokens,
    const float* __restrict__ dloss, int T, int E, int k, float coef,
    float* dlogits) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = *tokens;
  const float kn = n > 0 ? 1.0f / ((float)k * (float)n) : 0.f;
  const float g = n > 0 ? *dloss * coef * (float)E / (float)n : 0.f;
  float f[EPL];
#pragma unroll
  for (int i = 0; i < EPL; i++)
    f[i] = lane + 64 * i < E ? (float)counts[lane + 64 * i] * kn : 0.f;
  for (int t = blockIdx.x * 4 + wave; t < T; t += gridDim.x * 4) {
    float z[EPL];
    if (mask && mask[t] == 0) {
#pragma unroll
      for (int i = 0; i < EPL; i++) z[i] = 0.f;
    } else {
      load_row<EPL>(logits + (size_t)t * E, E, z);
      softmax_row<EPL>(z);
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; i++) dot += z[i] * f[i];
      dot = wave_sum(dot);
#pragma unroll
      for (int i = 0; i < EPL; i++) z[i] = g * z[i] * (f[i] - dot);
    }
    float* out = dlogits + (size_t)t * E;
#pragma unroll
    for (int i = 0; i < EPL; i++)
      if (lane + 64 * i < E) out[lane + 64 * i] = z[i];
  }
}

}  // namespace

// A wave takes a token at a time whatever E is, so what the one block costs goes
// by its tokens: up to six per wave it is done before the second launch of the
// other form would be.  One block / two launches, us on the GPU, by tokens:
//   experts        16           64           96          112          4096
//   8           3.1 / 5.7    4.8 / 5.8    6.0 / 6.0    6.4 / 5.9    140 / 7.0
//   256         3.2 / 7.4    5.2 / 7.7    6.8 / 7.8    7.3 / 7.7
//   1024        4.6 / 11.3   8.8 / 11.5  11.7 / 11.6  13.1 / 11.6
bool balance_small(int T) { return T <= 6 * kSmallWaves; }
int balance_blocks(int T) {
  const int need = (T + kWaves - 1) / kWaves;
  return need < 1 ? 1 : need > 256 ? 256 : need;
}

#define QMOE_BALANCE_EPL(CALL) \
  if (E <= 64) CALL(1)         \
  else if (E <= 128) CALL(2)   \
  else if (E <= 256) CALL(4)   \
  else if (E <= 512) CALL(8)   \
  else CALL(16)

hipError_t launch_balance(const float* logits, const int32_t* ids, const uint8_t* mask, int T,
                          int E, int k, float coef, float* loss, int32_t* counts, float* probs,
                          int32_t* tokens, const BalanceParts& w, hipStream_t s) {
  if (balance_small(T)) {
#define QMOE_CALL(EPL)                                                                           \
  hipLaunchKernelGGL(balance_small_kernel<EPL>, dim3(1), dim3(64 * kSmallWaves), 0, s, logits,    \
                     ids, mask, T, E, k, coef, loss, counts, probs, tokens);
    QMOE_BALANCE_EPL(QMOE_CALL)
#undef QMOE_CALL
    return hipGetLastError();
  }
  const int nb = balance_blocks(T);
#define QMOE_CALL(EPL)                                                                          \
  hipLaunchKernelGGL(balance_partial_kernel<EPL>, dim3(nb), dim3(64 * kWaves), 0, s, logits, ids, \
                     mask, T, E, k, w);
  QMOE_BALANCE_EPL(QMOE_CALL)
#undef QMOE_CALL
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(balance_finish_kernel, dim3((E + kFinish - 1) / kFinish), dim3(1024), 0, s,
                     w, nb, E, k, coef, loss, counts, probs, tokens);
  return hipGetLastError();
}

hipError_t launch_balance_backward(const float* logits, const uint8_t* mask,
                                   const int32_t* counts, const int32_t* tokens,
                                   const float* dloss, int T, int E, int k, float coef,
                                   float* dlogits, hipStream_t s) {
  // A token per wave up to 8192 of them: many waves hide the loads better than
  // several tokens per wave do (8192 x 512: 11 against 14 us).
  const int nb = T < 4 * 2048 ? (T + 3) / 4 : 2048;
#define QMOE_CALL(EPL)                                                                        \
  hipLaunchKernelGGL(balance_backward_kernel<EPL>, dim3(nb), dim3(256), 0, s, logits, mask,    \
                     counts, tokens, dloss, T, E, k, coef, dlogits);
  QMOE_BALANCE_EPL(QMOE_CALL)
#undef QMOE_CALL
  return hipGetLastError();
}

}  // namespace qmoe
