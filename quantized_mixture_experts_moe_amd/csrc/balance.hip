// Balance loss of the router with per-expert counts, and its gradient.
//
//   p[t] = softmax(logits[t]) over the E experts, for the n kept tokens
//   f_e  = count_e / (k n),  P_e = sum_t p[t,e] / n
//   loss = coef * E * sum_e f_e P_e
//   dlogits[t,e] = dloss * coef * E / n * p[t,e] * (f_e - sum_j f_j p[t,j])
//
// The counts carry no gradient (they are whole numbers).  One wave holds a
// token's logits in registers, EPL per lane, as in the routing kernel.  The
// sums run in a fixed order (per wave over its tokens, over a block's waves,
// then over the blocks in fp64), the counts are integer atomics, whose order
// does not matter: results are the same bits on every run.
#include "block_common.h"

namespace qmoe {
namespace {
using namespace bk;

// Softmax of one row held as z[EPL] (expert e = lane + 64 i; missing experts
// hold -inf): p in place.  A row of -inf alone (every expert masked) has no
// softmax and gives zeros; a NaN or +inf gives NaN.
template <int EPL>
__device__ inline void softmax_row(float z[EPL]) {
  float mx = z[0];
#pragma unroll
  for (int i = 1; i < EPL; i++) mx = fmaxf(mx, z[i]);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off, 64));
  const float m0 = mx == -INFINITY ? 0.f : mx;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < EPL; i++) {
    z[i] = expf(z[i] - m0);
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

// One block's share of the tokens: partial probability sums psum[block][E],
// counts csum[block][E] and kept tokens nsum[block].
template <int EPL>
__global__ __launch_bounds__(256) void balance_partial_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids,
    const uint8_t* __restrict__ mask, int T, int E, int k, float* __restrict__ psum,
    int32_t* __restrict__ csum, int32_t* __restrict__ nsum) {
  __shared__ float ps[4][64 * EPL];
  __shared__ int hist[64 * EPL];
  __shared__ int kept[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < 64 * EPL; e += 256) hist[e] = 0;
  __syncthreads();
  float acc[EPL];
#pragma unroll
  for (int i = 0; i < EPL; i++) acc[i] = 0.f;
  int n = 0;
  for (int t = blockIdx.x * 4 + wave; t < T; t += gridDim.x * 4) {
    if (mask && mask[t] == 0) continue;  // the same for the whole wave
    n++;
    float z[EPL];
    load_row<EPL>(logits + (size_t)t * E, E, z);
    if (lane < k) {
      const int e = ids[(size_t)t * k + lane];
      if (e >= 0 && e < E) atomicAdd(&hist[e], 1);
    }
    softmax_row<EPL>(z);
#pragma unroll
    for (int i = 0; i < EPL; i++) acc[i] += z[i];
  }
#pragma unroll
  for (int i = 0; i < EPL; i++) ps[wave][lane + 64 * i] = acc[i];
  if (lane == 0) kept[wave] = n;
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 256) {
    psum[(size_t)blockIdx.x * E + e] = (ps[0][e] + ps[1][e]) + (ps[2][e] + ps[3][e]);
    csum[(size_t)blockIdx.x * E + e] = hist[e];
  }
  if (threadIdx.x == 0) nsum[blockIdx.x] = kept[0] + kept[1] + kept[2] + kept[3];
}

// Sums the partials of nb blocks (one block of 1024 threads, one expert per
// thread) and forms the loss.
__global__ __launch_bounds__(1024) void balance_finish_kernel(
    const float* __restrict__ psum, const int32_t* __restrict__ csum,
    const int32_t* __restrict__ nsum, int nb, int E, int k, float coef, float* __restrict__ loss,
    int32_t* __restrict__ counts, float* __restrict__ probs, int32_t* __restrict__ tokens) {
  __shared__ double terms[16];
  int n = 0;
  for (int b = 0; b < nb; b++) n += nsum[b];
  double term = 0.0;
  for (int e = threadIdx.x; e < E; e += 1024) {
    double p = 0.0;
    int c = 0;
    for (int b = 0; b < nb; b++) {
      p += (double)psum[(size_t)b * E + e];
      c += csum[(size_t)b * E + e];
    }
    p = n > 0 ? p / n : 0.0;
    counts[e] = c;
    probs[e] = (float)p;
    if (n > 0) term += (double)c / ((double)k * n) * p;
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) term += __shfl_xor(term, off, 64);
  if ((threadIdx.x & 63) == 0) terms[threadIdx.x >> 6] = term;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < 16; w++) s += terms[w];
    *loss = (float)((double)coef * E * s);
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
    float* out = dlogits + (size_t)t * E;
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
#pragma unroll
    for (int i = 0; i < EPL; i++)
      if (lane + 64 * i < E) out[lane + 64 * i] = z[i];
  }
}

}  // namespace

int balance_blocks(int T) {
  const int need = (T + 3) / 4;
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
                          int32_t* tokens, float* psum, int32_t* csum, int32_t* nsum,
                          hipStream_t s) {
  const int nb = balance_blocks(T);
#define QMOE_CALL(EPL)                                                                         \
  hipLaunchKernelGGL(balance_partial_kernel<EPL>, dim3(nb), dim3(256), 0, s, logits, ids, mask, \
                     T, E, k, psum, csum, nsum);
  QMOE_BALANCE_EPL(QMOE_CALL)
#undef QMOE_CALL
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(balance_finish_kernel, dim3(1), dim3(1024), 0, s, psum, csum, nsum, nb, E, k,
                     coef, loss, counts, probs, tokens);
  return hipGetLastError();
}

hipError_t launch_balance_backward(const float* logits, const uint8_t* mask,
                                   const int32_t* counts, const int32_t* tokens,
                                   const float* dloss, int T, int E, int k, float coef,
                                   float* dlogits, hipStream_t s) {
  const int nb = T < 4 * 2048 ? (T + 3) / 4 : 2048;
#define QMOE_CALL(EPL)                                                                        \
  hipLaunchKernelGGL(balance_backward_kernel<EPL>, dim3(nb), dim3(256), 0, s, logits, mask,    \
                     counts, tokens, dloss, T, E, k, coef, dlogits);
  QMOE_BALANCE_EPL(QMOE_CALL)
#undef QMOE_CALL
  return hipGetLastError();
}

}  // namespace qmoe
