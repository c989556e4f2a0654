// Internal declarations of the operators around the experts: fp8 quantizer
// and products, balance loss, norms (not installed).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "qmoe.h"

namespace qmoe {

// Status of a HIP call; remembers a failing hipError_t for the thread.
qmoe_status hip_status(hipError_t e);

struct Fp8QuantArgs {
  const void* x;  // [B, M, K], or [M, 2K] with act
  bool f32, block, act;
  int B, M, K;  // B > 1 only with block
  uint8_t* codes;    // [B, M, KB*128] or nullptr
  float* scale;      // [KB, M]; block [B, MB, KB]
  uint8_t* codes_t;  // [B, K, MB*128] or nullptr
  float* scale_t;    // [MB, K]; block [B, KB, MB]
};
hipError_t launch_fp8_quant(const Fp8QuantArgs& a, hipStream_t s);

struct Fp8MatmulArgs {
  const uint8_t* a;      // [Ma, K]
  const float* a_scale;  // [KB, Ma]
  const uint8_t* b;      // [N, K]; grouped [E, N, K]
  const float* b_scale;  // b_block [ceil(N/128), KB] (grouped: per expert), else [KB, N]
  void* out;             // [M, N]; grouped [P, N]
  int M, Ma, N, K, KB;   // grouped: M = capacity of the sorted list
  bool b_block, out_f32;
  // grouped
  const int32_t* sorted;
  const int32_t* tile_expert;
  const int32_t* expert_offsets;
  const int32_t* num_padded;
  int P, k, block_m, E;
  bool pair_rows;
  // dense: sums of a K split in parts [splits, M, N] fp32
  float* parts;
  int split_kb;  // K blocks per part (set by the launcher)
};
size_t fp8_matmul_parts_bytes(int M, int N, int K);
hipError_t launch_fp8_matmul(const Fp8MatmulArgs& g, hipStream_t s);
hipError_t launch_fp8_grouped_matmul(const Fp8MatmulArgs& g, hipStream_t s);

// Workspace of the balance loss: per block (balance_blocks) the probability
// sums and counts [E] and kept tokens; per 32 experts a term of the loss; the
// blocks that have arrived.  A small batch needs none.
struct BalanceParts {
  float* psum;
  int32_t* csum;
  int32_t* nsum;
  double* terms;
  int32_t* arrived;
};
bool balance_small(int T);
int balance_blocks(int T);
hipError_t launch_balance(const float* logits, const int32_t* ids, const uint8_t* mask, int T,
                          int E, int k, float coef, float* loss, int32_t* counts, float* probs,
                          int32_t* tokens, const BalanceParts& w, hipStream_t s);
hipError_t launch_balance_backward(const float* logits, const uint8_t* mask,
                                   const int32_t* counts, const int32_t* tokens,
                                   const float* dloss, int T, int E, int k, float coef,
                                   float* dlogits, hipStream_t s);

struct NormForm {
  int form;      // qmoe_form
  void* n;
  float* scale;
};
struct PostNormArgs {
  const void *y, *x;
  bool f32;
  const float* w;
  const void* gate;
  int gate_kind;
  float alpha, eps;
  int T, H;
  void* out;
  const float* w2;  // nullptr: no next norm
  NormForm f;
};
struct PreNormBwdArgs {
  const void *dn, *x;
  bool f32;
  const float* w;
  const void* dres;
  float eps;
  int T, H;
  void* dx;
  float* dw;
  float* part;  // [norm_partial_rows(), H]
};
struct PostNormBwdArgs {
  const void *dout, *y;
  bool f32;
  const float* w;
  const void* gate;
  int gate_kind;
  float alpha, eps;
  int T, H;
  void *dy, *dres;
  float* dw;
  void* dgate;
  float* part;  // [norm_partial_rows(), H], twice with a column gate
};
int norm_partial_rows();
int norm_max_columns();
// Without 16-byte loads (norm_vec_ok: H a multiple of 8, arrays aligned).
int norm_max_scalar_columns();
bool norm_vec_ok(int H, std::initializer_list<const void*> arrays);
hipError_t launch_pre_norm(const void* x, bool f32, const float* w, float eps, int T, int H,
                           const NormForm& f, hipStream_t s);
hipError_t launch_post_norm(const PostNormArgs& a, hipStream_t s);
hipError_t launch_pre_norm_backward(const PreNormBwdArgs& a, hipStream_t s);
hipError_t launch_post_norm_backward(const PostNormBwdArgs& a, hipStream_t s);

}  // namespace qmoe
