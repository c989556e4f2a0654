// Host side of the operators around the experts declared in include/qmoe.h:
// argument validation, workspace layout and dispatch.  Nothing here allocates
// device memory or synchronises.
#include <hip/hip_runtime.h>

#include <math.h>

#include "block_internal.h"
#include "qmoe.h"

namespace qmoe {
namespace {

size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool valid_dtype(int32_t d) { return d == QMOE_DT_BF16 || d == QMOE_DT_F32; }
size_t elem(int32_t dtype) { return dtype == QMOE_DT_F32 ? 4 : 2; }
bool valid_eps(float eps) { return eps > 0.0f && std::isfinite(eps); }

// Workspace of qmoe_balance (none for a small batch).
struct BalanceWs {
  size_t psum, csum, nsum, terms, arrived, total;
};
BalanceWs balance_ws_layout(int T, int E) {
  BalanceWs w{};
  if (balance_small(T)) return w;
  const size_t nb = balance_blocks(T);
  w.csum = align_up(nb * E * 4, 256);
  w.nsum = align_up(w.csum + nb * E * 4, 256);
  w.terms = align_up(w.nsum + nb * 4, 256);
  w.arrived = align_up(w.terms + (size_t)((E + 31) / 32) * 8, 256);
  w.total = w.arrived + 256;
  return w;
}

// A tile's rows of K bytes are addressed with 31-bit byte offsets.
constexpr int kMaxK = 1 << 22;

bool valid_form(int32_t form) { return form >= QMOE_FORM_BF16 && form <= QMOE_FORM_E4M3_B128; }
bool form_scaled(int32_t form) { return form >= QMOE_FORM_INT8; }
// `arrays`: those of H columns (nullptr for one that is not given).
qmoe_status check_norm(int32_t dtype, int32_t T, int32_t H, float eps,
                       std::initializer_list<const void*> arrays) {
  if (!valid_dtype(dtype) || T < 0 || H < 1 || !valid_eps(eps)) return QMOE_ERR_INVALID_ARG;
  if (H > norm_max_columns()) return QMOE_ERR_UNSUPPORTED;
  if (H > norm_max_scalar_columns() && !norm_vec_ok(H, arrays)) return QMOE_ERR_UNSUPPORTED;
  return QMOE_OK;
}
bool gate_wide(int32_t kind) { return kind == QMOE_GATE_COLUMN || kind == QMOE_GATE_FULL; }

}  // namespace
}  // namespace qmoe

using namespace qmoe;

extern "C" {

qmoe_status qmoe_fp8_quant(const void* x, int32_t dtype, int32_t B, int32_t M, int32_t K,
                           int32_t block, int32_t act, uint8_t* codes, float* scale,
                           uint8_t* codes_t, float* scale_t, void* stream) {
  if (!valid_dtype(dtype) || B < 0 || M < 0 || K < 1 || block < 0 || block > 1 || act < 0 ||
      act > 1)
    return QMOE_ERR_INVALID_ARG;
  if ((!block && B > 1) || (block && act)) return QMOE_ERR_INVALID_ARG;
  if ((codes == nullptr) != (scale == nullptr) || (codes_t == nullptr) != (scale_t == nullptr))
    return QMOE_ERR_INVALID_ARG;
  if (B > 65535 || M > 65535 * 128 || K > (1 << 29)) return QMOE_ERR_UNSUPPORTED;
  if (B == 0 || M == 0) return QMOE_OK;
  if (x == nullptr || (codes == nullptr && codes_t == nullptr)) return QMOE_ERR_INVALID_ARG;
  if (!aligned(x, elem(dtype)) || !aligned(codes, 16) || !aligned(codes_t, 16) ||
      !aligned(scale, 4) || !aligned(scale_t, 4))
    return QMOE_ERR_INVALID_ARG;
  const Fp8QuantArgs a{x, dtype == QMOE_DT_F32, block != 0, act != 0, B,      M,
                       K, codes,                scale,      codes_t,  scale_t};
  return hip_status(launch_fp8_quant(a, (hipStream_t)stream));
}

size_t qmoe_fp8_matmul_workspace(int32_t M, int32_t N, int32_t K) {
  if (M < 0 || N < 1 || K < 128 || K % 128 != 0) return 0;
  return align_up(fp8_matmul_parts_bytes(M, N, K), 256);
}

qmoe_status qmoe_fp8_matmul(const uint8_t* a, const float* a_scale, const uint8_t* b,
                            const float* b_scale, int32_t b_block, int32_t M, int32_t N,
                            int32_t K, void* out, int32_t out_dtype, void* ws, size_t ws_bytes,
                            void* stream) {
  if (M < 0 || N < 1 || K < 128 || K % 128 != 0 || b_block < 0 || b_block > 1 ||
      !valid_dtype(out_dtype))
    return QMOE_ERR_INVALID_ARG;
  if (M > (1 << 24) || N > (1 << 24) || K > kMaxK) return QMOE_ERR_UNSUPPORTED;
  if (M == 0) return QMOE_OK;
  if (!a || !a_scale || !b || !b_scale || !out) return QMOE_ERR_INVALID_ARG;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(a_scale, 4) || !aligned(b_scale, 4) ||
      !aligned(out, elem(out_dtype)))
    return QMOE_ERR_INVALID_ARG;
  const size_t need = qmoe_fp8_matmul_workspace(M, N, K);
  if (need > 0 && (!ws || ws_bytes < need || !aligned(ws, 256))) return QMOE_ERR_INVALID_ARG;
  Fp8MatmulArgs g{};
  g.a = a;
  g.a_scale = a_scale;
  g.b = b;
  g.b_scale = b_scale;
  g.out = out;
  g.M = g.Ma = M;
  g.N = N;
  g.K = K;
  g.KB = K / 128;
  g.b_block = b_block != 0;
  g.out_f32 = out_dtype == QMOE_DT_F32;
  g.parts = reinterpret_cast<float*>(ws);
  return hip_status(launch_fp8_matmul(g, (hipStream_t)stream));
}

qmoe_status qmoe_fp8_grouped_matmul(const uint8_t* a, const float* a_scale, int32_t pair_rows,
                                    const uint8_t* b, const float* b_scale,
                                    const int32_t* sorted_pair_ids, const int32_t* tile_expert,
                                    const int32_t* expert_offsets, const int32_t* num_padded,
                                    int32_t T, int32_t k, int32_t E,
                                    int32_t block_m, int32_t N, int32_t K, void* out,
                                    int32_t out_dtype, void* stream) {
  if (T < 0 || k < 1 || E < 1 || k > E || N < 1 || K < 128 || K % 128 != 0 || pair_rows < 0 ||
      pair_rows > 1 || !valid_dtype(out_dtype))
    return QMOE_ERR_INVALID_ARG;
  if (block_m != 16 && block_m != 32 && block_m != 64 && block_m != 128)
    return QMOE_ERR_INVALID_ARG;
  if ((long long)T * k > (1ll << 30)) return QMOE_ERR_INVALID_ARG;
  if (E > 1024 || N > (1 << 24) || K > kMaxK) return QMOE_ERR_UNSUPPORTED;
  // Gathered rows are addressed with 32-bit byte offsets below 3 GiB (the
  // kernel's offset of no row).
  if ((uint64_t)T * (pair_rows ? k : 1) * K > (3ull << 30)) return QMOE_ERR_UNSUPPORTED;
  if (T == 0) return QMOE_OK;
  if (!a || !a_scale || !b || !b_scale || !sorted_pair_ids || !tile_expert || !expert_offsets ||
      !num_padded || !out)
    return QMOE_ERR_INVALID_ARG;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(a_scale, 4) || !aligned(b_scale, 4) ||
      !aligned(out, elem(out_dtype)))
    return QMOE_ERR_INVALID_ARG;
  Fp8MatmulArgs g{};
  g.a = a;
  g.a_scale = a_scale;
  g.b = b;
  g.b_scale = b_scale;
  g.out = out;
  g.M = (int)qmoe_align_capacity(T, k, E, block_m);
  g.Ma = pair_rows ? T * k : T;
  g.N = N;
  g.K = K;
  g.KB = K / 128;
  g.b_block = true;
  g.out_f32 = out_dtype == QMOE_DT_F32;
  g.sorted = sorted_pair_ids;
  g.tile_expert = tile_expert;
  g.expert_offsets = expert_offsets;
  g.num_padded = num_padded;
  g.P = T * k;
  g.k = k;
  g.block_m = block_m;
  g.E = E;
  g.pair_rows = pair_rows != 0;
  return hip_status(launch_fp8_grouped_matmul(g, (hipStream_t)stream));
}

size_t qmoe_balance_workspace(int32_t T, int32_t E) {
  if (T < 0 || E < 1) return 0;
  return balance_ws_layout(T, E).total;
}

qmoe_status qmoe_balance(const float* logits, const int32_t* topk_ids, const uint8_t* mask,
                         int32_t T, int32_t E, int32_t k, float coef, float* loss,
                         int32_t* counts, float* probs, int32_t* tokens, void* ws,
                         size_t ws_bytes, void* stream) {
  if (T < 0 || E < 1 || k < 1 || k > E || k > 16 || !std::isfinite(coef))
    return QMOE_ERR_INVALID_ARG;
  if ((long long)T * k > (1ll << 30)) return QMOE_ERR_INVALID_ARG;
  if (E > 1024) return QMOE_ERR_UNSUPPORTED;
  if ((T > 0 && (!logits || !topk_ids)) || !loss || !counts || !probs || !tokens)
    return QMOE_ERR_INVALID_ARG;
  const BalanceWs lay = balance_ws_layout(T, E);
  if (lay.total > 0 && (!ws || ws_bytes < lay.total || !aligned(ws, 256)))
    return QMOE_ERR_INVALID_ARG;
  uint8_t* w = reinterpret_cast<uint8_t*>(ws);
  const BalanceParts parts{reinterpret_cast<float*>(w + lay.psum),
                           reinterpret_cast<int32_t*>(w + lay.csum),
                           reinterpret_cast<int32_t*>(w + lay.nsum),
                           reinterpret_cast<double*>(w + lay.terms),
                           reinterpret_cast<int32_t*>(w + lay.arrived)};
  return hip_status(launch_balance(logits, topk_ids, mask, T, E, k, coef, loss, counts, probs,
                                   tokens, parts, (hipStream_t)stream));
}

qmoe_status qmoe_balance_backward(const float* logits, const uint8_t* mask, const int32_t* counts,
                                  const int32_t* tokens, const float* dloss, int32_t T, int32_t E,
                                  int32_t k, float coef, float* dlogits, void* stream) {
  if (T < 0 || E < 1 || k < 1 || k > E || k > 16 || !std::isfinite(coef))
    return QMOE_ERR_INVALID_ARG;
  if ((long long)T * k > (1ll << 30)) return QMOE_ERR_INVALID_ARG;
  if (E > 1024) return QMOE_ERR_UNSUPPORTED;
  if (T == 0) return QMOE_OK;
  if (!logits || !counts || !tokens || !dloss || !dlogits) return QMOE_ERR_INVALID_ARG;
  return hip_status(launch_balance_backward(logits, mask, counts, tokens, dloss, T, E, k, coef,
                                            dlogits, (hipStream_t)stream));
}

qmoe_status qmoe_pre_norm(const void* x, int32_t dtype, const float* w, float eps, int32_t T,
                          int32_t H, int32_t form, void* n, float* scale, void* stream) {
  const qmoe_status st = check_norm(dtype, T, H, eps, {x, w, n});
  if (st != QMOE_OK) return st;
  if (!valid_form(form)) return QMOE_ERR_INVALID_ARG;
  if (T == 0) return QMOE_OK;
  if (!x || !w || !n || (form_scaled(form) && !scale)) return QMOE_ERR_INVALID_ARG;
  return hip_status(launch_pre_norm(x, dtype == QMOE_DT_F32, w, eps, T, H,
                                    NormForm{form, n, scale}, (hipStream_t)stream));
}

size_t qmoe_norm_backward_workspace(int32_t H) {
  if (H < 1 || H > norm_max_columns()) return 0;
  return align_up((size_t)2 * norm_partial_rows() * H * 4, 256);
}

qmoe_status qmoe_pre_norm_backward(const void* dn, const void* x, int32_t dtype, const float* w,
                                   float eps, const void* dres, int32_t T, int32_t H, void* dx,
                                   float* dw, void* ws, size_t ws_bytes, void* stream) {
  const qmoe_status st = check_norm(dtype, T, H, eps, {dn, x, w, dres, dx});
  if (st != QMOE_OK) return st;
  if ((T > 0 && (!dn || !x || !w || !dx)) || !dw || !ws) return QMOE_ERR_INVALID_ARG;
  if (ws_bytes < qmoe_norm_backward_workspace(H) || !aligned(ws, 256))
    return QMOE_ERR_INVALID_ARG;
  const PreNormBwdArgs a{dn, x, dtype == QMOE_DT_F32, w, dres, eps, T, H, dx, dw,
                         reinterpret_cast<float*>(ws)};
  return hip_status(launch_pre_norm_backward(a, (hipStream_t)stream));
}

static bool gate_ok(int32_t kind, const void* gate, int32_t T) {
  return kind == QMOE_GATE_NONE || gate != nullptr || T == 0;
}

qmoe_status qmoe_post_norm(const void* y, const void* x, int32_t dtype, const float* w,
                           const void* gate, int32_t gate_kind, float alpha, float eps, int32_t T,
                           int32_t H, void* out, const float* next_w, int32_t form, void* n,
                           float* scale, void* stream) {
  const qmoe_status st = check_norm(
      dtype, T, H, eps,
      {y, x, w, out, gate_wide(gate_kind) ? gate : nullptr, next_w, next_w ? n : nullptr});
  if (st != QMOE_OK) return st;
  if (gate_kind < QMOE_GATE_NONE || gate_kind > QMOE_GATE_FULL || !std::isfinite(alpha))
    return QMOE_ERR_INVALID_ARG;
  if (next_w && !valid_form(form)) return QMOE_ERR_INVALID_ARG;
  if (T == 0) return QMOE_OK;
  if (!y || !x || !w || !out || !gate_ok(gate_kind, gate, T)) return QMOE_ERR_INVALID_ARG;
  if (next_w && (!n || (form_scaled(form) && !scale))) return QMOE_ERR_INVALID_ARG;
  const PostNormArgs a{y, x, dtype == QMOE_DT_F32, w, gate, gate_kind, alpha, eps, T, H, out,
                       next_w, NormForm{form, n, scale}};
  return hip_status(launch_post_norm(a, (hipStream_t)stream));
}

qmoe_status qmoe_post_norm_backward(const void* dout, const void* y, int32_t dtype,
                                    const float* w, const void* gate, int32_t gate_kind,
                                    float alpha, float eps, int32_t T, int32_t H, void* dy,
                                    void* dres, float* dw, void* dgate, void* ws, size_t ws_bytes,
                                    void* stream) {
  const qmoe_status st = check_norm(dtype, T, H, eps,
                                    {dout, y, w, dy, dres, gate_wide(gate_kind) ? gate : nullptr,
                                     gate_wide(gate_kind) ? dgate : nullptr});
  if (st != QMOE_OK) return st;
  if (gate_kind < QMOE_GATE_NONE || gate_kind > QMOE_GATE_FULL || !std::isfinite(alpha))
    return QMOE_ERR_INVALID_ARG;
  if ((T > 0 && (!dout || !y || !w || !dy || !dres)) || !dw || !ws || !gate_ok(gate_kind, gate, T))
    return QMOE_ERR_INVALID_ARG;
  if (gate_kind != QMOE_GATE_NONE && !dgate && (T > 0 || gate_kind == QMOE_GATE_COLUMN))
    return QMOE_ERR_INVALID_ARG;
  if (ws_bytes < qmoe_norm_backward_workspace(H) || !aligned(ws, 256))
    return QMOE_ERR_INVALID_ARG;
  const PostNormBwdArgs a{dout, y,  dtype == QMOE_DT_F32, w,     gate,
                          gate_kind, alpha, eps,          T,     H,
                          dy,   dres, dw,                 dgate, reinterpret_cast<float*>(ws)};
  return hip_status(launch_post_norm_backward(a, (hipStream_t)stream));
}

}  // extern "C"
