// C ABI of the 8-bit product, the teacher's top logits and the distillation
// loss: argument validation on the host, then the kernels on the caller's
// stream.
#include <cmath>
#include <limits>

#include "kq_internal.h"

using namespace kq;

namespace {

constexpr int64_t ROWS_MAX = 1 << 20;
constexpr int64_t D_IN_MAX = 65536;  // 127 * 255 * d_in stays below 2^31

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t elem(kq_dtype dt) { return dt == KQ_BF16 ? 2 : 4; }
bool bad_dtype(kq_dtype dt) { return dt != KQ_BF16 && dt != KQ_F32; }

kq_status check_scratch(const void* ws, size_t have, size_t need, const char* who) {
  if (need == 0) return KQ_OK;
  if (!ws || have < need)
    return fail(KQ_ERR_WORKSPACE, "%s: workspace of %zu bytes required, got %zu", who, need, ws ? have : size_t(0));
  if (!aligned(ws, 16)) return fail(KQ_ERR_ARG, "%s: workspace must be 16-byte aligned", who);
  return KQ_OK;
}

kq_status check_i8_sizes(int64_t n, int64_t d_out, int64_t d_in, const char* who) {
  if (n < 0 || n > ROWS_MAX) return fail(KQ_ERR_SHAPE, "%s: 0 <= n_tok <= 1048576", who);
  if (d_out < 1 || d_out > ROWS_MAX) return fail(KQ_ERR_SHAPE, "%s: 1 <= d_out <= 1048576", who);
  if (d_in < 1 || d_in > D_IN_MAX) return fail(KQ_ERR_SHAPE, "%s: 1 <= d_in <= 65536", who);
  return KQ_OK;
}

// the checks that a product shares, given tokens or their codes
kq_status check_product(const int8_t* w, const float* w_scale, int64_t d_out, const void* y, kq_dtype dt,
                        int64_t ldy, const char* who) {
  if (!w || !w_scale || !y) return fail(KQ_ERR_ARG, "%s: NULL argument", who);
  if (bad_dtype(dt)) return fail(KQ_ERR_ARG, "%s: bad dtype %d of y", who, int(dt));
  if (ldy < d_out) return fail(KQ_ERR_SHAPE, "%s: ldy must be at least d_out", who);
  if (!aligned(w, 16)) return fail(KQ_ERR_ARG, "%s: codes must be 16-byte aligned", who);
  if (!aligned(y, elem(dt))) return fail(KQ_ERR_ARG, "%s: y must be aligned to its type", who);
  return KQ_OK;
}

kq_status check_logits(kq_dtype dt, int64_t n, int64_t vocab, int64_t ld, int32_t k, float temperature,
                       const char* who) {
  if (bad_dtype(dt)) return fail(KQ_ERR_ARG, "%s: bad dtype %d", who, int(dt));
  if (n < 0 || n > ROWS_MAX) return fail(KQ_ERR_SHAPE, "%s: 0 <= n <= 1048576", who);
  if (vocab < 1 || ld < vocab) return fail(KQ_ERR_SHAPE, "%s: 1 <= vocab <= ld", who);
  if (k < 1 || k > logits_max_k()) return fail(KQ_ERR_SHAPE, "%s: 1 <= k <= %d", who, logits_max_k());
  // (the reciprocal of a smaller number may be infinite)
  if (!(std::isfinite(temperature) && temperature >= std::numeric_limits<float>::min()))
    return fail(KQ_ERR_ARG, "%s: temperature must be finite and at least 2^-126", who);
  return KQ_OK;
}

kq_status check_distill(const void* logits, kq_dtype dt, int64_t n, int64_t vocab, int64_t ld,
                        const float* t_values, const int32_t* t_index, int32_t k, float temperature,
                        const char* who) {
  KQ_TRY(check_logits(dt, n, vocab, ld, k, temperature, who));
  if (vocab > distill_max_vocab())
    return fail(KQ_ERR_UNSUPPORTED, "%s: vocab above %lld", who, (long long)distill_max_vocab());
  if (n == 0) return KQ_OK;
  if (!logits || !t_values || !t_index) return fail(KQ_ERR_ARG, "%s: NULL argument", who);
  if (!aligned(logits, elem(dt))) return fail(KQ_ERR_ARG, "%s: logits must be aligned to their type", who);
  return KQ_OK;
}

kq_status check_grad(const void* logits, kq_dtype dt, int64_t vocab, int64_t ld, const void* grad, int64_t ldg,
                     const char* who) {
  if (!grad) return fail(KQ_ERR_ARG, "%s: NULL argument", who);
  if (ldg < vocab) return fail(KQ_ERR_SHAPE, "%s: ldg must be at least vocab", who);
  if (grad == logits && ldg != ld) return fail(KQ_ERR_ARG, "%s: in place, ldg must be ld", who);
  if (!aligned(grad, elem(dt))) return fail(KQ_ERR_ARG, "%s: grad must be aligned to its type", who);
  return KQ_OK;
}

}  // namespace

extern "C" {

kq_status kq_i8_row_bytes(int64_t d_in, int64_t* bytes) {
  clear_error();
  if (!bytes) return fail(KQ_ERR_ARG, "i8_row_bytes: bytes is NULL");
  if (d_in < 1 || d_in > D_IN_MAX) return fail(KQ_ERR_SHAPE, "i8_row_bytes: 1 <= d_in <= 65536");
  *bytes = i8_row_bytes(d_in);
  return KQ_OK;
}

kq_status kq_quantize_rows(const void* x, kq_dtype dt, int64_t n, int64_t d_in, int64_t ldx, float clip,
                           int8_t* codes, float* scale, int32_t* sums, hipStream_t stream) {
  clear_error();
  KQ_TRY(check_i8_sizes(n, 1, d_in, "quantize_rows"));
  if (bad_dtype(dt)) return fail(KQ_ERR_ARG, "quantize_rows: bad dtype %d", int(dt));
  if (!(clip > 0.f && clip <= 1.f)) return fail(KQ_ERR_ARG, "quantize_rows: clip must be in (0, 1]");
  if (ldx < d_in) return fail(KQ_ERR_SHAPE, "quantize_rows: ldx must be at least d_in");
  if (n == 0) return KQ_OK;
  if (!x || !codes || !scale || !sums) return fail(KQ_ERR_ARG, "quantize_rows: NULL argument");
  if (!aligned(x, elem(dt))) return fail(KQ_ERR_ARG, "quantize_rows: x must be aligned to its type");
  if (!aligned(codes, 16)) return fail(KQ_ERR_ARG, "quantize_rows: codes must be 16-byte aligned");
  return quantize_rows_run(x, dt, n, d_in, ldx, clip, codes, scale, sums, stream);
}

kq_status kq_pack_i8(const uint8_t* codes, const float* zero, int64_t d_out, int64_t d_in, int8_t* packed,
                     float* zero_out, hipStream_t stream) {
  clear_error();
  KQ_TRY(check_i8_sizes(1, d_out, d_in, "pack_i8"));
  if (!codes || !zero || !packed || !zero_out) return fail(KQ_ERR_ARG, "pack_i8: NULL argument");
  if (!aligned(packed, 16)) return fail(KQ_ERR_ARG, "pack_i8: packed must be 16-byte aligned");
  return pack_i8_run(codes, zero, d_out, d_in, packed, zero_out, stream);
}

kq_status kq_matmul_i8(const int8_t* a, const float* a_scale, const int32_t* a_sum, const int8_t* w,
                       const float* w_scale, const float* w_zero, const float* bias, int64_t n_tok,
                       int64_t d_out, int64_t d_in, void* y, kq_dtype dt, int64_t ldy, void* ws,
                       size_t ws_bytes, hipStream_t stream) {
  clear_error();
  KQ_TRY(check_i8_sizes(n_tok, d_out, d_in, "matmul_i8"));
  if (n_tok == 0) return KQ_OK;
  KQ_TRY(check_product(w, w_scale, d_out, y, dt, ldy, "matmul_i8"));
  if (!a || !a_scale) return fail(KQ_ERR_ARG, "matmul_i8: NULL argument");
  if (w_zero && !a_sum) return fail(KQ_ERR_ARG, "matmul_i8: w_zero needs a_sum");
  if (!aligned(a, 16)) return fail(KQ_ERR_ARG, "matmul_i8: codes must be 16-byte aligned");
  KQ_TRY(check_scratch(ws, ws_bytes, matmul_i8_ws_bytes(d_out, d_in, n_tok), "matmul_i8"));
  Arena ar{static_cast<char*>(ws), ws_bytes, 0};
  return matmul_i8_run(a, a_scale, a_sum, w, w_scale, w_zero, bias, n_tok, d_out, d_in, y, dt, ldy, ar, stream);
}

kq_status kq_linear_i8(const void* x, kq_dtype dt, int64_t ldx, float clip, const int8_t* w,
                       const float* w_scale, const float* w_zero, const float* bias, int64_t n_tok,
                       int64_t d_out, int64_t d_in, void* y, kq_dtype y_dt, int64_t ldy, void* ws,
                       size_t ws_bytes, hipStream_t stream) {
  clear_error();
  KQ_TRY(check_i8_sizes(n_tok, d_out, d_in, "linear_i8"));
  if (bad_dtype(dt)) return fail(KQ_ERR_ARG, "linear_i8: bad dtype %d of x", int(dt));
  if (!(clip > 0.f && clip <= 1.f)) return fail(KQ_ERR_ARG, "linear_i8: clip must be in (0, 1]");
  if (ldx < d_in) return fail(KQ_ERR_SHAPE, "linear_i8: ldx must be at least d_in");
  if (n_tok == 0) return KQ_OK;
  KQ_TRY(check_product(w, w_scale, d_out, y, y_dt, ldy, "linear_i8"));
  if (!x) return fail(KQ_ERR_ARG, "linear_i8: NULL argument");
  if (!aligned(x, elem(dt))) return fail(KQ_ERR_ARG, "linear_i8: x must be aligned to its type");
  KQ_TRY(check_scratch(ws, ws_bytes, linear_i8_ws_bytes(d_out, d_in, n_tok), "linear_i8"));
  Arena ar{static_cast<char*>(ws), ws_bytes, 0};
  return linear_i8_run(x, dt, ldx, clip, w, w_scale, w_zero, bias, n_tok, d_out, d_in, y, y_dt, ldy, ar, stream);
}

kq_status kq_top_logits(const void* logits, kq_dtype dt, int64_t n, int64_t vocab, int64_t ld, int32_t k,
                        float temperature, float* values, int32_t* index, float* lse, hipStream_t stream) {
  clear_error();
  KQ_TRY(check_logits(dt, n, vocab, ld, k, temperature, "top_logits"));
  if (k > vocab || vocab > (int64_t(1) << 30)) return fail(KQ_ERR_SHAPE, "top_logits: k <= vocab <= 2^30");
  if (n == 0) return KQ_OK;
  if (!logits || !values || !index) return fail(KQ_ERR_ARG, "top_logits: NULL argument");
  if (!aligned(logits, elem(dt))) return fail(KQ_ERR_ARG, "top_logits: logits must be aligned to their type");
  return top_logits_run(logits, dt, n, vocab, ld, k, temperature, values, index, lse, stream);
}

kq_status kq_distill_loss(const void* logits, kq_dtype dt, int64_t n, int64_t vocab, int64_t ld,
                          const float* t_values, const int32_t* t_index, const float* t_lse, int32_t k,
                          float temperature, const float* weight, float* loss, float* stats,
                          hipStream_t stream) {
  clear_error();
  KQ_TRY(check_distill(logits, dt, n, vocab, ld, t_values, t_index, k, temperature, "distill_loss"));
  if (n == 0) return KQ_OK;
  if (!loss) return fail(KQ_ERR_ARG, "distill_loss: NULL argument");
  return distill_run(logits, dt, n, vocab, ld, t_values, t_index, t_lse, k, temperature, weight, loss, stats,
                     nullptr, 0, stream);
}

kq_status kq_distill_grad(const void* logits, kq_dtype dt, int64_t n, int64_t vocab, int64_t ld,
                          const float* t_values, const int32_t* t_index, const float* t_lse, int32_t k,
                          float temperature, const float* stats, const float* dloss, void* grad, int64_t ldg,
                          hipStream_t stream) {
  clear_error();
  KQ_TRY(check_distill(logits, dt, n, vocab, ld, t_values, t_index, k, temperature, "distill_grad"));
  if (n == 0) return KQ_OK;
  if (!stats || !dloss) return fail(KQ_ERR_ARG, "distill_grad: NULL argument");
  KQ_TRY(check_grad(logits, dt, vocab, ld, grad, ldg, "distill_grad"));
  return distill_run(logits, dt, n, vocab, ld, t_values, t_index, t_lse, k, temperature, dloss, nullptr,
                     const_cast<float*>(stats), grad, ldg, stream);
}

kq_status kq_distill_loss_grad(const void* logits, kq_dtype dt, int64_t n, int64_t vocab, int64_t ld,
                               const float* t_values, const int32_t* t_index, const float* t_lse, int32_t k,
                               float temperature, const float* weight, float* loss, float* stats, void* grad,
                               int64_t ldg, hipStream_t stream) {
  clear_error();
  KQ_TRY(check_distill(logits, dt, n, vocab, ld, t_values, t_index, k, temperature, "distill_loss_grad"));
  if (n == 0) return KQ_OK;
  if (!loss) return fail(KQ_ERR_ARG, "distill_loss_grad: NULL argument");
  KQ_TRY(check_grad(logits, dt, vocab, ld, grad, ldg, "distill_loss_grad"));
  return distill_run(logits, dt, n, vocab, ld, t_values, t_index, t_lse, k, temperature, weight, loss, stats,
                     grad, ldg, stream);
}

}  // extern "C"
