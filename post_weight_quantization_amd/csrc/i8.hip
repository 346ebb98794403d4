// Product in 8-bit integers with a scale for each token and each channel.
//
//   s_t  = clip max_k |x_tk| / 127,  a_tk = clamp(rint(x_tk / s_t), -127, 127)
//   y_to = s_t w_o (sum_k a_tk (q_ok - z_o)) + b_o
//
// The sum is integer arithmetic on the matrix cores: |a (q - z)| <= 127 * 255
// and d_in <= 65536 keep it inside an int32, so it is exact and its order does
// not matter (sum a q and z sum a may each wrap; their difference does not).
// The scales and the bias are applied in fp32, and y is rounded once.
//
// Code rows (tokens and channels alike) are padded with zeros to a multiple of
// 128 bytes, so the products read whole rows without a tail.
#include "kq_internal.h"

namespace kq {

typedef int v4i __attribute__((ext_vector_type(4)));

namespace {

constexpr int I8_PAD = 128;  // code rows are padded to this many bytes

__device__ inline float bf16_f32(uint16_t v) { return __uint_as_float(uint32_t(v) << 16); }

// nearest even; a NaN stays a NaN
__device__ inline uint16_t f32_bf16(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return uint16_t((u >> 16) | 0x40);
  return uint16_t((u + 0x7fff + ((u >> 16) & 1)) >> 16);
}

template <class T>
__device__ inline float load_f32(const T* p);
template <>
__device__ inline float load_f32<uint16_t>(const uint16_t* p) { return bf16_f32(*p); }
template <>
__device__ inline float load_f32<float>(const float* p) { return *p; }

__device__ inline void store_y(uint16_t* p, float v) { *p = f32_bf16(v); }
__device__ inline void store_y(float* p, float v) { *p = v; }

// the code of one value; s > 0 and finite
__device__ inline int i8_code(float v, float s) {
  return int(fminf(fmaxf(rintf(v / s), -127.f), 127.f));
}

// One workgroup per row: largest magnitude, then codes and their sum. A row
// with a NaN or an infinity gets scale NaN and codes 0, so that its products
// are NaN; one whose scale is 0 gets codes 0.
template <class T>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const T* __restrict__ x, int64_t d, int64_t ldx,
                                                            int64_t row_bytes, float clip,
                                                            int8_t* __restrict__ codes,
                                                            float* __restrict__ scale,
                                                            int32_t* __restrict__ sums) {
  __shared__ float pm[4];
  __shared__ int pn[4], ps[4];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const int64_t row = blockIdx.x;
  const T* xr = x + row * ldx;
  float m = 0.f;
  int bad = 0;
  for (int64_t k = t; k < d; k += 256) {
    const float v = fabsf(load_f32(xr + k));
    bad |= !(v < __builtin_inff());
    m = fmaxf(m, v);
  }
  for (int o = 32; o > 0; o >>= 1) {
    m = fmaxf(m, __shfl_xor(m, o));
    bad |= __shfl_xor(bad, o);
  }
  if (lane == 0) pm[w] = m, pn[w] = bad;
  __syncthreads();
  m = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
  bad = pn[0] | pn[1] | pn[2] | pn[3];
  const float s = bad ? __builtin_nanf("") : clip * m / 127.f;
  int8_t* cr = codes + row * row_bytes;
  int sum = 0;
  for (int64_t k = t; k < row_bytes; k += 256) {
    const int c = k < d && s > 0.f ? i8_code(load_f32(xr + k), s) : 0;
    cr[k] = int8_t(c);
    sum += c;
  }
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  if (lane == 0) ps[w] = sum;
  __syncthreads();
  if (t == 0) {
    scale[row] = s;
    sums[row] = ps[0] + ps[1] + ps[2] + ps[3];
  }
}

// codes of the sweep (0 .. 255) as signed bytes q - 128, rows padded with 0
__global__ __launch_bounds__(256) void pack_i8_kernel(const uint8_t* __restrict__ codes,
                                                      const float* __restrict__ zero, int64_t d,
                                                      int64_t row_bytes, int8_t* __restrict__ packed,
                                                      float* __restrict__ zero_out) {
  const int64_t row = blockIdx.x;
  for (int64_t k = threadIdx.x; k < row_bytes; k += 256)
    packed[row * row_bytes + k] = k < d ? int8_t(int(codes[row * d + k]) - 128) : int8_t(0);
  if (threadIdx.x == 0) zero_out[row] = zero[row] - 128.f;
}

struct I8Epi {
  const float* a_scale;
  const int32_t* a_sum;
  const float* w_scale;
  const float* w_zero;  // NULL: symmetric
  const float* bias;    // NULL: none
  int64_t n, m, ldy;
};

template <class Y>
__device__ inline void i8_finish(const I8Epi& e, int64_t t, int64_t o, int acc, Y* y) {
  if (e.w_zero) acc -= int(rintf(e.w_zero[o])) * e.a_sum[t];
  float v = float(acc) * e.a_scale[t] * e.w_scale[o];
  if (e.bias) v += e.bias[o];
  store_y(y + t * e.ldy + o, v);
}

// One wave per 16 tokens x 16 channels, operands straight from memory.
// v_mfma_i32_16x16x64_i8: lane 16 g + i holds 16 bytes of row i (A: channel,
// B: token) at k = 16 g; register r of the result is channel 4 g + r of
// token i.
template <class Y>
__global__ __launch_bounds__(256) void matmul_i8_kernel(const int8_t* __restrict__ a,
                                                        const int8_t* __restrict__ w, int64_t row_bytes,
                                                        I8Epi e, Y* __restrict__ y) {
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int64_t t0 = int64_t(blockIdx.x) * 16;
  const int64_t o0 = (int64_t(blockIdx.y) * 4 + (threadIdx.x >> 6)) * 16;
  if (o0 >= e.m) return;
  const int64_t tr = min(t0 + i, e.n - 1), wr = min(o0 + i, e.m - 1);
  const int8_t* ap = a + tr * row_bytes + 16 * g;
  const int8_t* wp = w + wr * row_bytes + 16 * g;
  v4i acc = {0, 0, 0, 0};
  for (int64_t k = 0; k < row_bytes; k += 64)
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(*reinterpret_cast<const v4i*>(wp + k),
                                                *reinterpret_cast<const v4i*>(ap + k), acc, 0, 0, 0);
  if (t0 + i >= e.n) return;
  for (int r = 0; r < 4; ++r)
    if (o0 + 4 * g + r < e.m) i8_finish(e, t0 + i, o0 + 4 * g + r, acc[r], y);
}

}  // namespace

int64_t i8_row_bytes(int64_t d_in) { return cdiv(d_in, I8_PAD) * I8_PAD; }

kq_status quantize_rows_run(const void* x, kq_dtype dt, int64_t n, int64_t d, int64_t ldx, float clip,
                            int8_t* codes, float* scale, int32_t* sums, hipStream_t s) {
  const int64_t rb = i8_row_bytes(d);
  if (dt == KQ_BF16)
    quantize_rows_kernel<<<unsigned(n), 256, 0, s>>>(static_cast<const uint16_t*>(x), d, ldx, rb, clip, codes,
                                                     scale, sums);
  else
    quantize_rows_kernel<<<unsigned(n), 256, 0, s>>>(static_cast<const float*>(x), d, ldx, rb, clip, codes,
                                                     scale, sums);
  KQ_HIP(hipGetLastError());
  return KQ_OK;
}

kq_status pack_i8_run(const uint8_t* codes, const float* zero, int64_t d_out, int64_t d_in, int8_t* packed,
                      float* zero_out, hipStream_t s) {
  pack_i8_kernel<<<unsigned(d_out), 256, 0, s>>>(codes, zero, d_in, i8_row_bytes(d_in), packed, zero_out);
  KQ_HIP(hipGetLastError());
  return KQ_OK;
}

size_t matmul_i8_ws_bytes(int64_t, int64_t, int64_t) { return 0; }

kq_status matmul_i8_run(const int8_t* a, const float* a_scale, const int32_t* a_sum, const int8_t* w,
                        const float* w_scale, const float* w_zero, const float* bias, int64_t n, int64_t m,
                        int64_t d, void* y, kq_dtype dt, int64_t ldy, Arena&, hipStream_t s) {
  const int64_t rb = i8_row_bytes(d);
  const I8Epi e{a_scale, a_sum, w_scale, w_zero, bias, n, m, ldy};
  const dim3 grid(unsigned(cdiv(n, 16)), unsigned(cdiv(m, 64)));
  if (dt == KQ_BF16)
    matmul_i8_kernel<<<grid, 256, 0, s>>>(a, w, rb, e, static_cast<uint16_t*>(y));
  else
    matmul_i8_kernel<<<grid, 256, 0, s>>>(a, w, rb, e, static_cast<float*>(y));
  KQ_HIP(hipGetLastError());
  return KQ_OK;
}

namespace {
struct LinearWs {
  int8_t* codes;
  float* scale;
  int32_t* sums;
};
LinearWs linear_take(Arena& ar, int64_t n, int64_t d) {
  LinearWs w;
  w.codes = ar.take<int8_t>(size_t(n) * i8_row_bytes(d));
  w.scale = ar.take<float>(size_t(n));
  w.sums = ar.take<int32_t>(size_t(n));
  return w;
}
}  // namespace

size_t linear_i8_ws_bytes(int64_t m, int64_t d, int64_t n) {
  Arena ar{nullptr, 0, 0};
  linear_take(ar, n, d);
  ar.take<char>(matmul_i8_ws_bytes(m, d, n));
  return ar.used;
}

kq_status linear_i8_run(const void* x, kq_dtype dt, int64_t ldx, float clip, const int8_t* w,
                        const float* w_scale, const float* w_zero, const float* bias, int64_t n, int64_t m,
                        int64_t d, void* y, kq_dtype ydt, int64_t ldy, Arena& ws, hipStream_t s) {
  const LinearWs l = linear_take(ws, n, d);
  if (!l.codes || !l.scale || !l.sums) return fail(KQ_ERR_WORKSPACE, "linear_i8: workspace too small");
  KQ_TRY(quantize_rows_run(x, dt, n, d, ldx, clip, l.codes, l.scale, l.sums, s));
  return matmul_i8_run(l.codes, l.scale, l.sums, w, w_scale, w_zero, bias, n, m, d, y, ydt, ldy, ws, s);
}

}  // namespace kq
