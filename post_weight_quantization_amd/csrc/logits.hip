// A teacher's top logits, and the distillation loss on them with its gradient.
//
// top_logits: the K largest logits of each row in descending order, ties to
// the lowest index, and the row's log sum exp(l / T).
//
// distill: with q = softmax(s / T) over the vocabulary and the teacher's
// probabilities p_k of its K listed columns (renormalised over the list, or
// exp(t_k / T - Z_t) with everything off the list as one bucket of mass
// r = 1 - sum p against the student's q_r),
//   L = w T^2 [ sum_k p_k (log p_k - log q_k) + r (log r - log q_r) ]
//   dL/ds_j = w T [ c_j q_j - p_j ],   c_j = P on the list, P - r / q_r off it,
//   P = sum p + r.
// What decides a small loss is kept from cancelling: the largest logit goes
// off before the scaling, and q_r is summed over the columns off the list
// (a bit per column in LDS says which are on it), never as 1 - sum q.
#include "kq_internal.h"

namespace kq {

namespace {

constexpr int TPB = 1024;             // threads per row
constexpr int NW = TPB / 64;
constexpr int K_MAX = 256;            // longest list
constexpr int64_t V_MAX = 1 << 19;    // largest vocabulary of the distillation (its bits fill 64 KB)
constexpr double REST_MIN = 1.0 / 65536.0;

__device__ inline float bf16_f32(uint16_t v) { return __uint_as_float(uint32_t(v) << 16); }
__device__ inline uint16_t f32_bf16(float f) {
  const uint32_t u = __float_as_uint(f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return uint16_t((u >> 16) | 0x40);
  return uint16_t((u + 0x7fff + ((u >> 16) & 1)) >> 16);
}
__device__ inline float load_f32(const uint16_t* p) { return bf16_f32(*p); }
__device__ inline float load_f32(const float* p) { return *p; }
__device__ inline void store_f32(uint16_t* p, float v) { *p = f32_bf16(v); }
__device__ inline void store_f32(float* p, float v) { *p = v; }

// Order of logits as unsigned keys: -inf lowest, both zeros equal, a NaN
// above everything.
__device__ inline uint32_t key_of(float v) {
  if (v != v) return 0xffffffffu;
  if (v == 0.f) v = 0.f;
  const uint32_t u = __float_as_uint(v);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <class T, class F>
__device__ inline T block_reduce(T v, T* part, F f) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = f(v, T(__shfl_xor(v, o)));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  T r = part[0];
  for (int w = 1; w < NW; ++w) r = f(r, part[w]);
  return r;
}

__device__ inline float fmax_nan(float a, float b) { return a > b || a != a ? a : b; }

struct Sum {
  template <class T>
  __device__ T operator()(T a, T b) const { return a + b; }
};
struct Max {
  __device__ float operator()(float a, float b) const { return fmax_nan(a, b); }
};

// One workgroup per row, K rounds of a block-wide maximum over (key, lowest
// index) below the last one taken.
template <class T>
__global__ __launch_bounds__(TPB) void top_logits_kernel(const T* __restrict__ logits, int64_t vocab,
                                                         int64_t ld, int k, float inv_t,
                                                         float* __restrict__ values,
                                                         int32_t* __restrict__ index,
                                                         float* __restrict__ lse) {
  __shared__ uint64_t part[NW];
  __shared__ float fpart[NW];
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x;
  const T* lr = logits + row * ld;
  // (key, ~index): larger is earlier
  uint64_t last = ~uint64_t(0);
  bool first = true;
  float top = 0.f;
  for (int r = 0; r < k; ++r) {
    uint64_t best = 0;
    for (int64_t j = t; j < vocab; j += TPB) {
      const uint64_t c = uint64_t(key_of(load_f32(lr + j))) << 32 | uint32_t(~uint32_t(j));
      if ((first || c < last) && c > best) best = c;
    }
    best = block_reduce(best, part, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
    const int64_t j = uint32_t(~uint32_t(best));
    const float v = load_f32(lr + j);
    if (first) top = v;
    if (t == 0) {
      values[row * k + r] = v;
      index[row * k + r] = int32_t(j);
    }
    last = best;
    first = false;
  }
  if (!lse) return;
  const float m = top == -__builtin_inff() ? 0.f : top;
  float s = 0.f;
  for (int64_t j = t; j < vocab; j += TPB) s += __expf((load_f32(lr + j) - m) * inv_t);
  s = block_reduce(s, fpart, Sum());
  if (t == 0) lse[row] = m * inv_t + logf(s);
}

struct DistillArgs {
  int64_t vocab, ld, ldg;
  const float* t_values;
  const int32_t* t_index;
  const float* t_lse;   // NULL: renormalise over the list
  int k;
  float temperature;
  const float* weight;  // NULL: ones
  float* loss;
  float* stats;         // n x 3: largest logit m, log sum exp((s - m) / T), log of the mass off the list
};

// One workgroup per row; the logits are read once for the largest, once for
// the sums and once for the gradient.
template <class T, bool LOSS, bool GRAD>
__global__ __launch_bounds__(TPB) void distill_kernel(const T* logits, DistillArgs d, T* grad) {
  extern __shared__ uint32_t bits[];  // a bit per column: on the list
  __shared__ double dpart[NW];
  __shared__ float fpart[NW];
  __shared__ float p_at[K_MAX];
  __shared__ int idx_at[K_MAX];
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x;
  const T* lr = logits + row * d.ld;
  T* gr = GRAD ? grad + row * d.ldg : nullptr;
  const float w = d.weight ? d.weight[row] : 1.f;
  const float inv_t = 1.f / d.temperature;
  if (w == 0.f) {  // a row without weight is not read
    if (GRAD)
      for (int64_t j = t; j < d.vocab; j += TPB) store_f32(gr + j, 0.f);
    if (LOSS && t == 0) d.loss[row] = 0.f;
    if (LOSS && d.stats && t < 3) d.stats[3 * row + t] = 0.f;
    return;
  }
  const int words = int(cdiv(d.vocab, 32));
  for (int j = t; j < words; j += TPB) bits[j] = 0;
  __syncthreads();
  // the teacher's side, in 64 bits: a small remainder 1 - sum p has to hold
  int idx = -1;
  double tv = -__builtin_inf();
  if (t < d.k) {
    idx = d.t_index[row * d.k + t];
    if (idx < 0 || idx >= d.vocab) idx = -1;
    idx_at[t] = idx;
    if (idx >= 0) {
      atomicOr(&bits[idx >> 5], 1u << (idx & 31));
      tv = double(d.t_values[row * d.k + t]) / double(d.temperature);
    }
  }
  double log_z, rest = 0.0;
  if (d.t_lse) {
    log_z = double(d.t_lse[row]);
  } else {
    double m = block_reduce(tv, dpart, [](double a, double b) { return a > b || a != a ? a : b; });
    if (m == -__builtin_inf()) m = 0.0;
    const double s = block_reduce(idx >= 0 ? exp(tv - m) : 0.0, dpart, Sum());
    log_z = s == 0.0 ? 0.0 : m + log(s);
  }
  const double log_p = tv - log_z;
  const double p = idx >= 0 ? exp(log_p) : 0.0;
  double mass = block_reduce(p, dpart, Sum());
  if (d.t_lse) {
    rest = 1.0 - mass;
    if (rest <= REST_MIN) rest = 0.0;
    mass += rest;
  }
  if (t < d.k) p_at[t] = float(p);
  __syncthreads();
  // the student's side
  float m = -__builtin_inff(), log_total = 0.f, off = 0.f;
  double log_off;
  if (LOSS) {
    for (int64_t j = t; j < d.vocab; j += TPB) m = fmax_nan(m, load_f32(lr + j));
    m = block_reduce(m, fpart, Max());
    if (m == -__builtin_inff()) m = 0.f;
    float on = 0.f;
    for (int64_t j = t; j < d.vocab; j += TPB) {
      const float e = __expf((load_f32(lr + j) - m) * inv_t);
      if (bits[j >> 5] >> (j & 31) & 1) on += e;
      else off += e;
    }
    off = block_reduce(off, fpart, Sum());
    on = block_reduce(on, fpart, Sum());
    const float total = on + off;
    // a row without a finite logit has q = 0 and log q = -inf
    log_total = total == 0.f ? 0.f : logf(total);
    log_off = total == 0.f ? -__builtin_inf() : log(double(off) / double(total));
    double term = 0.0;
    if (p > 0.0) {
      const float z = (load_f32(lr + idx) - m) * inv_t;
      term = p * (log_p - (double(z) - (total == 0.f ? 0.0 : log(double(total)))));
    }
    term = block_reduce(term, dpart, Sum());
    if (rest > 0.0) term += rest * (log(rest) - log_off);
    if (t == 0) {
      d.loss[row] = float(double(w) * d.temperature * d.temperature * term);
      if (d.stats) {
        d.stats[3 * row] = m;
        d.stats[3 * row + 1] = log_total;
        d.stats[3 * row + 2] = float(log_off);
      }
    }
  } else {
    m = d.stats[3 * row];
    log_total = d.stats[3 * row + 1];
    log_off = double(d.stats[3 * row + 2]);
  }
  if (!GRAD) return;
  const float gain = w * d.temperature;
  const float c_on = float(mass);
  const float c_off = rest > 0.0 && log_off > -__builtin_inf() ? float(mass - rest * exp(-log_off)) : c_on;
  for (int64_t j = t; j < d.vocab; j += TPB) {
    const float z = load_f32(lr + j);
    const float q = __expf((z - m) * inv_t - log_total);
    float g = q * ((bits[j >> 5] >> (j & 31) & 1) ? c_on : c_off);
    if (bits[j >> 5] >> (j & 31) & 1)
      for (int l = 0; l < d.k; ++l)
        if (idx_at[l] == j) g -= p_at[l];
    store_f32(gr + j, g * gain);
  }
}

template <class T>
kq_status distill_launch(const void* logits, int64_t n, const DistillArgs& d, void* grad, bool loss,
                         hipStream_t s) {
  const T* l = static_cast<const T*>(logits);
  T* g = static_cast<T*>(grad);
  const unsigned lds = unsigned(cdiv(d.vocab, 32) * 4);
  auto go = [&](auto kernel) -> kq_status {
    if (lds > 49152)
      KQ_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                 hipFuncAttributeMaxDynamicSharedMemorySize, int(lds)));
    kernel<<<unsigned(n), TPB, lds, s>>>(l, d, g);
    KQ_HIP(hipGetLastError());
    return KQ_OK;
  };
  if (loss && grad) return go(distill_kernel<T, true, true>);
  if (loss) return go(distill_kernel<T, true, false>);
  return go(distill_kernel<T, false, true>);
}

}  // namespace

int64_t distill_max_vocab() { return V_MAX; }
int32_t logits_max_k() { return K_MAX; }

kq_status top_logits_run(const void* logits, kq_dtype dt, int64_t n, int64_t vocab, int64_t ld, int k,
                         float temperature, float* values, int32_t* index, float* lse, hipStream_t s) {
  const float inv_t = 1.f / temperature;
  if (dt == KQ_BF16)
    top_logits_kernel<<<unsigned(n), TPB, 0, s>>>(static_cast<const uint16_t*>(logits), vocab, ld, k, inv_t,
                                                  values, index, lse);
  else
    top_logits_kernel<<<unsigned(n), TPB, 0, s>>>(static_cast<const float*>(logits), vocab, ld, k, inv_t,
                                                  values, index, lse);
  KQ_HIP(hipGetLastError());
  return KQ_OK;
}

kq_status distill_run(const void* logits, kq_dtype dt, int64_t n, int64_t vocab, int64_t ld,
                      const float* t_values, const int32_t* t_index, const float* t_lse, int k,
                      float temperature, const float* weight, float* loss, float* stats, void* grad,
                      int64_t ldg, hipStream_t s) {
  const DistillArgs d{vocab, ld, ldg, t_values, t_index, t_lse, k, temperature, weight, loss, stats};
  if (dt == KQ_BF16) return distill_launch<uint16_t>(logits, n, d, grad, loss != nullptr, s);
  return distill_launch<float>(logits, n, d, grad, loss != nullptr, s);
}

}  // namespace kq
