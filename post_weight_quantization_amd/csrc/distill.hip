// The distillation loss on a teacher's top logits, and its gradient.
//
// With q = softmax(s / T) over the vocabulary and the teacher's probabilities
// p_k of its K listed columns (renormalised over the list, or
// exp(t_k / T - Z_t) with everything off the list as one bucket of mass
// r = 1 - sum p against the student's q_r),
//   L = w T^2 [ sum_k p_k (log p_k - log q_k) + r (log r - log q_r) ]
//   dL/ds_j = w T [ c_j q_j - p_j ],   c_j = P on the list, P - r / q_r off it,
//   P = sum p + r.
//
// A workgroup takes a row (logits_rows.h). One pass finds the largest logit m'
// off the list and the sum of e_j = exp((s_j - m') / T) there; the K listed
// logits make the sum on it, from a maximum of their own, and both join to
// the sum of the row. e_j again times one factor of the row,
//   w T (P q_r - r) / sum of e off the list,
// is the gradient of every column off the list; the K columns on it
// are written again after a barrier. (Without a bucket every column counts as
// off the list, and the factor is w T P / sum e.) For loss and gradient in one call rows of
// up to 128 KB stay in registers between the passes, so the logits are read
// once and the gradient written once: memory bounds it (4096 x 32000 bf16: 109
// us, 4.8 TB/s; copying runs at 5.2). Longer rows are read twice (8192 x 128256
// bf16: 911 us, 4.6 TB/s of one read and one write, the second read beside
// them). The teacher's side is computed by the first K threads while the row
// is on its way.
//
// What decides a small loss is kept from cancelling: the maxima go off before the
// scaling, e is summed apart for the columns on and off the list (a bit per
// column in LDS says which), never as a difference of sums, and the remainder
// 1 - sum p, the sum of the loss's terms and the factors of the gradient are
// joined in 64 bits. And from vanishing: off the list e is taken against the
// largest there, so q_r may be as small as the distance of the two maxima makes it
// (against the row's largest it was 0, and the loss +inf, from 87 T on).
// Exponentials and logarithms are the hardware's in fp32.
#include "logits_rows.h"

namespace kq {

using namespace rows;

namespace {

constexpr int K_MAX = 256;          // longest list
constexpr int V_MAX = 1 << 19;      // largest vocabulary: its bits fill 64 KB
constexpr double REST_MIN = 1.0 / 65536.0;
constexpr float LOG2E = 1.44269504088896340736f;
constexpr double LN2 = 0.69314718055994530942;

// a value that all lanes share, in a scalar register
__device__ inline float uniform(float v) {
  return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(v)));
}
__device__ inline double uniform(double v) {
  return __hiloint2double(__builtin_amdgcn_readfirstlane(__double2hiint(v)),
                          __builtin_amdgcn_readfirstlane(__double2loint(v)));
}

__device__ inline float masked(float v, uint32_t keep) { return __uint_as_float(__float_as_uint(v) & keep); }

// one value of the columns off the list, one of those on it
struct Pair {
  float off, on;
};

// f over the workgroup's pairs (see block_reduce); the second halves of waves
// that `lists` does not name are `none`
template <int TPB, class F>
__device__ inline Pair block_reduce_pairs(Pair v, bool lists, float none, Pair* part, F f) {
  v.off = wave_reduce(v.off, f);
  v.on = lists ? wave_reduce(v.on, f) : none;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  Pair r = part[0];
#pragma unroll
  for (int w = 1; w < TPB / 64; ++w) r = {f(r.off, part[w].off), f(r.on, part[w].on)};
  return r;
}

struct DistillArgs {
  int64_t n, ld, ldg;
  int vocab, k;
  const float* t_values;
  const int32_t* t_index;
  const float* t_lse;   // NULL: renormalise over the list
  float temperature;
  const float* weight;  // NULL: ones
  float* loss;
  float* stats;         // n x 3: m, log sum exp((s - m) / T), log of the mass off the list
};

template <class T, class V, bool LOSS, bool GRAD>
__global__ __launch_bounds__(V::TPB, V::WAVES) void distill_kernel(const T* logits, DistillArgs d, T* grad) {
  constexpr int CH = V::CH, TPB = V::TPB;
  extern __shared__ uint32_t bits[];  // a bit per column: on the list
  __shared__ double dpart[2][TPB / 64];
  __shared__ float fpart[4][TPB / 64];
  __shared__ Pair pair[2][TPB / 64];
  __shared__ int twice;  // a column is on the list more than once (known with the bucket)
  __shared__ __align__(16) int idx_at[K_MAX];
  __shared__ __align__(16) float p_at[K_MAX];
  static_assert(K_MAX <= TPB, "one thread per entry of the list");
  const int t = threadIdx.x;
  const int full = d.vocab / E<T>;
  const float inv_t = 1.f / d.temperature, c = LOG2E / d.temperature;
  const bool bucket = d.t_lse != nullptr;
  if (bucket)
    for (int j = t; j < int(cdiv(d.vocab, 32)); j += TPB) bits[j] = 0;
  for (int j = t; j < K_MAX; j += TPB) idx_at[j] = -1, p_at[j] = 0.f;
  if (t == 0) twice = bucket ? 0 : 1;
  __syncthreads();
  Row<T, V> r;
  r.load(logits + int64_t(blockIdx.x) * d.ld, full, d.vocab);
  for (int64_t row = blockIdx.x; row < d.n; row += gridDim.x) {
    const T* lr = logits + row * d.ld;
    T* gr = GRAD ? grad + row * d.ldg : nullptr;
    const bool more = row + gridDim.x < d.n;
    const int ahead = more ? full : 0;
    const T* nr = lr + (more ? int64_t(gridDim.x) * d.ld : 0);
    const float w = d.weight ? uniform(d.weight[row]) : 1.f;
    // a row without weight goes along (whatever its logits hold), and zeros
    // are written for it
    const uint32_t keep = w == 0.f ? 0u : ~0u;
    // ---- the teacher's side
    int idx = -1;
    float at_idx = 0.f;  // the student's logit there
    float tv = -__builtin_inff();
    if (t < d.k) {
      idx = d.t_index[row * d.k + t];
      if (uint32_t(idx) >= uint32_t(d.vocab)) idx = -1;
      idx_at[t] = idx;
      if (idx >= 0) {
        at_idx = to_f32(lr[idx]);
        tv = d.t_values[row * d.k + t];
        if (bucket && atomicOr(&bits[idx >> 5], 1u << (idx & 31)) >> (idx & 31) & 1) twice = 1;
      }
    }
    double mass = 1.0, rest = 0.0;
    float log_p;  // to base 2
    if (bucket) {
      // t / T rounds by itself, as in the log-sum-exp that top logits come with: of a
      // list that holds almost all of it, the rounding is then in both and goes off
      // (Z's own is left). In one operation with Z it would stay in p alone, up to
      // 2e-6 at t / T = 50, and 1 - sum p, which counts from 2^-16 on, would be off by
      // as much.
      float scaled = tv * inv_t;
      asm volatile("" : "+v"(scaled));
      log_p = (scaled - d.t_lse[row]) * LOG2E;
    } else {
      float tm = block_reduce<TPB>(tv, fpart[0], Max());
      if (tm == -__builtin_inff()) tm = 0.f;
      const float z = (tv - tm) * c;
      const float total = block_reduce<TPB>(__builtin_amdgcn_exp2f(z), fpart[1], Sum());
      log_p = z - __builtin_amdgcn_logf(total);
      if (total == 0.f) mass = 0.0;
    }
    const float p = idx >= 0 ? __builtin_amdgcn_exp2f(log_p) : 0.f;
    if (GRAD && t < d.k) p_at[t] = p;
    if (bucket) {
      mass = uniform(block_reduce<TPB>(double(p), dpart[0], Sum()));
      rest = 1.0 - mass;
      if (rest <= REST_MIN) rest = 0.0;
      mass += rest;
    } else {
      __syncthreads();
    }
    // Entries of one column: the first counts and writes for all. All are compared
    // with all only where the bits have met such a column (loss of 20000 x 4000
    // with lists of 256: 74 us, 370 where every row is).
    float p_col = p;
    bool first = (GRAD || bucket) && idx >= 0;
    if (first && twice) {
      p_col = 0.f;
      for (int l = 0; l < d.k; l += 4) {
        const int4 other = *reinterpret_cast<const int4*>(idx_at + l);
        if (GRAD) {
          const float4 po = *reinterpret_cast<const float4*>(p_at + l);
          p_col += (other.x == idx ? po.x : 0.f) + (other.y == idx ? po.y : 0.f) +
                   (other.z == idx ? po.z : 0.f) + (other.w == idx ? po.w : 0.f);
        }
        if ((other.x == idx && l < t) || (other.y == idx && l + 1 < t) || (other.z == idx && l + 2 < t) ||
            (other.w == idx && l + 3 < t))
          first = false;
      }
    }
    // ---- the student's side
    // listed elements of a chunk become -inf (in registers for good: their
    // gradient comes from the list)
    auto without_listed = [&](int ch, Raw& q) {
      if (!bucket || ch >= full) return;
      const int j = ch * E<T>;
      const uint32_t mark = bits[j >> 5] >> (j & 31) & ((1u << E<T>) - 1);
      if (mark)
        for (int i = 0; i < 4; ++i) {
          uint32_t listed = uint32_t(__builtin_amdgcn_sbfe(int(mark), E<T> / 4 * i, 1));
          if (E<T> == 8) {  // two halves
            const uint32_t upper = uint32_t(__builtin_amdgcn_sbfe(int(mark), 2 * i + 1, 1));
            listed = __builtin_amdgcn_perm(upper, listed, 0x05040100u);
          }
          q[i] = (q[i] & ~listed) | (neg_inf_word<T>() & listed);
        }
    };
    // m: the row's largest logit, total: the sum of exp((s - m) / T), q_r: the mass
    // off the list. There a column's share of q_r is exp2((s - ref) c - log_ref) / off.
    float m, total, q_r, off, ref, log_ref;
    if (LOSS) {
      Online o;
      float top = LOWEST;
      off = 0.f;
      auto rescale = [&](float f) { off *= f; };
      r.template each<!GRAD>(
          lr, full,
          [&](int, int, const float(&x)[E<T>], Raw) {
            const float here = max_of(x);
            top = max3(top, here, here);
            o.raise(here, c, rescale);
            float part = 0.f;
            for (int i = 0; i < E<T>; ++i) part += __builtin_amdgcn_exp2f((x[i] - o.m) * c);
            off += part;
            // computed here, not where the sum is used: the elements would be kept
            asm volatile("" : "+v"(off));
          },
          without_listed);
      const int j = full * E<T> + t;
      const bool tail_on = bucket && j < d.vocab && bits[j >> 5] >> (j & 31) & 1;
      const float tail = tail_on ? -__builtin_inff() : r.tail;
      top = max3(top, tail, tail);
      o.raise(tail, c, rescale);
      off += __builtin_amdgcn_exp2f((tail - o.m) * c);
      if (!GRAD && more) r.load_tail(nr, full, d.vocab);
      float top_off, scaled_off;  // (LOWEST is the maximum of no logit, and its sum 0)
      if (bucket) {
        const float listed = first ? at_idx : -__builtin_inff();
        const bool lists = (t & ~63) < d.k;  // whether the wave has entries
        const Pair tops =
            block_reduce_pairs<TPB>(Pair{top, max3(listed, LOWEST, LOWEST)}, lists, LOWEST, pair[0], Max());
        rescale(__builtin_amdgcn_exp2f((o.m - tops.off) * c));
        const float on = __builtin_amdgcn_exp2f((listed - tops.on) * c);
        const Pair sums = block_reduce_pairs<TPB>(Pair{off, on}, lists, 0.f, pair[1], Sum());
        top_off = uniform(tops.off), off = uniform(sums.off);
        m = uniform(Max()(tops.off, tops.on));
        scaled_off = off * __builtin_amdgcn_exp2f((top_off - m) * c);
        total = uniform(scaled_off + sums.on * __builtin_amdgcn_exp2f((tops.on - m) * c));
      } else {
        m = top_off = uniform(block_reduce<TPB>(top, fpart[2], Max()));
        rescale(__builtin_amdgcn_exp2f((o.m - m) * c));
        off = total = scaled_off = uniform(block_reduce<TPB>(off, fpart[3], Sum()));
      }
      if (total == 0.f) m = 0.f;
      // to base 2; a row without a finite logit has q = 0 and log q = -inf
      const float log_total = total == 0.f ? 0.f : __builtin_amdgcn_logf(total);
      if (GRAD) q_r = scaled_off / total;
      ref = top_off, log_ref = 0.f;
      double term = 0.0;
      if (p > 0.f) term = double(p) * ((double(log_p) - double(at_idx - m) * double(c)) + double(log_total));
      term = block_reduce<TPB>(term, dpart[1], Sum());
      if (t == 0) {
        const double log_q_r = off == 0.f ? -double(__builtin_inff())
                                          : (double(top_off) - double(m)) * double(c) +
                                                double(__builtin_amdgcn_logf(off)) - double(log_total);
        if (rest > 0.0) term += rest * (double(__builtin_amdgcn_logf(float(rest))) - log_q_r);
        d.loss[row] = masked(float(double(w) * d.temperature * d.temperature * LN2 * term), keep);
        if (d.stats) {
          // (of the logits alone: a row without weight here may have some in
          // the backward pass)
          d.stats[3 * row] = m;
          d.stats[3 * row + 1] = total == 0.f ? -__builtin_inff() : log_total * float(LN2);
          d.stats[3 * row + 2] = float(log_q_r * LN2);
        }
      }
    } else {
      m = d.stats[3 * row];
      const float log_total = d.stats[3 * row + 1] * LOG2E;
      total = __builtin_amdgcn_exp2f(log_total);
      const float log_q_r = d.stats[3 * row + 2] * LOG2E;
      q_r = __builtin_amdgcn_exp2f(log_q_r);
      off = log_q_r == -__builtin_inff() ? 0.f : 1.f;
      ref = m, log_ref = log_total + log_q_r;
    }
    // ---- the gradient
    if (GRAD) {
      const double gain = double(w) * d.temperature;
      const float f_on = float(total == 0.f ? 0.0 : gain * mass / total);
      // Off the list P q_j - r q_j / q_r is taken as (q_j / q_r) (P q_r - r): the
      // first factor is at most 1, however small q_r.
      float f_off = f_on;
      if (rest > 0.0 && off > 0.f) f_off = float(gain * (mass * q_r - rest) / off);
      else ref = m, log_ref = 0.f;
      auto exps = [&](float x) {
        if constexpr (LOSS) return __builtin_amdgcn_exp2f((x - ref) * c);
        // (what the stats round off may take it past 1, by their |log q_r| 2^-24)
        return __builtin_amdgcn_fmed3f(__builtin_amdgcn_exp2f(fmaf(x - ref, c, -log_ref)), 0.f, 1.f);
      };
      r.template each<true>(lr, full, [&](int i, int ch, const float(&x)[E<T>], Raw) {
        float g[E<T>];
        for (int e = 0; e < E<T>; ++e) g[e] = exps(x[e]) * f_off;
        Raw q = pack(g);
        q &= keep;
        if (ch < full) store_once(CH > 0 ? r.chunk_at(gr, i) : gr + int64_t(ch) * E<T>, q);
        if constexpr (CH > 0) r.load_chunk(i, nr, ahead);
      });
      if (full * E<T> + t < d.vocab)
        put(gr + full * E<T> + t, masked(exps(r.tail) * f_off, keep));
      if (more) r.load_tail(nr, full, d.vocab);
      __syncthreads();
      if (first)
        put(gr + idx, masked(__builtin_amdgcn_exp2f((at_idx - m) * c) * f_on - float(gain) * p_col, keep));
    } else {
      __syncthreads();
    }
    if (bucket && idx >= 0) bits[idx >> 5] = 0;
    if (bucket && t == 0) twice = 0;
    __syncthreads();
  }
}

}  // namespace

int64_t distill_max_vocab() { return V_MAX; }

kq_status distill_run(const void* logits, kq_dtype dt, int64_t n, int64_t vocab, int64_t ld,
                      const float* t_values, const int32_t* t_index, const float* t_lse, int k,
                      float temperature, const float* weight, float* loss, float* stats, void* grad,
                      int64_t ldg, hipStream_t s) {
  const DistillArgs d{n, ld, ldg, int(vocab), k, t_values, t_index, t_lse, temperature, weight, loss, stats};
  // the bits are of use with the bucket alone
  const size_t lds = t_lse ? size_t(cdiv(vocab, 32)) * 4 : 0;
  auto launch = [&](auto* p) -> kq_status {
    using T = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    const int64_t chunks = cdiv(vocab, E<T>);
    auto go = [&](auto v, auto with_loss, auto with_grad) -> kq_status {
      using V = decltype(v);
      const auto kernel = distill_kernel<T, V, decltype(with_loss)::value, decltype(with_grad)::value>;
      if (lds > 49152)
        KQ_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                   hipFuncAttributeMaxDynamicSharedMemorySize, int(lds)));
      kernel<<<row_groups<V>(n), V::TPB, lds, s>>>(p, d, static_cast<T*>(grad));
      KQ_HIP(hipGetLastError());
      return KQ_OK;
    };
    const std::true_type yes;
    const std::false_type no;
    // What is chosen goes by the row's length alone, so that a row's sums, and
    // their rounding, are the same in whatever company.
    // One pass, nothing to hold: loss of 20000 x 4000 bf16 without a bucket 57 us
    // with 256 threads and room for 8 waves, which spills 12 bytes a lane, 58.5
    // with 7, 67 with 6; with a bucket and lists of 256 74 with 8 and 72 with 7, of
    // 8192 x 8000 and 200 46.6 and 43.2; of 4096 x 32000 54 with 256 and 6, 59 with
    // 8, 66 with 512 threads; of 1 x 128256 24 with 256, 16 with 512, and of 4096
    // of them 162 and 172.
    if (!grad) {
      if (chunks <= 1024) return t_lse ? go(Variant<0, 256, 7>(), yes, no) : go(Variant<0, 256, 8>(), yes, no);
      if (chunks <= 4096) return go(Variant<0, 256, 6>(), yes, no);
      return go(Variant<0, 512, 6>(), yes, no);
    }
    if (!loss) {
      // gradient of 8192 x 4000 bf16: 52 us with 256 threads, 75 with 512; 4096
      // x 32000: 107, 103; 4096 x 128256: 417, 405, 392 with 1024
      if (chunks <= 2048) return go(Variant<0, 256, 6>(), no, yes);
      if (chunks <= 8192) return go(Variant<0, 512, 6>(), no, yes);
      return go(Variant<0, 1024, 8>(), no, yes);
    }
    // Loss and gradient: two passes. Rows of up to 128 KB are held in
    // registers (4096 x 32000 bf16, the same rows each time: 115 us, read twice
    // 121; 4096 x 65536: 215, 229); of longer ones a CU holds too few at once to
    // keep the memory busy, and the second pass finds them in the cache beside it
    // (4096 x 128256: 451 us, in registers 493).
    if (chunks <= 512) return go(Variant<2, 256, 6>(), yes, yes);
    if (chunks <= 1024) return go(Variant<4, 256, 6>(), yes, yes);
    if (chunks <= 2048) return go(Variant<8, 256, 5>(), yes, yes);
    if (chunks <= 4096) return go(Variant<16, 256, 4>(), yes, yes);
    if (chunks <= 6144) return go(Variant<24, 256, 3>(), yes, yes);
    if (chunks <= 8192) return go(Variant<16, 512, 4>(), yes, yes);
    return go(Variant<0, 512, 6>(), yes, yes);
  };
  if (dt == KQ_BF16) return launch(static_cast<const uint16_t*>(logits));
  return launch(static_cast<const float*>(logits));
}

}  // namespace kq
