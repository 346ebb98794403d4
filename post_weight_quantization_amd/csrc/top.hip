// A teacher's top logits: the K largest logits of each row in descending
// order, equal ones by lowest index, and log sum exp(l / T) of the whole row.
//
// A workgroup holds its row on chip (logits_rows.h) and goes through it twice.
//   1. Each thread's largest value over its chunks (for long lists up to
//      four, of as many interleaved shares of them): 256 to 1024 group maxima. The K-th
//      largest of these, tau, has at least K elements at or above it, and few
//      more: the groups interleave over the row, so the K largest elements
//      seldom share one (64 of 1024 groups: 66 elements on average).
//      Only the upper 16 bits of tau's key are sought, 4 bits a round, the
//      waves counting for 16 pivots side by side.
//   2. Chunks with an element at or above tau go to LDS, each wave's to a
//      part of its own (places by ballot, no atomics to wait for), while the
//      exponentials are summed and the next row is loaded in their place (with
//      the sums in the first pass, after which the loads begin later, 64 of 4096
//      x 128256 bf16 took 329 us where this order took 268); their elements at
//      or above tau then make a list. An element is the 64-bit key (order of its
//      value, complement of its index), so no two are equal, and its rank is the
//      number of larger keys on the list.
// Should either overflow (128 chunks of a wave, 1024 elements: many equal
// logits), a second pass takes what is above the largest key that begins like
// tau's, and of the first K columns what equals it: enough where that makes K
// of them, as in a row whose mask, of whatever value, leaves few columns (256 x
// 100000 with 5 left: 71 us bf16, 128 fp32; searched, 1770 and 3370).
// What that does not settle (and a row with a NaN or +inf)
// is searched bit by bit for the K-th largest key, counting.
//
// The log-sum-exp is that of the quotients l / T as the distillation rounds
// them: of a list with nearly all of the mass, what it leaves is a difference of
// numbers that both round alike (T = 0.7, l / T near 60: within 2e-6, else up to
// 4e-6). The candidates are corrected for it, to first order, each by its share
// times its quotient's rounding; where a list has nearly all of the mass, the
// others have little.
//
// 64 of 4096 x 128256 bf16 take 207 us, 5.1 TB/s; vector instructions bound it:
// they keep the SIMDs busy 83 % of the time, half of that an exponential per
// element, at a quarter of the rate of the others. One row alone takes its CU 13
// us, spent the same way; it is not shared among CUs (which would have to join
// its waves' sums in their order here, for a row to be the same bits in whatever
// company).
#include <type_traits>

#include "logits_rows.h"

namespace kq {

using namespace rows;

namespace {

constexpr int K_MAX = 256;        // longest list
constexpr int CHUNKS = 128;       // chunks with a candidate of one wave, in LDS
constexpr int LIST = 1024;        // candidates in LDS
constexpr int GROUPS = 1024;      // group maxima

// Order of logits as unsigned keys: -inf lowest, both zeros equal, a NaN
// above everything.
__device__ inline uint32_t key_of(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t u = __float_as_uint(v == 0.f ? 0.f : v);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ inline float value_of(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
constexpr uint32_t KEY_NEG_INF = 0x007fffffu;

__device__ inline uint64_t entry_of(float v, int j) { return uint64_t(key_of(v)) << 32 | uint32_t(~uint32_t(j)); }

// how many of the lanes in `mask` lie below this one
__device__ inline int lanes_below(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi(uint32_t(mask >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(mask), 0));
}

// v / T as the distillation takes it, v times 1 / T rounded to fp32, and what
// that is above the exact product
__device__ inline float quotient(float v, float inv_t) {
  float z = v * inv_t;
  asm volatile("" : "+v"(z));  // (by itself, not within a sum)
  return z;
}
__device__ inline float quotient_error(float v, float inv_t) { return -fmaf(v, inv_t, -quotient(v, inv_t)); }

// the sum of a row's exponentials, and of candidates' exponentials times what
// the rounding of their quotients adds
struct Sums {
  float all, moved;
};
struct Join {
  __device__ Sums operator()(Sums a, Sums b) const { return {a.all + b.all, a.moved + b.moved}; }
};

template <int NW>
struct TopLds {
  __align__(16) uint64_t list[LIST + 2];
  uint32_t rank[LIST];
  Raw chunk[NW][CHUNKS];
  int chunk_no[NW][CHUNKS];
  __align__(16) uint16_t group[GROUPS];
  int pivots[2][16];
  float part[NW];
  // apart from `part`, which a wave may still read when another is done with the row
  float sum[NW];
  Sums sums[NW];
  int ipart[2][NW];
  int count, overflow;
};

// Appends the entries among this thread's elements that `take` names.
template <class T, int TPB, class F>
__device__ inline void gather(const T* row, int vocab, TopLds<TPB / 64>& s, F take) {
#pragma unroll 1
  for (int j = threadIdx.x; j < vocab; j += TPB) {
    const float v = to_f32(row[j]);
    if (take(v, j)) {
      const int at = atomicAdd(&s.count, 1);
      if (at < LIST) s.list[at] = entry_of(v, j);
    }
  }
}

// The exact search: the K-th largest key by its bits, then, among the
// elements of that key, the index up to which they belong to the K.
template <class T, int TPB>
__device__ void search(const T* row, int vocab, int k, TopLds<TPB / 64>& s) {
  auto count = [&](int flip, auto f) {
    int c = 0;
#pragma unroll 1
    for (int j = threadIdx.x; j < vocab; j += TPB) c += f(key_of(to_f32(row[j])), j);
    return block_reduce<TPB>(c, s.ipart[flip & 1], Sum());
  };
  uint32_t key = 0;
  int flip = 0;
  // a bfloat16's key has ones or zeros alone in its lower half
#pragma unroll 1
  for (int b = 31; b >= 0; --b) {
    const uint32_t probe = key | 1u << b;
    if (count(flip++, [&](uint32_t q, int) { return int(q >= probe); }) >= k) key = probe;
  }
  const int above = count(flip++, [&](uint32_t q, int) { return int(q > key); });
  // the lowest bound such that enough elements of this key lie below it
  int bound = 0;
#pragma unroll 1
  for (int b = 30; b >= 0; --b) {
    const int probe = bound | 1 << b;
    if (probe <= vocab &&
        count(flip++, [&](uint32_t q, int j) { return int(q == key && j < probe); }) < k - above)
      bound = probe;
  }
  if (threadIdx.x == 0) s.count = 0;
  __syncthreads();
  gather<T, TPB>(row, vocab, s, [&](float v, int j) {
    const uint32_t q = key_of(v);
    return q > key || (q == key && j <= bound);
  });
  __syncthreads();
}

template <class T, class V>
__global__ __launch_bounds__(V::TPB, V::WAVES) void top_logits_kernel(const T* __restrict__ logits, int n, int vocab,
                                                         int64_t ld, int k, float inv_t,
                                                         float* __restrict__ values,
                                                         int32_t* __restrict__ index,
                                                         float* __restrict__ lse) {
  constexpr int CH = V::CH, TPB = V::TPB;
  constexpr int GP = GROUPS / TPB;  // groups of a thread
  constexpr int NW = TPB / 64;
  __shared__ TopLds<NW> s;
  const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int full = vocab / E<T>;
  const float c = inv_t * 1.44269504088896340736f;
  // whether quotients round, and someone asks for their sum
  const bool rounds = lse && (__float_as_uint(inv_t) & 0x7fffffu) != 0;
  Row<T, V> r;
  r.load(logits + int64_t(blockIdx.x) * ld, full, vocab);
  for (int row = blockIdx.x; row < n; row += gridDim.x) {
    const T* lr = logits + int64_t(row) * ld;
    const bool more = row + int(gridDim.x) < n;
    const int ahead = more ? full : 0;
    const T* nr = lr + (more ? int64_t(gridDim.x) * ld : 0);
    // ---- the largest of each group
    float g[GP];
    for (int i = 0; i < GP; ++i) g[i] = -__builtin_inff();
    r.each(lr, full, [&](int i, int, const float(&x)[E<T>], Raw) {
      // Rows of a chunk a thread or less: a group for every two elements, for
      // there may be fewer chunks than K (of up to 1024 elements all may go on
      // the list).
      if constexpr (E<T> == 8 && CH == 4 && GP == 4) {
        if (i == 0 && full <= TPB) {
          for (int e = 0; e < GP; ++e) g[e] = max3(x[2 * e], x[2 * e + 1], x[2 * e + 1]);
          return;
        }
      }
      const float top = max_of(x);
      g[i % GP] = max3(g[i % GP], top, top);
    });
    g[0] = max3(g[0], r.tail, r.tail);
    float mine = g[0];
    for (int i = 1; i < GP; ++i) mine = max3(mine, g[i], g[i]);
    // a group for each thread will do for lists of up to a quarter as many
    const bool few = k <= TPB / 4;
    if (few)
      s.group[t] = uint16_t(key_of(mine) >> 16);
    else
      for (int i = 0; i < GP; ++i) s.group[i * TPB + t] = uint16_t(key_of(g[i]) >> 16);
    // m, and a bound below tau: the lowest of the largest of K sets of threads
    // or more, the sets as large as that leaves them
    float m = mine, least = mine;
    auto wider = [&](auto step) {
      m = wave_step<decltype(step)::value>(m, Max());
      if (TPB >> (decltype(step)::value + 1) >= k) least = m;
    };
    wider(std::integral_constant<int, 0>());
    wider(std::integral_constant<int, 1>());
    wider(std::integral_constant<int, 2>());
    wider(std::integral_constant<int, 3>());
    wider(std::integral_constant<int, 4>());
    wider(std::integral_constant<int, 5>());
    m = max3(m, LOWEST, LOWEST);
    uint32_t low = wave_reduce(key_of(least) >> 16, Min());
    if (lane == 0) s.part[w] = m, s.ipart[0][w] = int(low);
    if (t == 0) s.count = 0, s.overflow = 0;
    __syncthreads();
    for (int i = 0; i < NW; ++i) m = max3(m, s.part[i], s.part[i]), low = min(low, uint32_t(s.ipart[0][i]));
    // ---- the K-th largest of them, from the top in steps of 4 bits, between
    // the lowest and the highest (which seldom lie more than 8 bits apart)
    uint32_t key = __builtin_amdgcn_readfirstlane(low);
    const uint32_t high = __builtin_amdgcn_readfirstlane(key_of(m) >> 16);
    const int bits = high > key ? 32 - __clz(int(high - key)) : 0;
    auto kth = [&](auto per_lane) {
      constexpr int G = decltype(per_lane)::value;
      uint32_t v[G];
      const uint32_t* pairs = reinterpret_cast<const uint32_t*>(s.group) + lane * (G / 2);
      for (int i = 0; i < G; i += 2) v[i] = pairs[i / 2] & 0xffffu, v[i + 1] = pairs[i / 2] >> 16;
#pragma unroll 1
      for (int step = (bits + 3) / 4 - 1; step >= 0; --step) {
#pragma unroll 1
        for (int p = w; p < 16; p += NW) {
          const uint32_t pivot = key + (uint32_t(p) << (4 * step));
          int cnt = 0;
          for (int i = 0; i < G; ++i) cnt += __popcll(__ballot(v[i] >= pivot));
          if (lane == 0) s.pivots[step & 1][p] = cnt;
        }
        __syncthreads();
        // the highest pivot with K groups at or above it; all are above the first
        const uint64_t enough = __ballot(s.pivots[step & 1][lane & 15] >= k) | 1;
        key += uint32_t(31 - __clz(int(uint32_t(enough) & 0xffffu))) << (4 * step);
      }
    };
    if (few) kth(std::integral_constant<int, TPB / 64>());
    else kth(std::integral_constant<int, GROUPS / 64>());
    // too few groups reach above -inf: so does tau
    const float tau = key <= (KEY_NEG_INF >> 16) ? -__builtin_inff() : value_of(key << 16);
    // ---- candidates, and the sum of exponentials: 2^(x c - ref), ref the whole
    // number next to m c, so that it is one operation and its rounding that of
    // x c. Where m c is past 2^30, neighbouring numbers differ by 2^7 and more,
    // and what is not equal to m counts for nothing: the same for any larger c,
    // and one that keeps m c below 2^31 has no overflow.
    float scale = c;
    if (!(fabsf(m * c) < 0x1p30f)) scale = ldexpf(1.f, 30 - (int(__float_as_uint(m) >> 23 & 255) - 127));
    const float ref = rintf(m * scale);
    float sum = 0.f;
    int held = 0;  // of this wave's chunks, in LDS
    r.template each<true>(lr, full, [&](int i, int ch, const float(&x)[E<T>], Raw q) {
      const bool hit = max_of(x) >= tau && ch < full;
      const uint64_t hits = __ballot(hit);
      if (hits) {
        const int at = held + lanes_below(hits);
        if (hit && at < CHUNKS) s.chunk[w][at] = q, s.chunk_no[w][at] = ch;
        held += __popcll(hits);
      }
      float part = __builtin_amdgcn_exp2f(fmaf(x[0], scale, -ref));
      for (int e = 1; e < E<T>; ++e) part += __builtin_amdgcn_exp2f(fmaf(x[e], scale, -ref));
      sum += part;
      // computed here, not where the sum is used: the elements would be kept
      asm volatile("" : "+v"(sum));
      if constexpr (CH > 0) r.load_chunk(i, nr, ahead);
    });
    // the elements of the wave's chunks, and the tail, at or above tau
    float moved = 0.f;
    auto append = [&](bool take, float v, int j) {
      const uint64_t takes = __ballot(take);
      if (!takes) return;
      if (rounds) {
        const float e = __builtin_amdgcn_exp2f(fmaf(v, scale, -ref));
        if (take && e > 0.f) moved += e * quotient_error(v, inv_t);
      }
      int base = 0;
      if (lane == 0) base = atomicAdd(&s.count, __popcll(takes));
      const int at = __builtin_amdgcn_readfirstlane(base) + lanes_below(takes);
      if (take && at < LIST) s.list[at] = entry_of(v, j);
    };
    append(r.tail >= tau && full * E<T> + t < vocab, r.tail, full * E<T> + t);
    sum += __builtin_amdgcn_exp2f(fmaf(r.tail, scale, -ref));
    if (more) r.load_tail(nr, full, vocab);
    if (held > CHUNKS) s.overflow = 1;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int items = min(held, CHUNKS) * E<T>;
#pragma unroll 1
    for (int i = lane; i - lane < items; i += 64) {
      const int at = min(i, items - 1) / E<T>, e = i % E<T>;
      const uint32_t word = reinterpret_cast<const uint32_t*>(&s.chunk[w][at])[E<T> == 8 ? e / 2 : e];
      const float v = __uint_as_float(E<T> == 4 ? word : e & 1 ? word & 0xffff0000u : word << 16);
      append(i < items && v >= tau, v, s.chunk_no[w][at] * E<T> + e);
    }
    if (rounds) {
      const Sums sums = block_reduce<TPB>(Sums{sum, moved}, s.sums, Join());
      sum = sums.all, moved = sums.moved;
    } else {
      sum = block_reduce<TPB>(sum, s.sum, Sum());
    }
    // (NaN: the row's largest, found below, is the answer; no finite logit: the sum
    // is 0; a quotient past fp32 is the answer)
    if (lse && t == 0 && sum == sum) {
      const float top = quotient(m, inv_t);
      const float rel = logf(sum) + fmaf(-m, scale, ref) * 0.69314718055994530942f;
      const float by = moved / sum - quotient_error(m, inv_t);
      lse[row] = sum == 0.f ? -__builtin_inff() : isinf(top) ? top : top + (rel + by);
    }
    int count = s.count;
    if (s.overflow || count > LIST || sum != sum) {
      __syncthreads();
      if (sum == sum) {
        if (t == 0) s.count = 0;
        __syncthreads();
        uint32_t most = 0;
        gather<T, TPB>(lr, vocab, s, [&](float v, int) {
          const uint32_t q = key_of(v);
          if (q >> 16 == key) most = max(most, q);
          return q >> 16 > key;
        });
        most = block_reduce<TPB>(most, reinterpret_cast<uint32_t*>(s.ipart[0]), Max());
        if (t < k && key_of(to_f32(lr[t])) == most) {
          const int at = atomicAdd(&s.count, 1);
          if (at < LIST) s.list[at] = entry_of(to_f32(lr[t]), t);
        }
        __syncthreads();
        count = s.count;
      }
      if (count > LIST || count < k || sum != sum) {
        search<T, TPB>(lr, vocab, k, s);
        count = s.count;
      }
    }
    // ---- ranks: threads t, t + width, ... share the comparisons of one candidate
    int width = 64;
    while (width < count && width < TPB) width *= 2;
#pragma unroll 1
    for (int i = t; i < count; i += TPB) s.rank[i] = 0;
    if (t == 0) s.list[count] = 0;  // (below every entry: the list is read in pairs)
    __syncthreads();
#pragma unroll 1
    for (int i = t & (width - 1); i < count; i += width) {
      const uint64_t mine = s.list[i];
      uint32_t before = 0;
      const int step = 2 * (TPB / width);
      auto count_above = [&](const ulonglong2& two) { before += (two.x > mine) + (two.y > mine); };
      auto pair_at = [&](int j) { return *reinterpret_cast<const ulonglong2*>(s.list + j); };
      int j = 2 * (t / width);
      // four pairs on their way before the first is compared (in turn, 256 of 4096
      // x 32000 took 133 us for 119)
#pragma unroll 1
      for (; j + 3 * step < count; j += 4 * step) {
        ulonglong2 pairs[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) pairs[u] = pair_at(j + u * step);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < 4; ++u) count_above(pairs[u]);
      }
#pragma unroll 1
      for (; j < count; j += step) count_above(pair_at(j));
      if (before) atomicAdd(&s.rank[i], before);
    }
    __syncthreads();
#pragma unroll 1
    for (int i = t; i < count; i += TPB) {
      const uint32_t at = s.rank[i];
      if (at < uint32_t(k)) {
        const float v = value_of(uint32_t(s.list[i] >> 32));
        values[int64_t(row) * k + at] = v;
        if (at == 0 && lse && sum != sum) lse[row] = v;  // +inf, or NaN, which is above it
        index[int64_t(row) * k + at] = int32_t(~uint32_t(s.list[i]));
      }
    }
    __syncthreads();
  }
}

}  // namespace

int32_t logits_max_k() { return K_MAX; }

kq_status top_logits_run(const void* logits, kq_dtype dt, int64_t n, int64_t vocab, int64_t ld, int k,
                         float temperature, float* values, int32_t* index, float* lse, hipStream_t s) {
  auto launch = [&](auto* p) -> kq_status {
    using T = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    const int64_t chunks = cdiv(vocab, E<T>);
    auto go = [&](auto v) -> kq_status {
      using V = decltype(v);
      top_logits_kernel<T, V><<<row_groups<V>(n), V::TPB, 0, s>>>(p, int(n), int(vocab), ld, k, 1.f / temperature,
                                                                  values, index, lse);
      KQ_HIP(hipGetLastError());
      return KQ_OK;
    };
    // Held in registers, in workgroups as small as take the row in 16 chunks
    // a thread (4096 x 32000 bf16: 64 us with 256 threads, 98 with 512; 512 x
    // 50001 fp32, lists of 200: 31.7 us with 16 chunks of 1024 threads, 34.1
    // with 32 of 512), and the largest rows that fit too (4096 x 128256 bf16:
    // 207 us, read twice 290). The number of rows has no say, so that a row's sum,
    // and its rounding, is the same in whatever company.
    if (chunks <= 1024) return go(Variant<4, 256, 6>());
    if (chunks <= 2048) return go(Variant<8, 256, 5>());
    if (chunks <= 4096) return go(Variant<16, 256, 4>());
    if (chunks <= 8192) return go(Variant<16, 512, 4>());
    if (chunks <= 16384) return go(Variant<16, 1024, 4>());
    return go(Variant<0, 512, 6>());
  };
  if (dt == KQ_BF16) return launch(static_cast<const uint16_t*>(logits));
  return launch(static_cast<const float*>(logits));
}

}  // namespace kq
