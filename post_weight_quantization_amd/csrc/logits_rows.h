// Rows of logits held on chip, shared by the top-logit and the distillation
// kernels.
//
// One workgroup takes a row. Its threads hold the row in registers, CH chunks
// of 16 bytes each (chunk c of the row is register c / TPB of thread c % TPB,
// so that a wave's loads are 1 KB of adjacent bytes), and the elements past
// the last full chunk as one value each of the first threads. The register
// file of a CU (512 KB) takes the largest rows here, up to 20 chunks a thread
// of 1024, which are read from memory once, whatever the number of passes
// over them; longer rows (CH = 0) are read again for each pass. A workgroup goes on to
// further rows and loads the next one, chunk by chunk, as the last pass
// frees the registers. Rows need no alignment beyond their element's: global
// loads and stores of 16 bytes take any.
#pragma once
#include "kq_internal.h"

namespace kq {
namespace rows {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

struct __attribute__((packed, aligned(2))) Raw {
  uint32_t w[4];
};

template <class T>
constexpr int E = 16 / int(sizeof(T));  // elements of a chunk

__device__ inline float to_f32(uint16_t v) { return __uint_as_float(uint32_t(v) << 16); }
__device__ inline float to_f32(float v) { return v; }

__device__ inline uint32_t pack_bf16(float lo, float hi) {
  const bf16x2 r = __builtin_convertvector(f32x2{lo, hi}, bf16x2);
  uint32_t u;
  __builtin_memcpy(&u, &r, 4);
  return u;
}
__device__ inline void put(uint16_t* p, float v) { *p = uint16_t(pack_bf16(v, v)); }
__device__ inline void put(float* p, float v) { *p = v; }

__device__ inline void unpack(const Raw& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(r.w[i] << 16);
    x[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
  }
}
__device__ inline void unpack(const Raw& r, float (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(r.w[i]);
}
__device__ inline Raw pack(const float (&x)[8]) {
  return {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
}
__device__ inline Raw pack(const float (&x)[4]) {
  return {__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
}

// Largest of three; a NaN is passed over (who needs to know finds it in a
// sum). fmaxf would first canonicalize every operand.
__device__ inline float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}
__device__ inline float max_of(const float (&x)[8]) {
  return max3(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), max3(x[6], x[7], x[7]));
}
__device__ inline float max_of(const float (&x)[4]) { return max3(max3(x[0], x[1], x[2]), x[3], x[3]); }

// The thread's number, hidden from the compiler: what is derived from it per
// chunk would otherwise be kept in registers from row to row.
__device__ __forceinline__ int thread_of_row() {
  int t = int(threadIdx.x);
  asm volatile("" : "+v"(t));
  return t;
}

template <class T>
__device__ constexpr uint32_t neg_inf_word() {
  return sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
}

// The part of a row that thread t holds (see above).
template <class T, int CH, int TPB>
struct Row {
  Raw reg[CH > 0 ? CH : 1];
  float tail;

  // Where this thread's chunk i lies: a scalar base and one offset for all i.
  // (The empty asm keeps the sum scalar: as a constant it would be added to
  // the offset, in two vector registers for each i.)
  static __device__ __forceinline__ T* chunk_at(T* row, int i) {
    uint32_t at = uint32_t(i) * TPB * 16;
    asm("" : "+s"(at));
    char* base = reinterpret_cast<char*>(row) + at;
    return reinterpret_cast<T*>(base + threadIdx.x * 16u);
  }
  // -inf everywhere; what no load reaches stays so.
  __device__ __forceinline__ void clear() {
    constexpr uint32_t ni = neg_inf_word<T>();
    for (Raw& q : reg) q = {ni, ni, ni, ni};
    tail = -__builtin_inff();
  }
  // Register i <- chunk i of this thread's, of the row's `full` chunks (0:
  // no load, the register is kept).
  __device__ __forceinline__ void load_chunk(int i, const T* row, int full) {
    if (i * TPB + thread_of_row() < full) reg[i] = *reinterpret_cast<const Raw*>(chunk_at(const_cast<T*>(row), i));
  }
  __device__ __forceinline__ void load_tail(const T* row, int full, int vocab) {
    const int j = full * E<T> + int(threadIdx.x);
    if (j < vocab) tail = to_f32(row[j]);
  }
  __device__ __forceinline__ void load(const T* row, int full, int vocab) {
    if constexpr (CH > 0) {
#pragma unroll
      for (int i = 0; i < CH; ++i) load_chunk(i, row, full);
    }
    load_tail(row, full, vocab);
  }
  // f(register, chunk, elements, chunk as it lies) for each of this thread's chunks. A pass
  // unpacks them anew (the empty asm hides that they have not changed):
  // kept from pass to pass, the unpacked row would be twice the registers.
  template <class F>
  __device__ __forceinline__ void each(const T* row, int full, F f) {
    if constexpr (CH > 0) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        Raw& q = reg[i];
        asm volatile("" : "+v"(q.w[0]), "+v"(q.w[1]), "+v"(q.w[2]), "+v"(q.w[3]));
        float x[E<T>];
        unpack(q, x);
        f(i, i * TPB + thread_of_row(), x, q);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
#pragma unroll 4
      for (int c = threadIdx.x; c < full; c += TPB) {
        float x[E<T>];
        const Raw q = *reinterpret_cast<const Raw*>(row + int64_t(c) * E<T>);
        unpack(q, x);
        f(0, c, x, q);
      }
    }
  }
};

// f over the workgroup's values, left in every thread. part: TPB / 64 values
// of LDS that no other reduction still reads (callers alternate two).
template <int TPB, class T, class F>
__device__ inline T block_reduce(T v, T* part, F f) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = f(v, T(__shfl_xor(v, o)));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  T r = part[0];
#pragma unroll
  for (int w = 1; w < TPB / 64; ++w) r = f(r, part[w]);
  return r;
}

struct Sum {
  template <class T>
  __device__ T operator()(T a, T b) const { return a + b; }
};
struct Max {
  __device__ float operator()(float a, float b) const { return max3(a, b, b); }
  __device__ double operator()(double a, double b) const { return a > b ? a : b; }
};

// Calls go(integral constants CH, TPB) for the variant that holds `chunks`:
// small rows take small workgroups, several to a CU.
template <int A, int B>
struct Variant {
  static constexpr int CH = A, TPB = B;
};
template <class G>
kq_status with_variant(int64_t chunks, G go) {
  if (chunks <= 256 * 2) return go(Variant<2, 256>());
  if (chunks <= 256 * 4) return go(Variant<4, 256>());
  if (chunks <= 256 * 8) return go(Variant<8, 256>());
  if (chunks <= 512 * 8) return go(Variant<8, 512>());
  if (chunks <= 512 * 16) return go(Variant<16, 512>());
  if (chunks <= 512 * 32) return go(Variant<32, 512>());
  if (chunks <= 512 * 40) return go(Variant<40, 512>());
  return go(Variant<0, 512>());
}

// Waves of a SIMD that the registers of a variant are to leave room for.
constexpr int min_waves(int ch) { return ch == 0 || ch > 16 ? 2 : 4; }

// Workgroups of a launch: as many as the 256 CUs hold at once, so that each
// goes through its share of the rows.
template <class V>
inline unsigned row_groups(int64_t n) {
  const int64_t at_once = 256 * (4 * min_waves(V::CH) / (V::TPB / 64));
  return unsigned(n < at_once ? n : at_once);
}

}  // namespace rows
}  // namespace kq
