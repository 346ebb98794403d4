// Rows of logits held on chip, shared by the top-logit and the distillation
// kernels.
//
// One workgroup takes a row. Its threads may hold the row in registers, CH
// chunks of 16 bytes each (chunk c of the row is register c / TPB of thread
// c % TPB, so that a wave's loads are 1 KB of adjacent bytes), and the elements
// past the last full chunk as one value each of the first threads; the row is
// then read from memory once, whatever the number of passes over it, and the
// workgroup loads its next one, chunk by chunk, as the last pass frees the
// registers. With CH = 0 each pass reads the row, the first from memory, later
// ones, as a rule, from the cache beside it. Rows need no alignment beyond
// their element's: global loads and stores of 16 bytes take any.
#pragma once
#include "kq_internal.h"
#include "lanes.h"

namespace kq {
namespace rows {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// 16 bytes of a row as they lie. One vector of four registers throughout: of
// four words, the compiler would keep each where it likes, and copy them there
// as soon as they come.
typedef uint32_t Raw __attribute__((ext_vector_type(4)));
typedef uint32_t RawMem __attribute__((ext_vector_type(4), aligned(2)));  // at any element

// What the kernel itself touches once goes past the caches' usual order
// (reading 2 GB so took 6.5 TB/s, else 5.9; copying them 5.2, else 4.7).
__device__ __forceinline__ Raw load_once(const void* p) {
  return __builtin_nontemporal_load(static_cast<const RawMem*>(p));
}
__device__ __forceinline__ Raw load_kept(const void* p) { return *static_cast<const RawMem*>(p); }
__device__ __forceinline__ void store_once(void* p, Raw q) {
  __builtin_nontemporal_store(RawMem(q), static_cast<RawMem*>(p));
}

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

__device__ inline void unpack(Raw r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(r[i] << 16);
    x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
  }
}
__device__ inline void unpack(Raw r, float (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(r[i]);
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
static __device__ const uint32_t neg_inf_chunks[2][4] = {{0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u},
                                                         {0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u}};
template <class T>
__device__ __forceinline__ const uint32_t* neg_inf_chunk() {
  return neg_inf_chunks[sizeof(T) == 2 ? 0 : 1];
}

// The part of a row that thread t holds (see above).
template <class T, class V>
struct Row {
  static constexpr int CH = V::CH, TPB = V::TPB;
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
  // Register i <- chunk i of this thread's, of the row's `full` chunks; past
  // the last one, -inf from a constant. (Loads of some lanes only would have
  // to be merged with what the others hold, and be waited for on the spot.)
  __device__ __forceinline__ void load_chunk(int i, const T* row, int full) {
    typedef const __attribute__((address_space(1))) RawMem* Global;  // either: both are global memory
    const uint64_t at = reinterpret_cast<uint64_t>(chunk_at(const_cast<T*>(row), i));
    const uint64_t none = reinterpret_cast<uint64_t>(neg_inf_chunk<T>());
    const bool have = i * TPB + thread_of_row() < full;
    reg[i] = __builtin_nontemporal_load(reinterpret_cast<Global>(have ? at : none));
  }
  __device__ __forceinline__ void load_tail(const T* row, int full, int vocab) {
    const int j = full * E<T> + int(threadIdx.x);
    tail = j < vocab ? to_f32(row[j]) : -__builtin_inff();
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
  // ONCE: without registers for the row, this is the last pass over it.
  // edit(chunk, it as it lies) may change elements first: for good in registers,
  // else for this pass.
  template <bool ONCE = false, class F>
  __device__ __forceinline__ void each(const T* row, int full, F f) {
    each<ONCE>(row, full, f, [](int, Raw&) {});
  }
  template <bool ONCE, class F, class G>
  __device__ __forceinline__ void each(const T* row, int full, F f, G edit) {
    if constexpr (CH > 0) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        Raw& q = reg[i];
        asm volatile("" : "+v"(q));
        edit(i * TPB + thread_of_row(), q);
        float x[E<T>];
        unpack(q, x);
        f(i, i * TPB + thread_of_row(), x, q);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      // every lane goes through every chunk of its wave (past the last one
      // with -inf), so that what f counts over the wave stays the same in all
      constexpr int U = V::UNROLL;
      constexpr uint32_t ni = neg_inf_word<T>();
      auto take = [&](int at, Raw& q) {
        edit(at, q);
        float x[E<T>];
        unpack(q, x);
        f(0, at, x, q);
      };
      auto get = [&](int at) {
        const T* src = row + int64_t(at) * E<T>;
        if constexpr (ONCE) return load_once(src);
        else return load_kept(src);
      };
      const int lane = int(threadIdx.x) & 63;
      int first = __builtin_amdgcn_readfirstlane(int(threadIdx.x) & ~63);
      for (; first + (U - 1) * TPB + 64 <= full; first += U * TPB) {
        Raw q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) q[u] = get(first + u * TPB + lane);
#pragma unroll
        for (int u = 0; u < U; ++u) take(first + u * TPB + lane, q[u]);
      }
      for (; first < full; first += TPB) {
        const int at = first + lane;
        Raw q = {ni, ni, ni, ni};
        if (at < full) q = get(at);
        take(at, q);
      }
    }
  }
};

// f over the workgroup's values, left in every thread. part: TPB / 64 values
// of LDS that no other reduction still reads (callers alternate two).
template <int TPB, class T, class F>
__device__ inline T block_reduce(T v, T* part, F f) {
  v = wave_reduce(v, f);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  T r = part[0];
#pragma unroll
  for (int w = 1; w < TPB / 64; ++w) r = f(r, part[w]);
  return r;
}

// What a thread's exponentials are taken against: not its running maximum
// but a value that the largest so far is at most 2^60 times of (in fp32 sums
// neither overflow nor lose digits by that), so that it seldom moves: of 64
// lanes, one or the other has a new maximum at almost every chunk. A chunk
// is taken when it has come, while later ones are on their way; with a pass
// for the maximum and one for the sum after it, the memory was idle during
// the second (loss and gradient of 4096 x 128256 bf16: 618 us so).
constexpr float LOWEST = -3.402823466e38f;
struct Online {
  float m = LOWEST;  // finite: -inf less it is -inf, never NaN

  // before the exponentials of elements up to `top`: the factor that the
  // sums so far take
  template <class F>
  __device__ __forceinline__ void raise(float top, float c, F scale) {
    if ((top - m) * c > 60.f) {
      scale(__builtin_amdgcn_exp2f((m - top) * c));
      m = top;
    }
  }
};

// How a kernel takes rows: chunks in a thread's registers, threads of a
// workgroup, and waves of a SIMD that its registers are to leave room for.
template <int CH_, int TPB_, int WAVES_>
struct Variant {
  static constexpr int CH = CH_, TPB = TPB_, WAVES = WAVES_;
  static constexpr int UNROLL = 4;
};

// Workgroups of a launch: as many as the 256 CUs hold at once, so that each
// goes through its share of the rows.
template <class V>
inline unsigned row_groups(int64_t n) {
  const int64_t at_once = 256 * (4 * V::WAVES / (V::TPB / 64));
  return unsigned(n < at_once ? n : at_once);
}

}  // namespace rows
}  // namespace kq
