// Reductions over the 64 lanes of a wave.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace kq {

struct Sum {
  template <class T>
  __device__ T operator()(T a, T b) const { return a + b; }
};
struct Min {
  __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return a < b ? a : b; }
};
struct Max {
  __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
  // a NaN is passed over (fmaxf would first canonicalize both)
  __device__ float operator()(float a, float b) const {
    float r;
    asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
  }
  __device__ double operator()(double a, double b) const { return a > b ? a : b; }
};

// Step S of f over a wave's values: v joined with those of the other lane of a
// pair, pair of a quad, half of 8 lanes, of a row of 16, of 32 and of the 64, by
// moves between lanes (through LDS, as by shuffles, six steps take some 700
// cycles).
template <int S, class T, class F>
__device__ __forceinline__ T wave_step(T v, F f) {
  constexpr int W = int(sizeof(T) / 4);
  struct Words {
    uint32_t w[W];
  };
  Words a = __builtin_bit_cast(Words, v);
  if constexpr (S < 4) {
    // within a quad 1 0 3 2, then 2 3 0 1; half a row mirrored, a row mirrored
    constexpr int ctrl = S == 0 ? 0xb1 : S == 1 ? 0x4e : S == 2 ? 0x141 : 0x140;
    for (int i = 0; i < W; ++i) a.w[i] = uint32_t(__builtin_amdgcn_mov_dpp(int(a.w[i]), ctrl, 0xf, 0xf, true));
    return f(v, __builtin_bit_cast(T, a));
  } else {
    Words b;  // the lower and the upper of each two, in both
    for (int i = 0; i < W; ++i) {
      const auto r = S == 4 ? __builtin_amdgcn_permlane16_swap(a.w[i], a.w[i], false, false)
                            : __builtin_amdgcn_permlane32_swap(a.w[i], a.w[i], false, false);
      a.w[i] = r[0], b.w[i] = r[1];
    }
    return f(__builtin_bit_cast(T, a), __builtin_bit_cast(T, b));
  }
}

// f over the wave's values, left in every lane.
template <class T, class F>
__device__ __forceinline__ T wave_reduce(T v, F f) {
  v = wave_step<0>(v, f);
  v = wave_step<1>(v, f);
  v = wave_step<2>(v, f);
  v = wave_step<3>(v, f);
  v = wave_step<4>(v, f);
  return wave_step<5>(v, f);
}

}  // namespace kq
