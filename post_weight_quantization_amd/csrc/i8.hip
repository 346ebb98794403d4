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
#include <algorithm>
#include <type_traits>

#include "kq_internal.h"
#include "lanes.h"

namespace kq {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v4i_any __attribute__((ext_vector_type(4), aligned(4)));  // at any word
typedef int v16i __attribute__((ext_vector_type(16)));

namespace {

constexpr int I8_PAD = 128;  // code rows are padded to this many bytes

__device__ inline float bf16_f32(uint16_t v) { return __uint_as_float(uint32_t(v) << 16); }

// nearest even; a NaN stays a NaN
__device__ inline uint16_t f32_bf16(float f) { return __builtin_bit_cast(uint16_t, __bf16(f)); }

template <class T>
__device__ inline float load_f32(const T* p);
template <>
__device__ inline float load_f32<uint16_t>(const uint16_t* p) { return bf16_f32(*p); }
template <>
__device__ inline float load_f32<float>(const float* p) { return *p; }

__device__ inline void store_y(uint16_t* p, float v) { *p = f32_bf16(v); }
__device__ inline void store_y(float* p, float v) { *p = v; }

struct __attribute__((packed, aligned(2))) Raw16 {
  uint32_t w[4];
};

// 16 bytes read once: past the caches' usual order (8192 tokens of 28672 bf16:
// 125 us, else 140)
typedef uint32_t Mem16 __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ Raw16 load_once(const void* p) {
  const Mem16 v = __builtin_nontemporal_load(static_cast<const Mem16*>(p));
  return {v.x, v.y, v.z, v.w};
}

// What a row's codes are made with. rint(v / s) asks for the correctly rounded
// quotient; v * (1 / s) is off from it by at most 127 * 2^-22 = 3e-5, so where it
// lies further than 1e-4 from a midpoint between two codes, both round to
// the same one, and the division (10 operations) is left for the few others.
struct I8Grid {
  float s, inv;  // s NaN or 0: all codes are 0

  __device__ explicit I8Grid(float scale) : s(scale), inv(scale >= 1e-37f ? 1.f / scale : 0.f) {}
  __device__ int code(float v) const {
    const float t = v * inv;
    float q = rintf(t);
    // (no reciprocal of a scale near the smallest numbers, or NaN)
    if (inv == 0.f || fabsf(fabsf(t - q) - 0.5f) < 1e-4f) q = s > 0.f ? rintf(v / s) : 0.f;
    return int(fminf(fmaxf(q, -127.f), 127.f));
  }
};

// scale of a row whose largest magnitude has the bits m: NaN if the row has an
// infinity or a NaN (they order above the numbers)
__device__ inline float i8_scale(uint32_t m, float clip) {
  return m >= 0x7f800000u ? __builtin_nanf("") : clip * __uint_as_float(m) / 127.f;
}

// 16 bytes of a row: the largest magnitude's bits so far, and the codes
template <class T>
struct I8Chunk {
  static constexpr int E = 16 / int(sizeof(T));
  static __device__ inline uint32_t largest(uint32_t m, const Raw16& q) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // (the upper half of a pair of bfloat16 is compared with the lower one
      // behind it, which own() takes away)
      m = max(m, q.w[k] & 0x7fffffffu);
      if (E == 8) m = max(m, (q.w[k] << 16) & 0x7fffffffu);
    }
    return m;
  }
  static __device__ inline uint32_t own(uint32_t m) { return E == 8 ? m & 0xffff0000u : m; }
  // codes of the elements, and their sum added to `sum`
  static __device__ inline void codes(const Raw16& q, const I8Grid& g, uint32_t (&out)[E / 4], int& sum) {
#pragma unroll
    for (int k = 0; k < E / 4; ++k) out[k] = 0;
#pragma unroll
    for (int k = 0; k < E; ++k) {
      const uint32_t u = q.w[E == 8 ? k / 2 : k];
      const int c = g.code(__uint_as_float(E == 4 ? u : k & 1 ? u & 0xffff0000u : u << 16));
      sum += c;
      out[k / 4] |= uint32_t(c & 255) << (8 * (k % 4));
    }
  }
};

// A row in registers: CH chunks of 16 bytes a thread, read once (chunk c is
// register c / TPB of thread c % TPB), rounded and written as 16-byte (fp32:
// 4-byte) pieces of codes. Rows need no alignment beyond their element's;
// elements past the last full chunk are one value each of the first threads.
// A row with a NaN or an infinity gets scale NaN and codes 0, so that its
// products are NaN; one whose scale is 0 gets codes 0.
template <class T, int CH, int TPB>
__global__ __launch_bounds__(TPB) void quantize_rows_kernel(const T* __restrict__ x, int d, int64_t ldx,
                                                            int row_bytes, float clip,
                                                            int8_t* __restrict__ codes,
                                                            float* __restrict__ scale,
                                                            int32_t* __restrict__ sums) {
  using Chunk = I8Chunk<T>;
  constexpr int E = Chunk::E, NW = TPB / 64;
  __shared__ uint32_t pm[NW];
  __shared__ int ps[NW];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const int64_t row = blockIdx.x;
  const T* xr = x + row * ldx;
  const int full = d / E;
  Raw16 q[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    q[i] = Raw16{};
    if (i * TPB + t < full) q[i] = load_once(xr + int64_t(i * TPB + t) * E);
  }
  float tail = 0.f;
  if (full * E + t < d) tail = load_f32(xr + full * E + t);
  uint32_t m = __float_as_uint(fabsf(tail));
#pragma unroll
  for (int i = 0; i < CH; ++i) m = Chunk::largest(m, q[i]);
  m = Chunk::own(m);
  m = wave_reduce(m, Max());
  if (lane == 0) pm[w] = m;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < NW; ++k) m = max(m, pm[k]);
  const float s = i8_scale(m, clip);
  const I8Grid grid(s);
  int8_t* cr = codes + row * row_bytes;
  int sum = 0;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = i * TPB + t;
    if (c < full) {
      uint32_t out[E / 4];
      Chunk::codes(q[i], grid, out, sum);
      __builtin_memcpy(__builtin_assume_aligned(cr + c * E, E), out, E);
    }
  }
  // the last elements, and the zeros up to the row's end
  for (int k = full * E + t; k < row_bytes; k += TPB) {
    const int code = k < d ? grid.code(tail) : 0;
    sum += code;
    cr[k] = int8_t(code);
  }
  sum = wave_reduce(sum, Sum());
  if (lane == 0) ps[w] = sum;
  __syncthreads();
  if (t == 0) {
#pragma unroll
    for (int k = 1; k < NW; ++k) sum += ps[k];
    scale[row] = s;
    sums[row] = sum;
  }
}

// codes of the sweep (0 .. 255) as signed bytes q - 128, rows padded with 0. Once
// for a layer: a byte a thread and step, 1.7 TB/s (8192 x 28672: 270 us, a copy
// 90).
__global__ __launch_bounds__(256) void pack_i8_kernel(const uint8_t* __restrict__ codes,
                                                      const float* __restrict__ zero, int64_t d,
                                                      int64_t row_bytes, int8_t* __restrict__ packed,
                                                      float* __restrict__ zero_out) {
  const int64_t row = blockIdx.x;
  for (int64_t k = threadIdx.x; k < row_bytes; k += 256)
    packed[row * row_bytes + k] = k < d ? int8_t(int(codes[row * d + k]) - 128) : int8_t(0);
  if (threadIdx.x == 0) zero_out[row] = zero[row] - 128.f;
}

// y of one exact sum (see the top of the file), the same bits whichever kernel
// made the sum: its conversion, the two scales and the bias each round once, and
// none of them is joined with another. No bias: -0, which changes nothing.
constexpr float NO_BIAS = -0.f;
__device__ __forceinline__ float i8_value(int sum, float a_scale, float w_scale, float bias) {
#pragma clang fp contract(off)
  return float(sum) * a_scale * w_scale + bias;
}

struct I8Epi {
  const float* a_scale;
  const int32_t* a_sum;
  const float* w_scale;
  const float* w_zero;  // NULL: symmetric
  const float* bias;    // NULL: none
  int64_t n, m, ldy;

  template <class Y>
  __device__ __forceinline__ void put(int sum, int64_t t, int64_t o, Y* y) const {
    if (w_zero) sum -= int(rintf(w_zero[o])) * a_sum[t];
    store_y(y + t * ldy + o, i8_value(sum, a_scale[t], w_scale[o], bias ? bias[o] : NO_BIAS));
  }
};

// ---------------------------------------------------------------- the GEMM
// Many tokens: a workgroup owns TM tokens x TN channels, each of its WT x WO
// waves a part of them in tiles of v_mfma_i32_32x32x32_i8 (A: channels, B:
// tokens; lane l holds 16 bytes of row l % 32 at k = 16 (l / 32), and of the
// result channels 8 (r / 4) + 4 (l / 32) + r % 4 of token l % 32 in register r).
//
// Stages of 128 bytes of K of all rows stream from memory straight into LDS
// through a ring of NST slots (64 bytes in a ring of 4: 10 % slower at 8192
// tokens, 28672 -> 8192). 16-byte chunk c of row r lies at c ^ (r / 2 % 8) of
// its 128 bytes, so that the 16 lanes that LDS serves together, 16 rows at one
// c, touch different groups of banks.
//
// At 8192 tokens, 28672 -> 8192, tiles of 256 x 256 reach 2.7 POP/s: a stage
// takes some 2600 cycles, its MFMAs 2048, at the 1.9 GHz that the part holds
// under this load; 8 waves (4 waves of 128 x 128 need fewer LDS reads but have
// nothing to run beside their own waits: 2.2 POP/s).

// 16 bytes per lane from base + off into LDS: lane l's at lds_addr + 16 l.
// Complete once vmcnt has counted the load down. (A write of m0 needs a wait
// state before the load that takes it; the compiler puts none within asm.)
__device__ inline void dma16(const int8_t* base, uint32_t off, uint32_t lds_addr) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(off), "s"(base), "s"(__builtin_amdgcn_readfirstlane(lds_addr))
               : "memory", "m0");
}

template <int N>
__device__ inline void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// orders a wave's own LDS accesses
__device__ inline void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <int TM_, int TN_, int WT_, int WO_, int NST_>
struct I8Tile {
  static constexpr int TM = TM_, TN = TN_;           // tokens, channels of a workgroup
  static constexpr int WT = WT_, WO = WO_;           // its waves along them
  static constexpr int KB = 128;                     // bytes of K of a stage
  static constexpr int NST = NST_;                   // slots of the ring
  static constexpr int NW = WT * WO, MI = TN / WO / 32, NJ = TM / WT / 32;
  static constexpr int STB = (TM + TN) * KB;
  static constexpr int PER = STB / 1024 / NW;        // loads of a wave for a stage
  static constexpr int RPL = 1024 / KB;              // rows of a load
  static constexpr int SLAB = 32 * (32 * MI * 4 + 16);  // bytes a wave turns its results round in
  static constexpr int LDS = NST * STB > NW * SLAB ? NST * STB : NW * SLAB;
  // the chunk swizzle of a row
  static __device__ int swz(int row) { return row >> 1 & 7; }
};

// y from the sums of a wave's tiles: 32 tokens at a time go through LDS as
// they are, so that a lane then has the same few channels of token after
// token, with their scales in registers, and a wave writes whole runs of a
// token's channels. Nothing is loaded
// within the passes (with the tokens' scales read there, and the sums rounded
// in software, a tile of 256 x 192 took 29000 cycles, now 19000), and y goes past
// the caches' usual order (14000: what 256 CUs write at once takes memory 11000).
template <int MI, int NJ, class Y>
__device__ inline void i8_store(const v16i (&acc)[MI][NJ], const I8Epi& e, int64_t t0, int64_t o0,
                                char* slab, Y* y, int32_t* partial) {
  constexpr int W = 32 * MI;                              // channels of a wave
  constexpr int ROWB = W * 4 + 16;                        // padded: rows start in other banks
  constexpr int CH = 16 / int(sizeof(Y));                 // channels of a lane: 16 bytes of y
  constexpr int LPR = W / CH, RPP = 64 / LPR;             // lanes of a token's channels, tokens of a pass
  const int lane = threadIdx.x & 63, lt = lane & 31, lh = lane >> 5;
  const int64_t o = o0 + lane % LPR * CH;
  // the tokens' scales and sums, a lane each
  constexpr int TR = (32 * NJ + 63) / 64;
  float as[TR];
  int32_t sums[TR];
#pragma unroll
  for (int r = 0; r < TR; ++r) {
    const int64_t tk = min(t0 + 64 * r + lane, e.n - 1);
    as[r] = partial ? 0.f : e.a_scale[tk];
    sums[r] = e.w_zero && !partial ? e.a_sum[tk] : 0;
  }
  float ws[CH], bias[CH];
  int32_t wz[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int64_t oc = min(o + k, e.m - 1);
    ws[k] = e.w_scale[oc];
    wz[k] = e.w_zero ? int(rintf(e.w_zero[oc])) : 0;
    bias[k] = e.bias ? e.bias[oc] : NO_BIAS;
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<v4i*>(slab + lt * ROWB + (32 * i + 8 * q + 4 * lh) * 4) =
            v4i{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    wave_sync();  // the slab is the wave's own
#pragma unroll 4
    for (int p = 0; p < (32 + RPP - 1) / RPP; ++p) {
      const int row = p * RPP + lane / LPR;
      const int64_t tk = t0 + 32 * j + row;
      const float a = __shfl(as[j / 2], 32 * (j % 2) + (row & 31));
      const int32_t sum = __shfl(sums[j / 2], 32 * (j % 2) + (row & 31));
      if (lane < RPP * LPR && row < 32 && tk < e.n) {
        const v4i* src = reinterpret_cast<const v4i*>(slab + row * ROWB + lane % LPR * CH * 4);
        if (partial) {  // a share of K: the sums as they are
          int32_t* dst = partial + tk * e.m + o;
#pragma unroll
          for (int q = 0; q < CH / 4; ++q) {
            if (o + 4 * q + 4 <= e.m) *reinterpret_cast<v4i_any*>(dst + 4 * q) = src[q];
            else
              for (int k = 0; k < 4; ++k)
                if (o + 4 * q + k < e.m) dst[4 * q + k] = src[q][k];
          }
          continue;
        }
        Y v[CH];
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          // (both factors have 24 bits)
          store_y(v + k, i8_value(src[k / 4][k % 4] - __mul24(wz[k], sum), a, ws[k], bias[k]));
        }
        Y* dst = y + tk * e.ldy + o;
        if (o + CH <= e.m) {
          Mem16 r;
          __builtin_memcpy(&r, v, 16);
          __builtin_nontemporal_store(r, reinterpret_cast<Mem16*>(dst));
        } else {
          for (int k = 0; k < CH; ++k)
            if (o + k < e.m) dst[k] = v[k];
        }
      }
    }
    wave_sync();
  }
}

// Workgroup b runs on XCD b % 8; each XCD takes a run of tiles in bands of 8
// token tiles, so that its 32 CUs work on 8 x 4 tiles at a time and share
// their 12 strips in its L2.
__device__ inline bool i8_tile(int nt, int no, int* ti, int* oi) {
  const int total = nt * no, per = (total + 7) / 8, in = int(blockIdx.x / 8);
  const int p = int(blockIdx.x % 8) * per + in;
  if (in >= per || p >= total) return false;
  const int band = p / (8 * no), h = min(nt - 8 * band, 8);
  const int q = p - band * 8 * no;
  *ti = __builtin_amdgcn_readfirstlane(band * 8 + q % h);
  *oi = __builtin_amdgcn_readfirstlane(q / h);
  return true;
}

template <class C, class Y>
__global__ __launch_bounds__(64 * C::NW) void gemm_i8_kernel(const int8_t* __restrict__ a,
                                                             const int8_t* __restrict__ w, int64_t rb, I8Epi e,
                                                             Y* __restrict__ y, int32_t* __restrict__ partial) {
  constexpr int TM = C::TM, TN = C::TN, KB = C::KB, KS = KB / 32;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int ti, oi;
  if (!i8_tile(int(cdiv(e.n, TM)), int(cdiv(e.m, TN)), &ti, &oi)) return;
  const int64_t t0 = int64_t(ti) * TM, o0 = int64_t(oi) * TN;
  // this share of the stages of K (of gridDim.y)
  const int all = int(rb / KB), s0 = int(int64_t(all) * blockIdx.y / gridDim.y);
  const int stages = int(int64_t(all) * (blockIdx.y + 1) / gridDim.y) - s0;
  // rows of a stage: TN channels, then TM tokens (the last one again where
  // the matrix ends)
  const int8_t* wb = w + o0 * rb + int64_t(s0) * KB;
  const int8_t* ab = a + t0 * rb + int64_t(s0) * KB;
  uint32_t off[C::PER];
#pragma unroll
  for (int j = 0; j < C::PER; ++j) {
    const int row = C::RPL * (wv * C::PER + j) + lane / (KB / 16);
    const int64_t src = row < TN ? min(int64_t(row), e.m - 1 - o0) : min(int64_t(row - TN), e.n - 1 - t0);
    off[j] = uint32_t(src * rb) + ((lane % (KB / 16) ^ C::swz(row)) << 4);
  }
  const uint32_t lds_base = uint32_t(reinterpret_cast<uintptr_t>(lds));
  auto issue = [&](int s, int slot) {
    const uint32_t sb = lds_base + uint32_t(slot * C::STB + wv * C::PER * 1024);
#pragma unroll
    for (int j = 0; j < C::PER; ++j) {
      const bool chan = C::RPL * (wv * C::PER + j) < TN;  // the same for the wave
      const int8_t* base = (chan ? wb : ab) + int64_t(s) * KB;
      dma16(base, off[j], sb + j * 1024);
    }
  };
  // operand reads of a wave: rows 32 i + l % 32 of its channels and tokens
  const int lr = lane & 31;
  const int so = (wv % C::WO) * (TN / C::WO) * KB, st = (TN + (wv / C::WO) * (TM / C::WT)) * KB;
  int at[KS];
  for (int ks = 0; ks < KS; ++ks) at[ks] = lr * KB + (((2 * ks + (lane >> 5)) ^ C::swz(lr)) << 4);
  struct Frags {
    v4i o[C::MI], t[C::NJ];
  };
  auto read = [&](Frags& f, int slot, int ks) {
    const char* p = lds + slot * C::STB + at[ks];
#pragma unroll
    for (int i = 0; i < C::MI; ++i) f.o[i] = *reinterpret_cast<const v4i*>(p + so + i * 32 * KB);
#pragma unroll
    for (int j = 0; j < C::NJ; ++j) f.t[j] = *reinterpret_cast<const v4i*>(p + st + j * 32 * KB);
  };
  v16i acc[C::MI][C::NJ];
#pragma unroll
  for (int i = 0; i < C::MI; ++i)
#pragma unroll
    for (int j = 0; j < C::NJ; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
  auto mma = [&](const Frags& f) {
#pragma unroll
    for (int i = 0; i < C::MI; ++i)
#pragma unroll
      for (int j = 0; j < C::NJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f.o[i], f.t[j], acc[i][j], 0, 0, 0);
  };
  // the next step's operand reads are issued between the first MFMAs of this one
  auto interleave = [&]() {
    constexpr int N = C::MI * C::NJ, R = C::MI + C::NJ;
    constexpr int PAIRED = R < N ? R : N;
#pragma unroll
    for (int k = 0; k < PAIRED; ++k) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    if constexpr (R > PAIRED) __builtin_amdgcn_sched_group_barrier(0x100, R - PAIRED, 0);
    if constexpr (N > PAIRED) __builtin_amdgcn_sched_group_barrier(0x008, N - PAIRED, 0);
  };
  // at most k stages stay in flight
  auto wait_stages = [&](int k) {
    if (k >= 4) wait_vm<4 * C::PER>();
    else if (k == 3) wait_vm<3 * C::PER>();
    else if (k == 2) wait_vm<2 * C::PER>();
    else if (k == 1) wait_vm<C::PER>();
    else wait_vm<0>();
  };
  static_assert(C::NST <= 5, "wait_stages covers at most 4 stages in flight");
  for (int k = 0; k < C::NST; ++k)
    if (k < stages) issue(k, k);
  wait_stages(min(stages, C::NST) - 1);
  __syncthreads();
  Frags f[2];
  read(f[0], 0, 0);
  int slot = 0;
  for (int s = 0; s + 1 < stages; ++s) {
    const int next = slot + 1 == C::NST ? 0 : slot + 1;
#pragma unroll
    for (int ks = 0; ks + 1 < KS; ++ks) {
      read(f[(ks + 1) & 1], slot, ks + 1);
      mma(f[ks & 1]);
      interleave();
    }
    // stage s + 1 has landed for every wave, and every read of this slot is
    // done (the barrier waits for the wave's own), so it is filled again
    wait_stages(min(stages, s + C::NST) - (s + 2));
    __syncthreads();
    if (s + C::NST < stages) issue(s + C::NST, slot);
    read(f[0], next, 0);
    mma(f[1]);
    interleave();
    slot = next;
  }
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    if (ks + 1 < KS) read(f[(ks + 1) & 1], slot, ks + 1);
    mma(f[ks & 1]);
  }
  __syncthreads();
  i8_store<C::MI, C::NJ>(acc, e, t0 + (wv / C::WO) * (TM / C::WT), o0 + (wv % C::WO) * (TN / C::WO),
                         lds + wv * C::SLAB, y,
                         gridDim.y > 1 ? partial + int64_t(blockIdx.y) * e.n * e.m : nullptr);
}

template <class C, class Y>
kq_status gemm_i8_launch(const int8_t* a, const int8_t* w, int64_t rb, const I8Epi& e, Y* y, int splits,
                         int32_t* partial, hipStream_t s) {
  const auto kernel = gemm_i8_kernel<C, Y>;
  static std::atomic<uint64_t> allowed{0};
  KQ_TRY(allow_lds(kernel, C::LDS, allowed));
  const dim3 grid(unsigned(8 * cdiv(cdiv(e.n, C::TM) * cdiv(e.m, C::TN), 8)), unsigned(splits));
  kernel<<<grid, 64 * C::NW, C::LDS, s>>>(a, w, rb, e, y, partial);
  KQ_HIP(hipGetLastError());
  return KQ_OK;
}

// ------------------------------------------------------- few tokens
// Up to 32 tokens: the channels' codes stream from memory through registers into
// the matrix cores (no LDS, no barrier, every byte read once), 16 channels a
// workgroup of SW waves, which share the 128-byte lines of a row and join their
// sums in LDS: integers, in any order the same. In v_mfma_i32_16x16x64_i8 A is
// the channels and B the tokens: lane l holds 16 bytes of row l % 16 at k = 16
// (l / 16), and of the result channels 4 (l / 16) + r of token l % 16 in register
// r. A wave's load is 16 rows of 64 bytes, four lines in flight (two with 32
// tokens), neighbouring waves on neighbouring lines. 1 token, 28672 -> 8192: 43
// us, 5.5 TB/s of codes: memory.
template <int TT, int SW>
struct StreamTile {
  v4i acc[TT];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = v4i{0, 0, 0, 0};
  }
  // A wave's sums for the others. part: SW * TT * 64 vectors of LDS.
  __device__ __forceinline__ void leave(v4i* part, int wv, int lane) const {
#pragma unroll
    for (int t = 0; t < TT; ++t) part[(wv * TT + t) * 64 + lane] = acc[t];
  }
  // The sums of all waves, joined: finish(sum, channel, token) by one thread each.
  template <class F>
  __device__ static __forceinline__ void join(const v4i* part, F finish) {
    for (int j = threadIdx.x; j < TT * 256; j += 64 * SW) {
      const int c = j % 16, tk = j / 16, ln = (c / 4) * 16 + tk % 16;
      int sum = 0;
#pragma unroll
      for (int k = 0; k < SW; ++k) sum += part[(k * TT + tk / 16) * 64 + ln][c % 4];
      finish(sum, c, tk);
    }
  }
};

// gridDim.y workgroups share the lines of a row of codes; with more than one,
// their sums go to `partial` (gridDim.y x n x m) and are joined afterwards.
template <int TT, int SW, class Y>
__global__ __launch_bounds__(64 * SW) void stream_i8_kernel(const int8_t* __restrict__ a,
                                                            const int8_t* __restrict__ w, int64_t rb, I8Epi e,
                                                            Y* __restrict__ y, int32_t* __restrict__ partial) {
  __shared__ v4i part[SW * TT * 64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  const int64_t o0 = int64_t(blockIdx.x) * 16;
  const int8_t* wp = w + min(o0 + i, e.m - 1) * rb + 16 * g;
  const int8_t* ap[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) ap[t] = a + min(int64_t(16 * t + i), e.n - 1) * rb + 16 * g;
  StreamTile<TT, SW> tile;
  tile.clear();
  constexpr int U = TT == 1 ? 4 : 2;  // 128-byte lines in flight
  const int lines = int(rb / 128), step = SW * int(gridDim.y);
  auto run = [&](int line, auto count) {
    constexpr int N = decltype(count)::value;
    v4i fw[N][2], fa[N][2][TT];
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t k = int64_t(line + u * step) * 128 + 64 * h;
        fw[u][h] = *reinterpret_cast<const v4i*>(wp + k);
#pragma unroll
        for (int t = 0; t < TT; ++t) fa[u][h][t] = *reinterpret_cast<const v4i*>(ap[t] + k);
      }
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < TT; ++t)
          tile.acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[u][h], fa[u][h][t], tile.acc[t], 0, 0, 0);
  };
  int line = int(blockIdx.y) * SW + wv;
  for (; line + (U - 1) * step < lines; line += U * step) run(line, std::integral_constant<int, U>());
  for (; line < lines; line += step) run(line, std::integral_constant<int, 1>());
  tile.leave(part, wv, lane);
  __syncthreads();
  tile.join(part, [&](int sum, int c, int tk) {
    const int64_t o = o0 + c;
    if (tk >= e.n || o >= e.m) return;
    if (gridDim.y > 1) partial[(int64_t(blockIdx.y) * e.n + tk) * e.m + o] = sum;
    else e.put(sum, tk, o, y);
  });
}

// The same where many channels meet several tokens. There every 16 channels
// read all tokens' codes once more, and from the caches that takes as long as
// the channels' own bytes do from memory (28672 -> 8192: 43 us with 1 token, 58
// with 12). So a workgroup keeps
// its share of the tokens in registers, U lines a wave, U * SW at most, and
// goes from 16 channels to the next, which are loaded while these are
// multiplied: 12 tokens 48 us, with the launch that joins the shares; without
// one (16 tokens, 4096 -> 32000) 27 us where each workgroup reads them 37.
template <int TT, int U, int SW, class Y>
__global__ __launch_bounds__(64 * SW) void kept_i8_kernel(const int8_t* __restrict__ a, const int8_t* __restrict__ w,
                                                          int64_t rb, I8Epi e, Y* __restrict__ y,
                                                          int32_t* __restrict__ partial) {
  __shared__ v4i part[2][SW * TT * 64];  // by turns: a barrier for each 16 channels
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lines = int(rb / 128), tiles = int(cdiv(e.m, 16));
  const int first = int(int64_t(lines) * blockIdx.y / gridDim.y);
  const int end = int(int64_t(lines) * (blockIdx.y + 1) / gridDim.y);
  // lines past the share: its last line of channels, zeros for tokens
  int at[U];
#pragma unroll
  for (int u = 0; u < U; ++u) at[u] = min(first + wv + u * SW, end - 1) * 128;
  auto load = [&](int t, v4i (&f)[U][2]) {
    const int8_t* p = w + min(int64_t(min(t, tiles - 1)) * 16 + i, e.m - 1) * rb + 16 * g;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) f[u][h] = *reinterpret_cast<const v4i*>(p + at[u] + 64 * h);
  };
  v4i fa[U][2][TT], f0[U][2], f1[U][2];
  int t = blockIdx.x;
  load(t, f0);
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < TT; ++q) {
        const int8_t* p = a + min(int64_t(16 * q + i), e.n - 1) * rb + 16 * g + at[u] + 64 * h;
        const v4i v = *reinterpret_cast<const v4i*>(p);
        fa[u][h][q] = first + wv + u * SW < end ? v : v4i{0, 0, 0, 0};
      }
  auto step = [&](v4i (&f)[U][2], v4i (&ahead)[U][2], v4i* mine) {
    load(t + int(gridDim.x), ahead);
    StreamTile<TT, SW> tile;
    tile.clear();
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < TT; ++q)
          tile.acc[q] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f[u][h], fa[u][h][q], tile.acc[q], 0, 0, 0);
    tile.leave(mine, wv, lane);
    // LDS alone: the loads stay in flight
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    tile.join(mine, [&](int sum, int c, int tk) {
      const int64_t o = int64_t(t) * 16 + c;
      if (tk >= e.n || o >= e.m) return;
      if (gridDim.y > 1) partial[(int64_t(blockIdx.y) * e.n + tk) * e.m + o] = sum;
      else e.put(sum, tk, o, y);
    });
    t += int(gridDim.x);
    return t < tiles;
  };
  while (step(f0, f1, part[0]) && step(f1, f0, part[1])) {
  }
}

// The smallest calls: the same with the tokens rounded on the way, by every
// workgroup for itself (into LDS, rows 16 bytes apart from a multiple of 128
// so that 16 tokens' chunks lie in different banks). The waves split the
// tokens among them; the first weights are on their way meanwhile.
constexpr int FUSED_CH(int size) { return size == 2 ? 4 : 8; }  // chunks of a thread
// waves for a token
__host__ __device__ constexpr int fused_waves(int64_t n) { return n <= 1 ? 16 : n <= 2 ? 8 : n <= 4 ? 4 : n <= 8 ? 2 : 1; }

template <class T, class Y>
__global__ __launch_bounds__(1024) void fused_i8_kernel(const T* __restrict__ x, int d, int64_t ldx,
                                                           float clip, const int8_t* __restrict__ w, int64_t rb,
                                                           I8Epi e, Y* __restrict__ y) {
  using Chunk = I8Chunk<T>;
  constexpr int E = Chunk::E, CH = FUSED_CH(sizeof(T)), U = 2, SW = 16;
  extern __shared__ __attribute__((aligned(16))) int8_t codes[];
  __shared__ v4i part[SW * 64];
  __shared__ uint32_t pm[SW];
  __shared__ int ps[SW];
  __shared__ float scale[16];
  __shared__ int sums[16];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  const int64_t o0 = int64_t(blockIdx.x) * 16;
  const int lines = int(rb / 128), rs = int(rb) + 16;
  const int8_t* wp = w + min(o0 + i, e.m - 1) * rb + 16 * g;
  // ---- the tokens: wave wv takes part of token wv / wpt
  const int wpt = fused_waves(e.n), tok = wv / wpt, at = (wv % wpt) * 64 + lane, step = 64 * wpt;
  const bool have = tok < e.n;
  const T* xr = x + (have ? tok : 0) * ldx;
  const int full = d / E;
  Raw16 q[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    q[k] = Raw16{};
    if (have && at + k * step < full) q[k] = *reinterpret_cast<const Raw16*>(xr + int64_t(at + k * step) * E);
  }
  float tail = 0.f;
  if (have && full * E + at < d) tail = load_f32(xr + full * E + at);
  v4i first[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      first[u][h] = *reinterpret_cast<const v4i*>(wp + int64_t(min(wv + u * SW, lines - 1)) * 128 + 64 * h);
  uint32_t m = __float_as_uint(fabsf(tail));
#pragma unroll
  for (int k = 0; k < CH; ++k) m = Chunk::largest(m, q[k]);
  m = Chunk::own(m);
  m = wave_reduce(m, Max());
  if (lane == 0) pm[wv] = m;
  __syncthreads();
  m = wave_reduce(pm[tok * wpt + (lane & (wpt - 1))], Max());
  const float s = i8_scale(m, clip);
  const I8Grid grid(s);
  int8_t* cr = codes + tok * rs;
  int sum = 0;
  if (have) {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = at + k * step;
      if (c < full) {
        uint32_t out[E / 4];
        Chunk::codes(q[k], grid, out, sum);
        __builtin_memcpy(__builtin_assume_aligned(cr + c * E, E), out, E);
      }
    }
    for (int k = full * E + at; k < rb; k += step) {
      const int code = k < d ? grid.code(tail) : 0;
      sum += code;
      cr[k] = int8_t(code);
    }
  }
  sum = wave_reduce(sum, Sum());
  if (lane == 0) ps[wv] = sum;
  __syncthreads();
  if (have && wv % wpt == 0) {
    sum = wave_reduce(lane < wpt ? ps[tok * wpt + lane] : 0, Sum());
    if (lane == 0) scale[tok] = s, sums[tok] = sum;
  }
  // ---- the product
  const int8_t* ap = codes + min(i, int(e.n) - 1) * rs + 16 * g;
  StreamTile<1, SW> tile;
  tile.clear();
  auto mma = [&](const v4i& fw, int line, int h) {
    const v4i fa = *reinterpret_cast<const v4i*>(ap + line * 128 + 64 * h);
    tile.acc[0] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw, fa, tile.acc[0], 0, 0, 0);
  };
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (wv + u * SW < lines) mma(first[u][h], wv + u * SW, h);
#pragma unroll 2
  for (int line = wv + U * SW; line < lines; line += SW) {
    const v4i f0 = *reinterpret_cast<const v4i*>(wp + int64_t(line) * 128);
    const v4i f1 = *reinterpret_cast<const v4i*>(wp + int64_t(line) * 128 + 64);
    mma(f0, line, 0);
    mma(f1, line, 1);
  }
  e.a_scale = scale;
  e.a_sum = sums;
  tile.leave(part, wv, lane);
  __syncthreads();
  tile.join(part, [&](int acc, int c, int tk) {
    if (tk < e.n && o0 + c < e.m) e.put(acc, tk, o0 + c, y);
  });
}

// y from the sums that `splits` workgroups left, 4 channels a thread
template <class Y>
__global__ __launch_bounds__(256) void join_i8_kernel(const int32_t* __restrict__ partial, int splits, I8Epi e,
                                                      Y* __restrict__ y) {
  const int64_t per = cdiv(e.m, 1024), t = blockIdx.x / per;
  const int64_t o = (blockIdx.x - t * per) * 1024 + 4 * threadIdx.x;
  if (o >= e.m) return;
  const int32_t* p = partial + t * e.m + o;
  const int64_t share = e.n * e.m;
  if (o + 4 <= e.m) {
    v4i sum = {0, 0, 0, 0};
#pragma unroll 4
    for (int k = 0; k < splits; ++k) sum += *reinterpret_cast<const v4i_any*>(p + k * share);
    for (int i = 0; i < 4; ++i) e.put(sum[i], t, o + i, y);
  } else {
    for (int i = 0; o + i < e.m; ++i) {
      int sum = 0;
      for (int k = 0; k < splits; ++k) sum += p[k * share + i];
      e.put(sum, t, o + i, y);
    }
  }
}

template <class Y>
kq_status join_i8_launch(const int32_t* partial, int splits, const I8Epi& e, Y* y, hipStream_t s) {
  join_i8_kernel<<<unsigned(cdiv(e.m, 1024) * e.n), 256, 0, s>>>(partial, splits, e, y);
  KQ_HIP(hipGetLastError());
  return KQ_OK;
}

}  // namespace

int64_t i8_row_bytes(int64_t d_in) { return cdiv(d_in, I8_PAD) * I8_PAD; }

kq_status quantize_rows_run(const void* x, kq_dtype dt, int64_t n, int64_t d, int64_t ldx, float clip,
                            int8_t* codes, float* scale, int32_t* sums, hipStream_t s) {
  auto launch = [&](auto* p) -> kq_status {
    using T = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    const int64_t chunks = cdiv(d * int64_t(sizeof(T)), 16);
    auto go = [&](auto kernel, int tpb) -> kq_status {
      kernel<<<unsigned(n), tpb, 0, s>>>(p, int(d), ldx, int(i8_row_bytes(d)), clip, codes, scale, sums);
      KQ_HIP(hipGetLastError());
      return KQ_OK;
    };
    // small workgroups, several to a CU, for short rows; 1024 threads for long ones
    if (chunks <= 256 * 2) return go(quantize_rows_kernel<T, 2, 256>, 256);
    if (chunks <= 512 * 4) return go(quantize_rows_kernel<T, 4, 512>, 512);
    if (chunks <= 1024 * 4) return go(quantize_rows_kernel<T, 4, 1024>, 1024);
    if (chunks <= 1024 * 8) return go(quantize_rows_kernel<T, 8, 1024>, 1024);
    if constexpr (sizeof(T) == 4) return go(quantize_rows_kernel<T, 16, 1024>, 1024);
    return fail(KQ_ERR_SHAPE, "quantize_rows: d_in");  // not reached: d_in <= 65536
  };
  if (dt == KQ_BF16) return launch(static_cast<const uint16_t*>(x));
  return launch(static_cast<const float*>(x));
}

kq_status pack_i8_run(const uint8_t* codes, const float* zero, int64_t d_out, int64_t d_in, int8_t* packed,
                      float* zero_out, hipStream_t s) {
  pack_i8_kernel<<<unsigned(d_out), 256, 0, s>>>(codes, zero, d_in, i8_row_bytes(d_in), packed, zero_out);
  KQ_HIP(hipGetLastError());
  return KQ_OK;
}

namespace {

// How a product is taken, by its sizes alone.
enum I8Kind { I8_STREAM, I8_KEPT, I8_64, I8_128, I8_128_256, I8_256_192, I8_256 };
struct I8Plan {
  I8Kind kind;
  int splits;  // shares of K
};

I8Plan i8_plan(int64_t n, int64_t m, int64_t d) {
  const int64_t lines = cdiv(d, I8_PAD);
  if (n <= 32) {
    // Few tokens: the channels' bytes are what counts, 16 channels a workgroup,
    // until the tokens' bytes, read for each, cost more than keeping them in
    // registers. That costs a second launch where the rows are longer than the
    // 32 lines that a workgroup keeps: it is worth it from about 300000 lines
    // of tokens on (4096 -> 14336, 112 lines: 10 tokens 17.6 us streamed and
    // kept, 16 tokens 19.4 and 18.3; 8192 -> 28672: 6 tokens 48 and 47, 16
    // tokens 64 and 48), else from 640 groups of channels on (1 token, 4096 ->
    // 11008: 13.8 and 12.0; 2048 -> 8192: 4.1 and 4.7).
    const int64_t groups = cdiv(m, 16), shares = cdiv(lines, 32);
    if (shares == 1 ? groups >= 640 : groups >= 256 && groups * lines * n >= 300000)
      return I8Plan{I8_KEPT, int(shares)};
    // Long rows of few channels are shared (16 tokens, 8192 -> 1024: 10.2 us,
    // shared by 4 7.6; 4096 -> 1024: 6.1, shared by 2 6.6).
    if (groups < 256 && lines >= 64) return I8Plan{I8_STREAM, int(std::min(256 / groups, lines / 16))};
    return I8Plan{I8_STREAM, 1};
  }
  // The tile (tokens x channels): the CU with most tiles takes k = ceil(tiles /
  // 256) of them, each some time for every 128-byte stage of K and some at
  // its ends; a CU's only tile has it for itself. Fitted to the times of every
  // tile at 54 sizes, three of them: 8192 tokens, 28672 -> 8192 (1442 us with
  // 256 x 256, 1683 with 256 x 192, 1621 and 1802 with 128 x 256 and 128 x 128),
  // 2048 tokens, 4096 -> 11008 (101, 88, 96, 95, and 150 with 64 x 64) and 512,
  // 4096 -> 4096 (45, 38, 29, 27 and 18). With fewer tiles than CUs the stages
  // are shared, for the launch that joins the sums and its traffic (600 tokens,
  // 20000 -> 600: 27 us with 4 shares, 46 with one). The chosen tile is the
  // fastest or within 3 % at 50 of the 54; the worst miss is 23 us for 21 (73
  // tokens, 7856 -> 4159).
  static const struct {
    I8Kind kind;
    int64_t tm, tn;
    double stage, ends, lone_stage;
  } tiles[] = {{I8_256, 256, 256, 1.2, 10.8, 1.4},
               {I8_256_192, 256, 192, 1.035, 8.0, 1.17},
               {I8_128_256, 128, 256, 0.785, 5.3, 0.89},
               {I8_128, 128, 128, 0.444, 3.25, 0.83},
               {I8_64, 64, 64, 0.267, 0.98, 0.293}};
  I8Plan best{I8_64, 1};
  double least = 1e30;
  for (const auto& t : tiles) {
    const int64_t count = cdiv(n, t.tm) * cdiv(m, t.tn);
    for (int64_t splits = 1; splits <= 8; splits *= 2) {
      if (splits > 1 && (count * splits > 512 || lines < 4 * splits)) break;
      const int64_t k = cdiv(count * splits, 256);
      const double stages = double(cdiv(lines, splits));
      double us = k == 1 ? stages * t.lone_stage + 3.0 : double(k) * (stages * t.stage + t.ends);
      if (splits > 1) us += 3.0 + double(splits) * double(n) * double(m) * 2.6e-6;
      if (us < least) least = us, best = I8Plan{t.kind, int(splits)};
    }
  }
  return best;
}

// Whether the tokens are rounded within the product: it takes the place of a
// launch (the host's time for it, 2.5 us, too) and a pass through memory, but
// every workgroup does it, 256 at a time, 16 channels each. us of the kernels
// rounded within, and apart:
//   1 token   4096 ->  4096   6.3,  9.9    4096 -> 12288  14.4, 16.7
//   1 token  16384 ->  6144  29.4, 32.3   16384 -> 12288  45.7, 42.3
//   2 tokens  4096 ->  8192  11.4, 13.1    4096 -> 12288  15.4, 16.8
//   2 tokens  8192 ->  6144  18.0, 18.2    8192 -> 12288  26.9, 24.2
//   4 tokens  4096 ->  4096   8.2, 10.4    4096 ->  5120  13.1, 12.8
//   8 tokens  2048 ->  4096   7.0,  7.4    2048 ->  5120  11.7,  8.8
//   8 tokens  1024 ->  8192   8.8,  7.4 (with the host's time 8.7, 10.7)
//   8 tokens  1024 -> 12288  13.0,  8.8
bool i8_fused(int64_t n, int64_t m, int64_t d) {
  if (n > 8 || (16 / fused_waves(n)) * d > 16384) return false;  // its registers
  if (m <= 4096) return true;
  if (m <= 8192) return n * d < 16384 || (n <= 2 && m <= 6144);
  return m <= 12288 && d > 2048 && n * d <= 8192;
}

}  // namespace

size_t matmul_i8_ws_bytes(int64_t m, int64_t d, int64_t n) {
  const I8Plan p = i8_plan(n, m, d);
  return p.splits > 1 ? size_t(p.splits) * n * m * sizeof(int32_t) : 0;
}

kq_status matmul_i8_run(const int8_t* a, const float* a_scale, const int32_t* a_sum, const int8_t* w,
                        const float* w_scale, const float* w_zero, const float* bias, int64_t n, int64_t m,
                        int64_t d, void* y, kq_dtype dt, int64_t ldy, Arena& ws, hipStream_t s) {
  const int64_t rb = i8_row_bytes(d);
  const I8Epi e{a_scale, a_sum, w_scale, w_zero, bias, n, m, ldy};
  const I8Plan p = i8_plan(n, m, d);
  int32_t* partial = nullptr;
  if (p.splits > 1) {
    partial = ws.take<int32_t>(size_t(p.splits) * n * m);
    if (!partial) return fail(KQ_ERR_WORKSPACE, "matmul_i8: workspace too small");
  }
  auto product = [&](auto* out) -> kq_status {
    using Y = std::remove_pointer_t<decltype(out)>;
    auto rows = [&](auto kernel, int waves, int64_t groups) -> kq_status {
      kernel<<<dim3(unsigned(groups), unsigned(p.splits)), 64 * waves, 0, s>>>(a, w, rb, e, out, partial);
      KQ_HIP(hipGetLastError());
      return KQ_OK;
    };
    const int64_t groups = cdiv(m, 16);
    switch (p.kind) {
      case I8_STREAM:
        if (n <= 16) return rows(stream_i8_kernel<1, 16, Y>, 16, groups);
        return rows(stream_i8_kernel<2, 8, Y>, 8, groups);
      case I8_KEPT: {
        // 16 waves a CU over all shares, each with 1 or 2 lines
        const int64_t share = cdiv(rb / I8_PAD, p.splits);
        const int64_t all = std::min<int64_t>(groups, 256 / p.splits);
        if (share <= 8) {
          if (n <= 16) return rows(kept_i8_kernel<1, 1, 8, Y>, 8, std::min<int64_t>(groups, 512));
          return rows(kept_i8_kernel<2, 1, 8, Y>, 8, std::min<int64_t>(groups, 512));
        }
        if (share <= 16) {
          if (n <= 16) return rows(kept_i8_kernel<1, 1, 16, Y>, 16, all);
          return rows(kept_i8_kernel<2, 1, 16, Y>, 16, all);
        }
        if (n <= 16) return rows(kept_i8_kernel<1, 2, 16, Y>, 16, all);
        return rows(kept_i8_kernel<2, 2, 16, Y>, 16, all);
      }
      case I8_256: return gemm_i8_launch<I8Tile<256, 256, 2, 4, 2>>(a, w, rb, e, out, p.splits, partial, s);
      case I8_256_192:
        return gemm_i8_launch<I8Tile<256, 192, 4, 2, 2>>(a, w, rb, e, out, p.splits, partial, s);
      case I8_128_256:
        return gemm_i8_launch<I8Tile<128, 256, 2, 4, 3>>(a, w, rb, e, out, p.splits, partial, s);
      case I8_128: return gemm_i8_launch<I8Tile<128, 128, 2, 2, 2>>(a, w, rb, e, out, p.splits, partial, s);
      default: return gemm_i8_launch<I8Tile<64, 64, 2, 2, 4>>(a, w, rb, e, out, p.splits, partial, s);
    }
  };
  auto go = [&](auto* out) -> kq_status {
    KQ_TRY(product(out));
    return p.splits > 1 ? join_i8_launch(partial, p.splits, e, out, s) : KQ_OK;
  };
  if (dt == KQ_BF16) return go(static_cast<uint16_t*>(y));
  return go(static_cast<float*>(y));
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
  if (i8_fused(n, m, d)) return 0;
  Arena ar{nullptr, 0, 0};
  linear_take(ar, n, d);
  ar.take<char>(matmul_i8_ws_bytes(m, d, n));
  return ar.used;
}

kq_status linear_i8_run(const void* x, kq_dtype dt, int64_t ldx, float clip, const int8_t* w,
                        const float* w_scale, const float* w_zero, const float* bias, int64_t n, int64_t m,
                        int64_t d, void* y, kq_dtype ydt, int64_t ldy, Arena& ws, hipStream_t s) {
  if (i8_fused(n, m, d)) {
    const int64_t rb = i8_row_bytes(d);
    const I8Epi e{nullptr, nullptr, w_scale, w_zero, bias, n, m, ldy};
    auto go = [&](auto* in, auto* out) -> kq_status {
      using T = std::remove_const_t<std::remove_pointer_t<decltype(in)>>;
      using Y = std::remove_pointer_t<decltype(out)>;
      fused_i8_kernel<T, Y><<<unsigned(cdiv(m, 16)), 1024, size_t(n) * (rb + 16), s>>>(in, int(d), ldx, clip, w,
                                                                                         rb, e, out);
      KQ_HIP(hipGetLastError());
      return KQ_OK;
    };
    auto with_y = [&](auto* in) -> kq_status {
      if (ydt == KQ_BF16) return go(in, static_cast<uint16_t*>(y));
      return go(in, static_cast<float*>(y));
    };
    if (dt == KQ_BF16) return with_y(static_cast<const uint16_t*>(x));
    return with_y(static_cast<const float*>(x));
  }
  const LinearWs l = linear_take(ws, n, d);
  if (!l.codes || !l.scale || !l.sums) return fail(KQ_ERR_WORKSPACE, "linear_i8: workspace too small");
  KQ_TRY(quantize_rows_run(x, dt, n, d, ldx, clip, l.codes, l.scale, l.sums, s));
  return matmul_i8_run(l.codes, l.scale, l.sums, w, w_scale, w_zero, bias, n, m, d, y, ydt, ldy, ws, s);
}

}  // namespace kq
