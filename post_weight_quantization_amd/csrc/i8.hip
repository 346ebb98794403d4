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
#include <type_traits>

#include "kq_internal.h"

namespace kq {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

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

struct __attribute__((packed, aligned(2))) Raw16 {
  uint32_t w[4];
};

// the code of one value; s > 0 and finite
__device__ inline int i8_code(float v, float s) {
  return int(fminf(fmaxf(rintf(v / s), -127.f), 127.f));
}

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
  constexpr int E = 16 / int(sizeof(T)), NW = TPB / 64;
  __shared__ uint32_t pm[NW];
  __shared__ int ps[NW];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const int64_t row = blockIdx.x;
  const T* xr = x + row * ldx;
  const int full = d / E;
  Raw16 q[CH];
  // magnitudes order as integers, an infinity and every NaN above the rest
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    q[i] = Raw16{};
    if (i * TPB + t < full) q[i] = *reinterpret_cast<const Raw16*>(xr + int64_t(i * TPB + t) * E);
  }
  float tail = 0.f;
  if (full * E + t < d) tail = load_f32(xr + full * E + t);
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t u = q[i].w[k];
      m = max(m, u & 0x7fffffffu);
      if (E == 8) m = max(m, (u << 16) & 0x7fffffffu);
    }
  // (the upper half of a pair carries the lower one's bits: a bfloat16's own
  // are cut out below)
  m = max(m, __float_as_uint(fabsf(tail)));
  if (E == 8) m &= 0xffff0000u;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = max(m, uint32_t(__shfl_xor(m, o)));
  if (lane == 0) pm[w] = m;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < NW; ++k) m = max(m, pm[k]);
  const float s = m >= 0x7f800000u ? __builtin_nanf("") : clip * __uint_as_float(m) / 127.f;
  int8_t* cr = codes + row * row_bytes;
  int sum = 0;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = i * TPB + t;
    if (c < full) {
      uint32_t out[E / 4] = {};
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const uint32_t u = q[i].w[E == 8 ? k / 2 : k];
        const float v = __uint_as_float(E == 4 ? u : k & 1 ? u & 0xffff0000u : u << 16);
        const int code = s > 0.f ? i8_code(v, s) : 0;
        sum += code;
        out[k / 4] |= uint32_t(code & 255) << (8 * (k % 4));
      }
      __builtin_memcpy(__builtin_assume_aligned(cr + c * E, E), out, E);
    }
  }
  // the last elements, and the zeros up to the row's end
  for (int k = full * E + t; k < row_bytes; k += TPB) {
    const int code = k < d && s > 0.f ? i8_code(tail, s) : 0;
    sum += code;
    cr[k] = int8_t(code);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  if (lane == 0) ps[w] = sum;
  __syncthreads();
  if (t == 0) {
#pragma unroll
    for (int k = 1; k < NW; ++k) sum += ps[k];
    scale[row] = s;
    sums[row] = sum;
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

// ---------------------------------------------------------------- the GEMM
// A workgroup of 4 waves owns TM tokens x TN channels, each wave a quarter of
// them in tiles of v_mfma_i32_32x32x32_i8 (A: channels, B: tokens; lane l
// holds 16 bytes of row l % 32 at k = 16 (l / 32), and of the result channels
// 8 (r / 4) + 4 (l / 32) + r % 4 of token l % 32 in register r).
//
// Stages of 64 bytes of K of all rows stream from memory straight into LDS
// through a ring of NST slots. 16-byte chunk c of row r lies at
// c ^ (r / 4 % 4) of its 64 bytes, so that the 16 lanes that LDS serves
// together, 16 rows at one c, touch 16 different groups of banks.
// 16 bytes per lane from base + off into LDS: lane l's at lds_addr + 16 l.
// Complete once vmcnt has counted the load down.
__device__ inline void dma16(const int8_t* base, uint32_t off, uint32_t lds_addr) {
  asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1"
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

template <int TM_, int TN_, int WT_, int WO_, int KB_, int NST_>
struct I8Tile {
  static constexpr int TM = TM_, TN = TN_;           // tokens, channels of a workgroup
  static constexpr int WT = WT_, WO = WO_;           // its waves along them
  static constexpr int KB = KB_;                     // bytes of K of a stage
  static constexpr int NST = NST_;                   // slots of the ring
  static constexpr int NW = WT * WO, MI = TN / WO / 32, NJ = TM / WT / 32;
  static constexpr int STB = (TM + TN) * KB;
  static constexpr int PER = STB / 1024 / NW;        // loads of a wave for a stage
  static constexpr int RPL = 1024 / KB;              // rows of a load
  static constexpr int SLAB = 32 * (32 * MI * 4 + 16);  // bytes a wave turns its results round in
  static constexpr int LDS = NST * STB > NW * SLAB ? NST * STB : NW * SLAB;
  // the chunk swizzle of a row
  static __device__ int swz(int row) { return KB == 64 ? row >> 2 & 3 : row >> 1 & 7; }
};

// y from the sums of a wave's tiles: 32 tokens at a time go through LDS as
// they are, so that a lane then has the same few channels of token after
// token, with their scales in registers, and a wave writes whole runs of a
// token's channels. The fp32 conversion of the sum, the two scales and the
// bias each round once; y is rounded to its type after that.
template <int MI, int NJ, class Y>
__device__ inline void i8_store(const v16i (&acc)[MI][NJ], const I8Epi& e, int64_t t0, int64_t o0,
                                char* slab, Y* y) {
  constexpr int W = 32 * MI;                              // channels of a wave
  constexpr int ROWB = W * 4 + 16;                        // padded: rows start in other banks
  constexpr int CH = 16 / int(sizeof(Y));                 // channels of a lane: 16 bytes of y
  constexpr int LPR = W / CH;                             // lanes for a token's channels
  const int lane = threadIdx.x & 63, lt = lane & 31, lh = lane >> 5;
  const int64_t o = o0 + lane % LPR * CH;
  float ws[CH], bias[CH];
  int32_t wz[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int64_t oc = min(o + k, e.m - 1);
    ws[k] = e.w_scale[oc];
    wz[k] = e.w_zero ? int(rintf(e.w_zero[oc])) : 0;
    bias[k] = e.bias ? e.bias[oc] : 0.f;
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
#pragma unroll 2
    for (int p = 0; p < 32 * LPR / 64; ++p) {
      const int row = p * (64 / LPR) + lane / LPR;
      const int64_t tk = t0 + 32 * j + row;
      if (tk < e.n) {
        const float as = e.a_scale[tk];
        const int32_t sum = e.w_zero ? e.a_sum[tk] : 0;
        const v4i* src = reinterpret_cast<const v4i*>(slab + row * ROWB + lane % LPR * CH * 4);
        Y v[CH];
#pragma unroll
        for (int k = 0; k < CH; ++k) {
          const float f = float(src[k / 4][k % 4] - wz[k] * sum) * as * ws[k];
          store_y(v + k, e.bias ? f + bias[k] : f);
        }
        Y* dst = y + tk * e.ldy + o;
        if (o + CH <= e.m) {
          Raw16 r;
          __builtin_memcpy(&r, v, 16);
          *reinterpret_cast<Raw16*>(dst) = r;
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
                                                             Y* __restrict__ y) {
  constexpr int TM = C::TM, TN = C::TN, KB = C::KB, KS = KB / 32;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int ti, oi;
  if (!i8_tile(int(cdiv(e.n, TM)), int(cdiv(e.m, TN)), &ti, &oi)) return;
  const int64_t t0 = int64_t(ti) * TM, o0 = int64_t(oi) * TN;
  const int stages = int(rb / KB);
  // rows of a stage: TN channels, then TM tokens (the last one again where
  // the matrix ends)
  const int8_t* wb = w + o0 * rb;
  const int8_t* ab = a + t0 * rb;
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
                         lds + wv * C::SLAB, y);
}

template <class C, class Y>
kq_status gemm_i8_launch(const int8_t* a, const int8_t* w, int64_t rb, const I8Epi& e, Y* y, hipStream_t s) {
  const auto kernel = gemm_i8_kernel<C, Y>;
  KQ_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                             C::LDS));
  kernel<<<unsigned(8 * cdiv(cdiv(e.n, C::TM) * cdiv(e.m, C::TN), 8)), 64 * C::NW, C::LDS, s>>>(a, w, rb, e, y);
  KQ_HIP(hipGetLastError());
  return KQ_OK;
}

// ------------------------------------------------------- few tokens
// The codes of 16 RT channels stream from memory through the registers of 16
// waves, which take the row's 128-byte lines in turn, and meet the codes of
// 16 TT tokens (from L2) in v_mfma_i32_16x16x64_i8 (A: channels, B: tokens;
// lane l holds 16 bytes of row l % 16 at k = 16 (l / 16), and of the result
// channels 4 (l / 16) + r of token l % 16 in register r). The waves' sums
// are joined in LDS: integers, in any order the same.
constexpr int SW = 16;  // waves of a workgroup

template <int RT, int TT, class Y>
__global__ __launch_bounds__(64 * SW) void stream_i8_kernel(const int8_t* __restrict__ a,
                                                            const int8_t* __restrict__ w, int64_t rb, I8Epi e,
                                                            Y* __restrict__ y) {
  __shared__ v4i part[SW][RT * TT][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
  const int64_t o0 = int64_t(blockIdx.x) * (16 * RT);
  const int8_t *wp[RT], *ap[TT];
#pragma unroll
  for (int r = 0; r < RT; ++r) wp[r] = w + min(o0 + 16 * r + i, e.m - 1) * rb + 16 * g;
#pragma unroll
  for (int t = 0; t < TT; ++t) ap[t] = a + min(int64_t(16 * t + i), e.n - 1) * rb + 16 * g;
  v4i acc[RT][TT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[r][t] = v4i{0, 0, 0, 0};
  constexpr int U = TT == 1 ? 4 : 2;  // 128-byte lines in flight
  const int lines = int(rb / 128);
  auto step = [&](int line, auto count) {
    constexpr int N = decltype(count)::value;
    v4i fw[N][2][RT], fa[N][2][TT];
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t k = int64_t(line + u * SW) * 128 + 64 * h;
#pragma unroll
        for (int r = 0; r < RT; ++r) fw[u][h][r] = *reinterpret_cast<const v4i*>(wp[r] + k);
#pragma unroll
        for (int t = 0; t < TT; ++t) fa[u][h][t] = *reinterpret_cast<const v4i*>(ap[t] + k);
      }
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int t = 0; t < TT; ++t)
            acc[r][t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[u][h][r], fa[u][h][t], acc[r][t], 0, 0, 0);
  };
  int line = wv;
  for (; line + (U - 1) * SW < lines; line += U * SW) step(line, std::integral_constant<int, U>());
  for (; line < lines; line += SW) step(line, std::integral_constant<int, 1>());
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) part[wv][r * TT + t][lane] = acc[r][t];
  __syncthreads();
  // one sum a thread: channel c of token tk
  for (int j = threadIdx.x; j < RT * TT * 256; j += 64 * SW) {
    const int c = j % (16 * RT), tk = j / (16 * RT);
    const int64_t o = o0 + c;
    if (tk >= e.n || o >= e.m) continue;
    const int tile = (c / 16) * TT + tk / 16, ln = (c % 16 / 4) * 16 + tk % 16;
    int sum = 0;
#pragma unroll
    for (int k = 0; k < SW; ++k) sum += part[k][tile][ln][c % 4];
    if (e.w_zero) sum -= int(rintf(e.w_zero[o])) * e.a_sum[tk];
    const float f = float(sum) * e.a_scale[tk] * e.w_scale[o];
    store_y(y + tk * e.ldy + o, e.bias ? f + e.bias[o] : f);
  }
}

template <int RT, int TT, class Y>
kq_status stream_i8_launch(const int8_t* a, const int8_t* w, int64_t rb, const I8Epi& e, Y* y, hipStream_t s) {
  stream_i8_kernel<RT, TT><<<unsigned(cdiv(e.m, 16 * RT)), 64 * SW, 0, s>>>(a, w, rb, e, y);
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

size_t matmul_i8_ws_bytes(int64_t, int64_t, int64_t) { return 0; }

kq_status matmul_i8_run(const int8_t* a, const float* a_scale, const int32_t* a_sum, const int8_t* w,
                        const float* w_scale, const float* w_zero, const float* bias, int64_t n, int64_t m,
                        int64_t d, void* y, kq_dtype dt, int64_t ldy, Arena&, hipStream_t s) {
  const int64_t rb = i8_row_bytes(d);
  const I8Epi e{a_scale, a_sum, w_scale, w_zero, bias, n, m, ldy};
  auto go = [&](auto* out) -> kq_status {
    // Few tokens: the weights' bytes are what counts. 32 channels a workgroup
    // where that still gives every CU one (12 tokens, 28672 -> 8192: 39.5 us
    // against 47.6 us with 16), else 16 (1 token, 4096 -> 4096: 5.8 us
    // against 6.5 us with 32).
    if (n <= 32) {
      const bool wide = m >= 32 * 256;
      if (n <= 16) return wide ? stream_i8_launch<2, 1>(a, w, rb, e, out, s) : stream_i8_launch<1, 1>(a, w, rb, e, out, s);
      return wide ? stream_i8_launch<2, 2>(a, w, rb, e, out, s) : stream_i8_launch<1, 2>(a, w, rb, e, out, s);
    }
    // The tile: the CU with most tiles takes ceil(tiles / 256) of them, one
    // after the other, and a stage of a tile took 1.74 us (256 x 256), 0.99
    // (128 x 256), 0.53 (128 x 128) and 0.23 us (64 x 64) at 8192 tokens,
    // 28672 -> 8192; 2048 tokens, 4096 -> 11008, for one, take 117 us, 123,
    // 123 and 183 with them, 512 tokens, 4096 -> 4096, 50, 32, 27 and 17 us.
    auto cost = [&](int64_t tm, int64_t tn, double t) {
      return double(cdiv(cdiv(n, tm) * cdiv(m, tn), 256)) * t;
    };
    const double c1 = cost(256, 256, 1.74), c2 = cost(128, 256, 0.99), c3 = cost(128, 128, 0.53),
                 c4 = cost(64, 64, 0.23);
    if (c1 <= c2 && c1 <= c3 && c1 <= c4) return gemm_i8_launch<I8Tile<256, 256, 2, 4, 128, 2>>(a, w, rb, e, out, s);
    if (c2 <= c3 && c2 <= c4) return gemm_i8_launch<I8Tile<128, 256, 2, 4, 128, 3>>(a, w, rb, e, out, s);
    if (c3 <= c4) return gemm_i8_launch<I8Tile<128, 128, 2, 2, 128, 2>>(a, w, rb, e, out, s);
    return gemm_i8_launch<I8Tile<64, 64, 2, 2, 128, 4>>(a, w, rb, e, out, s);
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
