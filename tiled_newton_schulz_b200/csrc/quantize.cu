// quantize.cu -- 8-bit codes of matrices, one scale per row or per column.
#include <algorithm>

#include "experts.hpp"
#include "layout.hpp"
#include "ptx.cuh"

namespace himuon {
namespace {

struct QuantArgs {
  const void *in[kMaxList];
  int8_t *codes[kMaxList];
  float *scale[kMaxList];
  int64_t rows[kMaxList], cols[kMaxList], ld[kMaxList], ldq[kMaxList];
  int32_t dtype[kMaxList];
  int32_t dim;
};

// code = round(127 x / top), ties to even.  With 127 / top = hi + lo (two fp32
// numbers, the second the division's remainder), p = x hi and e = what p lost, plus
// x lo, p + e is the quotient up to 2^-39 and its fp32 sum s the quotient rounded
// once.  Adding 1.5 * 2^23 then rounds to an integer and leaves it in the low bits.
// Five operations per element: the kernel is bound by its instructions (the plain
// division took 464 us for 8192 x 11008 bf16).  A quotient that is no
// tie lies 2 * 127 x - (2 k + 1) top, at least one last place of x, over 2 top from
// one.  For 16-bit x and a quotient in 2^m .. 2^(m + 1) that is 2^(m - 20), sixteen
// times what s is off, and rounding twice is exact.  For fp32 it may be 2^-33, where
// s is the tie itself; what s lost then decides.  A maximum
// so small or large that hi or x hi could leave fp32's range is multiplied by a power
// of two first, and x with it (an x that loses bits by that has the code 0).
constexpr float kToInt = 12582912.f;
template <int DT>
__device__ __forceinline__ uint32_t exact_code(float x, float hi, float lo) {   // the code in the low byte
  const float p = x * hi, e = fmaf(x, lo, fmaf(x, hi, -p)), s = p + e;
  if (DT != HIMUON_FP32) return __float_as_uint(s + kToInt);
  const float n = s + kToInt - kToInt, d = s - n, lost = e - (s - p);
  const bool next = fabsf(d) == 0.5f && fabsf(lost) > 0x1p-36f && (lost > 0.f) == (d > 0.f);
  return __float_as_uint(n + (next ? 2.f * d : 0.f) + kToInt);
}
// fp32, two at a time (packed arithmetic, 9 instructions a pair): the same codes but
// where s is a tie, of which `ties` tells: it is multiplied by d^2 - 1/4, d being s's
// distance from its integer, which is 0 there (and where the product underflows).
// Those elements are read and coded again.  (8192 x 11008: 73 us; 79 with exact_code
// for every element, 69 without a look at ties.)
struct Pair {
  uint64_t v;
  __device__ __forceinline__ Pair(float a, float b) {
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(__float_as_uint(a)), "r"(__float_as_uint(b)));
  }
  __device__ __forceinline__ explicit Pair(uint64_t bits) : v(bits) {}
  __device__ __forceinline__ void split(uint32_t &a, uint32_t &b) const { asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v)); }
  __device__ __forceinline__ bool any_zero() const {
    uint32_t a, b;
    split(a, b);
    return __uint_as_float(a) == 0.f || __uint_as_float(b) == 0.f;
  }
};
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a.v), "l"(b.v));
  return Pair(d);
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a.v), "l"(b.v));
  return Pair(d);
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a.v), "l"(b.v), "l"(c.v));
  return Pair(d);
}
__device__ __forceinline__ void near_codes(Pair x, Pair hi, Pair minus_hi, Pair minus_lo, uint32_t &c0, uint32_t &c1,
                                           Pair &ties) {
  const Pair minus(-1.f, -1.f), up(kToInt, kToInt), down(-kToInt, -kToInt), quarter(-0.25f, -0.25f);
  const Pair p = x * hi, s = fma2(fma2(x, minus_lo, fma2(x, minus_hi, p)), minus, p);
  const Pair u = s + up, d = fma2(u + down, minus, s);
  ties = ties * fma2(d, d, quarter);
  u.split(c0, c1);
}
struct Coder {
  float hi, lo, mul;
  __device__ explicit Coder(float top) {
    mul = top > 0x1p60f ? 0x1p-100f : top < 0x1p-60f ? 0x1p100f : 1.f;
    const float t = top * mul;
    hi = __fdiv_rn(127.f, t);
    lo = __fdiv_rn(fmaf(-t, hi, 127.f), t);
  }
  __device__ __forceinline__ bool in_range() const { return mul == 1.f; }   // (its codes take x itself)
  template <int DT>
  __device__ __forceinline__ uint32_t code(float x) const {
    return exact_code<DT>(x * mul, hi, lo);
  }
};
__device__ __forceinline__ uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// What the scale and the codes of a line with this maximum are: a line that
// holds an infinity or a NaN has `top` infinite here (the maximum of the bits of
// |x|: a NaN's are above infinity's).
__device__ __forceinline__ bool line_ok(uint32_t top_bits) { return top_bits > 0 && top_bits < 0x7f800000u; }
__device__ __forceinline__ float line_scale(uint32_t top_bits) {
  return top_bits < 0x7f800000u ? __fdiv_rn(__uint_as_float(top_bits), 127.f) : __uint_as_float(0x7fffffffu);
}
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// One scale per row: TPR threads per row.  The row stays in registers between
// the two passes (kHold runs of 8 elements per thread, all loads in flight
// together; longer rows are read again, from L2).  HBM-bound: 3 bytes per
// 16-bit element; 16384 x 4096 bf16 takes 38 us (5.3 TB/s), fp32 50 us (6.7
// TB/s, four fifths of it reads).
__device__ __forceinline__ uint32_t max_s16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.s16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <int DT>
struct Run8 {   // 8 consecutive elements as loaded (16 bits)
  uint4 u;
  __device__ __forceinline__ void load(const char *p, int64_t i) { u = *reinterpret_cast<const uint4 *>(p + 16 * i); }
  // |x| of 16-bit floats orders as an integer: two maxima at a time
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = 0x7fff7fffu;
    return max_s16x2(max_s16x2(u.x & m, u.y & m), max_s16x2(u.z & m, u.w & m));
  }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max_s16x2(a, b); }
  __device__ __forceinline__ float get(int j) const {
    const uint32_t w = j < 2 ? u.x : j < 4 ? u.y : j < 6 ? u.z : u.w;
    if (DT == HIMUON_BF16) return __uint_as_float(j & 1 ? w & 0xffff0000u : w << 16);
    const __half2 h = *reinterpret_cast<const __half2 *>(&w);
    return j & 1 ? __high2float(h) : __low2float(h);
  }
  __device__ __forceinline__ void clear() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load_some(const char *p, int64_t i, int n) {   // n < 8 elements from element i on
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) w[j / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(p)[i + j]) << (16 * (j & 1));
    u = make_uint4(w[0], w[1], w[2], w[3]);
  }
  // the 8 columns' maxima, in pairs until unpack()
  __device__ __forceinline__ void tops(uint32_t (&t)[8]) const {
    const uint32_t m = 0x7fff7fffu;
    t[0] = max_s16x2(t[0], u.x & m);
    t[1] = max_s16x2(t[1], u.y & m);
    t[2] = max_s16x2(t[2], u.z & m);
    t[3] = max_s16x2(t[3], u.w & m);
  }
  static __device__ __forceinline__ void unpack(uint32_t (&t)[8]) {
#pragma unroll
    for (int j = 7; j >= 0; --j) {
      const uint16_t h = static_cast<uint16_t>(j & 1 ? t[j / 2] >> 16 : t[j / 2] & 0xffffu);
      t[j] = DT == HIMUON_FP16 ? abs_bits(__half2float(*reinterpret_cast<const __half *>(&h))) : uint32_t(h) << 16;
    }
  }
};
template <>
struct Run8<HIMUON_FP32> {
  float4 a, b;
  __device__ __forceinline__ void load(const char *p, int64_t i) {
    a = *reinterpret_cast<const float4 *>(p + 32 * i);
    b = *reinterpret_cast<const float4 *>(p + 32 * i + 16);
  }
  __device__ __forceinline__ uint32_t top() const {
    return max(max(max(abs_bits(a.x), abs_bits(a.y)), max(abs_bits(a.z), abs_bits(a.w))),
               max(max(abs_bits(b.x), abs_bits(b.y)), max(abs_bits(b.z), abs_bits(b.w))));
  }
  static __device__ __forceinline__ uint32_t larger(uint32_t x, uint32_t y) { return max(x, y); }
  __device__ __forceinline__ float get(int j) const {
    const float4 &f = j < 4 ? a : b;
    return (j & 3) == 0 ? f.x : (j & 3) == 1 ? f.y : (j & 3) == 2 ? f.z : f.w;
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load_some(const char *p, int64_t i, int n) {
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = j < n ? reinterpret_cast<const float *>(p)[i + j] : 0.f;
    a = make_float4(w[0], w[1], w[2], w[3]);
    b = make_float4(w[4], w[5], w[6], w[7]);
  }
  __device__ __forceinline__ void tops(uint32_t (&t)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = max(t[j], abs_bits(get(j)));
  }
  static __device__ __forceinline__ void unpack(uint32_t (&)[8]) {}
};
template <int DT>
constexpr int kHold = DT == HIMUON_FP32 ? 4 : 8;

template <int DT, int TPR>
__global__ void __launch_bounds__(256, 4) quantize_rows_kernel(const __grid_constant__ QuantArgs a) {
  __shared__ uint32_t part[8];
  grid_start_next();
  grid_wait();
  const int32_t z = blockIdx.y;
  if (a.dtype[z] != DT) return;
  const int64_t row = blockIdx.x * static_cast<int64_t>(256 / TPR) + threadIdx.x / TPR;
  const int t = threadIdx.x % TPR;
  const int64_t cols = a.cols[z];
  const int32_t runs = static_cast<int32_t>(cols / 8);
  const bool live = row < a.rows[z];
  const char *in = static_cast<const char *>(a.in[z]) + (live ? row * a.ld[z] : 0) * (DT == HIMUON_FP32 ? 4 : 2);
  Run8<DT> v[kHold<DT>];
  uint32_t top = 0;   // fp32: bits of the maximum; else two 16-bit maxima
  if (live) {
#pragma unroll
    for (int h = 0; h < kHold<DT>; ++h)
      if (t + h * TPR < runs) v[h].load(in, t + h * TPR);
#pragma unroll
    for (int h = 0; h < kHold<DT>; ++h)
      if (t + h * TPR < runs) top = Run8<DT>::larger(top, v[h].top());
    for (int32_t i = t + kHold<DT> * TPR; i < runs; i += TPR) {
      Run8<DT> w;
      w.load(in, i);
      top = Run8<DT>::larger(top, w.top());
    }
  }
  if (DT != HIMUON_FP32) {   // the 16-bit maximum as an fp32's bits
    const uint32_t m = max(top >> 16, top & 0xffffu);
    const uint16_t h = static_cast<uint16_t>(m);
    top = DT == HIMUON_FP16 ? abs_bits(__half2float(*reinterpret_cast<const __half *>(&h))) : m << 16;
  }
  if (live)
    for (int64_t i = 8ll * runs + t; i < cols; i += TPR) top = max(top, abs_bits(ld_any(in, DT, i)));
  top = __reduce_max_sync(0xffffffffu, top);
  if (TPR > 32) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
    __syncthreads();
    constexpr int kWarps = TPR / 32;
    const int w0 = threadIdx.x / TPR * kWarps;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = max(top, part[w0 + w]);
  }
  if (!live) return;
  if (t == 0) a.scale[z][row] = line_scale(top);
  int8_t *out = a.codes[z] + row * a.ldq[z];
  const bool ok = line_ok(top);
  const Coder code(ok ? __uint_as_float(top) : 1.f);
  if (!ok || !code.in_range()) {   // (rare: one element at a time)
    for (int64_t i = t; i < cols; i += TPR) out[i] = ok ? static_cast<int8_t>(code.template code<DT>(ld_any(in, DT, i))) : 0;
    return;
  }
  auto put8 = [&](int32_t i, const uint32_t (&u)[8]) {
    *reinterpret_cast<uint2 *>(out + 8 * i) = make_uint2(bytes4(u[0], u[1], u[2], u[3]), bytes4(u[4], u[5], u[6], u[7]));
  };
  auto exact8 = [&](int32_t i, const Run8<DT> &x) {
    uint32_t u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = exact_code<DT>(x.get(j), code.hi, code.lo);
    put8(i, u);
  };
  auto near8 = [&](int32_t i, const Run8<DT> &x) {   // fp32; true: to be done again
    const Pair hi(code.hi, code.hi), minus_hi(-code.hi, -code.hi), minus_lo(-code.lo, -code.lo);
    Pair ties(1.f, 1.f);
    uint32_t u[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2)
      near_codes(Pair(x.get(j), x.get(j + 1)), hi, minus_hi, minus_lo, u[j], u[j + 1], ties);
    put8(i, u);
    return ties.any_zero();
  };
  auto again = [&](int32_t i) {
    Run8<DT> w;
    w.load(in, i);
    exact8(i, w);
  };
  uint32_t ties = 0;
#pragma unroll
  for (int h = 0; h < kHold<DT>; ++h)
    if (t + h * TPR < runs) {
      if (DT != HIMUON_FP32) exact8(t + h * TPR, v[h]);
      else if (near8(t + h * TPR, v[h])) ties |= 1u << h;
    }
  for (int32_t i = t + kHold<DT> * TPR, h = kHold<DT>; i < runs; i += TPR, ++h) {
    Run8<DT> w;
    w.load(in, i);
    if (DT != HIMUON_FP32) exact8(i, w);
    else if (near8(i, w)) ties |= 1u << (h & 31);
  }
  for (; ties; ties &= ties - 1)   // (one run in 2^14 of normal values; past 32 runs a bit stands for every 32nd)
    for (int64_t i = t + (__ffs(ties) - 1) * TPR; i < runs; i += 32 * TPR) again(static_cast<int32_t>(i));
  for (int64_t i = 8ll * runs + t; i < cols; i += TPR) out[i] = static_cast<int8_t>(exact_code<DT>(ld_any(in, DT, i), code.hi, code.lo));
}

// One scale per column, codes transposed.  A cluster takes 64 columns (128 bytes
// of a 16-bit row) and deals their rows, 128 at a time, over its CTAs (up to
// eight: a matrix of 4096 x 1024 has only 16 such column blocks).  The first pass
// finds the columns' maxima, joined over distributed shared memory; the second,
// from L2, codes the same rows: a thread takes 8 columns of 4 rows, packs each
// column's four codes into a word and the words are turned through shared
// memory, so that a warp stores 128 rows of a column at once.
constexpr int kTurnPitch = 33;   // words; with the columns' rotation below free of bank conflicts
template <int DT>
__global__ void __launch_bounds__(256, 3)
    quantize_cols_kernel(const __grid_constant__ QuantArgs a) {
  __shared__ uint32_t tops[64];
  __shared__ uint32_t turn[64 * kTurnPitch];
  grid_start_next();
  grid_wait();
  const int32_t z = blockIdx.z;
  if (a.dtype[z] != DT) return;   // (the same for the whole cluster)
  const int64_t c0 = blockIdx.x * 64ll;
  const int64_t rows = a.rows[z], cols = a.cols[z], ld = a.ld[z];
  if (c0 >= cols) return;
  const int32_t part = blockIdx.y, parts = gridDim.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c8 = lane & 7, rg = warp * 4 + (lane >> 3);   // 8 columns, rows 4 rg .. 4 rg + 3 of a block
  const int64_t c = c0 + 8 * c8;
  const bool whole = c + 8 <= cols;
  const char *in = static_cast<const char *>(a.in[z]) + c * (DT == HIMUON_FP32 ? 4 : 2);
  auto load = [&](int64_t r, Run8<DT> &x) {   // (zeros where there is nothing)
    if (r >= rows) x.clear();
    else if (whole) x.load(in + r * ld * (DT == HIMUON_FP32 ? 4 : 2), 0);
    else x.load_some(static_cast<const char *>(a.in[z]), r * ld + c, static_cast<int>(cols - c));
  };
  if (threadIdx.x < 64) tops[threadIdx.x] = 0;
  __syncthreads();
  {
    uint32_t top[8] = {};   // 16 bits: pairs of columns in the first four
    for (int64_t b = part * 128ll; b < rows; b += parts * 128ll) {
      Run8<DT> x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) load(b + 4 * rg + k, x[k]);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k].tops(top);
    }
    Run8<DT>::unpack(top);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      top[j] = max(top[j], __shfl_xor_sync(0xffffffffu, top[j], 8));
      top[j] = max(top[j], __shfl_xor_sync(0xffffffffu, top[j], 16));
      if (lane < 8) atomicMax(&tops[8 * c8 + j], top[j]);
    }
  }
  cluster_sync_all();
  uint32_t mine = 0;
  if (threadIdx.x < 64)
    for (int32_t p = 0; p < parts; ++p) {
      uint32_t v;
      asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(&tops[threadIdx.x]), p)));
      mine = max(mine, v);
    }
  cluster_sync_all();
  if (threadIdx.x < 64) {
    tops[threadIdx.x] = mine;
    if (part == 0 && c0 + threadIdx.x < cols) a.scale[z][c0 + threadIdx.x] = line_scale(mine);
  }
  __syncthreads();
  float hi[8], lo[8];
  bool near = true;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t top = tops[8 * c8 + j];
    const Coder code(line_ok(top) ? __uint_as_float(top) : 1.f);
    hi[j] = code.hi;
    lo[j] = code.lo;
    near = near && (line_ok(top) || top == 0) && code.in_range();   // (top 0: all zeros, whose codes are 0)
  }
  for (int64_t b = part * 128ll; b < rows; b += parts * 128ll) {
    Run8<DT> x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) load(b + 4 * rg + k, x[k]);
    uint32_t pairs = 0;   // fp32: to be done again
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      uint32_t u[2][4];
      if (near && DT == HIMUON_FP32) {
        const Pair h(hi[j], hi[j + 1]), minus_h(-hi[j], -hi[j + 1]), minus_l(-lo[j], -lo[j + 1]);
        Pair ties(1.f, 1.f);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          near_codes(Pair(x[k].get(j), x[k].get(j + 1)), h, minus_h, minus_l, u[0][k], u[1][k], ties);
        if (ties.any_zero()) pairs |= 1u << j;
      } else if (near) {
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k / 4][k % 4] = exact_code<DT>(x[k % 4].get(j + k / 4), hi[j + k / 4], lo[j + k / 4]);
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t top = tops[8 * c8 + j + i];
          const Coder code(line_ok(top) ? __uint_as_float(top) : 1.f);
#pragma unroll
          for (int k = 0; k < 4; ++k) u[i][k] = line_ok(top) ? code.template code<DT>(x[k].get(j + i)) : 0;
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        turn[(8 * c8 + j + i) * kTurnPitch + ((rg + 4 * (c8 >> 2)) & 31)] = bytes4(u[i][0], u[i][1], u[i][2], u[i][3]);
    }
    for (; pairs; pairs &= pairs - 1) {   // (rare)
      const int j = __ffs(pairs) - 1;
#pragma unroll 1
      for (int i = j; i < j + 2 && c + i < cols; ++i) {
        const uint32_t top = tops[8 * c8 + i];
        const Coder code(line_ok(top) ? __uint_as_float(top) : 1.f);
        uint32_t u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int64_t r = b + 4 * rg + k;
          u[k] = exact_code<DT>(r < rows ? ld_any(a.in[z], DT, r * ld + c + i) : 0.f, code.hi, code.lo);
        }
        turn[(8 * c8 + i) * kTurnPitch + ((rg + 4 * (c8 >> 2)) & 31)] = bytes4(u[0], u[1], u[2], u[3]);
      }
    }
    __syncthreads();
    const int64_t r = b + 4 * lane;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = 8 * warp + j;
      const uint32_t w = turn[col * kTurnPitch + ((lane + 4 * (warp >> 2)) & 31)];
      if (c0 + col >= cols || r >= rows) continue;
      int8_t *out = a.codes[z] + (c0 + col) * a.ldq[z] + r;
      if (r + 4 <= rows) *reinterpret_cast<uint32_t *>(out) = w;
      else
        for (int k = 0; r + k < rows; ++k) out[k] = static_cast<int8_t>(w >> (8 * k));
    }
    __syncthreads();
  }
}

template <typename Kern>
void launch_quant(Kern kern, dim3 grid, unsigned cluster_y, const QuantArgs &a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = attr[1].val.clusterDim.z = 1;
  attr[1].val.clusterDim.y = cluster_y;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  count_launch();
  cudaLaunchKernelEx(&cfg, kern, a);   // (its error is read by the caller)
}

// Columns of matrices of at most `most` columns and `tallest` rows.
template <int DT>
void quantize_cols(const QuantArgs &a, int64_t most, int64_t tallest, unsigned zs, cudaStream_t st) {
  // rows are dealt out only as far as the column blocks leave SMs without work
  unsigned parts = 1;
  while (parts < 8 && parts * 128ll < tallest && (most + 63) / 64 * zs * parts < 4 * sm_count()) parts *= 2;
  launch_quant(quantize_cols_kernel<DT>, dim3(static_cast<unsigned>((most + 63) / 64), parts, zs), parts, a, st);
}

template <int DT>
bool load_quant_kernels() {
  cudaFuncAttributes f;
  return cudaFuncGetAttributes(&f, quantize_rows_kernel<DT, 32>) == cudaSuccess &&
         cudaFuncGetAttributes(&f, quantize_rows_kernel<DT, 64>) == cudaSuccess &&
         cudaFuncGetAttributes(&f, quantize_rows_kernel<DT, 128>) == cudaSuccess &&
         cudaFuncGetAttributes(&f, quantize_rows_kernel<DT, 256>) == cudaSuccess &&
         cudaFuncGetAttributes(&f, quantize_cols_kernel<DT>) == cudaSuccess;
}

// Rows of at most `widest` columns: the fewest threads per row that hold it.
template <int DT>
void quantize_rows(const QuantArgs &a, int64_t most, int64_t widest, unsigned zs, cudaStream_t st) {
  const int64_t per = 8 * kHold<DT>;
  auto go = [&](auto kern, int tpr) {
    launch_quant(kern, dim3(static_cast<unsigned>((most + 256 / tpr - 1) / (256 / tpr)), zs), 1, a, st);
  };
  if (widest <= 32 * per) go(quantize_rows_kernel<DT, 32>, 32);
  else if (widest <= 64 * per) go(quantize_rows_kernel<DT, 64>, 64);
  else if (widest <= 128 * per) go(quantize_rows_kernel<DT, 128>, 128);
  else go(quantize_rows_kernel<DT, 256>, 256);
}

}  // namespace

bool load_quantize() {
  return load_quant_kernels<HIMUON_BF16>() && load_quant_kernels<HIMUON_FP16>() && load_quant_kernels<HIMUON_FP32>();
}

}  // namespace himuon

using namespace himuon;

extern "C" {

int himuon_quantize(const himuon_mat *in, int32_t n, int32_t dim, const himuon_mat *codes, const himuon_mat *scale,
                    void *stream) {
  if (!in || !codes || !scale || n < 1 || (dim != 0 && dim != 1)) return HIMUON_ERR_INVALID;
  for (int32_t e = 0; e < n; ++e) {
    int rc = check_operand(in[e], 0);
    if (!rc && dim == 1 && in[e].rows < 1) rc = HIMUON_ERR_INVALID;
    if (!rc) rc = check_operand(codes[e], 0);
    if (!rc) rc = check_scale(scale + e, 1, dim ? in[e].cols : in[e].rows);
    if (rc) return rc;
    if (!is_float(in[e].dtype) || codes[e].dtype != HIMUON_I8) return HIMUON_ERR_UNSUPPORTED;
    if (codes[e].rows != (dim ? in[e].cols : in[e].rows) || codes[e].cols != (dim ? in[e].rows : in[e].cols))
      return HIMUON_ERR_INVALID;
  }
  const int rc = expert_device();
  if (rc) return rc;
  for (int32_t e0 = 0; e0 < n; e0 += kMaxList) {
    const int32_t cnt = std::min(n - e0, kMaxList);
    QuantArgs a;
    a.dim = dim;
    int64_t most = 0, widest = 0, tallest = 0;
    bool any[3] = {false, false, false};
    for (int32_t e = 0; e < cnt; ++e) {
      const himuon_mat &m = in[e0 + e];
      a.in[e] = m.data;
      a.codes[e] = static_cast<int8_t *>(codes[e0 + e].data);
      a.scale[e] = static_cast<float *>(scale[e0 + e].data);
      a.rows[e] = m.rows;
      a.cols[e] = m.cols;
      a.ld[e] = m.ld;
      a.ldq[e] = codes[e0 + e].ld;
      a.dtype[e] = m.dtype;
      most = std::max(most, dim ? m.cols : m.rows);
      widest = std::max(widest, m.cols);
      tallest = std::max(tallest, m.rows);
      any[m.dtype] = true;
    }
    if (most == 0) continue;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const unsigned zs = static_cast<unsigned>(cnt);
    // one launch per storage type among the call's matrices
    if (dim) {
      if (any[HIMUON_BF16]) quantize_cols<HIMUON_BF16>(a, most, tallest, zs, st);
      if (any[HIMUON_FP16]) quantize_cols<HIMUON_FP16>(a, most, tallest, zs, st);
      if (any[HIMUON_FP32]) quantize_cols<HIMUON_FP32>(a, most, tallest, zs, st);
    } else {
      if (any[HIMUON_BF16]) quantize_rows<HIMUON_BF16>(a, most, widest, zs, st);
      if (any[HIMUON_FP16]) quantize_rows<HIMUON_FP16>(a, most, widest, zs, st);
      if (any[HIMUON_FP32]) quantize_rows<HIMUON_FP32>(a, most, widest, zs, st);
    }
    if (cudaGetLastError() != cudaSuccess) return HIMUON_ERR_CUDA;
  }
  return HIMUON_OK;
}

}  // extern "C"
