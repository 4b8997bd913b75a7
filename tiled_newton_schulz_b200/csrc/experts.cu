// experts.cu -- products over row groups: expert forward and input-gradient
// products, weight gradients, 8-bit codes and the 8-bit product.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>
#include <atomic>
#include <vector>

#include "himuon.h"
#include "layout.hpp"
#include "ptx.cuh"

namespace himuon {

int device_usable();         // api.cu: HIMUON_OK or HIMUON_ERR_NO_DEVICE for the current device
int *device_status_word();   // api.cu: the current device's status word

namespace {

__device__ __forceinline__ float ld_any(const void *p, int32_t dtype, int64_t i) {
  if (dtype == HIMUON_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
  if (dtype == HIMUON_FP16) return __half2float(static_cast<const __half *>(p)[i]);
  return static_cast<const float *>(p)[i];
}
__device__ __forceinline__ void st_any(void *p, int32_t dtype, int64_t i, float v) {
  if (dtype == HIMUON_BF16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
  else if (dtype == HIMUON_FP16) static_cast<__half *>(p)[i] = __float2half_rn(v);
  else static_cast<float *>(p)[i] = v;
}

// One launch takes the matrices of up to kMaxStack groups when they lie at
// equal distances (one tensor map, or a base and a stride), else a list of up
// to kMaxList in the kernel's parameters; longer calls run as several
// launches, each on its own stretch of the offsets.
constexpr int kMaxList = 64;
constexpr int kMaxStack = 256;

// ---------------------------------------------------------------- the product kernel
// Both directions are one tcgen05 product per output tile, D (256 x up to 256,
// fp32 or int32 in tensor memory) = A B^T over 128-byte stretches of K:
//   product:  A = W_e (256 channels), B = X (up to 256 rows of group e), so the
//             ragged side is the MMA's N, which is any multiple of 32: a group
//             of 5 rows costs a 32-column tile, not a 128-row one.
//   gradient: A = 256 columns of operand A, B = 256 columns of operand B,
//             K = the group's rows (both operands MN-major).
constexpr uint32_t kABytes = 16384;     // 128 rows (or 2 x 64 MN columns) x 128 bytes of K
constexpr uint32_t kBoxBytes = 2048;    // 16 rows of X x 128 bytes
constexpr uint32_t kData = 229376;      // operand ring and the epilogue's buffers
constexpr int kMaxStages = 10;
constexpr uint32_t kStageOut = 4096;    // an epilogue warp's buffer: 32 x 32 fp32, swizzled
constexpr int kEpiWarps = 8;
constexpr int kTileM = 256, kTileN = 256;   // a CTA pair's tile of D
constexpr int kThreads = 128 + 32 * kEpiWarps;   // three warpgroups: loads and MMAs (warps 0, 1), epilogue (4..11)
// fp32 results of 16-bit operands: the tensor core's accumulator truncates at
// every K = 16 step, which costs an fp32 result about 1e-8 of itself per step
// (K = 1100: 1.1e-6 against 2.6e-7 for rounded fp32 sums).  Their sums are cut
// every kChunk blocks of 64; the epilogue adds the pieces in fp32 registers.
constexpr int kChunk = 8;
constexpr uint32_t kBarBytes = 448;
constexpr uint32_t kSmem = kData + kBarBytes + 4 * (kMaxStack + 4) + 1024;
static_assert(kSmem <= 232448, "shared memory of one CTA");

// NMAP, NOUT: tensor maps of W, and of G and C (the product writes Y without
// one): 1, over matrices at equal distances, or one for each of a list.
template <int NMAP, int NOUT>
struct MmaArgs {
  CUtensorMap w[NMAP];     // product: W; gradient: operand A
  // product: X in boxes of 128, 64, 32 and 16 rows; gradient: operand B, and the
  // windows (make_window_map) of B and A
  CUtensorMap x[4];
  const int32_t *offsets;
  int64_t rows;
  int32_t n;
  int32_t K;               // product: length of the sums
  int32_t M, N;            // product: M channels; gradient: G is M x N
  int32_t mt_m, mt_n;      // tiles along M; gradient: along N
  int32_t cap;             // gradient: columns of a tile (a multiple of 32); product: log2 of a tile's most rows
  int32_t split;           // pairs that share a tile's sum (the cluster's)
  uint32_t idesc;          // without the N field
  int *status;
  const float *x_scale, *w_scale;
  int64_t ld_scale;
  CUtensorMap g[NOUT], c[NOUT];   // gradient: G and C in boxes of 32 rows x box_cols columns
  char *out[NOUT];                // product: Y; gradient: G
  int64_t ldo, out_stride;        // (NOUT = 1: bytes between consecutive matrices of G)
  int32_t odtype, cdtype, has_c;
  int32_t buffers;                // of kStageOut per epilogue warp
  int32_t box_cols;               // 32, or 64 where G and C are 16-bit
  float alpha, beta;
};

// Pair forms (CTA pairs, issued by the even CTA): both operands from shared
// memory at the same offsets in both CTAs.
__device__ __forceinline__ void mma_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_i8_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// TMA loads into this CTA's shared memory that complete on an mbarrier of
// either CTA of the pair (a shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map, int32_t x, int32_t y,
                                                 uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(bar_cluster)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(void *dst, const CUtensorMap *map, int32_t x, int32_t y, int32_t z,
                                                 uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
      "%4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar_cluster)
      : "memory");
}
// Launches of this file follow one another without a gap: a kernel lets the next
// one start as soon as its CTAs have (its first part, which touches no memory of
// the stream's, runs under this one's end), and waits for everything before it
// in the stream to have completed ahead of its first access.
__device__ __forceinline__ void grid_start_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// One thread of the converged warp (the same one every time).  The loops that
// issue copies and MMAs are run by whole warps, with only the instruction
// itself in the elected thread's branch: their addresses and descriptors then
// stay in uniform registers.  (Run by lane 0 alone, each stage's copies took
// about 500 cycles to issue and its MMAs 450, which bounded every case.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// A bounded wait by a whole warp: its lanes agree on the outcome.  CLUSTER:
// for phases that the pair's other CTA also arrives on.
template <bool CLUSTER = false>
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t phase, int *status) {
  auto ready = [&] {
    return __all_sync(0xffffffffu, CLUSTER ? mbar_try_wait_cluster(bar, phase) : mbar_try_wait(bar, phase));
  };
  if (ready()) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (ready()) return true;
    if ((i & 255u) == 0 && __any_sync(0xffffffffu, globaltimer_ns() - t0 > kWaitLimitNs)) break;
  }
  set_status(status, HIMUON_ERR_TIMEOUT_DEV);
  return false;
}

// Bound i of the groups, clamped into 0 .. rows.
__device__ __forceinline__ int32_t bound_at(const int32_t *offsets, int32_t i, int64_t rows) {
  if (!offsets) return i == 0 ? 0 : static_cast<int32_t>(rows);
  return static_cast<int32_t>(min(max((int64_t)offsets[i], (int64_t)0), rows));
}

__device__ __forceinline__ int32_t round32(int32_t x) { return (x + 31) / 32 * 32; }
// A group of cnt rows runs as ceil(cnt / 2^shift) tiles, its units of 32 rows
// (the pair's CTAs hold half of them each, in boxes of 16) dealt out as evenly
// as they go: tiles of equal width would pad up to 31 rows each (16381 rows of 61
// experts, 1024 -> 4096, a tenth of the MMAs' columns).
__device__ __forceinline__ int32_t row_tiles(int32_t cnt, int32_t shift) { return (cnt + (1 << shift) - 1) >> shift; }
__device__ __forceinline__ int32_t tile_width(int32_t cnt, int32_t shift) {   // the widest
  const int32_t mt = row_tiles(cnt, shift), units = (cnt + 31) / 32;
  return 32 * (mt <= 1 ? units : (units + mt - 1) / mt);
}

struct Tile {
  int32_t e;        // group
  int32_t m0;       // first row of D in the output: channel (product) or row of G
  int32_t n0;       // product: first row of X; gradient: first column of G
  int32_t width;    // columns of D: a multiple of 32
  int32_t valid;    // of them, inside the output
  int32_t k0, len;  // the sums' stretch: product, of K; gradient, rows (of the slice, where a tile is split)
};

// Tile `idx` of the launch, found by a whole warp.  `from`: a group not after
// the tile's (the last one found: a role's tiles come in order).
template <int GRAD, int SPLIT, int kElems, typename Args>
__device__ __forceinline__ Tile tile_at(const Args &a, const int32_t *start, int32_t slice, int32_t idx, int32_t from) {
  Tile t;
  const int32_t mt_m = a.mt_m;
  if (GRAD) {
    const int32_t u = idx / mt_m;
    t.e = u / a.mt_n;
    t.m0 = (idx - u * mt_m) * kTileM;
    t.n0 = (u - t.e * a.mt_n) * a.cap;
    t.valid = min(a.cap, a.N - t.n0);
    t.width = round32(t.valid);
    t.k0 = bound_at(a.offsets, t.e, a.rows);
    t.len = max(0, bound_at(a.offsets, t.e + 1, a.rows) - t.k0);
  } else {
    // the group whose row tiles hold row tile idx / mt_m: the last with start[e] <= it
    const int32_t u = idx / mt_m, lane = threadIdx.x & 31;
    for (;; from += 32) {
      const uint32_t before = __ballot_sync(0xffffffffu, from + 1 + lane < a.n && start[from + 1 + lane] <= u);
      if (before != 0xffffffffu) {
        t.e = from + __popc(before);
        break;
      }
    }
    const int32_t lo = bound_at(a.offsets, t.e, a.rows), hi = max(lo, bound_at(a.offsets, t.e + 1, a.rows));
    const int32_t cnt = hi - lo, mt = row_tiles(cnt, a.cap);
    // bands of up to 8 row tiles, row tile fastest: the tiles in flight share
    // a few panels of W and of X
    const int32_t r = idx - start[t.e] * mt_m;
    const int32_t g = mt <= 8 ? 0 : r / (8 * mt_m), rr = r - g * 8 * mt_m;
    const int32_t gm = min(8, mt - 8 * g), mc = gm == 1 ? rr : rr / gm;
    const int32_t tt = 8 * g + rr - mc * gm;
    t.m0 = mc * kTileM;
    const int32_t units = (cnt + 31) / 32, each = mt <= 1 ? units : units / mt, more = units - each * mt;
    t.width = 32 * (each + (tt < more ? 1 : 0));
    t.n0 = lo + 32 * (tt * each + min(tt, more));
    t.valid = min(t.width, hi - t.n0);
    t.k0 = 0;
    t.len = a.K;
  }
  if (SPLIT) {   // this pair's blocks of the sum
    const int32_t nb = (t.len + kElems - 1) / kElems;
    const int32_t b0 = nb * slice / a.split, b1 = nb * (slice + 1) / a.split;
    t.k0 += b0 * kElems;
    t.len = min(t.len, b1 * kElems) - b0 * kElems;
  }
  return t;
}

// The product's output: 32 rows of Y x 32 channels, of which `rows` x `cols`
// are inside.  A lane comes with one channel of every row and leaves with runs
// of a row: the block is turned through the warp's buffer (16-byte chunk c of
// line r at chunk c ^ (r & 7): free of bank conflicts both ways), so that every
// row is written as one 64- or 128-byte run.  (A group's last rows end inside a
// tile, where a tensor map could not stop.)
template <typename T2>
__device__ __forceinline__ uint32_t two16(float x, float y);
template <>
__device__ __forceinline__ uint32_t two16<__half2>(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t *>(&h);
}
template <>
__device__ __forceinline__ uint32_t two16<__nv_bfloat162>(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t *>(&h);
}
// 16-bit: line k holds rows 2 k and 2 k + 1, a 32-bit word per channel.
template <typename T2>
__device__ __forceinline__ void put_rows16(uint32_t *st, int lane, const float (&v)[32], uint16_t *out, int64_t ldo,
                                           int32_t rows, int32_t cols) {
  __syncwarp();   // the last block's readers are done
#pragma unroll
  for (int k = 0; k < 16; ++k)
    st[k * 32 + (((lane >> 2) ^ (k & 7)) << 2) + (lane & 3)] = two16<T2>(v[2 * k], v[2 * k + 1]);
  __syncwarp();
  const int32_t col = (lane & 3) * 8;
  uint16_t *o = out + (lane >> 2) * 2 * ldo + col;
#pragma unroll
  for (int p = 0; p < 2; ++p, o += 16 * ldo) {
    const int k = (lane >> 2) + 8 * p;
    const uint4 x = *reinterpret_cast<const uint4 *>(st + k * 32 + (((col >> 2) ^ (k & 7)) << 2));
    const uint4 y = *reinterpret_cast<const uint4 *>(st + k * 32 + ((((col >> 2) + 1) ^ (k & 7)) << 2));
    const uint4 a = make_uint4(__byte_perm(x.x, x.y, 0x5410), __byte_perm(x.z, x.w, 0x5410),
                               __byte_perm(y.x, y.y, 0x5410), __byte_perm(y.z, y.w, 0x5410));
    const uint4 b = make_uint4(__byte_perm(x.x, x.y, 0x7632), __byte_perm(x.z, x.w, 0x7632),
                               __byte_perm(y.x, y.y, 0x7632), __byte_perm(y.z, y.w, 0x7632));
    if (col + 8 <= cols) {
      if (2 * k < rows) *reinterpret_cast<uint4 *>(o) = a;
      if (2 * k + 1 < rows) *reinterpret_cast<uint4 *>(o + ldo) = b;
    } else {
      const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (col + j >= cols) break;
        if (2 * k < rows) o[j] = static_cast<uint16_t>(wa[j / 2] >> (16 * (j & 1)));
        if (2 * k + 1 < rows) o[ldo + j] = static_cast<uint16_t>(wb[j / 2] >> (16 * (j & 1)));
      }
    }
  }
}
// fp32: line r holds row r.
__device__ __forceinline__ void put_rows32(float *st, int lane, const float (&v)[32], float *out, int64_t ldo,
                                           int32_t rows, int32_t cols) {
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 32; ++k) st[k * 32 + (((lane >> 2) ^ (k & 7)) << 2) + (lane & 3)] = v[k];
  __syncwarp();
  const int32_t col = (lane & 7) * 4;
  float *o = out + (lane >> 3) * ldo + col;
#pragma unroll
  for (int p = 0; p < 8; ++p, o += 4 * ldo) {
    const int r = (lane >> 3) + 4 * p;
    const float4 f = *reinterpret_cast<const float4 *>(st + r * 32 + (((col >> 2) ^ (r & 7)) << 2));
    if (r >= rows) continue;
    if (col + 4 <= cols) {
      *reinterpret_cast<float4 *>(o) = f;
    } else {
      const float w[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (col + j < cols) o[j] = w[j];
    }
  }
}

// The gradient's epilogue buffers hold a box as TMA moves it: 32 rows of 128
// bytes (32 columns of fp32, 64 of 16 bits; 128-byte swizzle) or of 64 bytes (32
// columns of 16 bits; 64-byte swizzle).  A lane owns a row; both patterns are
// free of bank conflicts.  Chunk k (16 bytes) of this lane's row:
__device__ __forceinline__ uint32_t box_at(int lane, int k, bool wide) {
  return wide ? lane * 128 + ((k ^ (lane & 7)) << 4) : lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4);
}
// v = alpha v + beta (32 columns of this lane's row, from the box's chunk k0)
__device__ __forceinline__ void box_combine(const uint8_t *buf, int lane, int32_t dtype, int k0, bool wide, float alpha,
                                            float beta, float (&v)[32]) {
  if (dtype == HIMUON_FP32) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float4 f = *reinterpret_cast<const float4 *>(buf + box_at(lane, k, true));
      v[4 * k] = fmaf(beta, f.x, alpha * v[4 * k]);
      v[4 * k + 1] = fmaf(beta, f.y, alpha * v[4 * k + 1]);
      v[4 * k + 2] = fmaf(beta, f.z, alpha * v[4 * k + 2]);
      v[4 * k + 3] = fmaf(beta, f.w, alpha * v[4 * k + 3]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint4 u = *reinterpret_cast<const uint4 *>(buf + box_at(lane, k0 + k, wide));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const float2 f = dtype == HIMUON_FP16 ? __half22float2(*reinterpret_cast<const __half2 *>(&w[h]))
                                              : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[h]));
        v[8 * k + 2 * h] = fmaf(beta, f.x, alpha * v[8 * k + 2 * h]);
        v[8 * k + 2 * h + 1] = fmaf(beta, f.y, alpha * v[8 * k + 2 * h + 1]);
      }
    }
  }
}
template <typename T2>
__device__ __forceinline__ void box_write16(uint8_t *buf, int lane, int k0, bool wide, const float (&v)[32]) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    *reinterpret_cast<uint4 *>(buf + box_at(lane, k0 + k, wide)) =
        make_uint4(two16<T2>(v[8 * k], v[8 * k + 1]), two16<T2>(v[8 * k + 2], v[8 * k + 3]),
                   two16<T2>(v[8 * k + 4], v[8 * k + 5]), two16<T2>(v[8 * k + 6], v[8 * k + 7]));
}
__device__ __forceinline__ void box_write(uint8_t *buf, int lane, int32_t dtype, int k0, bool wide,
                                          const float (&v)[32]) {
  if (dtype == HIMUON_FP32) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      *reinterpret_cast<float4 *>(buf + box_at(lane, k, true)) =
          make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
  } else if (dtype == HIMUON_FP16) {
    box_write16<__half2>(buf, lane, k0, wide, v);
  } else {
    box_write16<__nv_bfloat162>(buf, lane, k0, wide, v);
  }
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *src, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
               "r"(x), "r"(y), "r"(z), "r"(smem_u32(src))
               : "memory");
}
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// Reports offsets that decrease or leave 0 .. rows (a whole warp).
template <typename Args>
__device__ __forceinline__ void check_offsets(const Args &a, int lane) {
  if (!a.offsets) return;
  for (int32_t e = lane; e < a.n; e += 32)
    if (a.offsets[e] < 0 || a.offsets[e + 1] < a.offsets[e] || a.offsets[e + 1] > a.rows)
      set_status(a.status, HIMUON_ERR_DEVICE);
}

// The product's tiles, from the groups' bounds (a whole warp): start[e], the
// row tiles of the groups before e, and the widest tile.
template <typename Args>
__device__ __forceinline__ void plan_rows(const Args &a, int32_t *start, int32_t *widest, int lane) {
  constexpr int kPer = kMaxStack / 32;
  int32_t cnt[kPer];   // of group lane + 32 i; all loads in flight together
  {
    int32_t o[kPer + 1];
#pragma unroll
    for (int i = 0; i <= kPer; ++i) {
      const int32_t e = lane + 32 * i;
      o[i] = e > a.n ? 0 : a.offsets ? a.offsets[e] : e == 0 ? 0 : static_cast<int32_t>(a.rows);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      cnt[i] = 0;
      if (32 * i >= a.n) continue;
      const int32_t e = lane + 32 * i;
      const int32_t down = __shfl_down_sync(0xffffffffu, o[i], 1), over = __shfl_sync(0xffffffffu, o[i + 1], 0);
      const int64_t lo = o[i], hi = lane == 31 ? over : down;
      if (e < a.n) {
        if (lo < 0 || hi < lo || hi > a.rows) set_status(a.status, HIMUON_ERR_DEVICE);
        const int64_t first = min(max(lo, (int64_t)0), a.rows), last = min(max(hi, (int64_t)0), a.rows);
        cnt[i] = static_cast<int32_t>(max(last - first, (int64_t)0));
      }
    }
  }
  int32_t base = 0, w = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (32 * i >= a.n) break;
    w = max(w, tile_width(cnt[i], a.cap));
    int32_t s = row_tiles(cnt[i], a.cap);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t up = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += up;
    }
    if (lane + 32 * i < a.n) start[lane + 32 * i + 1] = base + s;
    base += __shfl_sync(0xffffffffu, s, 31);
  }
  w = __reduce_max_sync(0xffffffffu, w);
  if (lane == 0) {
    start[0] = 0;
    *widest = w;
  }
}

// PREC: an epilogue warp's column groups half, half + 2, .. (below `in`) of
// accumulator piece p, added to its running sums.
template <int PREC>
__device__ __forceinline__ void read_pieces(float (&sum)[PREC ? 4 : 1][32], uint32_t taddr, int half, int32_t in,
                                            int32_t p, bool none) {
#pragma unroll
  for (int g = 0; g < (PREC ? 4 : 1); ++g) {
    const int32_t i = half + 2 * g;
    if (i >= in) continue;
    if (none) {
#pragma unroll
      for (int k = 0; k < 32; ++k) sum[g][k] = 0.f;
    } else if (p == 0) {
      tmem_ld32(taddr + 32 * i, sum[g]);
      tmem_wait_ld();
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[16];
        tmem_ld16(taddr + 32 * i + 16 * h, v);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k) sum[g][16 * h + k] += v[k];
      }
    }
  }
}

// SPLIT: adds up the slices' sums of a tile.  Column group g of a warp belongs
// to the pair g % split; every other pair's warp sends it its part over
// distributed shared memory, into the ring (free by then: the first cluster
// barrier follows every pair's last MMA), and the owner adds the parts in the
// order of the slices, whatever their order of arrival.  4 KB per part: chunk k
// (16 bytes) of lane l at k * 512 + 16 l.
template <int KIND, int PREC>
__device__ __forceinline__ void join_slices(float (&sum)[PREC ? 4 : 1][32], uint8_t *ring, int w, int lane, int half,
                                            int32_t in, int32_t rank, int32_t slice, int32_t split) {
  const int per = 4 / split;   // groups that a warp owns
  __syncwarp();
  cluster_sync_all();
#pragma unroll
  for (int g = 0; g < (PREC ? 4 : 1); ++g) {
    const int owner = g % split;
    if (half + 2 * g >= in || owner == slice) continue;
    const uint32_t to =
        mapa_shared(smem_u32(ring + ((slice * per + g / split) * kEpiWarps + w) * kStageOut), 2 * owner + rank) + 16 * lane;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      st_cluster_v4(to + 512 * k, make_uint4(__float_as_uint(sum[g][4 * k]), __float_as_uint(sum[g][4 * k + 1]),
                                             __float_as_uint(sum[g][4 * k + 2]), __float_as_uint(sum[g][4 * k + 3])));
  }
  __syncwarp();
  cluster_sync_all();
#pragma unroll
  for (int g = 0; g < (PREC ? 4 : 1); ++g) {
    if (half + 2 * g >= in || g % split != slice) continue;
    float total[32];
    for (int from = 0; from < split; ++from) {
      const uint8_t *part = ring + ((from * per + g / split) * kEpiWarps + w) * kStageOut + 16 * lane;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float4 f = from == slice ? make_float4(sum[g][4 * k], sum[g][4 * k + 1], sum[g][4 * k + 2], sum[g][4 * k + 3])
                                       : *reinterpret_cast<const float4 *>(part + 512 * k);
        const float x[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float &t = total[4 * k + c];
          if (from == 0) t = x[c];
          else if (KIND) t = __int_as_float(__float_as_int(t) + __float_as_int(x[c]));
          else t += x[c];
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 32; ++k) sum[g][k] = total[k];
  }
}

// KIND 0: 16-bit operands (kind::f16); 1: int8 (kind::i8).  A_MN: A is
// MN-major (W stored K x channels; the gradient's operands).  PREC: sums in
// pieces of kChunk blocks (fp32 results).
// SPLIT: the cluster's pairs share one tile, each a stretch of its sum (calls of
// few tiles); comes with PREC's running sums in registers.
//
// A pair of CTAs (cluster of 2) works on one 256-row tile of D: each CTA holds
// 128 of its rows (in its tensor memory) and of A's, and half of B's columns;
// the even CTA issues the MMAs for both.  A single CTA with the same 128 x 256
// tile writes and reads 96 + 96 bytes of operands per cycle of MMA in its
// shared memory, more than its 128 bytes per cycle; the pair needs 64 + 64.
// Persistent: warp 0 streams its CTA's operands through a ring of stages (TMA,
// completing on the even CTA's barriers), warp 1 of the even CTA issues each
// tile's MMAs into one of two accumulators, warps 4..11 of both drain the other
// one meanwhile.
template <int KIND, int A_MN, int GRAD, int NMAP, int NOUT, int PREC, int SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    expert_kernel(const __grid_constant__ MmaArgs<NMAP, NOUT> a) {
  constexpr int kElems = KIND ? 128 : 64;   // K elements per block of 128 bytes
  constexpr int kSub = GRAD && PREC ? 1 : 2;   // blocks per stage
  constexpr int kStageK = kElems * kSub;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t ring = kData - a.buffers * kEpiWarps * kStageOut;   // (a multiple of 1024)
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + kData);   // even CTA: both CTAs' loads
  uint64_t *empty = full + kMaxStages;        // each CTA: the stage's MMAs have read it
  uint64_t *acc_full = empty + kMaxStages;    // [2] each CTA: accumulator b holds a finished tile
  uint64_t *acc_empty = acc_full + 2;              // [2] even CTA: accumulator b drained by both CTAs
  uint64_t *drained = acc_empty + 2;               // [2] odd CTA: accumulator b drained by its warps
  uint64_t *done = drained + 2;                    // even CTA: every MMA issued has completed
  uint64_t *c_full = done + 1;                     // [3 per epilogue warp] a box of C has landed
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(c_full + 3 * kEpiWarps);
  int32_t *widest = reinterpret_cast<int32_t *>(tmem_slot + 1);   // product: columns of the widest tile
  int32_t *start = reinterpret_cast<int32_t *>(sm + kData + kBarBytes);   // [n + 1]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr bool kPieces = PREC && !KIND;   // (int32 sums are exact)
  const int32_t cta = static_cast<int32_t>(cluster_ctarank());
  const int32_t rank = cta & 1, even = cta & ~1, slice = SPLIT ? cta >> 1 : 0;
  const uint16_t pair_mask = static_cast<uint16_t>(3u << even);
  const int32_t ctas = SPLIT ? 2 * a.split : 2;
  const int32_t first = static_cast<int32_t>(blockIdx.x) / ctas, step = static_cast<int32_t>(gridDim.x) / ctas;
  grid_start_next();

  if (warp == 0) {
    // one barrier per lane and round: full, empty, acc_full, acc_empty, drained, done, c_full
    constexpr int kAcc = 2 * kMaxStages, kBars = kAcc + 7 + 3 * kEpiWarps;
    for (int i = lane; i < kBars; i += 32)
      mbar_init(full + i, i >= kAcc + 2 && i < kAcc + 4   ? kEpiWarps + 1
                          : i >= kAcc + 4 && i < kAcc + 6 ? kEpiWarps
                                                          : 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  grid_wait();   // nothing above reads or writes what earlier work of the stream does
  if (!GRAD && warp == 2) plan_rows(a, start, widest, lane);
  if (GRAD && warp == 2) check_offsets(a, lane);
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();   // barriers of both CTAs are ready before either is signalled
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int32_t all_tiles = (GRAD ? a.n * a.mt_n : start[a.n]) * a.mt_m;
  const int32_t n_tiles = SPLIT ? min(all_tiles, step) : all_tiles;   // (split: one tile per cluster)
  // a stage holds 128 rows of A and half of the widest tile's columns of B;
  // narrow tiles (few rows per expert) get more stages, so that enough of W is
  // in flight
  const uint32_t b_bytes =
      GRAD ? (a.cap / 2 + 63) / 64 * 8192u : (*widest + 31) / 32 * kBoxBytes;
  const uint32_t block_bytes = (kABytes + b_bytes + 1023) / 1024 * 1024, stage_bytes = kSub * block_bytes;
  const int stages = min(static_cast<int>(ring / stage_bytes), kMaxStages);

  // PREC: the epilogue's running sums take 128 registers per thread: 3 x 168
  // per thread of the three warpgroups become 56 + 2 x 224
  if (warp == 0) {
    if (PREC) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    const uint32_t full0 = mapa_shared(smem_u32(full), even);
    int s = 0;
    uint32_t phase = 1;   // parity of the stage's last release; the first round finds it free
    bool ok = true;
    int64_t issued = 0;
    Tile t, next;
    if (first < n_tiles) next = tile_at<GRAD, SPLIT, kElems>(a, start, slice, first, 0);
    for (int32_t idx = first; idx < n_tiles && ok; idx += step) {
      t = next;
      const bool more = idx + step < n_tiles;   // the next tile is looked up behind this one's first block
      if (more && t.len == 0) next = tile_at<GRAD, SPLIT, kElems>(a, start, slice, idx + step, t.e);
      const int32_t len = t.len;
      const CUtensorMap *mw = NMAP > 1 ? &a.w[t.e] : &a.w[0];
      const int32_t z = NMAP > 1 ? 0 : t.e;
      const int32_t half = t.width / 2;
      const int32_t m0 = t.m0 + 128 * rank, n0 = t.n0 + half * rank;
      const int32_t boxes = GRAD ? (half + 63) / 64 : half / 16;
      const uint32_t bytes = kABytes + boxes * (GRAD ? 8192u : kBoxBytes);
      for (int32_t k = 0; k < len; k += kStageK) {
        if (!(ok = warp_wait(empty + s, phase, a.status))) break;
        uint8_t *As = sm + s * stage_bytes, *Bs = As + kABytes;
        const uint32_t bar = full0 + 8 * s;
        if (GRAD) {
          // a group's last rows, fewer than a block: they go to the block's end,
          // behind rows of zeros (rows -(64 - left) .. of their window), so that
          // no row of another group, whatever it holds, meets the MMAs
          if (elect_one()) {
            const bool both = kSub > 1 && k + kElems < len;
            if (rank == 0) mbar_arrive_expect_tx(full + s, both ? 4 * bytes : 2 * bytes);
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
              if (u > 0 && !both) break;
              uint8_t *Au = As + u * block_bytes, *Bu = Bs + u * block_bytes;
              const int32_t y = t.k0 + k + u * kElems, left = len - k - u * kElems;
              if (left < kElems) {
                tma_load_3d_pair(Au, &a.x[2], m0, left - kElems, y, bar);
                tma_load_3d_pair(Au + 8192, &a.x[2], m0 + 64, left - kElems, y, bar);
                tma_load_3d_pair(Bu, &a.x[1], n0, left - kElems, y, bar);
                if (boxes > 1) tma_load_3d_pair(Bu + 8192, &a.x[1], n0 + 64, left - kElems, y, bar);
              } else {
                tma_load_2d_pair(Au, &a.w[0], m0, y, bar);
                tma_load_2d_pair(Au + 8192, &a.w[0], m0 + 64, y, bar);
                tma_load_2d_pair(Bu, &a.x[0], n0, y, bar);
                if (boxes > 1) tma_load_2d_pair(Bu + 8192, &a.x[0], n0 + 64, y, bar);
              }
            }
          }
        } else if (elect_one()) {
          const bool both = kSub > 1 && k + kElems < len;
          if (rank == 0) mbar_arrive_expect_tx(full + s, both ? 4 * bytes : 2 * bytes);
#pragma unroll
          for (int u = 0; u < kSub; ++u) {
            if (u > 0 && !both) break;
            uint8_t *Au = As + u * block_bytes, *Bu = Bs + u * block_bytes;
            const int32_t ku = t.k0 + k + u * kElems;
            if (A_MN) {
              tma_load_3d_pair(Au, mw, m0, ku, z, bar);
              tma_load_3d_pair(Au + 8192, mw, m0 + 64, ku, z, bar);
            } else {
              tma_load_3d_pair(Au, mw, ku, m0, z, bar);
            }
            // this CTA's rows of the tile in at most four boxes, the largest first
            int32_t at = 0;
#pragma unroll
            for (int32_t i = 0; i < 4; ++i)
              if (boxes & (8 >> i)) {
                tma_load_2d_pair(Bu + kBoxBytes * at, &a.x[i], ku, n0 + 16 * at, bar);
                at += 8 >> i;
              }
          }
        }
        __syncwarp();
        if (k == 0 && more) next = tile_at<GRAD, SPLIT, kElems>(a, start, slice, idx + step, t.e);
        ++issued;
        if (++s == stages) {
          s = 0;
          phase ^= 1;
        }
      }
    }
    // the last loads have landed before the CTA ends, also when something gave
    // up (the even CTA's barriers see both CTAs' loads; the CTAs leave together)
    if (rank == 0)
      for (int64_t i = max((int64_t)0, issued - stages); i < issued; ++i)
        warp_wait(full + i % stages, static_cast<uint32_t>((i / stages) & 1), a.status);
  } else if (warp == 1) {
    if (PREC) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (rank == 0) {
      // descriptors of stage 0, without the address
      const uint64_t a_bits = A_MN ? sw128_desc(0, 8192, 1024) : sw128_desc(0, 16, 1024);
      const uint64_t b_bits = GRAD ? sw128_desc(0, 8192, 1024) : sw128_desc(0, 16, 1024);
      constexpr uint32_t kStepA = (A_MN ? 2048 : 32) >> 4, kStepB = (GRAD ? 2048 : 32) >> 4;
      int s = 0;
      uint32_t phase = 0;
      int32_t j = 0;
      bool ok = true;
      Tile t, next;
      if (first < n_tiles) next = tile_at<GRAD, SPLIT, kElems>(a, start, slice, first, 0);
      for (int32_t idx = first; idx < n_tiles && ok; idx += step) {
        t = next;
        const bool more = idx + step < n_tiles;
        if (more && t.len == 0) next = tile_at<GRAD, SPLIT, kElems>(a, start, slice, idx + step, t.e);
        const int32_t len = t.len;
        const uint32_t idesc = a.idesc | (static_cast<uint32_t>(t.width >> 3) << 17);
        uint32_t d = 0;
        // the next accumulator, once the epilogue has drained it
        auto acquire = [&] {
          const int b = j & 1;
          d = tmem + static_cast<uint32_t>(b * kTileN);
          const bool free = j < 2 || warp_wait<true>(acc_empty + b, static_cast<uint32_t>(((j >> 1) - 1) & 1), a.status);
          tc_fence_after();
          return free;
        };
        auto hand_over = [&] {
          if (elect_one()) mma_commit_pair(acc_full + (j & 1), pair_mask);
          __syncwarp();
          ++j;
        };
        if (len == 0) {
          if (!(ok = acquire())) break;
          hand_over();
        }
        for (int32_t k = 0; k < len; k += kStageK) {
          const uint32_t as = smem_u32(sm) + s * stage_bytes;
          const int32_t left = len - k;
          const bool fresh = kPieces ? k % (kChunk * kElems) == 0 : k == 0;
          if (fresh && !(ok = acquire())) break;
          if (!(ok = warp_wait(full + s, phase, a.status))) break;
          tc_fence_after();
          // (a shared-memory address carries the CTA's rank above the descriptor's field)
          const uint64_t ad = a_bits | ((as >> 4) & 0x3FFF), bd = b_bits | (((as + kABytes) >> 4) & 0x3FFF);
          const int32_t begin = GRAD ? (kElems - min(left, kElems)) / 16 : 0;
          if (elect_one()) {
#pragma unroll
            for (int32_t kk = 0; kk < 4 * kSub; ++kk) {
              // 16 (int8: 32) elements of K at a time; of a block that is not
              // full, the product's lie at its start, the gradient's at its end
              if (kk > 0 && (GRAD ? kk / 4 * kElems : kk * (kElems / 4)) >= left) break;
              if (GRAD && kk % 4 < (kElems - min(left - kk / 4 * kElems, kElems)) / 16) continue;
              const uint32_t off = (kk / 4) * (block_bytes >> 4);
              const uint64_t au = ad + off + (kk % 4) * kStepA, bu = bd + off + (kk % 4) * kStepB;
              const uint32_t add = !fresh || kk > begin ? 1u : 0u;
              if (KIND) mma_i8_ss_pair(d, au, bu, idesc, add);
              else mma_ss_pair(d, au, bu, idesc, add);
            }
            mma_commit_pair(empty + s, pair_mask);   // the stage is free in both CTAs once these MMAs have read it
          }
          __syncwarp();
          if (left <= kStageK || (kPieces && (k + kStageK) % (kChunk * kElems) == 0)) hand_over();
          if (k == 0 && more) next = tile_at<GRAD, SPLIT, kElems>(a, start, slice, idx + step, t.e);
          if (++s == stages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      // nothing is in flight when the pair leaves and releases its tensor memory
      if (elect_one()) mma_commit_pair(done, static_cast<uint16_t>(1u << even));
      __syncwarp();
      warp_wait(done, 0, a.status);
    }
  } else if (warp < 4) {
    if (PREC) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 3 && rank == 1) {
      // Passes the odd CTA's "drained" on to the even one.  An arrival there
      // waits for the thread's earlier stores to be performed (cluster scope,
      // 1 to 2.5 thousand cycles beside a tile's stores); the epilogue's warps
      // arrive in their own CTA instead.
      const uint32_t free0 = mapa_shared(smem_u32(acc_empty), even);
      const int32_t from = 0;
      int32_t j = 0;
      bool ok = true;
      for (int32_t idx = first; idx < n_tiles && ok; idx += step) {
        const int32_t len = GRAD || SPLIT ? tile_at<GRAD, SPLIT, kElems>(a, start, slice, idx, from).len : a.K;
        const int32_t pieces = kPieces ? max(1, (len + kChunk * kElems - 1) / (kChunk * kElems)) : 1;
        for (int32_t p = 0; p < pieces && ok; ++p, ++j) {
          const int b = j & 1;
          ok = warp_wait(drained + b, static_cast<uint32_t>((j >> 1) & 1), a.status);
          tc_fence_after();
          tc_fence_before();
          if (ok && elect_one()) mbar_arrive_cluster(free0 + 8 * b);
          __syncwarp();
        }
      }
    }
  } else if (GRAD) {
    if (PREC) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    // This warp's boxes of G, 32 rows x 32 or 64 columns, in the order of its tiles
    // and, inside one, of the columns.  With C, the boxes of C come by TMA up
    // to two ahead of the one at work, also from the next tile, and the result
    // takes their place: three buffers, so that a buffer is loaded again one
    // box after its store was issued.
    const int q = warp & 3;             // TMEM lanes 32 q .. 32 q + 31
    const int half = (warp - 4) >> 2;   // the warp's column groups: half, half + 2, .. (split: its slice's)
    const int32_t i0 = SPLIT ? half + 2 * slice : half, di = SPLIT ? 2 * a.split : 2;
    const int32_t bc = PREC ? 32 : a.box_cols;
    uint8_t *buf = sm + ring + (warp - 4) * a.buffers * kStageOut;
    uint64_t *landed = c_full + 3 * (warp - 4);
    uint64_t *freed = rank == 0 ? acc_empty : drained;
    const uint32_t c_bytes = bc * (a.cdtype == HIMUON_FP32 ? 128 : 64);
    // A box that reaches over the last column is stored up to the end of that
    // column's 16 bytes (observed: columns behind it in the row's pitch were
    // overwritten); where G's width is no multiple of 16 bytes the last boxes
    // are stored element by element.
    const bool whole_runs = a.N % (a.odtype == HIMUON_FP32 ? 4 : 8) == 0;
    struct Box {
      int32_t idx, i;   // tile, column group; idx >= n_tiles: none left
      Tile t;
    };
    auto groups = [&](const Tile &t) {   // of this tile that are inside G
      return t.m0 + 128 * rank + 32 * q < a.M ? (t.valid + bc - 1) / bc : 0;
    };
    auto settle = [&](Box &x) {   // to the first box at or after (idx, i)
      while (x.idx < n_tiles && x.i >= groups(x.t)) {
        x.idx += step;
        x.i = i0;
        if (x.idx < n_tiles) x.t = tile_at<GRAD, SPLIT, kElems>(a, start, slice, x.idx, 0);
      }
    };
    auto load_c = [&](Box &x, int at) {   // box x into buffer `at`, then on to the next box
      if (x.idx >= n_tiles) return;
      if (elect_one()) {
        mbar_arrive_expect_tx(landed + at, c_bytes);
        tma_load_3d(buf + at * kStageOut, NOUT > 1 ? &a.c[x.t.e] : &a.c[0], x.t.n0 + bc * x.i,
                    x.t.m0 + 128 * rank + 32 * q, NOUT > 1 ? 0 : x.t.e, landed + at);
      }
      __syncwarp();
      x.i += di;
      settle(x);
    };
    Box ahead{first, i0, {}};
    if (a.has_c && first < n_tiles) {
      ahead.t = tile_at<GRAD, SPLIT, kElems>(a, start, slice, first, 0);
      settle(ahead);
      load_c(ahead, 0);
      load_c(ahead, 1);
    }
    int at = 0;                  // buffer of the box at work
    uint32_t c_phase = 0;        // per buffer
    bool ok = true;
    int32_t j = 0;
    for (int32_t idx = first; idx < n_tiles && ok; idx += step) {
      const Tile t = tile_at<GRAD, SPLIT, kElems>(a, start, slice, idx, 0);
      const int32_t in = groups(t);
      // column group i: combine with C, store.  fetch(h, v): its 32-column
      // part h from the accumulator or the running sums.
      auto emit = [&](int32_t i, auto fetch) {
        const int32_t m = t.m0 + 128 * rank + 32 * q, n0 = t.n0 + bc * i;
        const bool by_box = n0 + bc <= a.N || whole_runs;
        uint8_t *box = buf + at * kStageOut;
        float v[32];
        fetch(0, v);
        if (a.has_c) {
          if (!(ok = warp_wait(landed + at, (c_phase >> at) & 1, a.status))) return;
          c_phase ^= 1u << at;
        } else {
          if (elect_one()) bulk_wait_read<0>();   // (the last box's store has read the buffer)
          __syncwarp();
        }
#pragma unroll
        for (int h = 0; h < (PREC ? 1 : 2); ++h) {
          if (32 * h >= bc) break;
          if (h > 0) fetch(h, v);
          if (a.has_c) {
            box_combine(box, lane, a.cdtype, 4 * h, bc == 64, a.alpha, a.beta, v);
            if (bc == 32) __syncwarp();   // (G's rows may lie where C's of other lanes did)
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] *= a.alpha;
          }
          if (by_box) {
            box_write(box, lane, a.odtype, 4 * h, bc == 64, v);
          } else if (m + lane < a.M) {
            char *o = (NOUT > 1 ? a.out[t.e] : a.out[0] + t.e * a.out_stride);
            const int64_t at0 = (m + lane) * a.ldo + n0 + 32 * h;
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (n0 + 32 * h + k < a.N) st_any(o, a.odtype, at0 + k, v[k]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (elect_one()) {
          if (by_box) tma_store_3d(NOUT > 1 ? &a.g[t.e] : &a.g[0], box, n0, m, NOUT > 1 ? 0 : t.e);
          bulk_commit();
          if (a.has_c) bulk_wait_read<1>();   // the store of the box before has read its buffer
        }
        __syncwarp();
        if (a.has_c) load_c(ahead, at == 0 ? 2 : at - 1);
        at = at + 1 == a.buffers ? 0 : at + 1;
      };
      const int32_t pieces = kPieces ? max(1, (t.len + kChunk * kElems - 1) / (kChunk * kElems)) : 1;
      float sum[PREC ? 4 : 1][32];
      for (int32_t p = 0; p < pieces && ok; ++p, ++j) {
        const int b = j & 1;
        if (!(ok = warp_wait(acc_full + b, static_cast<uint32_t>((j >> 1) & 1), a.status))) break;
        tc_fence_after();
        const uint32_t taddr = tmem + static_cast<uint32_t>(b * kTileN) + (static_cast<uint32_t>(q * 32) << 16);
        auto release = [&] {
          tc_fence_before();
          __syncwarp();
          if (elect_one()) mbar_arrive(freed + b);
        };
        if (PREC && (SPLIT || pieces > 1)) {
          read_pieces<PREC>(sum, taddr, half, in, p, t.len == 0);
          release();
          if (!SPLIT && p + 1 == pieces) {
#pragma unroll
            for (int g = 0; g < (PREC ? 4 : 1); ++g)
              if (half + 2 * g < in && ok)
                emit(half + 2 * g, [&](int, float(&v)[32]) {
#pragma unroll
                  for (int k = 0; k < 32; ++k) v[k] = sum[g][k];
                });
          }
        } else {
          for (int32_t i = half; i < in && ok; i += 2) {
            emit(i, [&](int h, float(&v)[32]) {
              if (t.len == 0) {
#pragma unroll
                for (int k = 0; k < 32; ++k) v[k] = 0.f;
              } else {
                tmem_ld32(taddr + bc * i + 32 * h, v);
                tmem_wait_ld();
              }
              if (i + 2 >= in && 32 * (h + 1) >= bc) release();   // the accumulator is read
            });
          }
          if (in <= half) release();   // no box of this warp's in the tile
        }
      }
      if (SPLIT) {
        join_slices<KIND, PREC>(sum, sm, warp - 4, lane, half, in, rank, slice, a.split);
#pragma unroll
        for (int g = 0; g < (PREC ? 4 : 1); ++g)
          if (half + 2 * g < in && g % a.split == slice && ok)
            emit(half + 2 * g, [&](int, float(&v)[32]) {
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] = sum[g][k];
            });
      }
    }
    if (SPLIT && first >= n_tiles) {   // the cluster has no tile: keep step with its barriers
      cluster_sync_all();
      cluster_sync_all();
    }
    if (!ok && a.has_c) {   // gave up: what was loaded ahead lands before the CTA ends (bounded)
      for (int k = 0; k < 3; ++k) warp_wait(landed + k, (c_phase >> k) & 1, a.status);
    }
    if (elect_one()) bulk_wait0();
  } else {
    if (PREC) asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int q = warp & 3;             // TMEM lanes 32 q .. 32 q + 31
    const int half = (warp - 4) >> 2;   // the warp's 32-column groups: half, half + 2, ..
    float *st = reinterpret_cast<float *>(sm + ring + (warp - 4) * kStageOut);
    uint64_t *freed = rank == 0 ? acc_empty : drained;
    int32_t j = 0, from = 0;
    bool ok = true;
    for (int32_t idx = first; idx < n_tiles && ok; idx += step) {
      const Tile t = tile_at<GRAD, SPLIT, kElems>(a, start, slice, idx, from);
      from = t.e;
      const int32_t m = t.m0 + 128 * rank + 32 * q;   // this warp's 32 channels
      const int32_t m_in = min(32, a.M - m);
      float chan = 1.f;
      if (KIND && lane < m_in) chan = a.w_scale[t.e * a.ld_scale + m + lane];
      const int32_t in = m_in > 0 ? (t.valid + 31) / 32 : 0;
      auto emit = [&](int32_t i, float(&v)[32]) {   // rows 32 i .. of the tile
        const int64_t r0 = t.n0 + 32 * i;
        const int32_t r_in = min(32, t.valid - 32 * i);
        if (KIND) {   // int32 sums: scales of this lane's channel and of each row
          const float mine = lane < r_in ? a.x_scale[r0 + lane] : 0.f;
#pragma unroll
          for (int k = 0; k < 32; ++k)
            v[k] = static_cast<float>(__float_as_int(v[k])) * chan * __shfl_sync(0xffffffffu, mine, k);
        }
        const int64_t o = r0 * a.ldo + m;
        if ((PREC && !SPLIT) || a.odtype == HIMUON_FP32)
          put_rows32(st, lane, v, reinterpret_cast<float *>(a.out[0]) + o, a.ldo, r_in, m_in);
        else if (a.odtype == HIMUON_FP16)
          put_rows16<__half2>(reinterpret_cast<uint32_t *>(st), lane, v, reinterpret_cast<uint16_t *>(a.out[0]) + o,
                              a.ldo, r_in, m_in);
        else
          put_rows16<__nv_bfloat162>(reinterpret_cast<uint32_t *>(st), lane, v,
                                     reinterpret_cast<uint16_t *>(a.out[0]) + o, a.ldo, r_in, m_in);
      };
      const int32_t pieces = kPieces ? (t.len + kChunk * kElems - 1) / (kChunk * kElems) : 1;
      float sum[PREC ? 4 : 1][32];
      for (int32_t p = 0; p < pieces && ok; ++p, ++j) {
        const int b = j & 1;
        if (!(ok = warp_wait(acc_full + b, static_cast<uint32_t>((j >> 1) & 1), a.status))) break;
        tc_fence_after();
        const uint32_t taddr = tmem + static_cast<uint32_t>(b * kTileN) + (static_cast<uint32_t>(q * 32) << 16);
        if (PREC && (SPLIT || pieces > 1)) {
          read_pieces<PREC>(sum, taddr, half, in, p, false);
        } else {
#pragma unroll 1
          for (int32_t i = half; i < in; i += 2) {
            tmem_ld32(taddr + 32 * i, sum[0]);
            tmem_wait_ld();
            emit(i, sum[0]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (elect_one()) mbar_arrive(freed + b);
        if (PREC && !SPLIT && pieces > 1 && p + 1 == pieces) {
#pragma unroll
          for (int g = 0; g < (PREC ? 4 : 1); ++g)
            if (half + 2 * g < in) emit(half + 2 * g, sum[g]);
        }
      }
      if (SPLIT) {
        join_slices<KIND, PREC>(sum, sm, warp - 4, lane, half, in, rank, slice, a.split);
#pragma unroll
        for (int g = 0; g < (PREC ? 4 : 1); ++g)
          if (half + 2 * g < in && g % a.split == slice) emit(half + 2 * g, sum[g]);
      }
    }
    if (SPLIT && first >= n_tiles) {   // the cluster has no tile: keep step with its barriers
      cluster_sync_all();
      cluster_sync_all();
    }
  }
  if (SPLIT && warp < 4) {   // the two barriers of join_slices
    __syncwarp();
    cluster_sync_all();
    cluster_sync_all();
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();   // the pair leaves together: neither's memory goes while the other may signal or read it
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// SMs of the current device (looked up once per device).
int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  int sms = known[dev].load(std::memory_order_relaxed);
  if (sms == 0) {
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    known[dev].store(sms, std::memory_order_relaxed);
  }
  return sms;
}

struct QuantArgs {
  const void *in[kMaxList];
  int8_t *codes[kMaxList];
  float *scale[kMaxList];
  int64_t rows[kMaxList], cols[kMaxList], ld[kMaxList], ldq[kMaxList];
  int32_t dtype[kMaxList];
  int32_t dim;
};

// code = round(127 x / top), ties to even.  With 127 / top = hi + lo (two fp32
// numbers, the second the division's remainder), x hi + x lo summed without
// losing the first product's low part is the quotient rounded once: ties of
// 16-bit x, which are short numbers, come out exactly.  Adding 1.5 * 2^23 then
// rounds to an integer and leaves it in the low bits.  Five operations per
// element: the kernel is bound by its instructions (the plain division took 464
// us for 8192 x 11008 bf16).  A maximum so small or large that hi or x hi could
// leave fp32's range takes the division, scaled by a power of two.
__device__ __forceinline__ uint32_t near_code(float x, float hi, float lo) {   // the code in the low byte
  const float p = x * hi;
  return __float_as_uint(p + fmaf(x, lo, fmaf(x, hi, -p)) + 12582912.f);
}
struct Coder {
  float hi, lo, top;
  __device__ explicit Coder(float t) {
    top = t;
    hi = __fdiv_rn(127.f, t);
    lo = __fdiv_rn(fmaf(-t, hi, 127.f), t);
  }
  __device__ __forceinline__ bool in_range() const { return top >= 0x1p-60f && top <= 0x1p60f; }
  __device__ __forceinline__ uint32_t far_code(float x) const {
    const float mul = top > 1.f ? 0x1p-100f : 0x1p100f;
    return __float_as_uint(__fdiv_rn(127.f * (x * mul), top * mul) + 12582912.f);
  }
  __device__ __forceinline__ uint32_t operator()(float x) const { return in_range() ? near_code(x, hi, lo) : far_code(x); }
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
// 16-bit element.
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
    for (int64_t i = t; i < cols; i += TPR) out[i] = ok ? static_cast<int8_t>(code.far_code(ld_any(in, DT, i))) : 0;
    return;
  }
  auto put8 = [&](int32_t i, const Run8<DT> &x) {
    uint32_t u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = near_code(x.get(j), code.hi, code.lo);
    *reinterpret_cast<uint2 *>(out + 8 * i) = make_uint2(bytes4(u[0], u[1], u[2], u[3]), bytes4(u[4], u[5], u[6], u[7]));
  };
#pragma unroll
  for (int h = 0; h < kHold<DT>; ++h)
    if (t + h * TPR < runs) put8(t + h * TPR, v[h]);
  for (int32_t i = t + kHold<DT> * TPR; i < runs; i += TPR) {
    Run8<DT> w;
    w.load(in, i);
    put8(i, w);
  }
  for (int64_t i = 8ll * runs + t; i < cols; i += TPR) out[i] = static_cast<int8_t>(near_code(ld_any(in, DT, i), code.hi, code.lo));
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
__global__ void __launch_bounds__(256) quantize_cols_kernel(const __grid_constant__ QuantArgs a) {
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
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t u[4];
      if (near) {
#pragma unroll
        for (int k = 0; k < 4; ++k) u[k] = near_code(x[k].get(j), hi[j], lo[j]);
      } else {
        const uint32_t top = tops[8 * c8 + j];
        const Coder code(line_ok(top) ? __uint_as_float(top) : 1.f);
#pragma unroll
        for (int k = 0; k < 4; ++k) u[k] = line_ok(top) ? code(x[k].get(j)) : 0;
      }
      turn[(8 * c8 + j) * kTurnPitch + ((rg + 4 * (c8 >> 2)) & 31)] = bytes4(u[0], u[1], u[2], u[3]);
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

// ---------------------------------------------------------------- argument checks
size_t size_of(int32_t dt) { return dt == HIMUON_FP32 ? 4 : dt == HIMUON_I8 ? 1 : 2; }
bool is16(int32_t dt) { return dt == HIMUON_BF16 || dt == HIMUON_FP16; }
bool is_float(int32_t dt) { return dt >= HIMUON_BF16 && dt <= HIMUON_FP32; }

// Longest side of an operand: a sum of that length still ends well inside the
// kernels' bounded waits (two seconds).
constexpr int64_t kMaxSide = (int64_t)1 << 27;
constexpr int32_t kMaxGroups = 1 << 16;

// A matrix operand: shape, pointer and 16-byte alignment of its rows.
// `min_rows` 0: a row operand, which may be empty (its pointer is not used).
int check_operand(const himuon_mat &m, int64_t min_rows) {
  if (m.rows < min_rows || m.cols < 1 || m.ld < m.cols || (m.rows > 0 && !m.data)) return HIMUON_ERR_INVALID;
  if (m.dtype < HIMUON_BF16 || m.dtype > HIMUON_I8) return HIMUON_ERR_UNSUPPORTED;
  if (m.rows > kMaxSide || m.cols > kMaxSide || m.ld > (int64_t)1 << 36) return HIMUON_ERR_UNSUPPORTED;
  if (m.rows > 0 && reinterpret_cast<uintptr_t>(m.data) % 16 != 0) return HIMUON_ERR_ALIGNMENT;
  // (the pitch of a single row is never used)
  if (m.rows > 1 && (m.ld * static_cast<int64_t>(size_of(m.dtype))) % 16 != 0) return HIMUON_ERR_ALIGNMENT;
  return HIMUON_OK;
}

// n matrices that differ in `data` alone.
int check_list(const himuon_mat *m, int32_t n) {
  for (int32_t e = 0; e < n; ++e) {
    const int rc = check_operand(m[e], 1);
    if (rc) return rc;
    if (m[e].rows != m[0].rows || m[e].cols != m[0].cols || m[e].ld != m[0].ld || m[e].dtype != m[0].dtype)
      return HIMUON_ERR_INVALID;
  }
  return HIMUON_OK;
}

// Scales: fp32, `rows` x `cols`, natural alignment.
int check_scale(const himuon_mat *m, int64_t rows, int64_t cols) {
  if (!m || m->rows != rows || m->cols != cols || m->ld < m->cols) return HIMUON_ERR_INVALID;
  if (m->dtype != HIMUON_FP32) return HIMUON_ERR_UNSUPPORTED;
  if (cols > 0 && rows > 0 && !m->data) return HIMUON_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(m->data) % 4 != 0) return HIMUON_ERR_ALIGNMENT;
  return HIMUON_OK;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    return cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                   q == cudaDriverEntryPointSuccess
               ? reinterpret_cast<EncodeTiledFn>(p)
               : nullptr;
  }();
  return fn;
}

// Map over `n` row-major matrices `stride` bytes apart (2-D when n = 0): boxes
// of box_rows x box_cols (0: as many as make 128 bytes) with the swizzle of the
// box's width (64 or 128 bytes), zeros outside.
bool make_map(CUtensorMap *map, const himuon_mat &m, int32_t n, int64_t stride, uint32_t box_rows,
              uint32_t box_cols = 0) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const int64_t es = static_cast<int64_t>(size_of(m.dtype));
  if (!box_cols) box_cols = static_cast<uint32_t>(128 / es);
  const CUtensorMapDataType dt = m.dtype == HIMUON_I8     ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : m.dtype == HIMUON_FP32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                 : m.dtype == HIMUON_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                          : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  // the pitch of a single row is never used and may be any number
  const int64_t pitch = m.rows > 1 ? m.ld * es : (m.cols * es + 15) / 16 * 16;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(m.cols), static_cast<cuuint64_t>(m.rows),
                        static_cast<cuuint64_t>(n > 0 ? n : 1)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(pitch), static_cast<cuuint64_t>(n > 1 ? stride : pitch * m.rows)};
  cuuint32_t box[3] = {box_cols, box_rows, 1};
  cuuint32_t es1[3] = {1, 1, 1};
  return enc(map, dt, n > 0 ? 3 : 2, m.data, dims, strides, box, es1, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_cols * es == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A row operand as overlapping windows: coordinates (column, r, row) are row `row`
// + r, r < 64, so that a box that begins at r = left - 64 holds 64 - left rows of
// zeros and then rows row .. row + left - 1.
bool make_window_map(CUtensorMap *map, const himuon_mat &m) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const int64_t es = static_cast<int64_t>(size_of(m.dtype));
  const CUtensorMapDataType dt =
      m.dtype == HIMUON_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint64_t pitch = static_cast<cuuint64_t>(m.rows > 1 ? m.ld * es : (m.cols * es + 15) / 16 * 16);
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(m.cols), 64, static_cast<cuuint64_t>(m.rows)};
  cuuint64_t strides[2] = {pitch, pitch};
  cuuint32_t box[3] = {64, 64, 1};
  cuuint32_t es1[3] = {1, 1, 1};
  return enc(map, dt, 3, m.data, dims, strides, box, es1, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Do the matrices lie one behind the other at equal distances, a multiple of
// their pitch in a tensor map's range?  `stride`: that distance.  (Anything else,
// such as column blocks of one fused matrix, runs as a list.)
bool stacked(const himuon_mat *m, int32_t n, int64_t *stride) {
  *stride = 0;
  if (n == 1) return true;
  const int64_t d = static_cast<const char *>(m[1].data) - static_cast<const char *>(m[0].data);
  const int64_t pitch = m->ld * static_cast<int64_t>(size_of(m->dtype));
  if (d < pitch * m->rows || d % pitch != 0 || pitch % 16 != 0 || d >= (int64_t)1 << 39) return false;
  for (int32_t e = 1; e < n; ++e)
    if (static_cast<const char *>(m[e].data) - static_cast<const char *>(m[e - 1].data) != d) return false;
  *stride = d;
  return true;
}

// Every variant of the kernel is loaded, and allowed its shared memory, at the
// first call on a device: a call captured into a graph later loads nothing.
template <int KIND, int A_MN, int GRAD, int PREC, int SPLIT>
bool load_variant() {
  return cudaFuncSetAttribute(expert_kernel<KIND, A_MN, GRAD, 1, 1, PREC, SPLIT>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) == cudaSuccess &&
         cudaFuncSetAttribute(expert_kernel<KIND, A_MN, GRAD, GRAD ? 1 : kMaxList, GRAD ? kMaxList : 1, PREC, SPLIT>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) == cudaSuccess;
}
bool load_kernels() {
  static std::atomic<uint64_t> loaded{0};   // a bit per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (loaded.load(std::memory_order_relaxed) & bit) return true;
  const bool ok =
      load_variant<0, 0, 0, 0, 0>() && load_variant<0, 0, 0, 1, 0>() && load_variant<0, 0, 0, 1, 1>() &&
      load_variant<0, 1, 0, 0, 0>() && load_variant<0, 1, 0, 1, 0>() && load_variant<0, 1, 0, 1, 1>() &&
      load_variant<1, 0, 0, 0, 0>() && load_variant<1, 0, 0, 1, 1>() && load_variant<0, 1, 1, 0, 0>() &&
      load_variant<0, 1, 1, 1, 0>() && load_variant<0, 1, 1, 1, 1>() && device_status_word() != nullptr &&
      load_quant_kernels<HIMUON_BF16>() && load_quant_kernels<HIMUON_FP16>() && load_quant_kernels<HIMUON_FP32>();
  if (ok) loaded.fetch_or(bit, std::memory_order_relaxed);
  return ok;
}
int expert_device() {
  const int rc = device_usable();
  if (rc) return rc;
  return load_kernels() ? HIMUON_OK : HIMUON_ERR_CUDA;
}

template <int KIND, int A_MN, int GRAD, int PREC, int SPLIT, int NMAP, int NOUT>
int launch_mma(const MmaArgs<NMAP, NOUT> &a, int64_t most_tiles, cudaStream_t stream) {
  auto kern = expert_kernel<KIND, A_MN, GRAD, NMAP, NOUT, PREC, SPLIT>;
  const unsigned ctas = 2 * static_cast<unsigned>(a.split);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas * static_cast<unsigned>(SPLIT ? most_tiles : std::min<int64_t>(most_tiles, sm_count() / 2)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  count_launch();
  return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? HIMUON_OK : HIMUON_ERR_CUDA;
}

// How many pairs share a tile (1, 2 or 4): as many as the call's tiles, at most
// `tiles`, leave pairs for, each with at least 4 blocks of the longest sum.
int32_t split_of(int64_t tiles, int64_t blocks) {
  const int64_t pairs = sm_count() / 2;
  for (int32_t s = 4; s > 1; s /= 2)
    if (tiles * s <= pairs && blocks >= 4 * s) return s;
  return 1;
}

template <int NMAP, int NOUT>
void common_args(MmaArgs<NMAP, NOUT> &a, const int32_t *offsets, int32_t e0, int32_t n, int64_t rows) {
  a.offsets = offsets ? offsets + e0 : nullptr;
  a.rows = rows;
  a.n = n;
  a.status = device_status_word();
  a.x_scale = a.w_scale = nullptr;
  a.ld_scale = 0;
  a.has_c = 0;
  a.ldo = a.out_stride = 0;
  a.buffers = 1;
  a.box_cols = 0;
  a.split = 1;
  a.cdtype = HIMUON_BF16;
  a.alpha = 1.f;
  a.beta = 0.f;
}

// D format and operand formats of the instruction descriptor (its N field is
// set per tile): f32 from bf16/fp16, or s32 from s8.
uint32_t idesc_of(int32_t dtype, uint32_t a_mn, uint32_t b_mn) {
  if (dtype == HIMUON_I8) return (2u << 4) | (1u << 7) | (1u << 10) | ((kTileM >> 4) << 24);
  return idesc_f16(kTileM, 0, dtype == HIMUON_FP16 ? 0u : 1u, a_mn, b_mn, 0);
}

template <int NMAP>
int product_launch(const himuon_mat *X, const float *x_scale, const himuon_mat *W, int64_t stride,
                   const himuon_mat *w_scale, int32_t e0, int32_t n, const int32_t *offsets, int32_t w_trans,
                   const himuon_mat *Y, cudaStream_t stream) {
  MmaArgs<NMAP, 1> a;
  common_args(a, offsets, e0, n, X->rows);
  const uint32_t w_rows = w_trans ? 128 : 64;
  for (int32_t i = 0; i < (NMAP > 1 ? n : 1); ++i)
    if (!make_map(&a.w[i], W[e0 + i], NMAP > 1 ? 1 : n, stride, w_rows)) return HIMUON_ERR_CUDA;
  // (boxes of more rows than half of the widest tile are never loaded)
  const int64_t half = (std::min<int64_t>(X->rows, kTileN) + 31) / 32 * 16;
  for (int i = 0; i < 4; ++i)
    if ((128 >> i) <= half && !make_map(&a.x[i], *X, 0, 0, 128 >> i)) return HIMUON_ERR_CUDA;
  a.K = static_cast<int32_t>(X->cols);
  a.M = static_cast<int32_t>(Y->cols);
  a.N = 0;
  a.idesc = idesc_of(X->dtype, w_trans ? 0 : 1, 0);
  if (x_scale) {
    a.x_scale = x_scale;
    a.w_scale = static_cast<const float *>(w_scale->data) + e0 * w_scale->ld;
    a.ld_scale = w_scale->ld;
  }
  a.out[0] = static_cast<char *>(Y->data);
  a.ldo = Y->ld;
  a.odtype = Y->dtype;
  // Row tiles of up to 256 rows move the fewest bytes.  Where even tiles of up to
  // 128 (below that a tile's loads of W bound it) cannot fill the pairs once,
  // whatever the groups' sizes, they are taken, and what pairs are left then
  // share the tiles' sums.  (One group of 512 rows, 4096 -> 4096: 28.7 us
  // with 256 rows, 20.5 with 128; where the cap lengthens the last round instead,
  // it costs: 1024 rows 28.7 us with 256, 32.9 with 128.)
  const int64_t mt_m = (Y->cols + kTileM - 1) / kTileM, pairs = sm_count() / 2;
  auto most_tiles = [&](int64_t cap) {
    return mt_m * (n == 1 ? (X->rows + cap - 1) / cap : X->rows / cap + std::min<int64_t>(n, X->rows));
  };
  a.cap = most_tiles(128) <= pairs ? 7 : 8;
  const int64_t most = most_tiles(1 << a.cap);
  a.mt_m = static_cast<int32_t>(mt_m);
  a.mt_n = 0;
  a.split = split_of(most, (X->cols * static_cast<int64_t>(size_of(X->dtype)) + 127) / 128);
  const bool fp32 = Y->dtype == HIMUON_FP32;
  if (X->dtype == HIMUON_I8)
    return a.split > 1 ? launch_mma<1, 0, 0, 1, 1>(a, most, stream) : launch_mma<1, 0, 0, 0, 0>(a, most, stream);
  if (w_trans)
    return a.split > 1 ? launch_mma<0, 0, 0, 1, 1>(a, most, stream)
           : fp32      ? launch_mma<0, 0, 0, 1, 0>(a, most, stream)
                       : launch_mma<0, 0, 0, 0, 0>(a, most, stream);
  return a.split > 1 ? launch_mma<0, 1, 0, 1, 1>(a, most, stream)
         : fp32      ? launch_mma<0, 1, 0, 1, 0>(a, most, stream)
                     : launch_mma<0, 1, 0, 0, 0>(a, most, stream);
}

int run_product(const himuon_mat *X, const float *x_scale, const himuon_mat *W, const himuon_mat *w_scale, int32_t n,
                const int32_t *offsets, int32_t w_trans, const himuon_mat *Y, cudaStream_t stream) {
  if (X->rows == 0) return HIMUON_OK;
  int64_t stride;
  const bool st = stacked(W, n, &stride);
  const int32_t cap = st ? kMaxStack : kMaxList;
  for (int32_t e0 = 0; e0 < n; e0 += cap) {
    const int32_t cnt = std::min(n - e0, cap);
    const int rc = st ? product_launch<1>(X, x_scale, W, stride, w_scale, e0, cnt, offsets, w_trans, Y, stream)
                      : product_launch<kMaxList>(X, x_scale, W, 0, w_scale, e0, cnt, offsets, w_trans, Y, stream);
    if (rc) return rc;
  }
  return HIMUON_OK;
}

template <int NOUT>
int gradient_launch(const himuon_mat *A, const himuon_mat *B, int32_t e0, int32_t n, const int32_t *offsets,
                    float alpha, float beta, const himuon_mat *C, int64_t c_stride, const himuon_mat *G,
                    int64_t g_stride, cudaStream_t stream) {
  MmaArgs<1, NOUT> a;
  common_args(a, offsets, e0, n, A->rows);
  if (A->rows == 0) {
    // no row is ever loaded: the maps only have to be valid, and G's memory is
    himuon_mat any = *G;
    any.dtype = A->dtype;
    any.rows = 1;
    any.cols = 8;
    if (!make_map(&a.w[0], any, 0, 0, 64)) return HIMUON_ERR_CUDA;
    a.x[0] = a.x[1] = a.x[2] = a.w[0];
  } else if (!make_map(&a.w[0], *A, 0, 0, 64) || !make_map(&a.x[0], *B, 0, 0, 64) ||
             !make_window_map(&a.x[1], *B) || !make_window_map(&a.x[2], *A)) {
    return HIMUON_ERR_CUDA;
  }
  a.K = 0;
  a.M = static_cast<int32_t>(A->cols);
  a.N = static_cast<int32_t>(B->cols);
  a.idesc = idesc_of(A->dtype, 1, 1);
  a.alpha = alpha;
  a.beta = beta;
  a.has_c = C != nullptr;
  // Columns of a tile: as few tiles as 256 columns allow, or more of equal
  // width where that fills the last round of the pairs better (a tile costs its
  // columns and about as much as 64 more), in whole boxes of the epilogue.
  const bool wide = G->dtype == HIMUON_FP32 || (C && C->dtype == HIMUON_FP32);
  a.box_cols = wide ? 32 : 64;
  const int64_t m_tiles = n * ((A->cols + kTileM - 1) / kTileM), pairs = sm_count() / 2;
  const int64_t fewest = (B->cols + kTileN - 1) / kTileN;
  int64_t best = INT64_MAX, most = 0;
  for (int64_t c = fewest; c <= 4 * fewest; ++c) {
    const int64_t w = ((B->cols + c - 1) / c + a.box_cols - 1) / a.box_cols * a.box_cols;
    const int64_t tiles = m_tiles * ((B->cols + w - 1) / w), cost = (tiles + pairs - 1) / pairs * (w + 64);
    if (cost < best) {
      best = cost;
      most = tiles;
      a.cap = static_cast<int32_t>(w);
      a.mt_n = static_cast<int32_t>(tiles / m_tiles);
    }
    if (tiles >= 6 * pairs) break;
  }
  a.mt_m = static_cast<int32_t>(m_tiles / n);
  a.split = split_of(most, (A->rows + 63) / 64);
  if (a.split > 1) a.box_cols = 32;
  for (int32_t i = 0; i < (NOUT > 1 ? n : 1); ++i) {
    if (!make_map(&a.g[i], G[e0 + i], NOUT > 1 ? 1 : n, g_stride, 32, a.box_cols)) return HIMUON_ERR_CUDA;
    a.out[i] = static_cast<char *>(G[e0 + i].data);
    if (C && !make_map(&a.c[i], C[e0 + i], NOUT > 1 ? 1 : n, c_stride, 32, a.box_cols)) return HIMUON_ERR_CUDA;
  }
  a.ldo = G->ld;
  a.out_stride = g_stride;
  a.odtype = G->dtype;
  if (C) a.cdtype = C->dtype;
  a.buffers = C ? 3 : 1;
  if (a.split > 1) return launch_mma<0, 1, 1, 1, 1>(a, most, stream);
  return G->dtype == HIMUON_FP32 ? launch_mma<0, 1, 1, 1, 0>(a, most, stream) : launch_mma<0, 1, 1, 0, 0>(a, most, stream);
}

}  // namespace
}  // namespace himuon

using namespace himuon;

extern "C" {

int himuon_expert_product(const himuon_mat *X, const himuon_mat *W, int32_t n, const int32_t *offsets, int32_t w_trans,
                          const himuon_mat *Y, void *stream) {
  if (!X || !W || !Y || n < 1 || n > kMaxGroups || (!offsets && n != 1) || (w_trans != 0 && w_trans != 1)) return HIMUON_ERR_INVALID;
  int rc = check_operand(*X, 0);
  if (!rc) rc = check_operand(*Y, 0);
  if (!rc) rc = check_list(W, n);
  if (rc) return rc;
  if (!is16(X->dtype) || !is_float(Y->dtype)) return HIMUON_ERR_UNSUPPORTED;
  if (W->dtype != X->dtype || Y->rows != X->rows) return HIMUON_ERR_INVALID;
  if ((w_trans ? W->cols : W->rows) != X->cols || (w_trans ? W->rows : W->cols) != Y->cols) return HIMUON_ERR_INVALID;
  rc = expert_device();
  if (rc) return rc;
  return run_product(X, nullptr, W, nullptr, n, offsets, w_trans, Y, static_cast<cudaStream_t>(stream));
}

int himuon_expert_product_i8(const himuon_mat *X, const himuon_mat *x_scale, const himuon_mat *W,
                             const himuon_mat *w_scale, int32_t n, const int32_t *offsets, const himuon_mat *Y,
                             void *stream) {
  if (!X || !W || !Y || n < 1 || n > kMaxGroups || (!offsets && n != 1)) return HIMUON_ERR_INVALID;
  int rc = check_operand(*X, 0);
  if (!rc) rc = check_operand(*Y, 0);
  if (!rc) rc = check_list(W, n);
  if (!rc) rc = check_scale(x_scale, 1, X->rows);
  if (!rc) rc = check_scale(w_scale, n, Y->cols);
  if (rc) return rc;
  if (X->dtype != HIMUON_I8 || W->dtype != HIMUON_I8 || !is_float(Y->dtype)) return HIMUON_ERR_UNSUPPORTED;
  if (W->cols != X->cols || W->rows != Y->cols || Y->rows != X->rows) return HIMUON_ERR_INVALID;
  if (X->cols > 131071) return HIMUON_ERR_UNSUPPORTED;   // 2^14 per term: the sum stays inside int32
  rc = expert_device();
  if (rc) return rc;
  return run_product(X, static_cast<const float *>(x_scale->data), W, w_scale, n, offsets, 1, Y,
                     static_cast<cudaStream_t>(stream));
}

int himuon_expert_gradient(const himuon_mat *A, const himuon_mat *B, int32_t n, const int32_t *offsets, float alpha,
                           float beta, const himuon_mat *C, const himuon_mat *G, void *stream) {
  if (!A || !B || !G || n < 1 || n > kMaxGroups || (!offsets && n != 1)) return HIMUON_ERR_INVALID;
  if (!isfinite(alpha) || !isfinite(beta) || (!C && beta != 0.f)) return HIMUON_ERR_INVALID;
  int rc = check_operand(*A, 0);
  if (!rc) rc = check_operand(*B, 0);
  if (!rc) rc = check_list(G, n);
  if (!rc && C) rc = check_list(C, n);
  if (rc) return rc;
  if (!is16(A->dtype) || !is_float(G->dtype) || (C && !is_float(C->dtype))) return HIMUON_ERR_UNSUPPORTED;
  if (B->dtype != A->dtype || B->rows != A->rows || G->rows != A->cols || G->cols != B->cols) return HIMUON_ERR_INVALID;
  if (C && (C->rows != G->rows || C->cols != G->cols)) return HIMUON_ERR_INVALID;
  if (C && beta != 0.f && (C->ld != G->ld || C->dtype != G->dtype))
    for (int32_t e = 0; e < n; ++e)
      if (C[e].data == G[e].data) return HIMUON_ERR_INVALID;
  int64_t g_stride, c_stride = 0;
  const bool g_stacked = stacked(G, n, &g_stride);
  if (!g_stacked) {   // (stacked ones differ)
    std::vector<const void *> seen(n);
    for (int32_t e = 0; e < n; ++e) seen[e] = G[e].data;
    std::sort(seen.begin(), seen.end());
    if (std::adjacent_find(seen.begin(), seen.end()) != seen.end()) return HIMUON_ERR_INVALID;
  }
  rc = expert_device();
  if (rc) return rc;
  if (beta == 0.f) C = nullptr;
  const bool st = g_stacked && (!C || stacked(C, n, &c_stride));
  const int32_t cap = st ? kMaxStack : kMaxList;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (int32_t e0 = 0; e0 < n; e0 += cap) {
    const int32_t cnt = std::min(n - e0, cap);
    rc = st ? gradient_launch<1>(A, B, e0, cnt, offsets, alpha, beta, C, c_stride, G, g_stride, s)
            : gradient_launch<kMaxList>(A, B, e0, cnt, offsets, alpha, beta, C, 0, G, 0, s);
    if (rc) return rc;
  }
  return HIMUON_OK;
}

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
