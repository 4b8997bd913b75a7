// experts.cu -- products over row groups: expert forward and input-gradient
// products, weight gradients, 8-bit codes and the 8-bit product.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>
#include <vector>

#include "himuon.h"
#include "layout.hpp"
#include "ptx.cuh"

namespace himuon {

int device_usable();         // api.cu: HIMUON_OK or HIMUON_ERR_NO_DEVICE for the current device
int *device_status_word();   // api.cu: the current device's status word

namespace {

// Matrices of one launch, by value in the kernel's parameters: a list of up to
// kMaxList pointers (a longer list runs as several launches, each on its own
// stretch of the offsets).
constexpr int kMaxList = 64;
struct PtrList {
  void *p[kMaxList];
};

__device__ __forceinline__ float ld_any(const void *p, int32_t dtype, int64_t i) {
  if (dtype == HIMUON_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
  if (dtype == HIMUON_FP16) return __half2float(static_cast<const __half *>(p)[i]);
  if (dtype == HIMUON_I8) return static_cast<float>(static_cast<const int8_t *>(p)[i]);
  return static_cast<const float *>(p)[i];
}
__device__ __forceinline__ void st_any(void *p, int32_t dtype, int64_t i, float v) {
  if (dtype == HIMUON_BF16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
  else if (dtype == HIMUON_FP16) static_cast<__half *>(p)[i] = __float2half_rn(v);
  else static_cast<float *>(p)[i] = v;
}

// Rows [lo, hi) of group e; a bound outside 0 .. rows or below the one before
// it is clamped and reported.
__device__ __forceinline__ void group_rows(const int32_t *offsets, int32_t e, int64_t rows, int *status, int64_t &lo,
                                           int64_t &hi) {
  if (!offsets) {
    lo = 0;
    hi = rows;
    return;
  }
  lo = offsets[e];
  hi = offsets[e + 1];
  if (lo < 0 || hi < lo || hi > rows) set_status(status, HIMUON_ERR_DEVICE);
  lo = min(max(lo, (int64_t)0), rows);
  hi = min(max(hi, lo), rows);
}

struct ProductArgs {
  const void *X;
  int64_t rows, ldx;
  PtrList W;
  int64_t ldw;
  const int32_t *offsets;
  int32_t n, dtype, w_trans;
  const float *x_scale;
  const float *w_scale;   // row e: group e's channel scales, ld_scale apart
  int64_t ld_scale;
  void *Y;
  int64_t ldy;
  int32_t ydtype;
  int64_t K, N;
  int *status;
};

// One thread per output element, blocks of 16 rows x 16 columns of a group.
template <typename Acc>
__global__ void __launch_bounds__(256) product_kernel(const __grid_constant__ ProductArgs a) {
  const int32_t e = blockIdx.z;
  int64_t lo, hi;
  group_rows(a.offsets, e, a.rows, a.status, lo, hi);
  const int64_t c = blockIdx.x * 16ll + (threadIdx.x & 15);
  for (int64_t r = lo + blockIdx.y * 16ll + (threadIdx.x >> 4); r < hi; r += 16ll * gridDim.y) {
    if (c >= a.N) continue;
    Acc acc = 0;
    for (int64_t k = 0; k < a.K; ++k) {
      const float w = ld_any(a.W.p[e], a.dtype, a.w_trans ? c * a.ldw + k : k * a.ldw + c);
      acc += static_cast<Acc>(ld_any(a.X, a.dtype, r * a.ldx + k)) * static_cast<Acc>(w);
    }
    float v = static_cast<float>(acc);
    if (a.x_scale) v = v * a.x_scale[r] * a.w_scale[e * a.ld_scale + c];
    st_any(a.Y, a.ydtype, r * a.ldy + c, v);
  }
}

struct GradientArgs {
  const void *A, *B;
  int64_t rows, lda, ldb;
  const int32_t *offsets;
  int32_t n, dtype;
  float alpha, beta;
  PtrList C, G;
  int64_t ldc, ldg;
  int32_t cdtype, gdtype, has_c;
  int64_t P, Q;
  int *status;
};

__global__ void __launch_bounds__(256) gradient_kernel(const __grid_constant__ GradientArgs a) {
  const int32_t e = blockIdx.z;
  int64_t lo, hi;
  group_rows(a.offsets, e, a.rows, a.status, lo, hi);
  const int64_t q = blockIdx.x * 16ll + (threadIdx.x & 15);
  for (int64_t p = blockIdx.y * 16ll + (threadIdx.x >> 4); p < a.P; p += 16ll * gridDim.y) {
    if (q >= a.Q) continue;
    float acc = 0.f;
    for (int64_t r = lo; r < hi; ++r)
      acc = fmaf(ld_any(a.A, a.dtype, r * a.lda + p), ld_any(a.B, a.dtype, r * a.ldb + q), acc);
    float v = a.alpha * acc;
    if (a.has_c) v = fmaf(a.beta, ld_any(a.C.p[e], a.cdtype, p * a.ldc + q), v);
    st_any(a.G.p[e], a.gdtype, p * a.ldg + q, v);
  }
}

struct QuantArgs {
  const void *in[kMaxList];
  int8_t *codes[kMaxList];
  float *scale[kMaxList];
  int64_t rows[kMaxList], cols[kMaxList], ld[kMaxList], ldq[kMaxList];
  int32_t dtype[kMaxList];
  int32_t dim;
};

// code = round(127 x / top), ties to even: 127 x is exact in fp32 for 16-bit
// x, and the division rounds correctly, so a tie in exact arithmetic is a tie
// here.
__device__ __forceinline__ int8_t code_of(float x, float top) {
  return static_cast<int8_t>(__float2int_rn(__fdiv_rn(127.f * x, top)));
}

// One warp per row (dim 0) or column (dim 1).
__global__ void __launch_bounds__(256) quantize_kernel(const __grid_constant__ QuantArgs a) {
  const int32_t z = blockIdx.y;
  const int64_t lines = a.dim ? a.cols[z] : a.rows[z], len = a.dim ? a.rows[z] : a.cols[z];
  const int64_t line = blockIdx.x * 8ll + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (line >= lines) return;
  const int64_t step = a.dim ? a.ld[z] : 1, base = a.dim ? line : line * a.ld[z];
  float top = 0.f;
  bool bad = false;
  for (int64_t i = lane; i < len; i += 32) {
    const float x = fabsf(ld_any(a.in[z], a.dtype[z], base + i * step));
    bad |= !(x <= 3.402823466e38f);
    top = fmaxf(top, x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  bad = __any_sync(0xffffffffu, bad);
  for (int64_t i = lane; i < len; i += 32) {
    const float x = ld_any(a.in[z], a.dtype[z], base + i * step);
    a.codes[z][line * a.ldq[z] + i] = (bad || top == 0.f) ? 0 : code_of(x, top);
  }
  if (lane == 0) a.scale[z][line] = bad ? __int_as_float(0x7fffffff) : top / 127.f;
}

// ---------------------------------------------------------------- argument checks
size_t size_of(int32_t dt) { return dt == HIMUON_FP32 ? 4 : dt == HIMUON_I8 ? 1 : 2; }
bool is16(int32_t dt) { return dt == HIMUON_BF16 || dt == HIMUON_FP16; }
bool is_float(int32_t dt) { return dt >= HIMUON_BF16 && dt <= HIMUON_FP32; }

// A matrix operand: shape, pointer and 16-byte alignment of its rows.
// `min_rows` 0: a row operand, which may be empty (its pointer is not used).
int check_operand(const himuon_mat &m, int64_t min_rows) {
  if (m.rows < min_rows || m.cols < 1 || m.ld < m.cols || (m.rows > 0 && !m.data)) return HIMUON_ERR_INVALID;
  if (m.dtype < HIMUON_BF16 || m.dtype > HIMUON_I8) return HIMUON_ERR_UNSUPPORTED;
  if (m.rows > (int64_t)1 << 30 || m.cols > (int64_t)1 << 30 || m.ld > (int64_t)1 << 36) return HIMUON_ERR_UNSUPPORTED;
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

int run_product(const himuon_mat *X, const float *x_scale, const himuon_mat *W, const himuon_mat *w_scale, int32_t n,
                const int32_t *offsets, int32_t w_trans, const himuon_mat *Y, cudaStream_t stream) {
  if (X->rows == 0) return HIMUON_OK;
  for (int32_t e0 = 0; e0 < n; e0 += kMaxList) {
    ProductArgs a;
    a.n = std::min(n - e0, kMaxList);
    a.X = X->data;
    a.rows = X->rows;
    a.ldx = X->ld;
    for (int32_t e = 0; e < a.n; ++e) a.W.p[e] = W[e0 + e].data;
    a.ldw = W->ld;
    a.offsets = offsets ? offsets + e0 : nullptr;
    a.dtype = X->dtype;
    a.w_trans = w_trans;
    a.x_scale = x_scale;
    a.w_scale = w_scale ? static_cast<const float *>(w_scale->data) + e0 * w_scale->ld : nullptr;
    a.ld_scale = w_scale ? w_scale->ld : 0;
    a.Y = Y->data;
    a.ldy = Y->ld;
    a.ydtype = Y->dtype;
    a.K = X->cols;
    a.N = Y->cols;
    a.status = device_status_word();
    const dim3 grid(static_cast<unsigned>((a.N + 15) / 16),
                    static_cast<unsigned>(std::min<int64_t>((a.rows + 15) / 16, 64)), static_cast<unsigned>(a.n));
    count_launch();
    if (X->dtype == HIMUON_I8) product_kernel<int32_t><<<grid, 256, 0, stream>>>(a);
    else product_kernel<float><<<grid, 256, 0, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return HIMUON_ERR_CUDA;
  }
  return HIMUON_OK;
}

}  // namespace
}  // namespace himuon

using namespace himuon;

extern "C" {

int himuon_expert_product(const himuon_mat *X, const himuon_mat *W, int32_t n, const int32_t *offsets, int32_t w_trans,
                          const himuon_mat *Y, void *stream) {
  if (!X || !W || !Y || n < 1 || (!offsets && n != 1) || (w_trans != 0 && w_trans != 1)) return HIMUON_ERR_INVALID;
  int rc = check_operand(*X, 0);
  if (!rc) rc = check_operand(*Y, 0);
  if (!rc) rc = check_list(W, n);
  if (rc) return rc;
  if (!is16(X->dtype) || !is_float(Y->dtype)) return HIMUON_ERR_UNSUPPORTED;
  if (W->dtype != X->dtype || Y->rows != X->rows) return HIMUON_ERR_INVALID;
  if ((w_trans ? W->cols : W->rows) != X->cols || (w_trans ? W->rows : W->cols) != Y->cols) return HIMUON_ERR_INVALID;
  rc = device_usable();
  if (rc) return rc;
  return run_product(X, nullptr, W, nullptr, n, offsets, w_trans, Y, static_cast<cudaStream_t>(stream));
}

int himuon_expert_product_i8(const himuon_mat *X, const himuon_mat *x_scale, const himuon_mat *W,
                             const himuon_mat *w_scale, int32_t n, const int32_t *offsets, const himuon_mat *Y,
                             void *stream) {
  if (!X || !W || !Y || n < 1 || (!offsets && n != 1)) return HIMUON_ERR_INVALID;
  int rc = check_operand(*X, 0);
  if (!rc) rc = check_operand(*Y, 0);
  if (!rc) rc = check_list(W, n);
  if (!rc) rc = check_scale(x_scale, 1, X->rows);
  if (!rc) rc = check_scale(w_scale, n, Y->cols);
  if (rc) return rc;
  if (X->dtype != HIMUON_I8 || W->dtype != HIMUON_I8 || !is_float(Y->dtype)) return HIMUON_ERR_UNSUPPORTED;
  if (W->cols != X->cols || W->rows != Y->cols || Y->rows != X->rows) return HIMUON_ERR_INVALID;
  if (X->cols > 131071) return HIMUON_ERR_UNSUPPORTED;   // 2^14 per term: the sum stays inside int32
  rc = device_usable();
  if (rc) return rc;
  return run_product(X, static_cast<const float *>(x_scale->data), W, w_scale, n, offsets, 1, Y,
                     static_cast<cudaStream_t>(stream));
}

int himuon_expert_gradient(const himuon_mat *A, const himuon_mat *B, int32_t n, const int32_t *offsets, float alpha,
                           float beta, const himuon_mat *C, const himuon_mat *G, void *stream) {
  if (!A || !B || !G || n < 1 || (!offsets && n != 1)) return HIMUON_ERR_INVALID;
  if (!isfinite(alpha) || !isfinite(beta) || (!C && beta != 0.f)) return HIMUON_ERR_INVALID;
  int rc = check_operand(*A, 0);
  if (!rc) rc = check_operand(*B, 0);
  if (!rc) rc = check_list(G, n);
  if (!rc && C) rc = check_list(C, n);
  if (rc) return rc;
  if (!is16(A->dtype) || !is_float(G->dtype) || (C && !is_float(C->dtype))) return HIMUON_ERR_UNSUPPORTED;
  if (B->dtype != A->dtype || B->rows != A->rows || G->rows != A->cols || G->cols != B->cols) return HIMUON_ERR_INVALID;
  if (C && (C->rows != G->rows || C->cols != G->cols)) return HIMUON_ERR_INVALID;
  std::vector<const void *> seen(n);
  for (int32_t e = 0; e < n; ++e) {
    seen[e] = G[e].data;
    if (C && beta != 0.f && C[e].data == G[e].data && (C->ld != G->ld || C->dtype != G->dtype)) return HIMUON_ERR_INVALID;
  }
  std::sort(seen.begin(), seen.end());
  if (std::adjacent_find(seen.begin(), seen.end()) != seen.end()) return HIMUON_ERR_INVALID;
  rc = device_usable();
  if (rc) return rc;
  for (int32_t e0 = 0; e0 < n; e0 += kMaxList) {
    GradientArgs a;
    a.n = std::min(n - e0, kMaxList);
    a.A = A->data;
    a.B = B->data;
    a.rows = A->rows;
    a.lda = A->ld;
    a.ldb = B->ld;
    a.offsets = offsets ? offsets + e0 : nullptr;
    a.dtype = A->dtype;
    a.alpha = alpha;
    a.beta = beta;
    a.has_c = beta != 0.f;
    for (int32_t e = 0; e < a.n; ++e) {
      a.G.p[e] = G[e0 + e].data;
      a.C.p[e] = a.has_c ? C[e0 + e].data : nullptr;
    }
    a.ldc = a.has_c ? C->ld : 0;
    a.cdtype = a.has_c ? C->dtype : 0;
    a.ldg = G->ld;
    a.gdtype = G->dtype;
    a.P = A->cols;
    a.Q = B->cols;
    a.status = device_status_word();
    const dim3 grid(static_cast<unsigned>((a.Q + 15) / 16),
                    static_cast<unsigned>(std::min<int64_t>((a.P + 15) / 16, 64)), static_cast<unsigned>(a.n));
    count_launch();
    gradient_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
    if (cudaGetLastError() != cudaSuccess) return HIMUON_ERR_CUDA;
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
  const int rc = device_usable();
  if (rc) return rc;
  for (int32_t e0 = 0; e0 < n; e0 += kMaxList) {
    const int32_t cnt = std::min(n - e0, kMaxList);
    QuantArgs a;
    a.dim = dim;
    int64_t most = 0;
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
    }
    if (most == 0) continue;
    const dim3 grid(static_cast<unsigned>((most + 7) / 8), static_cast<unsigned>(cnt));
    count_launch();
    quantize_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
    if (cudaGetLastError() != cudaSuccess) return HIMUON_ERR_CUDA;
  }
  return HIMUON_OK;
}

}  // extern "C"
