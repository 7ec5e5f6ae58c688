// Dense layer on rows, y = act(x W^T + b) + residual, and its gradient.
#pragma once
#include "rows.cuh"

namespace emp {
namespace dense {

// ------------------------------------------------------------------ the epilogue
// From a product's sum acc at (m, n): z = acc (x_scale_m w_scale_n) + b_n, y = act(z) + residual.
struct Epi {
  int act, y_dtype, bias_dtype;
  const float *x_scale, *w_scale;
  const void *bias, *residual;
  long long ldr;
  void *y, *z;
  long long ldy, ldz;
};

__device__ __forceinline__ void put_one(const Epi& e, long long m, int n, float acc) {
  float v = acc;
  if (e.x_scale) v *= e.x_scale[m] * e.w_scale[n];
  if (e.bias) v += load_any(e.bias, n, e.bias_dtype);
  if (e.z) store_any(e.z, (size_t)m * e.ldz + n, e.y_dtype, v);
  v = act_f(e.act, v);
  if (e.residual) v += load_any(e.residual, (size_t)m * e.ldr + n, e.y_dtype);
  store_any(e.y, (size_t)m * e.ldy + n, e.y_dtype, v);
}

// ------------------------------------------------------------------ a product in FP32 on SIMT
// out[m][n] = sum_k A(m, k) B(n, k), A(m, k) = a[m am + k ak], B(n, k) = b[n bn + k bk]: any strides,
// any type.  64 x 64 tiles, 4 x 4 outputs a thread.  Splits of the k axis (gridDim.z) leave partial
// products in part[z][M][N], joined in order by k_join.
struct Prod {
  long long M, K;
  int N, dtype;
  const void *a, *b;
  long long am, ak, bn, bk;
  float* part;
};
constexpr int T_M = 64, T_K = 16;

__global__ void __launch_bounds__(256) k_dense_simt(const Prod p, const Epi e) {
  __shared__ float as[T_K][T_M + 1], bs[T_K][T_M + 1];
  const long long m0 = (long long)blockIdx.x * T_M;
  const int n0 = blockIdx.y * T_M;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const long long per = ((p.K + gridDim.z - 1) / gridDim.z + T_K - 1) / T_K * T_K;
  const long long k_first = per * blockIdx.z, k_end = k_first + per < p.K ? k_first + per : p.K;
  float acc[4][4] = {};
  for (long long k0 = k_first; k0 < k_end; k0 += T_K) {
    for (int i = threadIdx.x; i < T_K * T_M; i += 256) {
      const int k = p.ak == 1 ? i % T_K : i / T_M, m = p.ak == 1 ? i / T_K : i % T_M;
      as[k][m] = m0 + m < p.M && k0 + k < k_end ? load_any(p.a, (size_t)((m0 + m) * p.am + (k0 + k) * p.ak), p.dtype) : 0.f;
    }
    for (int i = threadIdx.x; i < T_K * T_M; i += 256) {
      const int k = p.bk == 1 ? i % T_K : i / T_M, n = p.bk == 1 ? i / T_K : i % T_M;
      bs[k][n] = n0 + n < p.N && k0 + k < k_end ? load_any(p.b, (size_t)((n0 + n) * p.bn + (k0 + k) * p.bk), p.dtype) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < T_K; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += as[k][ty + 16 * i] * bs[k][tx + 16 * j];
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const long long m = m0 + ty + 16 * i;
      const int n = n0 + tx + 16 * j;
      if (m >= p.M || n >= p.N) continue;
      if (p.part) p.part[((size_t)blockIdx.z * p.M + m) * p.N + n] = acc[i][j];
      else put_one(e, m, n, acc[i][j]);
    }
}

__global__ void k_join(long long M, int N, int splits, const float* __restrict__ part, const Epi e) {
  const size_t total = (size_t)M * N;
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (size_t)gridDim.x * blockDim.x) {
    float s = 0.f;
    for (int z = 0; z < splits; ++z) s += part[(size_t)z * total + i];
    put_one(e, (long long)(i / N), (int)(i % N), s);
  }
}

// ------------------------------------------------------------------ g act'(z) and the bias gradient
// gz = g act'(z), rounded to the operands' type (it is an operand of both products, which take that
// type), and part[block][n] = the block's column sums of the unrounded values (bias gradient).
constexpr int GZ_ROWS = 8;
struct GzArgs {
  long long rows;
  int cols, dtype, act;
  const void *g, *z;
  long long ldg, ldz, ldo;
  void* gz;                    // null without an activation
  float* part;                 // null without a bias gradient
};
__global__ void __launch_bounds__(32 * GZ_ROWS) k_dense_gz(const GzArgs p) {
  __shared__ float sm[GZ_ROWS][33];
  const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int c = blockIdx.y * 32 + lane;
  float s = 0.f;
  if (c < p.cols)
    for (long long m = (long long)blockIdx.x * GZ_ROWS + r; m < p.rows; m += (long long)gridDim.x * GZ_ROWS) {
      float v = load_any(p.g, (size_t)(m * p.ldg + c), p.dtype);
      // a rounded product (no contraction into the sum), so that g_bias has the same bits with and without gz
      if (p.z) v = __fmul_rn(v, dact_f(p.act, load_any(p.z, (size_t)(m * p.ldz + c), p.dtype)));
      if (p.gz) store_any(p.gz, (size_t)(m * p.ldo + c), p.dtype, v);
      s += v;
    }
  if (!p.part) return;
  sm[r][lane] = s;
  __syncthreads();
  if (r == 0 && c < p.cols) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < GZ_ROWS; ++i) t += sm[i][lane];
    p.part[(size_t)blockIdx.x * p.cols + c] = t;
  }
}

}  // namespace dense
}  // namespace emp
