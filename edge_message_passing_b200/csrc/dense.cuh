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

// ------------------------------------------------------------------ few rows
// Up to FEW_ROWS rows: the product reads W once and little else, so it runs on SIMT with a warp on
// FEW_COLS columns of the output and up to 8 rows at a time (x in shared memory as floats, K_PART of k at
// once; a lane takes V elements of k, 32 V apart), in FP32 throughout.
constexpr int FEW_ROWS = 16, FEW_COLS = 2, FEW_WARPS = 4, FEW_M = 8, K_PART = 1024;

struct Few {
  int M, N, K;
  const void *x, *w;
  long long ldx, ldw;
};

template <typename T, int V>
__global__ void __launch_bounds__(32 * FEW_WARPS) k_dense_few(const Few p, const Epi e) {
  __shared__ __align__(16) float xs[FEW_M][K_PART];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = (blockIdx.x * FEW_WARPS + warp) * FEW_COLS, m0 = blockIdx.y * FEW_M;
  float acc[FEW_COLS][FEW_M] = {};
  for (int k0 = 0; k0 < p.K; k0 += K_PART) {
    const int kn = min(K_PART, p.K - k0);
    if (k0) __syncthreads();
    for (int i = threadIdx.x * V; i < FEW_M * K_PART; i += 32 * FEW_WARPS * V) {
      const int r = i / K_PART, k = i % K_PART;
      float v[V];
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = 0.f;
      if (m0 + r < p.M && k < kn) load_v<T, V>(static_cast<const T*>(p.x) + (m0 + r) * p.ldx + k0 + k, v);
#pragma unroll
      for (int j = 0; j < V; ++j) xs[r][k + j] = v[j];
    }
    __syncthreads();
    for (int k = lane * V; k < kn; k += 32 * V) {
      float w[FEW_COLS][V];
#pragma unroll
      for (int c = 0; c < FEW_COLS; ++c) {
#pragma unroll
        for (int j = 0; j < V; ++j) w[c][j] = 0.f;
        if (n0 + c < p.N) load_v<T, V>(static_cast<const T*>(p.w) + (n0 + c) * p.ldw + k0 + k, w[c]);
      }
#pragma unroll
      for (int r = 0; r < FEW_M; ++r)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float x = xs[r][k + j];
#pragma unroll
          for (int c = 0; c < FEW_COLS; ++c) acc[c][r] += w[c][j] * x;
        }
    }
  }
  float mine = 0.f;                       // lane c FEW_M + r keeps output (r, c)
#pragma unroll
  for (int c = 0; c < FEW_COLS; ++c)
#pragma unroll
    for (int r = 0; r < FEW_M; ++r) {
      float a = acc[c][r];
#pragma unroll
      for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
      if (lane == c * FEW_M + r) mine = a;
    }
  const int m = m0 + lane % FEW_M, n = n0 + lane / FEW_M;
  if (lane < FEW_COLS * FEW_M && m < p.M && n < p.N) put_one(e, m, n, mine);
}

// ------------------------------------------------------------------ operands TMA cannot read
// Rows whose start or pitch is not a multiple of 16 bytes are copied once to rows that are.
template <typename B>
__global__ void k_pack(long long rows, int cols, const B* __restrict__ src, long long ld, B* __restrict__ dst, long long ldd) {
  const long long total = rows * cols;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (long long)gridDim.x * blockDim.x) {
    const long long r = i / cols;
    const int c = (int)(i - r * cols);
    dst[r * ldd + c] = src[r * ld + c];
  }
}

// ------------------------------------------------------------------ join of the k splits, in order
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
