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

struct EpiIn {                 // what the epilogue of one output reads
  float scale, bias, residual;
};
__device__ __forceinline__ EpiIn epi_in(const Epi& e, long long m, int n) {
  EpiIn i;
  i.scale = e.x_scale ? e.x_scale[m] * e.w_scale[n] : 1.f;
  i.bias = e.bias ? load_any(e.bias, n, e.bias_dtype) : 0.f;
  i.residual = e.residual ? load_any(e.residual, (size_t)m * e.ldr + n, e.y_dtype) : 0.f;
  return i;
}
__device__ __forceinline__ void put_one(const Epi& e, long long m, int n, float acc, const EpiIn& in) {
  float v = acc * in.scale + in.bias;
  if (e.z) store_any(e.z, (size_t)m * e.ldz + n, e.y_dtype, v);
  store_any(e.y, (size_t)m * e.ldy + n, e.y_dtype, act_f(e.act, v) + in.residual);
}
__device__ __forceinline__ void put_one(const Epi& e, long long m, int n, float acc) { put_one(e, m, n, acc, epi_in(e, m, n)); }

// ------------------------------------------------------------------ few rows
// Up to 16 rows of a short k and a small W: the product reads W once per 8 rows and little else, so it runs on SIMT with
// a warp on FEW_COLS columns of the output and up to 8 rows at a time (x in shared memory as floats, K_PART of
// k at once; a lane takes V elements of k, 32 V apart, and where V is 1 eight of those at a time, for as many loads in flight), in FP32 throughout.  Against the tensor-core kernel, whose
// set-up costs more: 8 rows, 256 -> 1024, FP32: 9.2 and 15.1 us; 2048 -> 2048: 14.9 and 24.4 (bf16 15.1 and 17.1); beyond,
// W's reads and a warp's long k lose: 16 rows, 2048 -> 2048 bf16 20.9 and 17.0, 8 rows, 8192 -> 128 51.7 and 17.4.
constexpr int FEW_COLS = 2, FEW_WARPS = 4, FEW_M = 8, K_PART = 1024;
inline bool few_rows(long long rows, long long N, long long K) {
  return rows <= 2 * FEW_M && K <= 2048 && (rows + FEW_M - 1) / FEW_M * N * K <= (1 << 22);
}

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
  // lane c FEW_M + r finishes output (r, c); what its epilogue reads, and the first of W, is on its way before x is staged
  const int m = m0 + lane % FEW_M, n = n0 + lane / FEW_M;
  const bool mine = lane < FEW_COLS * FEW_M && m < p.M && n < p.N;
  EpiIn in{};
  if (mine) in = epi_in(e, m, n);
  constexpr int B = V == 1 ? 8 : 1, STEP = 32 * V * B;            // B groups of V elements, 32 V apart
  Raw<T, 1> wu[FEW_COLS][B];                                      // V = 1
  float w[FEW_COLS][B][V];
  auto load_w = [&](int k) {
#pragma unroll
    for (int c = 0; c < FEW_COLS; ++c)
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const T* at = static_cast<const T*>(p.w) + (n0 + c) * p.ldw + k + 32 * V * b;
        const bool in = n0 + c < p.N && k + 32 * V * b < p.K;
        if constexpr (V == 1) {
          wu[c][b].load(at, in);
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) w[c][b][j] = 0.f;
          if (in) load_v<T, V>(at, w[c][b]);
        }
      }
  };
  load_w(lane * V);
  float acc[FEW_COLS][FEW_M] = {};
  for (int k0 = 0; k0 < p.K; k0 += K_PART) {
    const int kn = min(K_PART, p.K - k0), kz = (kn + STEP - 1) / STEP * STEP;     // V divides K (or is 1)
    if (k0) __syncthreads();
    for (int r = warp; r < FEW_M; r += FEW_WARPS) {
      const T* x = static_cast<const T*>(p.x) + (m0 + r) * p.ldx + k0;
      if constexpr (V == 1) {
        for (int k1 = lane; k1 < kz; k1 += STEP) {                // zeros behind the last of k
          Raw<T, 1> u[B];
#pragma unroll
          for (int b = 0; b < B; ++b) u[b].load(x + k1 + 32 * b, m0 + r < p.M && k1 + 32 * b < kn);
#pragma unroll
          for (int b = 0; b < B; ++b) xs[r][k1 + 32 * b] = u[b].one(T());
        }
      } else {
#pragma unroll 8
        for (int k = lane * V; k < kn; k += 32 * V) {
          float v[V];
#pragma unroll
          for (int j = 0; j < V; ++j) v[j] = 0.f;
          if (m0 + r < p.M) load_v<T, V>(x + k, v);
#pragma unroll
          for (int j = 0; j < V; ++j) xs[r][k + j] = v[j];
        }
      }
    }
    __syncthreads();
    for (int k = lane * V; k < kn; k += STEP) {
      if constexpr (V == 1) {
#pragma unroll
        for (int c = 0; c < FEW_COLS; ++c)
#pragma unroll
          for (int b = 0; b < B; ++b) w[c][b][0] = wu[c][b].one(T());
      }
#pragma unroll
      for (int r = 0; r < FEW_M; ++r)
#pragma unroll
        for (int b = 0; b < B; ++b)
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float x = xs[r][k + 32 * V * b + j];
#pragma unroll
            for (int c = 0; c < FEW_COLS; ++c) acc[c][r] += w[c][b][j] * x;
          }
      load_w(k0 + k + STEP < k0 + kn ? k0 + k + STEP : k0 + K_PART + lane * V);           // the next of this part, or of the next part
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int c = 0; c < FEW_COLS; ++c)
#pragma unroll
    for (int r = 0; r < FEW_M; ++r) {
      float a = acc[c][r];
#pragma unroll
      for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
      if (lane == c * FEW_M + r) sum = a;
    }
  if (mine) put_one(e, m, n, sum, in);
}

// ------------------------------------------------------------------ operands TMA cannot read
// Rows whose start or pitch is not a multiple of 16 bytes are copied once to rows that are.  A thread
// writes 16 bytes, put together by funnel shifts from the (up to five) aligned words that hold them; words
// past the row's last byte are not read (of the first and the last word, the bytes beside the row are, and dropped).
// x: 16-byte chunks of a row, y: rows.  Bound by the latency of its one wave: 20011 x 515 bf16 takes 13 us, 3.2 TB/s.
struct Pack {                  // up to two matrices (blockIdx.z)
  int n = 0;
  long long rows[2], pitch[2], pitch_d[2];
  int row_bytes[2];
  const unsigned char* src[2];
  unsigned char* dst[2];
};
constexpr int PACK_ROWS = 4;   // rows of a thread whose loads are in flight together
__global__ void __launch_bounds__(256) k_pack(const Pack p) {
  // (chosen by value: an index into the parameters would put them into local memory)
  const bool second = blockIdx.z != 0;
  const long long rows = second ? p.rows[1] : p.rows[0], pitch = second ? p.pitch[1] : p.pitch[0];
  const long long pitch_d = second ? p.pitch_d[1] : p.pitch_d[0];
  const int row_bytes = second ? p.row_bytes[1] : p.row_bytes[0], at = (blockIdx.x * blockDim.x + threadIdx.x) * 16;
  const unsigned char* __restrict__ src = second ? p.src[1] : p.src[0];
  unsigned char* __restrict__ dst = second ? p.dst[1] : p.dst[0];
  if (at >= row_bytes) return;
  const long long step = (long long)gridDim.y * blockDim.y;
  for (long long r0 = (long long)blockIdx.y * blockDim.y + threadIdx.y; r0 < rows; r0 += PACK_ROWS * step) {
    uint32_t v[PACK_ROWS][5];
    unsigned off[PACK_ROWS];
#pragma unroll
    for (int k = 0; k < PACK_ROWS; ++k) {
      const long long r = r0 + k * step;
      const unsigned char* s = src + r * pitch + at;
      const unsigned char* end = src + r * pitch + row_bytes;
      off[k] = (unsigned)(reinterpret_cast<uintptr_t>(s) & 3);
      const uint32_t* w = reinterpret_cast<const uint32_t*>(s - off[k]);
#pragma unroll
      for (int i = 0; i < 5; ++i) v[k][i] = r < rows && reinterpret_cast<const unsigned char*>(w + i) < end ? w[i] : 0u;
    }
#pragma unroll
    for (int k = 0; k < PACK_ROWS; ++k) {
      const long long r = r0 + k * step;
      if (r >= rows) break;
      uint4 o;
      o.x = __funnelshift_r(v[k][0], v[k][1], off[k] * 8);
      o.y = __funnelshift_r(v[k][1], v[k][2], off[k] * 8);
      o.z = __funnelshift_r(v[k][2], v[k][3], off[k] * 8);
      o.w = __funnelshift_r(v[k][3], v[k][4], off[k] * 8);
      *reinterpret_cast<uint4*>(dst + r * pitch_d + at) = o;
    }
  }
}

// ------------------------------------------------------------------ join of the k splits, in order
// V consecutive elements a thread (4 where N allows), JOIN_Z splits' loads in flight together.  Bound by the latency of
// those loads: 37 splits of 512 x 128 take 8 us.
constexpr int JOIN_Z = 8;
template <int V>
__global__ void __launch_bounds__(256) k_join(long long M, int N, int splits, const float* __restrict__ part, const Epi e) {
  const size_t total = (size_t)M * N;
  for (size_t i = ((size_t)blockIdx.x * blockDim.x + threadIdx.x) * V; i < total; i += (size_t)gridDim.x * blockDim.x * V) {
    float s[V];
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = 0.f;
    for (int z0 = 0; z0 < splits; z0 += JOIN_Z) {
      float v[JOIN_Z][V];
#pragma unroll
      for (int k = 0; k < JOIN_Z; ++k) {
#pragma unroll
        for (int j = 0; j < V; ++j) v[k][j] = 0.f;
        if (z0 + k < splits) load_v<float, V>(part + (size_t)(z0 + k) * total + i, v[k]);
      }
#pragma unroll
      for (int k = 0; k < JOIN_Z; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] += v[k][j];
    }
    const long long m = (long long)(i / N);
    const int n = (int)(i % N);
#pragma unroll
    for (int j = 0; j < V; ++j) put_one(e, m, n + j, s[j]);
  }
}

// ------------------------------------------------------------------ g act'(z) and the bias gradient
// gz = g act'(z), rounded to the operands' type (it is an operand of both products, which take that
// type), and part[block][n] = the block's column sums of the unrounded values (bias gradient).
// A warp takes 32 V neighbouring columns of every 8 gridDim.x-th row, a few rows' loads at a time.
// Bound by HBM: g and z in, gz out (80896 x 512: FP32 80 us, 6.2 TB/s; bf16 43 us, 5.8 TB/s), at widths off 16 bytes by the
// instructions of its narrow loads (80896 x 515: FP32 90 us, bf16 104 us; 514 in bf16, by words, 59).
// Four blocks per SM, and as many rows in flight as their registers hold: two of 16-byte vectors (bf16 one 52 us, two 47,
// four 47), four of 32-bit words, eight single floats (four 107 us at 80896 x 515, eight 94) or four single 16-bit
// elements (two 134 us, four 108, eight 122).
constexpr int GZ_WARPS = 8, GZ_PER_SM = 4;
struct GzArgs {
  long long rows;
  int cols, act;
  const void *g, *z;
  long long ldg, ldz, ldo;
  void* gz;                    // null: the bias gradient alone
  float* part;                 // null without a bias gradient ...
  void* g_b;                   // ... which a single block per column writes itself
};
template <typename T, int V>
__global__ void __launch_bounds__(32 * GZ_WARPS, GZ_PER_SM) k_dense_gz(const GzArgs p) {
  constexpr int GZ_BATCH = V >= 4 ? 2 : V == 2 || sizeof(T) == 2 ? 4 : 8;
  __shared__ float sm[GZ_WARPS][32 * V];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = (blockIdx.y * 32 + lane) * V;
  float s[V];
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] = 0.f;
  if (c < p.cols) {
    const int step = gridDim.x * GZ_WARPS, first = blockIdx.x * GZ_WARPS + w;
    const T* g = static_cast<const T*>(p.g) + first * p.ldg + c;
    const T* z = static_cast<const T*>(p.z) + first * p.ldz + c;
    T* o = static_cast<T*>(p.gz) + first * p.ldo + c;
    const long long sg = step * p.ldg, sz = step * p.ldz, so = step * p.ldo;
    // the lane's rows; the pointers go along (a 64-bit product per load would cost as much as the rest)
    for (int left = first < p.rows ? ((int)p.rows - first - 1) / step + 1 : 0; left > 0; left -= GZ_BATCH) {
      Raw<T, V> rg[GZ_BATCH], rz[GZ_BATCH];
#pragma unroll
      for (int k = 0; k < GZ_BATCH; ++k) {
        rg[k].load(g, k < left);
        rz[k].load(z, k < left && p.z);
        g += sg;
        z += sz;
      }
#pragma unroll
      for (int k = 0; k < GZ_BATCH; ++k) {
        if (k >= left) break;
        float a[V], b[V];
        rg[k].get(a);
        rz[k].get(b);
        // a rounded product (no contraction into the sum), so that g_bias has the same bits with and without gz
        if (p.act == EMP_ACT_SILU) {
#pragma unroll
          for (int i = 0; i < V; ++i) a[i] = __fmul_rn(a[i], dact<EMP_ACT_SILU, T>(b[i]));
        } else if (p.act == EMP_ACT_GELU) {
#pragma unroll
          for (int i = 0; i < V; ++i) a[i] = __fmul_rn(a[i], dact<EMP_ACT_GELU, T>(b[i]));
        }
        if (p.gz) store_v<T, V>(o, a);
        o += so;
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] += a[i];
      }
    }
  }
  if (!p.g_b) return;
#pragma unroll
  for (int i = 0; i < V; ++i) sm[w][i * 32 + lane] = s[i];
  __syncthreads();
  for (int j = threadIdx.x; j < 32 * V; j += 32 * GZ_WARPS) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < GZ_WARPS; ++i) t += sm[i][j];
    const int col = (blockIdx.y * 32 + (j & 31)) * V + (j >> 5);
    if (col >= p.cols) continue;
    if (gridDim.x == 1) static_cast<T*>(p.g_b)[col] = from_f<T>(t);
    else p.part[(size_t)blockIdx.x * p.cols + col] = t;
  }
}

}  // namespace dense
}  // namespace emp
