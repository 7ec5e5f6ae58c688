// Root-mean-square norm of rows with the residual's addition, and its gradient.
//
//   s = x + residual,  rstd = 1 / sqrt(mean_j s_j^2 + eps),  y_j = s_j rstd w_j
//   h = g w,  n = s rstd:  g_x = g_s + rstd (h - n mean_j(h_j n_j)),  g_w = sum over rows of g n
//
// A row is one pass: its elements stay in registers between the sum of squares and the output, so
// every input is read once and every output written once; the kernels are bound by HBM (or, for few
// rows, by latency).  G threads (a multiple of 32) share a row, each holding SL vectors of V
// elements; short rows share a block of 256 threads.  Sums are FP32: a thread's elements in order,
// the warp by an xor tree, the warps in order.
//
// y in 8 bits: scale = max_j |y_j| / 448 per row, q = RN_e4m3(y / scale).  max |y| = rstd max |s w|
// (rstd is one positive factor of the row), so the maximum is taken together with the sum of squares
// and the row still needs one block-wide reduction.  The maximum is taken on the bits of |s w| as
// unsigned integers, where a NaN is larger than every number, so a row with a NaN comes out as NaN.
#pragma once
#include "rows.cuh"

namespace emp {
namespace norm {

constexpr int MAX_COLS = EMP_NORM_MAX_COLS;
constexpr int MAX_THREADS = 512;                  // G at the most columns: 8192 / (16 elements a thread)
constexpr float TINY = 7.7037197775489434e-34f;   // 2^-110: below it a row's scale is 1 and 1 / scale stays finite

struct Args {
  long long rows;
  int cols, degrees;
  float eps;
  const void *x, *residual, *w;
  void *y, *s;
  float* scale;
  long long ldx, ldr, ldy, lds;
};
struct GradArgs {
  long long rows;
  int cols, degrees;
  float eps;
  const void *g, *s, *g_s, *w;
  void* g_x;
  float* part;                 // [gridDim.x][weights] sums of g n (null: no weight gradient)
  long long ldg, lds, ldgs, ldgx;
};

__device__ __forceinline__ int weight_at(int col, int C, int degrees) {
  if (!degrees) return col;
  const int lm = col / C;
  return degree_of(lm) * C + (col - lm * C);
}

// sum of a and maximum (as unsigned) of b over the G threads of a row; red: 32 float2-sized slots per row
__device__ __forceinline__ void row_reduce(float& a, uint32_t& b, int G, int t, float* red_a, uint32_t* red_b) {
#pragma unroll
  for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  b = __reduce_max_sync(0xffffffffu, b);
  if (G > 32) {
    const int nw = G >> 5, w = t >> 5;
    if ((t & 31) == 0) { red_a[w] = a; red_b[w] = b; }
    __syncthreads();
    a = 0.f;
    for (int i = 0; i < nw; ++i) { a += red_a[i]; b = max(b, red_b[i]); }
  }
}

template <typename T, int V, int SL, bool QUANT>
__global__ void __launch_bounds__(MAX_THREADS) k_rms_norm(const Args p) {
  __shared__ float red_a[32];
  __shared__ uint32_t red_b[32];
  const int G = blockDim.x, t = threadIdx.x, r = threadIdx.y;
  const long long row = (long long)blockIdx.x * blockDim.y + r;
  const bool live = row < p.rows;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* res = p.residual ? static_cast<const T*>(p.residual) + row * p.ldr : nullptr;
  const T* w = static_cast<const T*>(p.w);
  const int C = p.cols / NCOMP;
  float v[SL][V], wv[SL][V];
  float ss = 0.f;
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < SL; ++k) {
    const int c = (k * G + t) * V;
    const bool in = live && c < p.cols;
#pragma unroll
    for (int i = 0; i < V; ++i) v[k][i] = 0.f;
    if (in) load_v<T, V>(x + c, v[k]);
  }
  if (res) {
#pragma unroll
    for (int k = 0; k < SL; ++k) {
      const int c = (k * G + t) * V;
      if (live && c < p.cols) {
        float a[V];
        load_v<T, V>(res + c, a);
#pragma unroll
        for (int i = 0; i < V; ++i) v[k][i] += a[i];
      }
    }
  }
#pragma unroll
  for (int k = 0; k < SL; ++k) {
    const int c = (k * G + t) * V;
#pragma unroll
    for (int i = 0; i < V; ++i) wv[k][i] = 1.f;
    if (w && c < p.cols) load_v<T, V>(w + weight_at(c, C, p.degrees), wv[k]);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      ss += v[k][i] * v[k][i];
      if (QUANT) top = max(top, __float_as_uint(v[k][i] * wv[k][i]) & 0x7fffffffu);
    }
  }
  const int slot = r * (G >> 5);
  row_reduce(ss, top, G, t, red_a + slot, red_b + slot);
  if (!live) return;
  const float rstd = rsqrtf(ss / (float)p.cols + p.eps);
  float inv = 1.f;
  if (QUANT) {
    const float m = __uint_as_float(top) * rstd;
    const float scale = m < TINY ? 1.f : m / 448.f;     // a NaN stays one
    inv = 1.f / scale;
    if (t == 0) p.scale[row] = scale;
  }
#pragma unroll
  for (int k = 0; k < SL; ++k) {
    const int c = (k * G + t) * V;
    if (c >= p.cols) continue;
    if (p.s) store_v<T, V>(static_cast<T*>(p.s) + row * p.lds + c, v[k]);
    float y[V];
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = v[k][i] * rstd * wv[k][i];
    if (QUANT) {
#pragma unroll
      for (int i = 0; i < V; ++i) y[i] *= inv;
      store_e4m3<V>(static_cast<__nv_fp8_storage_t*>(p.y) + row * p.ldy + c, y);
    } else {
      store_v<T, V>(static_cast<T*>(p.y) + row * p.ldy + c, y);
    }
  }
}

// Persistent: block b takes row groups b, b + gridDim.x, ...; a thread's columns are the same in
// every row, so its part of g_w stays in registers until the end.
template <typename T, int V, int SL>
__global__ void __launch_bounds__(MAX_THREADS) k_rms_norm_grad(const GradArgs p) {
  extern __shared__ float acc_sm[];              // [cols] when the block has several rows or there are degrees
  __shared__ float red[2][2][32];
  const int G = blockDim.x, t = threadIdx.x, r = threadIdx.y, R = blockDim.y;
  const int C = p.cols / NCOMP;
  const T* w = static_cast<const T*>(p.w);
  float acc[SL][V];
#pragma unroll
  for (int k = 0; k < SL; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) acc[k][i] = 0.f;
  const long long groups = (p.rows + R - 1) / R;
  int par = 0;
  for (long long b = blockIdx.x; b < groups; b += gridDim.x, par ^= 1) {
    const long long row = b * R + r;
    const bool live = row < p.rows;
    float g[SL][V], s[SL][V];
    float ss = 0.f, hs = 0.f;
#pragma unroll
    for (int k = 0; k < SL; ++k) {
      const int c = (k * G + t) * V;
#pragma unroll
      for (int i = 0; i < V; ++i) g[k][i] = s[k][i] = 0.f;
      if (live && c < p.cols) {
        load_v<T, V>(static_cast<const T*>(p.g) + row * p.ldg + c, g[k]);
        load_v<T, V>(static_cast<const T*>(p.s) + row * p.lds + c, s[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < SL; ++k) {
      const int c = (k * G + t) * V;
      float wv[V];
#pragma unroll
      for (int i = 0; i < V; ++i) wv[i] = 1.f;
      if (w && c < p.cols) load_v<T, V>(w + weight_at(c, C, p.degrees), wv);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        ss += s[k][i] * s[k][i];
        hs += g[k][i] * wv[i] * s[k][i];
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      hs += __shfl_xor_sync(0xffffffffu, hs, o);
    }
    if (G > 32) {
      // two sets of slots in turn: one barrier per row keeps a set's readers and its next writers apart
      const int nw = G >> 5, w0 = r * nw;
      if ((t & 31) == 0) { red[par][0][w0 + (t >> 5)] = ss; red[par][1][w0 + (t >> 5)] = hs; }
      __syncthreads();
      ss = hs = 0.f;
      for (int i = 0; i < nw; ++i) { ss += red[par][0][w0 + i]; hs += red[par][1][w0 + i]; }
    }
    if (!live) continue;
    const float rstd = rsqrtf(ss / (float)p.cols + p.eps);
    const float q = hs * rstd * rstd / (float)p.cols;      // mean(h n) rstd: n mean(h n) = s q
#pragma unroll
    for (int k = 0; k < SL; ++k) {
      const int c = (k * G + t) * V;
      if (c >= p.cols) continue;
      float wv[V], o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) { wv[i] = 1.f; o[i] = 0.f; }
      if (w) load_v<T, V>(w + weight_at(c, C, p.degrees), wv);
      if (p.g_s) load_v<T, V>(static_cast<const T*>(p.g_s) + row * p.ldgs + c, o);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        o[i] += rstd * (g[k][i] * wv[i] - s[k][i] * q);
        acc[k][i] += g[k][i] * (s[k][i] * rstd);
      }
      store_v<T, V>(static_cast<T*>(p.g_x) + row * p.ldgx + c, o);
    }
  }
  if (!p.part) return;
  const int nout = p.degrees ? 4 * C : p.cols;
  float* part = p.part + (size_t)blockIdx.x * nout;
  const bool direct = R == 1 && !p.degrees;
  // the block's row groups, added in order
  for (int q = 0; q < R; ++q) {
    if (q) __syncthreads();
    if (r != q) continue;
#pragma unroll
    for (int k = 0; k < SL; ++k) {
      const int c = (k * G + t) * V;
      if (c >= p.cols) continue;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (direct) part[c + i] = acc[k][i];
        else acc_sm[c + i] = q ? acc_sm[c + i] + acc[k][i] : acc[k][i];
      }
    }
  }
  if (direct) return;
  __syncthreads();
  for (int o = r * G + t; o < nout; o += G * R) {
    if (!p.degrees) {
      part[o] = acc_sm[o];
    } else {                                     // the 2 l + 1 components of degree l
      const int l = o / C, c = o - l * C;
      float a = 0.f;
      for (int q = l * l; q < (l + 1) * (l + 1); ++q) a += acc_sm[q * C + c];
      part[o] = a;
    }
  }
}

// Launch shape: a row's V-element vectors fill a warp first, then each thread takes up to `most` of
// them, then the row gets more warps; short rows share a block of up to 256 threads, fewer when there
// are not enough rows for two blocks on every SM.
struct Shape {
  int V, SL, G, R;
};
inline Shape shape_for(int cols, int V, int most, long long rows) {
  Shape s;
  s.V = V;
  const int n = (cols + V - 1) / V;
  s.SL = 1;
  while (s.SL < most && n > 32 * s.SL) s.SL *= 2;
  if (s.SL == 8) s.SL = 16;                          // the element-wise form has 1, 2, 4 or 16
  s.G = (n + 32 * s.SL - 1) / (32 * s.SL) * 32;
  s.R = (int)std::max<long long>(1, std::min<long long>(256 / s.G, rows / 296));
  return s;
}

// 16-byte vectors need every pointer and row pitch in use to allow them
inline bool vec_ok(const void* p, long long ld, int es) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * es % 16 == 0);
}

template <typename T, int V, int SL>
void launch_fwd2(const Args& a, const Shape& h, bool quant, cudaStream_t st) {
  const dim3 block(h.G, h.R);
  const unsigned grid = (unsigned)((a.rows + h.R - 1) / h.R);
  if (quant) k_rms_norm<T, V, SL, true><<<grid, block, 0, st>>>(a);
  else k_rms_norm<T, V, SL, false><<<grid, block, 0, st>>>(a);
}
template <typename T>
void launch_fwd(const Args& a, bool quant, cudaStream_t st) {
  constexpr int ES = sizeof(T), V = 16 / ES;
  const bool yv = quant ? reinterpret_cast<uintptr_t>(a.y) % V == 0 && a.ldy % V == 0 : vec_ok(a.y, a.ldy, ES);
  const bool vec = a.cols % V == 0 && yv && vec_ok(a.x, a.ldx, ES) && vec_ok(a.residual, a.ldr, ES) &&
                   vec_ok(a.s, a.lds, ES) && vec_ok(a.w, 0, ES) && (!a.degrees || a.cols / NCOMP % V == 0);
  const Shape h = shape_for(a.cols, vec ? V : 1, vec ? 16 / V : 16, a.rows);
  if (vec) {
    if (h.SL == 1) launch_fwd2<T, V, 1>(a, h, quant, st);
    else if (h.SL == 2) launch_fwd2<T, V, 2>(a, h, quant, st);
    else launch_fwd2<T, V, 16 / V>(a, h, quant, st);
  } else {
    if (h.SL == 1) launch_fwd2<T, 1, 1>(a, h, quant, st);
    else if (h.SL == 2) launch_fwd2<T, 1, 2>(a, h, quant, st);
    else if (h.SL == 4) launch_fwd2<T, 1, 4>(a, h, quant, st);
    else launch_fwd2<T, 1, 16>(a, h, quant, st);
  }
}

// blocks of the gradient (each leaves one row of column sums): up to four per SM
inline int grad_blocks(long long rows, int R) { return (int)std::min<long long>((rows + R - 1) / R, 4 * 148); }

template <typename T, int V, int SL>
void launch_grad2(const GradArgs& a, const Shape& h, cudaStream_t st) {
  k_rms_norm_grad<T, V, SL><<<grad_blocks(a.rows, h.R), dim3(h.G, h.R), h.R > 1 || a.degrees ? a.cols * 4 : 0, st>>>(a);
}
template <typename T>
Shape grad_shape(const GradArgs& a) {
  constexpr int ES = sizeof(T), V = 16 / ES;
  const bool vec = a.cols % V == 0 && vec_ok(a.g, a.ldg, ES) && vec_ok(a.s, a.lds, ES) && vec_ok(a.g_s, a.ldgs, ES) &&
                   vec_ok(a.g_x, a.ldgx, ES) && vec_ok(a.w, 0, ES) && (!a.degrees || a.cols / NCOMP % V == 0);
  return shape_for(a.cols, vec ? V : 1, vec ? 16 / V : 16, a.rows);
}
template <typename T>
int launch_grad(const GradArgs& a, cudaStream_t st) {          // returns the rows of a.part
  constexpr int V = 16 / sizeof(T);
  const Shape h = grad_shape<T>(a);
  if (h.V == V) {
    if (h.SL == 1) launch_grad2<T, V, 1>(a, h, st);
    else if (h.SL == 2) launch_grad2<T, V, 2>(a, h, st);
    else launch_grad2<T, V, 16 / V>(a, h, st);
  } else {
    if (h.SL == 1) launch_grad2<T, 1, 1>(a, h, st);
    else if (h.SL == 2) launch_grad2<T, 1, 2>(a, h, st);
    else if (h.SL == 4) launch_grad2<T, 1, 4>(a, h, st);
    else launch_grad2<T, 1, 16>(a, h, st);
  }
  return grad_blocks(a.rows, h.R);
}

}  // namespace norm
}  // namespace emp
