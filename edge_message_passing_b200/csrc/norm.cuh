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
// and the row still needs one block-wide reduction.  The maximum keeps a NaN, so a row with one comes out as NaN.
//
// The squares of a whole row would leave FP32 at |s| of 1.8e19 / sqrt(cols), and 1 / sqrt of infinity would turn the row into
// zeros.  So a thread's sum (of 176 elements at the most) is multiplied by `unit`, a power of two of 1 / cols at most, before it
// is added to the others: |s| up to 1.3e18 then stays in range at any width, and the factor changes no bit.  (On every square
// it would allow 1.8e19 and cost up to 5 %: 80896 x 515 bf16 43 us instead of 41.)
#pragma once
#include <atomic>
#include <type_traits>
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
  float unit, count;           // set by the launch: a power of two of 1 / cols at most, and cols unit
};
struct GradArgs {
  long long rows;
  int cols, degrees;
  float eps;
  const void *g, *s, *g_s, *w;
  void* g_x;
  float* part;                 // [gridDim.x][weights] sums of g n (null: no weight gradient)
  long long ldg, lds, ldgs, ldgx;
  float unit, count;           // as in Args
};

__device__ __forceinline__ int weight_at(int col, int C, int degrees) {
  if (!degrees) return col;
  const int lm = col / C;
  return degree_of(lm) * C + (col - lm * C);
}

// max(a, |b|), a NaN if either is one
__device__ __forceinline__ float max_abs(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(fabsf(b)));
  return m;
}

// sum of a and max_abs of b over the G threads of a row; red_a, red_b: a slot per warp of the row
template <bool MAX>
__device__ __forceinline__ void row_reduce(float& a, float& b, int G, int t, float* red_a, float* red_b) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    if (MAX) b = max_abs(b, __shfl_xor_sync(0xffffffffu, b, o));
  }
  if (G > 32) {
    const int nw = G >> 5, w = t >> 5;
    if ((t & 31) == 0) { red_a[w] = a; red_b[w] = b; }
    __syncthreads();
    a = 0.f;
    for (int i = 0; i < nw; ++i) {
      a += red_a[i];
      if (MAX) b = max_abs(b, red_b[i]);
    }
  }
}

// a column's sums over the 2 l + 1 components of weight o = (l, c)
__device__ __forceinline__ float degree_sum(const float* sums, int o, int C) {
  const int l = o / C, c = o - l * C;
  float a = 0.f;
  for (int q = l * l; q < (l + 1) * (l + 1); ++q) a += sums[q * C + c];
  return a;
}

// Rows of 16-byte vectors.  Bound by HBM (from L2's side: the loads of many small blocks in flight): 4096 x 2048 FP32 with
// a residual 26.5 us, 5.1 TB/s; 16384 x 2048 bf16 with a residual to 8 bits 46 us, 5.1 TB/s.
// (FP32 with 16 elements a thread: 42 registers at most; the compiler would take 50 and 27.2 us.)
template <typename T, int V, int SL, bool QUANT>
__global__ void __launch_bounds__(MAX_THREADS, V == 4 && SL == 4 && !QUANT ? 3 : 0) k_rms_norm(const Args p) {
  __shared__ float red_a[32], red_b[32];
  const int G = blockDim.x, t = threadIdx.x, r = threadIdx.y;
  const long long row = (long long)blockIdx.x * blockDim.y + r;
  const bool live = row < p.rows;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* res = p.residual ? static_cast<const T*>(p.residual) + row * p.ldr : nullptr;
  const T* w = static_cast<const T*>(p.w);
  const int C = p.cols / NCOMP;
  float v[SL][V];
  float ss = 0.f, top = 0.f;
#pragma unroll
  for (int k = 0; k < SL; ++k) {
    const int c = (k * G + t) * V;
#pragma unroll
    for (int i = 0; i < V; ++i) v[k][i] = 0.f;
    if (live && c < p.cols) load_v<T, V>(x + c, v[k]);
  }
  if (res) {
    float a[SL][V];
#pragma unroll
    for (int k = 0; k < SL; ++k) {
      const int c = (k * G + t) * V;
#pragma unroll
      for (int i = 0; i < V; ++i) a[k][i] = 0.f;
      if (live && c < p.cols) load_v<T, V>(res + c, a[k]);
    }
#pragma unroll
    for (int k = 0; k < SL; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] += a[k][i];
  }
  // s needs no reduction: it is written now, and only the products s w are kept
#pragma unroll
  for (int k = 0; k < SL; ++k) {
    const int c = (k * G + t) * V;
    if (p.s && live && c < p.cols) store_v<T, V>(static_cast<T*>(p.s) + row * p.lds + c, v[k]);
#pragma unroll
    for (int i = 0; i < V; ++i) ss += v[k][i] * v[k][i];
    if (w && c < p.cols) {
      float wv[V];
      load_v<T, V>(w + weight_at(c, C, p.degrees), wv);
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] *= wv[i];
    }
    if (QUANT) {
#pragma unroll
      for (int i = 0; i < V; ++i) top = max_abs(top, v[k][i]);
    }
  }
  const int slot = r * (G >> 5);
  ss *= p.unit;
  row_reduce<QUANT>(ss, top, G, t, red_a + slot, red_b + slot);
  if (!live) return;
  const float rstd = rsqrtf(ss / p.count + p.eps);
  float inv = 1.f;
  if (QUANT) {
    const float m = top * rstd;
    const float scale = m < TINY ? 1.f : m / 448.f;     // a NaN stays one
    inv = 1.f / scale;
    if (t == 0) p.scale[row] = scale;
  }
#pragma unroll
  for (int k = 0; k < SL; ++k) {
    const int c = (k * G + t) * V;
    if (c >= p.cols) continue;
    float y[V];
#pragma unroll
    for (int i = 0; i < V; ++i) y[i] = v[k][i] * rstd;
    if (QUANT) {
#pragma unroll
      for (int i = 0; i < V; ++i) y[i] *= inv;
      store_e4m3<V>(static_cast<__nv_fp8_storage_t*>(p.y) + row * p.ldy + c, y);
    } else {
      store_v<T, V>(static_cast<T*>(p.y) + row * p.ldy + c, y);
    }
  }
}

// ------------------------------------------------------------------ contiguous rows off 16-byte boundaries
// Rows whose size is no multiple of 16 bytes but that follow one another without gaps: R of them are
// (R cols sizeof(T) is), so a block moves R rows at once between memory and shared memory in 16-byte
// vectors, and a warp takes whole rows there.  (Element-wise loads from memory instead took 350 us for
// 80896 x 515 in bf16.)
constexpr int ODD_THREADS = 256, ODD_SMEM = 110 * 1024, SM_SMEM = 227 * 1024;   // two blocks per SM at least

// `bytes` from src to dst, one of them in shared memory; both 16-byte aligned
__device__ __forceinline__ void copy_rows(void* dst, const void* src, int bytes) {
  const int n = bytes >> 4;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += ODD_THREADS) reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(src)[i];
  for (int i = (n << 4) + threadIdx.x; i < bytes; i += ODD_THREADS)
    reinterpret_cast<unsigned char*>(dst)[i] = reinterpret_cast<const unsigned char*>(src)[i];
}

// In shared memory a warp reads a row by 32-bit words, two elements each of a 16-bit type: a row that begins inside a
// word leaves out its first element, one that ends inside a word its last, and lane 0 takes that one by itself (for an
// odd number of columns there is exactly one, for an even number none): 80896 x 515 in bf16 took 56 us by elements
// and takes 46, 3.6 TB/s, bound by instructions.  Persistent where shared memory has room for a second buffer, into which the
// next rows are on their way (cp.async) meanwhile: with a residual 82 us without that, 74 (4.5 TB/s) with it.  Rows behind
// the last one are computed from whatever the shared memory holds and not written.
template <typename T> struct Word {                               // fp32: an element is a word
  static constexpr int N = 1;
  static __device__ __forceinline__ void get(uint32_t u, float (&v)[1]) { v[0] = __uint_as_float(u); }
  static __device__ __forceinline__ uint32_t put(const float (&v)[1]) { return __float_as_uint(v[0]); }
};
template <typename T> struct Word16 {
  static constexpr int N = 2;
  static __device__ __forceinline__ void get(uint32_t u, float (&v)[2]) { unpack2<T>(u, v[0], v[1]); }
  static __device__ __forceinline__ uint32_t put(const float (&v)[2]) { return pack2<T>(v[0], v[1]); }
};
template <> struct Word<__nv_bfloat16> : Word16<__nv_bfloat16> {};
template <> struct Word<__half> : Word16<__half> {};

inline __host__ __device__ int round16(int bytes) { return (bytes + 15) & ~15; }

// the same into shared memory without waiting (up to cp.async.wait_all)
__device__ __forceinline__ void copy_rows_async(void* dst, const void* src, int bytes) {
  const int n = bytes >> 4;
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  for (int i = threadIdx.x; i < n; i += ODD_THREADS)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d + i * 16), "l"(reinterpret_cast<const uint4*>(src) + i) : "memory");
  for (int i = (n << 4) + threadIdx.x; i < bytes; i += ODD_THREADS)
    reinterpret_cast<unsigned char*>(dst)[i] = reinterpret_cast<const unsigned char*>(src)[i];
}

template <typename T, bool QUANT, bool RES, int RW>               // RW rows of a warp, side by side
__global__ void __launch_bounds__(ODD_THREADS) k_rms_norm_odd(const Args p, int bufs) {
  extern __shared__ __align__(16) unsigned char odd_sm[];
  using Wd = Word<T>;
  constexpr int WARPS = ODD_THREADS / 32, R = RW * WARPS, N = Wd::N;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, C = p.cols / NCOMP;
  const int area = round16(R * p.cols * (int)sizeof(T)), half = RES ? 2 * area : area;
  float* wf = reinterpret_cast<float*>(odd_sm);                   // the weights, one per column
  unsigned char* cur = odd_sm + round16(4 * p.cols);
  unsigned char* other = cur + (bufs - 1) * half;
  __nv_fp8_storage_t* qs = reinterpret_cast<__nv_fp8_storage_t*>(cur + bufs * half);
  const T* w = static_cast<const T*>(p.w);
  const long long groups = (p.rows + R - 1) / R;
  auto rows_of = [&](long long b) { return (int)min((long long)R, p.rows - b * R); };
  auto fetch = [&](long long b, unsigned char* to) {
    const long long at = b * R * p.cols;
    const int bytes = rows_of(b) * p.cols * (int)sizeof(T);
    copy_rows_async(to, static_cast<const T*>(p.x) + at, bytes);
    if (RES) copy_rows_async(to + area, static_cast<const T*>(p.residual) + at, bytes);
  };
  fetch(blockIdx.x, cur);
  for (int c = threadIdx.x; c < p.cols; c += ODD_THREADS) wf[c] = w ? to_f(w[weight_at(c, C, p.degrees)]) : 1.f;
  const int first = warp * RW, n = p.cols / N;
  const bool loose = N == 2 && (p.cols & 1) && lane == 0;         // this lane takes the row's loose element
  for (long long b = blockIdx.x; b < groups; b += gridDim.x) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();                                                // cur has landed, other's rows have been copied out
    if (b + gridDim.x < groups) fetch(b + gridDim.x, other);        // (with one buffer there is no second turn)
    const long long row0 = b * R;
    const int rows = rows_of(b), bytes = rows * p.cols * (int)sizeof(T);
    T* xs = reinterpret_cast<T*>(cur);
    T* rs = reinterpret_cast<T*>(RES ? cur + area : cur);
    const uint32_t *xw[RW], *rw[RW];                                // the row's first whole word
    int head[RW];                                                   // and its column
#pragma unroll
    for (int j = 0; j < RW; ++j) {
      const int start = (first + j) * p.cols;
      head[j] = N == 2 ? start & 1 : 0;
      xw[j] = reinterpret_cast<const uint32_t*>(xs + start + head[j]);
      rw[j] = reinterpret_cast<const uint32_t*>(rs + start + head[j]);
    }
    float ss[RW], top[RW];
#pragma unroll
    for (int j = 0; j < RW; ++j) {
      ss[j] = top[j] = 0.f;
      if (loose) {
        const int c = head[j] ? 0 : p.cols - 1, i = (first + j) * p.cols + c;
        float v = to_f(xs[i]);
        if (RES) v += to_f(rs[i]);
        ss[j] = v * v;
        if (QUANT) top[j] = max_abs(0.f, v * wf[c]);
      }
    }
#pragma unroll 4
    for (int k = lane; k < n; k += 32) {
#pragma unroll
      for (int j = 0; j < RW; ++j) {
        float v[N], r[N];
        Wd::get(xw[j][k], v);
        if (RES) Wd::get(rw[j][k], r);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          if (RES) v[e] += r[e];
          ss[j] = fmaf(v[e], v[e], ss[j]);
          if (QUANT) top[j] = max_abs(top[j], v[e] * wf[head[j] + k * N + e]);
        }
      }
    }
    float rstd[RW], inv[RW];
#pragma unroll
    for (int j = 0; j < RW; ++j) {
      ss[j] *= p.unit;
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        ss[j] += __shfl_xor_sync(0xffffffffu, ss[j], o);
        if (QUANT) top[j] = max_abs(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
      }
      rstd[j] = rsqrtf(ss[j] / p.count + p.eps);
      inv[j] = 1.f;
      if (QUANT) {
        const float m = top[j] * rstd[j];
        const float scale = m < TINY ? 1.f : m / 448.f;
        inv[j] = 1.f / scale;
        if (lane == 0 && first + j < rows) p.scale[row0 + first + j] = scale;
      }
    }
#pragma unroll 4
    for (int k = lane; k < n; k += 32) {
#pragma unroll
      for (int j = 0; j < RW; ++j) {
        float v[N], r[N];
        Wd::get(xw[j][k], v);
        if (RES) {
          Wd::get(rw[j][k], r);
#pragma unroll
          for (int e = 0; e < N; ++e) v[e] += r[e];
          const_cast<uint32_t*>(rw[j])[k] = Wd::put(v);             // s
        }
#pragma unroll
        for (int e = 0; e < N; ++e) {
          v[e] = v[e] * rstd[j] * wf[head[j] + k * N + e];
          if (QUANT) v[e] *= inv[j];
        }
        if (!QUANT) const_cast<uint32_t*>(xw[j])[k] = Wd::put(v);
        else
#pragma unroll
          for (int e = 0; e < N; ++e) store_e4m3<1>(qs + (first + j) * p.cols + head[j] + k * N + e, {v[e]});
      }
    }
#pragma unroll
    for (int j = 0; j < RW; ++j) {
      if (!loose) continue;
      const int c = head[j] ? 0 : p.cols - 1, i = (first + j) * p.cols + c;
      float v = to_f(xs[i]);
      if (RES) {
        v += to_f(rs[i]);
        rs[i] = from_f<T>(v);
      }
      v = v * rstd[j] * wf[c];
      if (QUANT) store_e4m3<1>(qs + i, {v * inv[j]});
      else xs[i] = from_f<T>(v);
    }
    __syncthreads();
    if (QUANT) copy_rows(static_cast<__nv_fp8_storage_t*>(p.y) + row0 * p.cols, qs, rows * p.cols);
    else copy_rows(static_cast<T*>(p.y) + row0 * p.cols, xs, bytes);
    if (RES && p.s) copy_rows(static_cast<T*>(p.s) + row0 * p.cols, rs, bytes);
    unsigned char* t = cur;
    cur = other;
    other = t;
  }
}

// The gradient of the same rows: persistent, a row per warp at a time, read by words in the same way.  Whether a row begins
// inside a word depends on the warp alone, so a lane's columns are the same in every row of its, and its part of g_w
// stays in registers (NS words, and the loose column of lane 0).  The next rows are on their way (cp.async) into the
// other half of the shared memory meanwhile: 80896 x 515 in bf16 104 us, 2.4 TB/s, bound by instructions (198 by elements and
// without it).
constexpr int ODD_GRAD_COLS = 1024;
template <typename T, int NS>
__global__ void __launch_bounds__(ODD_THREADS) k_rms_norm_grad_odd(const GradArgs p) {
  extern __shared__ __align__(16) unsigned char odd_sm[];
  using Wd = Word<T>;
  constexpr int R = ODD_THREADS / 32, N = Wd::N;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, C = p.cols / NCOMP;
  const int area = R * p.cols * (int)sizeof(T);                   // a multiple of 16: R = 8
  const int half = area * (p.g_s ? 3 : 2);                        // g, s and g_s of R rows
  const T* w = static_cast<const T*>(p.w);
  const int start = warp * p.cols, head = N == 2 ? start & 1 : 0, n = p.cols / N;
  const bool loose = N == 2 && (p.cols & 1) && lane == 0;
  const int lc = head ? 0 : p.cols - 1;                           // the loose column
  auto weight = [&](int c) { return w ? to_f(w[weight_at(c, C, p.degrees)]) : 1.f; };
  float acc[NS][N], wv[NS][N], accl = 0.f, wl = loose ? weight(lc) : 0.f;
#pragma unroll
  for (int k = 0; k < NS; ++k)
#pragma unroll
    for (int e = 0; e < N; ++e) {
      acc[k][e] = 0.f;
      wv[k][e] = lane + 32 * k < n ? weight(head + (lane + 32 * k) * N + e) : 0.f;
    }
  const long long groups = (p.rows + R - 1) / R;
  auto rows_of = [&](long long b) { return (int)min((long long)R, p.rows - b * R); };
  auto fetch = [&](long long b, unsigned char* to) {
    const long long at = b * R * p.cols;
    const int bytes = rows_of(b) * p.cols * (int)sizeof(T);
    copy_rows_async(to, static_cast<const T*>(p.g) + at, bytes);
    copy_rows_async(to + area, static_cast<const T*>(p.s) + at, bytes);
    if (p.g_s) copy_rows_async(to + 2 * area, static_cast<const T*>(p.g_s) + at, bytes);
  };
  unsigned char* cur = odd_sm;
  unsigned char* other = odd_sm + half;
  if (blockIdx.x < groups) fetch(blockIdx.x, cur);
  for (long long b = blockIdx.x; b < groups; b += gridDim.x) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();                                              // cur has landed, other's rows have been copied out
    if (b + gridDim.x < groups) fetch(b + gridDim.x, other);
    const int rows = rows_of(b);
    T* gs = reinterpret_cast<T*>(cur);
    const T* ss_ = reinterpret_cast<const T*>(cur + area);
    const T* ts = reinterpret_cast<const T*>(cur + 2 * area);
    uint32_t* gw = reinterpret_cast<uint32_t*>(gs + start + head) + lane;
    const uint32_t* sw = reinterpret_cast<const uint32_t*>(ss_ + start + head) + lane;
    const uint32_t* tw = reinterpret_cast<const uint32_t*>(ts + start + head) + lane;
    if (warp < rows) {
      const int li = start + lc;
      float s2 = 0.f, hs = 0.f;
      if (loose) {
        const float s = to_f(ss_[li]);
        s2 = s * s;
        hs = to_f(gs[li]) * wl * s;
      }
#pragma unroll
      for (int k = 0; k < NS; ++k)
        if (lane + 32 * k < n) {
          float s[N], g[N];
          Wd::get(sw[32 * k], s);
          Wd::get(gw[32 * k], g);
#pragma unroll
          for (int e = 0; e < N; ++e) {
            s2 += s[e] * s[e];
            hs += g[e] * wv[k][e] * s[e];
          }
        }
      s2 *= p.unit;
      hs *= p.unit;
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        s2 += __shfl_xor_sync(0xffffffffu, s2, o);
        hs += __shfl_xor_sync(0xffffffffu, hs, o);
      }
      const float rstd = rsqrtf(s2 / p.count + p.eps), q = hs * rstd * rstd / p.count;
#pragma unroll
      for (int k = 0; k < NS; ++k)
        if (lane + 32 * k < n) {
          float s[N], g[N], o[N];
          Wd::get(sw[32 * k], s);
          Wd::get(gw[32 * k], g);
#pragma unroll
          for (int e = 0; e < N; ++e) {
            o[e] = rstd * (g[e] * wv[k][e] - s[e] * q);
            acc[k][e] += g[e] * (s[e] * rstd);
          }
          if (p.g_s) {
            float t[N];
            Wd::get(tw[32 * k], t);
#pragma unroll
            for (int e = 0; e < N; ++e) o[e] += t[e];
          }
          gw[32 * k] = Wd::put(o);
        }
      if (loose) {
        const float s = to_f(ss_[li]), g = to_f(gs[li]);
        float o = rstd * (g * wl - s * q);
        if (p.g_s) o += to_f(ts[li]);
        accl += g * (s * rstd);
        gs[li] = from_f<T>(o);
      }
    }
    __syncthreads();
    copy_rows(static_cast<T*>(p.g_x) + b * R * p.cols, gs, rows * p.cols * (int)sizeof(T));
    unsigned char* t = cur;
    cur = other;
    other = t;
  }
  if (!p.part) return;
  __syncthreads();
  float* sum = reinterpret_cast<float*>(odd_sm);                  // [cols]; the warps in order
  for (int q = 0; q < R; ++q) {
    if (q) __syncthreads();
    if (warp != q) continue;
    auto add = [&](int c, float a) { sum[c] = q ? sum[c] + a : a; };
#pragma unroll
    for (int k = 0; k < NS; ++k)
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (lane + 32 * k < n) add(head + (lane + 32 * k) * N + e, acc[k][e]);
    if (loose) add(lc, accl);
  }
  __syncthreads();
  const int nout = p.degrees ? 4 * C : p.cols;
  float* part = p.part + (size_t)blockIdx.x * nout;
  for (int o = threadIdx.x; o < nout; o += ODD_THREADS) part[o] = p.degrees ? degree_sum(sum, o, C) : sum[o];
}

// ------------------------------------------------------------------ any rows
// The rest (pitches or starts off 16 bytes, or contiguous rows too long for the form above) is staged in
// shared memory at the offset from a 16-byte boundary that a row has in memory, so that all but its first and
// last bytes still move in 16-byte vectors.  Persistent teams of tw warps (1 to 8, so that a thread has at most 16 of a
// row's columns, 32 beyond 4096), each with its own rows and no barrier but its own: while a row is
// computed the next one is on its way (cp.async) into the team's other input slots.  A thread's columns are the
// same in every row, so its weights, and its part of g_w, stay in registers.  Bound by instructions, some hundreds a row
// and warp beside its elements: 80896 x 515 in bf16 at a pitch of 518 takes 135 us, its gradient with g_s 236.
constexpr int ST_THREADS = 256, ST_WARPS = ST_THREADS / 32;

__host__ __device__ constexpr int slot_bytes(int row_bytes) { return (row_bytes + 15) / 16 * 16 + 16; }
__device__ __forceinline__ int phase_of(const void* p) { return (int)(reinterpret_cast<uintptr_t>(p) & 15); }

struct Team {
  int tw, n, r, t;                 // warps, threads, the team's number in the block, the thread's in the team
  __device__ __forceinline__ explicit Team(int tw_) : tw(tw_), n(32 * tw_), r(threadIdx.x / (32 * tw_)), t(threadIdx.x % (32 * tw_)) {}
  __device__ __forceinline__ void sync() const {
    if (tw == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(r + 1), "r"(n) : "memory");
  }
};

// A row's copy into its slot: 16-byte bodies by cp.async, the up to 15 bytes before and behind them as at most one
// element each per thread, kept in registers until they are written.
template <typename T>
struct RowIn {
  T head, tail;
  __device__ __forceinline__ void issue(unsigned char* slot, const T* row, int cols, const Team& m) {
    const int ph = phase_of(row), end = ph + cols * (int)sizeof(T);
    const unsigned char* base = reinterpret_cast<const unsigned char*>(row) - ph;
    const int first = ph ? 1 : 0, last = end >> 4;                     // whole chunks: first .. last - 1
    const uint32_t dst = (uint32_t)__cvta_generic_to_shared(slot);
    for (int i = first + m.t; i < last; i += m.n)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + i * 16), "l"(base + i * 16) : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");
    const int h = head_at(ph, end, m.t), l = tail_at(ph, end, m.t);
    if (h >= 0) head = *reinterpret_cast<const T*>(base + h);
    if (l >= 0) tail = *reinterpret_cast<const T*>(base + l);
  }
  __device__ __forceinline__ void finish(unsigned char* slot, const T* row, int cols, const Team& m) const {
    const int ph = phase_of(row), end = ph + cols * (int)sizeof(T);
    const int h = head_at(ph, end, m.t), l = tail_at(ph, end, m.t);
    if (h >= 0) *reinterpret_cast<T*>(slot + h) = head;
    if (l >= 0) *reinterpret_cast<T*>(slot + l) = tail;
  }
  // byte offset of thread t's element before the first whole chunk and behind the last, or -1
  static __device__ __forceinline__ int head_at(int ph, int end, int t) {
    const int at = ph + t * (int)sizeof(T);
    return ph && at < 16 && at < end ? at : -1;
  }
  static __device__ __forceinline__ int tail_at(int ph, int end, int t) {
    const int from = end & ~15, at = from + t * (int)sizeof(T);
    return at < end && !(from == 0 && ph) ? at : -1;                   // a row inside one chunk is all head
  }
};
template <typename U>
__device__ __forceinline__ void row_out(const unsigned char* slot, U* row, int cols, const Team& m) {
  const int ph = phase_of(row), end = ph + cols * (int)sizeof(U);
  unsigned char* base = reinterpret_cast<unsigned char*>(row) - ph;
  for (int i = (ph ? 1 : 0) + m.t; i < (end >> 4); i += m.n) *reinterpret_cast<uint4*>(base + i * 16) = *reinterpret_cast<const uint4*>(slot + i * 16);
  const int h = RowIn<U>::head_at(ph, end, m.t), l = RowIn<U>::tail_at(ph, end, m.t);
  if (h >= 0) *reinterpret_cast<U*>(base + h) = *reinterpret_cast<const U*>(slot + h);
  if (l >= 0) *reinterpret_cast<U*>(base + l) = *reinterpret_cast<const U*>(slot + l);
}
__device__ __forceinline__ void rows_landed() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// sums (MAX: the second is max_abs) over a team
template <bool MAX>
__device__ __forceinline__ void team_reduce(float& a, float& b, const Team& m, float (*red)[2]) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    const float c = __shfl_xor_sync(0xffffffffu, b, o);
    b = MAX ? max_abs(b, c) : b + c;
  }
  if (m.tw == 1) return;
  const int w0 = m.r * m.tw;
  if ((m.t & 31) == 0) { red[w0 + (m.t >> 5)][0] = a; red[w0 + (m.t >> 5)][1] = b; }
  m.sync();
  a = red[w0][0];
  b = red[w0][1];
  for (int i = 1; i < m.tw; ++i) {
    a += red[w0 + i][0];
    b = MAX ? max_abs(b, red[w0 + i][1]) : b + red[w0 + i][1];
  }
}

// Shared memory of a team: `stages` sets of input slots (two where they fit), then the output slots.
template <typename T, bool QUANT, int NA>
__global__ void __launch_bounds__(ST_THREADS, NA > 16 ? 2 : 4) k_rms_norm_staged(const Args p, int tw, int stages) {
  extern __shared__ __align__(16) unsigned char st_sm[];
  __shared__ float red[ST_WARPS][2];
  const Team m(tw);
  const int C = p.cols / NCOMP, R = ST_WARPS / tw, slot = slot_bytes(p.cols * (int)sizeof(T)), ni = p.residual ? 2 : 1;
  unsigned char* in = st_sm + m.r * slot * (stages * ni + (p.s ? 2 : 1));
  unsigned char* ys = in + stages * ni * slot;
  unsigned char* ss_ = ys + slot;
  const T* w = static_cast<const T*>(p.w);
  float wv[NA];
#pragma unroll
  for (int k = 0; k < NA; ++k) {
    const int c = m.t + m.n * k;
    wv[k] = w && c < p.cols ? to_f(w[weight_at(c, C, p.degrees)]) : 1.f;
  }
  auto x_row = [&](long long row) { return static_cast<const T*>(p.x) + row * p.ldx; };
  auto r_row = [&](long long row) { return static_cast<const T*>(p.residual) + row * p.ldr; };
  RowIn<T> xi, ri;
  auto issue = [&](long long row, int st) {
    if (row >= p.rows) return;
    xi.issue(in + st * ni * slot, x_row(row), p.cols, m);
    if (p.residual) ri.issue(in + (st * ni + 1) * slot, r_row(row), p.cols, m);
  };
  const long long step = (long long)gridDim.x * R;
  long long row = (long long)blockIdx.x * R + m.r;
  int st = 0;
  issue(row, 0);
  for (; row < p.rows; row += step) {
    unsigned char* xs = in + st * ni * slot;
    unsigned char* rs = xs + slot;
    xi.finish(xs, x_row(row), p.cols, m);
    if (p.residual) ri.finish(rs, r_row(row), p.cols, m);
    rows_landed();
    m.sync();
    if (stages == 2) issue(row + step, st ^ 1);
    const T* xv = reinterpret_cast<const T*>(xs + phase_of(x_row(row)));
    const T* rv = reinterpret_cast<const T*>(rs + phase_of(r_row(row)));
    T* srow = static_cast<T*>(p.s) + row * p.lds;
    T* sv = reinterpret_cast<T*>(ss_ + phase_of(srow));
    float v[NA], ss = 0.f, top = 0.f;
#pragma unroll
    for (int k = 0; k < NA; ++k) {
      const int c = m.t + m.n * k;
      v[k] = 0.f;
      if (c < p.cols) {
        v[k] = to_f(xv[c]);
        if (p.residual) v[k] += to_f(rv[c]);
        if (p.s) sv[c] = from_f<T>(v[k]);
      }
      ss += v[k] * v[k];
      v[k] *= wv[k];
      if (QUANT) top = max_abs(top, v[k]);
    }
    ss *= p.unit;
    team_reduce<true>(ss, top, m, red);
    const float rstd = rsqrtf(ss / p.count + p.eps);
    float inv = 1.f;
    if (QUANT) {
      const float big = top * rstd;
      const float scale = big < TINY ? 1.f : big / 448.f;
      inv = 1.f / scale;
      if (m.t == 0) p.scale[row] = scale;
    }
    T* yrow = static_cast<T*>(p.y) + row * p.ldy;
    __nv_fp8_storage_t* qrow = static_cast<__nv_fp8_storage_t*>(p.y) + row * p.ldy;
    T* yv = reinterpret_cast<T*>(ys + phase_of(yrow));
    __nv_fp8_storage_t* qv = ys + phase_of(qrow);
#pragma unroll
    for (int k = 0; k < NA; ++k) {
      const int c = m.t + m.n * k;
      if (c >= p.cols) continue;
      if (QUANT) qv[c] = __nv_cvt_float_to_fp8(v[k] * rstd * inv, __NV_SATFINITE, __NV_E4M3);
      else yv[c] = from_f<T>(v[k] * rstd);
    }
    m.sync();
    if (stages == 1) issue(row + step, 0);
    if (QUANT) row_out<__nv_fp8_storage_t>(ys, qrow, p.cols, m);
    else row_out<T>(ys, yrow, p.cols, m);
    if (p.s) row_out<T>(ss_, srow, p.cols, m);
    if (stages == 2) st ^= 1;
  }
}

template <typename T, int NA>
__global__ void __launch_bounds__(ST_THREADS, NA > 16 ? 2 : 3) k_rms_norm_grad_staged(const GradArgs p, int tw, int stages) {
  extern __shared__ __align__(16) unsigned char st_sm[];
  __shared__ float red[ST_WARPS][2];
  const Team m(tw);
  const int C = p.cols / NCOMP, R = ST_WARPS / tw, slot = slot_bytes(p.cols * (int)sizeof(T)), ni = p.g_s ? 3 : 2;
  unsigned char* in = st_sm + m.r * slot * (stages * ni + 1);
  unsigned char* os = in + stages * ni * slot;
  const T* w = static_cast<const T*>(p.w);
  float acc[NA], wv[NA];
#pragma unroll
  for (int k = 0; k < NA; ++k) {
    const int c = m.t + m.n * k;
    acc[k] = 0.f;
    wv[k] = w && c < p.cols ? to_f(w[weight_at(c, C, p.degrees)]) : 1.f;
  }
  auto g_row = [&](long long row) { return static_cast<const T*>(p.g) + row * p.ldg; };
  auto s_row = [&](long long row) { return static_cast<const T*>(p.s) + row * p.lds; };
  auto t_row = [&](long long row) { return static_cast<const T*>(p.g_s) + row * p.ldgs; };
  RowIn<T> gi, si, ti;
  auto issue = [&](long long row, int st) {
    if (row >= p.rows) return;
    unsigned char* a = in + st * ni * slot;
    gi.issue(a, g_row(row), p.cols, m);
    si.issue(a + slot, s_row(row), p.cols, m);
    if (p.g_s) ti.issue(a + 2 * slot, t_row(row), p.cols, m);
  };
  const long long step = (long long)gridDim.x * R;
  long long row = (long long)blockIdx.x * R + m.r;
  int st = 0;
  issue(row, 0);
  for (; row < p.rows; row += step) {
    unsigned char* a = in + st * ni * slot;
    gi.finish(a, g_row(row), p.cols, m);
    si.finish(a + slot, s_row(row), p.cols, m);
    if (p.g_s) ti.finish(a + 2 * slot, t_row(row), p.cols, m);
    rows_landed();
    m.sync();
    if (stages == 2) issue(row + step, st ^ 1);
    const T* gv = reinterpret_cast<const T*>(a + phase_of(g_row(row)));
    const T* sv = reinterpret_cast<const T*>(a + slot + phase_of(s_row(row)));
    const T* tv = reinterpret_cast<const T*>(a + 2 * slot + phase_of(t_row(row)));
    float s2 = 0.f, hs = 0.f;
#pragma unroll
    for (int k = 0; k < NA; ++k) {
      const int c = m.t + m.n * k;
      if (c >= p.cols) continue;
      const float v = to_f(sv[c]);
      s2 += v * v;
      hs += to_f(gv[c]) * wv[k] * v;
    }
    s2 *= p.unit;
    hs *= p.unit;
    team_reduce<false>(s2, hs, m, red);
    const float rstd = rsqrtf(s2 / p.count + p.eps), q = hs * rstd * rstd / p.count;
    T* out = static_cast<T*>(p.g_x) + row * p.ldgx;
    T* ov = reinterpret_cast<T*>(os + phase_of(out));
#pragma unroll
    for (int k = 0; k < NA; ++k) {
      const int c = m.t + m.n * k;
      if (c >= p.cols) continue;
      const float v = to_f(sv[c]), g = to_f(gv[c]);
      float o = rstd * (g * wv[k] - v * q);
      if (p.g_s) o += to_f(tv[c]);
      acc[k] += g * (v * rstd);
      ov[c] = from_f<T>(o);
    }
    m.sync();
    if (stages == 1) issue(row + step, 0);
    row_out<T>(os, out, p.cols, m);
    if (stages == 2) st ^= 1;
  }
  if (!p.part) return;
  __syncthreads();
  float* sum = reinterpret_cast<float*>(st_sm);                // [cols]; the block's teams in order
  for (int q = 0; q < R; ++q) {
    if (q) __syncthreads();
    if (m.r == q) {
#pragma unroll
      for (int k = 0; k < NA; ++k) {
        const int c = m.t + m.n * k;
        if (c < p.cols) sum[c] = q ? sum[c] + acc[k] : acc[k];
      }
    }
  }
  __syncthreads();
  const int nout = p.degrees ? 4 * C : p.cols;
  float* part = p.part + (size_t)blockIdx.x * nout;
  for (int o = threadIdx.x; o < nout; o += ST_THREADS) part[o] = p.degrees ? degree_sum(sum, o, C) : sum[o];
}

// Persistent: block b takes row groups b, b + gridDim.x, ...; a thread's columns are the same in
// every row, so its part of g_w stays in registers until the end.  The next row's loads are issued before
// the current row's reduction, so that some are always in flight.
// Two blocks of 256 threads per SM and two vectors a thread: 4096 x 2048 FP32 takes 28 us, 4.8 TB/s, and 80896 x 512 bf16
// 67 us, 4.9 TB/s; three blocks spill (33 us), one vector with four blocks 40 us (both at 4096 x 2048).
constexpr int GRAD_PER_SM = 2;
template <typename T, int V, int SL, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? GRAD_PER_SM : 1) k_rms_norm_grad(const GradArgs p) {
  extern __shared__ float acc_sm[];              // [cols] when the block has several rows or there are degrees
  __shared__ float red[2][2][32];
  const int G = blockDim.x, t = threadIdx.x, r = threadIdx.y, R = blockDim.y;
  const int C = p.cols / NCOMP;
  const T* w = static_cast<const T*>(p.w);
  float acc[SL][V];
  Raw<T, V> g_[SL], s_[SL], t_[SL];
  int at[SL];                                    // where a vector's weights are
#pragma unroll
  for (int k = 0; k < SL; ++k) {
    const int c = (k * G + t) * V;
    at[k] = c < p.cols ? weight_at(c, C, p.degrees) : 0;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[k][i] = 0.f;
  }
  auto fetch = [&](long long row) {
    const bool live = row < p.rows;
#pragma unroll
    for (int k = 0; k < SL; ++k) {
      const int c = (k * G + t) * V;
      const bool in = live && c < p.cols;
      g_[k].load(static_cast<const T*>(p.g) + row * p.ldg + c, in);
      s_[k].load(static_cast<const T*>(p.s) + row * p.lds + c, in);
      if (p.g_s) t_[k].load(static_cast<const T*>(p.g_s) + row * p.ldgs + c, in);
    }
  };
  const long long groups = (p.rows + R - 1) / R;
  int par = 0;
  fetch((long long)blockIdx.x * R + r);
  for (long long b = blockIdx.x; b < groups; b += gridDim.x, par ^= 1) {
    const long long row = b * R + r;
    const bool live = row < p.rows;
    float g[SL][V], s[SL][V];
    Raw<T, V> th[SL];
    float ss = 0.f, hs = 0.f;
#pragma unroll
    for (int k = 0; k < SL; ++k) {
      g_[k].get(g[k]);
      s_[k].get(s[k]);
      th[k] = t_[k];
    }
    fetch(row + (long long)gridDim.x * R);
#pragma unroll
    for (int k = 0; k < SL; ++k) {
      float wv[V];
#pragma unroll
      for (int i = 0; i < V; ++i) wv[i] = 1.f;
      if (w) load_v<T, V>(w + at[k], wv);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        ss += s[k][i] * s[k][i];
        hs += g[k][i] * wv[i] * s[k][i];
      }
    }
    ss *= p.unit;
    hs *= p.unit;
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
    const float rstd = rsqrtf(ss / p.count + p.eps);
    const float q = hs * rstd * rstd / p.count;      // mean(h n) rstd: n mean(h n) = s q
#pragma unroll
    for (int k = 0; k < SL; ++k) {
      const int c = (k * G + t) * V;
      if (c >= p.cols) continue;
      float wv[V], o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) { wv[i] = 1.f; o[i] = 0.f; }
      if (w) load_v<T, V>(w + at[k], wv);
      if (p.g_s) th[k].get(o);
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
    part[o] = p.degrees ? degree_sum(acc_sm, o, C) : acc_sm[o];
  }
}

// Launch shape of the vector kernels: a row's vectors fill a warp first, then each thread takes up to `most` of
// them, then the row gets more warps; short rows share a block of up to 256 threads, fewer when there
// are not enough rows for two blocks on every SM.
struct Shape {
  int SL, G, R;
};
inline Shape shape_for(int cols, int V, int most, long long rows) {
  Shape s;
  const int n = (cols + V - 1) / V;
  s.SL = 1;
  while (s.SL < most && n > 32 * s.SL) s.SL *= 2;
  s.G = (n + 32 * s.SL - 1) / (32 * s.SL) * 32;
  s.R = (int)std::max<long long>(1, std::min<long long>(256 / s.G, rows / 296));
  return s;
}

// 16-byte vectors need every pointer and row pitch in use to allow them
inline bool vec_ok(const void* p, long long ld, long long rows, int es) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows == 1 || ld * es % 16 == 0));
}
// a kernel's dynamic shared memory above 48 KB has to be allowed, once per device
template <auto KERNEL>
cudaError_t allow_smem(int bytes) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load() & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit);
  return e;
}
constexpr int ST_SMEM = 220 * 1024;                            // one row of the most columns, its inputs and outputs, fits

template <typename T, int V, int SL>
void launch_fwd2(const Args& a, const Shape& h, bool quant, cudaStream_t st) {
  const dim3 block(h.G, h.R);
  const unsigned grid = (unsigned)((a.rows + h.R - 1) / h.R);
  if (quant) k_rms_norm<T, V, SL, true><<<grid, block, 0, st>>>(a);
  else k_rms_norm<T, V, SL, false><<<grid, block, 0, st>>>(a);
}
// blocks of the persistent kernels (the gradient's each leave one row of column sums): up to four per SM
inline int grad_blocks(long long rows, int R) { return (int)std::min<long long>((rows + R - 1) / R, 4 * 148); }

struct Staged {
  int tw, R, stages, smem, NA;
};
inline Staged staged_for(int cols, int es, int ins, int outs) {
  Staged h;
  h.tw = 1;
  while (h.tw < ST_WARPS && cols > 32 * 16 * h.tw) h.tw *= 2;
  h.R = ST_WARPS / h.tw;
  const int per = h.R * slot_bytes(cols * es);
  h.stages = per * (2 * ins + outs) <= ST_SMEM / 2 ? 2 : 1;            // two where two blocks fit on an SM
  h.smem = std::max(per * (h.stages * ins + outs), cols * 4);
  h.NA = cols <= 128 ? 4 : cols <= 32 * 16 * h.tw ? 16 : 32;
  return h;
}
template <auto KERNEL, typename A>
cudaError_t launch_staged(const A& a, const Staged& h, int blocks, cudaStream_t st) {
  const cudaError_t e = allow_smem<KERNEL>(ST_SMEM);
  if (e != cudaSuccess) return e;
  KERNEL<<<blocks, ST_THREADS, h.smem, st>>>(a, h.tw, h.stages);
  return cudaGetLastError();
}
template <typename T, bool QUANT>
cudaError_t launch_fwd_staged(const Args& a, cudaStream_t st) {
  const Staged h = staged_for(a.cols, sizeof(T), a.residual ? 2 : 1, a.s ? 2 : 1);
  const int blocks = grad_blocks(a.rows, h.R);
  if (h.NA == 4) return launch_staged<k_rms_norm_staged<T, QUANT, 4>>(a, h, blocks, st);
  if (h.NA == 16) return launch_staged<k_rms_norm_staged<T, QUANT, 16>>(a, h, blocks, st);
  return launch_staged<k_rms_norm_staged<T, QUANT, 32>>(a, h, blocks, st);
}
template <typename T, bool QUANT, bool RES, int RW>
bool launch_odd4(const Args& a, int rows_smem, int smem, cudaStream_t st) {
  if (allow_smem<k_rms_norm_odd<T, QUANT, RES, RW>>(ODD_SMEM) != cudaSuccess) return false;
  const long long groups = (a.rows + RW * ODD_THREADS / 32 - 1) / (RW * ODD_THREADS / 32);
  // a block per group of rows where they are all at work at once (5374 x 794 bf16 with a residual: 12.3 us, 14.3 with two
  // buffers) or two buffers do not fit, else persistent
  auto at_once = [](int bytes) { return (long long)tc::num_sms() * std::min(8, SM_SMEM / (bytes + 1024)); };
  const int bufs = groups > at_once(smem) && smem + rows_smem <= ODD_SMEM ? 2 : 1;
  if (bufs == 2) smem += rows_smem;
  const long long grid = bufs == 2 ? at_once(smem) : groups;
  k_rms_norm_odd<T, QUANT, RES, RW><<<(unsigned)grid, ODD_THREADS, smem, st>>>(a, bufs);
  return true;
}
template <typename T, bool QUANT, int RW>
bool launch_odd3(const Args& a, cudaStream_t st) {
  const int rows_smem = round16(RW * ODD_THREADS / 32 * a.cols * (int)sizeof(T)) * (a.residual ? 2 : 1);
  const int smem = round16(4 * a.cols) + rows_smem + (QUANT ? RW * ODD_THREADS / 32 * a.cols : 0);
  if (smem > ODD_SMEM) return false;
  return a.residual ? launch_odd4<T, QUANT, true, RW>(a, rows_smem, smem, st) : launch_odd4<T, QUANT, false, RW>(a, rows_smem, smem, st);
}
inline bool packed_rows(const void* p, long long ld, const Args& a) {       // contiguous, on a 16-byte boundary
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld == a.cols || a.rows == 1));
}
template <typename T>
bool launch_odd(const Args& a, bool quant, cudaStream_t st) {
  if (!packed_rows(a.x, a.ldx, a) || !packed_rows(a.residual, a.ldr, a) || !packed_rows(a.y, a.ldy, a) ||
      !packed_rows(a.s, a.lds, a) || (a.s && !a.residual))
    return false;
  if (quant) return launch_odd3<T, true, 2>(a, st);                 // 16 rows of 8 bits are whole 16 bytes
  // two rows a warp where there are enough of them for every SM, else (or where they do not fit) one
  const bool many = a.rows > 2 * ODD_THREADS / 32 * tc::num_sms();
  return (many && launch_odd3<T, false, 2>(a, st)) || launch_odd3<T, false, 1>(a, st);
}

template <typename A>
A with_unit(A a) {
  a.unit = 1.f;
  while (a.unit * a.cols > 1.f) a.unit *= 0.5f;
  a.count = a.unit * a.cols;
  return a;
}

template <typename T>
cudaError_t launch_fwd(const Args& args, bool quant, cudaStream_t st) {
  const Args a = with_unit(args);
  constexpr int ES = sizeof(T), V = 16 / ES;
  const bool yv = quant ? reinterpret_cast<uintptr_t>(a.y) % V == 0 && (a.rows == 1 || a.ldy % V == 0) : vec_ok(a.y, a.ldy, a.rows, ES);
  const bool vec = a.cols % V == 0 && yv && vec_ok(a.x, a.ldx, a.rows, ES) && vec_ok(a.residual, a.ldr, a.rows, ES) &&
                   vec_ok(a.s, a.lds, a.rows, ES) && vec_ok(a.w, 0, 1, ES) && (!a.degrees || a.cols / NCOMP % V == 0);
  if (!vec && launch_odd<T>(a, quant, st)) return cudaGetLastError();
  if (!vec) return quant ? launch_fwd_staged<T, true>(a, st) : launch_fwd_staged<T, false>(a, st);
  // at most 16 elements a thread (16384 x 2048 bf16 to e4m3: 59 us with 8, 50 with 16, 68 with 32)
  const Shape h = shape_for(a.cols, V, 16 / V, a.rows);
  if (h.SL == 1) launch_fwd2<T, V, 1>(a, h, quant, st);
  else if (h.SL == 2) launch_fwd2<T, V, 2>(a, h, quant, st);
  else if constexpr (V == 4) launch_fwd2<T, V, 4>(a, h, quant, st);
  return cudaGetLastError();
}

template <typename T, int V, int SL>
void launch_grad2(const GradArgs& a, const Shape& h, int blocks, cudaStream_t st) {
  const int smem = h.R > 1 || a.degrees ? a.cols * 4 : 0;
  if constexpr (SL < 4) {                // rows of four vectors a thread are above 4096 columns, which takes 288 threads at least
    if (h.G * h.R <= 256) {
      k_rms_norm_grad<T, V, SL, 256><<<blocks, dim3(h.G, h.R), smem, st>>>(a);
      return;
    }
  }
  k_rms_norm_grad<T, V, SL, MAX_THREADS><<<blocks, dim3(h.G, h.R), smem, st>>>(a);
}
template <typename T, int NS>
int launch_grad_odd3(const GradArgs& a, int smem, cudaStream_t st) {
  if (allow_smem<k_rms_norm_grad_odd<T, NS>>(ODD_SMEM) != cudaSuccess) return 0;
  const int blocks = grad_blocks(a.rows, ODD_THREADS / 32);
  k_rms_norm_grad_odd<T, NS><<<blocks, ODD_THREADS, smem, st>>>(a);
  return blocks;
}
template <typename T>
int launch_grad_odd(const GradArgs& a, cudaStream_t st) {      // 0: not for these rows
  auto packed = [&](const void* p, long long ld) {
    return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld == a.cols || a.rows == 1));
  };
  const int smem = 2 * ODD_THREADS / 32 * a.cols * (int)sizeof(T) * (a.g_s ? 3 : 2);      // (the final sums, 4 cols, fit too)
  if (a.cols > ODD_GRAD_COLS || smem > ODD_SMEM || !packed(a.g, a.ldg) || !packed(a.s, a.lds) || !packed(a.g_s, a.ldgs) ||
      !packed(a.g_x, a.ldgx))
    return 0;
  const int words = (a.cols / Word<T>::N + 31) / 32;                // of a lane
  if (words <= 2) return launch_grad_odd3<T, 2>(a, smem, st);
  if (words <= 4) return launch_grad_odd3<T, 4>(a, smem, st);
  if (words <= 8) return launch_grad_odd3<T, 8>(a, smem, st);
  if (words <= 12) return launch_grad_odd3<T, 12>(a, smem, st);
  if (words <= 16) return launch_grad_odd3<T, 16>(a, smem, st);
  if constexpr (Word<T>::N == 1) return launch_grad_odd3<T, 32>(a, smem, st);
  return 0;
}
template <typename T>
cudaError_t launch_grad(const GradArgs& args, int* blocks, cudaStream_t st) {       // *blocks: the rows of part
  const GradArgs a = with_unit(args);
  constexpr int ES = sizeof(T), V = 16 / ES;
  const bool vec = a.cols % V == 0 && vec_ok(a.g, a.ldg, a.rows, ES) && vec_ok(a.s, a.lds, a.rows, ES) &&
                   vec_ok(a.g_s, a.ldgs, a.rows, ES) && vec_ok(a.g_x, a.ldgx, a.rows, ES) && vec_ok(a.w, 0, 1, ES) &&
                   (!a.degrees || a.cols / NCOMP % V == 0);
  if (!vec) {
    if ((*blocks = launch_grad_odd<T>(a, st)) > 0) return cudaGetLastError();
    const Staged h = staged_for(a.cols, ES, a.g_s ? 3 : 2, 1);
    *blocks = grad_blocks(a.rows, h.R);
    if (h.NA == 4) return launch_staged<k_rms_norm_grad_staged<T, 4>>(a, h, *blocks, st);
    if (h.NA == 16) return launch_staged<k_rms_norm_grad_staged<T, 16>>(a, h, *blocks, st);
    return launch_staged<k_rms_norm_grad_staged<T, 32>>(a, h, *blocks, st);
  }
  const Shape h = shape_for(a.cols, V, a.cols > MAX_THREADS * 2 * V ? 4 : 2, a.rows);
  *blocks = grad_blocks(a.rows, h.R);
  if (h.SL == 1) launch_grad2<T, V, 1>(a, h, *blocks, st);
  else if (h.SL == 2) launch_grad2<T, V, 2>(a, h, *blocks, st);
  else if constexpr (V == 4) launch_grad2<T, V, 4>(a, h, *blocks, st);      // 16-bit rows of the most columns take two
  return cudaGetLastError();
}

}  // namespace norm
}  // namespace emp
