// Typed rows for the row-wise operators (norm.cuh, dense.cuh): loads and stores of fp32, bf16, fp16 and
// e4m3 elements as fp32 values, the activations, and the fixed-order join of per-block column sums.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <type_traits>
#include "emp_common.cuh"

namespace emp {

__host__ __device__ constexpr int dtype_size(int t) { return t == EMP_F32 ? 4 : t == EMP_E4M3 ? 1 : 2; }

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// two neighbouring elements of a 32-bit word (16-bit types) as floats, and back; by value throughout, so that
// no array of them ends up in local memory
template <typename T> __device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b);
template <> __device__ __forceinline__ void unpack2<__nv_bfloat16>(uint32_t w, float& a, float& b) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xffff0000u);
}
template <> __device__ __forceinline__ void unpack2<__half>(uint32_t w, float& a, float& b) {
  a = __half2float(__ushort_as_half((unsigned short)(w & 0xffffu)));
  b = __half2float(__ushort_as_half((unsigned short)(w >> 16)));
}
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);      // one conversion for both
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 16 bytes as floats: four of fp32 or eight of a 16-bit type
template <typename T, int V>
__device__ __forceinline__ void unpack16(const uint4& u, float (&v)[V]) {
  if constexpr (V == 4) {
    v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y); v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
  } else {
    unpack2<T>(u.x, v[0], v[1]); unpack2<T>(u.y, v[2], v[3]); unpack2<T>(u.z, v[4], v[5]); unpack2<T>(u.w, v[6], v[7]);
  }
}
// V consecutive elements as floats; V > 1: 16 bytes (4 for V = 2, 8 of e4m3), p aligned to them
template <typename T, int V>
__device__ __forceinline__ void load_v(const T* p, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = to_f(*p);
  } else if constexpr (sizeof(T) == 1) {
    static_assert(V == 8, "vector bytes");
    const uint2 u = *reinterpret_cast<const uint2*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      __nv_fp8_e4m3 e;
      e.__x = (unsigned char)((i < 4 ? u.x : u.y) >> (8 * (i & 3)));
      v[i] = (float)e;
    }
  } else if constexpr (V == 2) {
    unpack2<T>(*reinterpret_cast<const uint32_t*>(p), v[0], v[1]);
  } else {
    static_assert(V * sizeof(T) == 16, "vector bytes");
    unpack16<T, V>(*reinterpret_cast<const uint4*>(p), v);
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    *p = from_f<T>(v[0]);
  } else if constexpr (V == 2) {
    *reinterpret_cast<uint32_t*>(p) = pack2<T>(v[0], v[1]);
  } else if constexpr (V == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
  }
}
// V elements as they are in memory (zeros where `in` is false): a load with its conversion in one branch would be
// waited for before the next one.  One element of 8 or 16 bits has a register to itself.
template <typename T, int V> struct Raw {
  using U = std::conditional_t<V * sizeof(T) == 16, uint4, uint32_t>;
  U u;
  __device__ __forceinline__ void load(const T* p, bool in) {
    u = U();
    if (!in) return;
    if constexpr (V > 1 || sizeof(T) == 4) u = *reinterpret_cast<const U*>(p);
    else if constexpr (sizeof(T) == 2) u = *reinterpret_cast<const unsigned short*>(p);
    else u = *reinterpret_cast<const unsigned char*>(p);
  }
  __device__ __forceinline__ void get(float (&v)[V]) const {
    if constexpr (V == 1) v[0] = one(T());
    else if constexpr (V == 2) unpack2<T>(u, v[0], v[1]);
    else unpack16<T, V>(u, v);
  }
  __device__ __forceinline__ float one(float) const { return __uint_as_float(u); }
  __device__ __forceinline__ float one(__nv_bfloat16) const { return __uint_as_float(u << 16); }
  __device__ __forceinline__ float one(__half) const { return __half2float(__ushort_as_half((unsigned short)u)); }
  __device__ __forceinline__ float one(__nv_fp8_e4m3 e) const {
    e.__x = (unsigned char)u;
    return (float)e;
  }
};
// V values rounded to e4m3 (to nearest even; beyond +-448 to +-448; NaN kept)
template <int V>
__device__ __forceinline__ void store_e4m3(__nv_fp8_storage_t* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    *p = __nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
  } else {
    uint32_t w[V / 4];
#pragma unroll
    for (int i = 0; i < V; i += 4)
      w[i / 4] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[i], v[i + 1]), __NV_SATFINITE, __NV_E4M3) |
                 (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[i + 2], v[i + 3]), __NV_SATFINITE, __NV_E4M3) << 16;
    if constexpr (V == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}

// one element of a buffer whose type, FP32, bf16 or fp16, is known at run time only (edges, small operands)
__device__ __forceinline__ float load_any(const void* p, size_t i, int t) {
  switch (t) {
    case EMP_F32: return static_cast<const float*>(p)[i];
    case EMP_BF16: return to_f(static_cast<const __nv_bfloat16*>(p)[i]);
    default: return to_f(static_cast<const __half*>(p)[i]);
  }
}
__device__ __forceinline__ void store_any(void* p, size_t i, int t, float v) {
  switch (t) {
    case EMP_F32: static_cast<float*>(p)[i] = v; break;
    case EMP_BF16: static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v); break;
    default: static_cast<__half*>(p)[i] = __float2half_rn(v); break;
  }
}

// degree of component lm = l*l + l + m
__device__ __forceinline__ int degree_of(int lm) { return (lm > 0) + (lm > 3) + (lm > 8); }

// ------------------------------------------------------------- activations
// SiLU z / (1 + exp(-z)) and GELU z Phi(z), and their derivatives, with e^x = 2^(x log2 e) by the special-function
// unit's 2^x and 1/x, both with results below 2^-126 as zero: __expf and __fdividef, which keep those, take 14
// instructions an element of SiLU instead of 5, and instructions bound a short-k epilogue (647168 x 64 -> 512 in FP32:
// 401 us so, 340 thus).  -inf and NaN give NaN.  Phi, the normal distribution function, is for z < 0
//   Phi(z) = exp(-z^2 / 2) t q(t),  t = 1 / (1 + p |z|),
// with q a polynomial fitted to exp(z^2 / 2) Phi(z) / t over -13.3 <= z <= 0 for the least largest RELATIVE error (least squares with
// Lawson's weights), so that GELU keeps its digits where it is small: 1/2 (1 + erf) has none there beyond z = -5, and erff costs
// more than twice as much.  For FP32 degree 7, within 1.2e-7: with the FP32 arithmetic Phi is within (32 + 1.5 z^2) 2^-24 of itself,
// the second term from the rounding of z^2 / 2 (SiLU's exponential has the same, |z| 2^-23).  For 16-bit types degree 5,
// within 1.2e-6 up to |z| = 1 and 5e-5 from 3 on, a tenth of half a step of fp16 (161792 x 64 -> 512 with GELU: bf16 90 us with
// degree 7, 85 with 5; FP32 106).  Below z = -13.2 (SiLU: -87) the results are zero.
__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_ftz(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float LOG2E = 1.4426950408889634f;

__device__ __forceinline__ float sigmoid_ftz(float z) { return rcp_ftz(1.0f + ex2_ftz(-LOG2E * z)); }
template <typename T> __device__ __forceinline__ float phi_ftz(float z, float gauss) {            // Phi(z); gauss = exp(-z^2 / 2)
  float t, q;
  if constexpr (sizeof(T) == 4) {
    t = rcp_ftz(fmaf(0.3f, fabsf(z), 1.f));
    q = fmaf(t, 0.0360362099f, -0.158713255f);
    q = fmaf(t, q, 0.208964023f);
    q = fmaf(t, q, -0.0560953968f);
    q = fmaf(t, q, 0.129843179f);
    q = fmaf(t, q, 0.0995231307f);
    q = fmaf(t, q, 0.120816882f);
    q = fmaf(t, q, 0.119625166f);
  } else {
    t = rcp_ftz(fmaf(0.29f, fabsf(z), 1.f));
    q = fmaf(t, -0.0867664392f, 0.278030956f);
    q = fmaf(t, q, -0.0844277764f);
    q = fmaf(t, q, 0.174245341f);
    q = fmaf(t, q, 0.102189743f);
    q = fmaf(t, q, 0.116728611f);
  }
  const float h = t * q * gauss;                          // Phi(-|z|)
  return z < 0.f ? h : 1.f - h;
}
__device__ __forceinline__ float gauss_ftz(float z) { return ex2_ftz(-0.5f * LOG2E * z * z); }

// T: the type that the result is rounded to
template <int ACT, typename T> __device__ __forceinline__ float act(float z) {
  if constexpr (ACT == EMP_ACT_SILU) return z * sigmoid_ftz(z);
  else if constexpr (ACT == EMP_ACT_GELU) return z * phi_ftz<T>(z, gauss_ftz(z));
  else return z;
}
template <int ACT, typename T> __device__ __forceinline__ float dact(float z) {
  if constexpr (ACT == EMP_ACT_SILU) {
    const float s = sigmoid_ftz(z);
    return s * (1.0f + z * (1.0f - s));
  } else if constexpr (ACT == EMP_ACT_GELU) {
    const float g = gauss_ftz(z);
    return phi_ftz<T>(z, g) + z * 0.39894228040143268f * g;
  } else {
    return 1.0f;
  }
}
__device__ __forceinline__ float act_f(int a, float z) {
  return a == EMP_ACT_SILU ? act<EMP_ACT_SILU, float>(z) : a == EMP_ACT_GELU ? act<EMP_ACT_GELU, float>(z) : z;
}

// ------------------------------------------------------------- join of column sums
// out[j] = sum over b of part[b][j].  32 columns per block, JOIN_WARPS warps over the rows (warp w takes
// rows w, w + JOIN_WARPS, ..., JOIN_BATCH loads at a time; the warps' sums are added in warp order), so the
// order is fixed.  Bound by the latency of its few loads.
constexpr int JOIN_WARPS = 32, JOIN_BATCH = 10;
__global__ void __launch_bounds__(32 * JOIN_WARPS)
    k_col_join(int nb, int cols, const float* __restrict__ part, void* __restrict__ out, int dtype) {
  __shared__ float sm[JOIN_WARPS][33];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = blockIdx.x * 32 + lane;
  float s = 0.f;
  for (int b0 = w; b0 < nb; b0 += JOIN_WARPS * JOIN_BATCH) {
    float v[JOIN_BATCH];
#pragma unroll
    for (int i = 0; i < JOIN_BATCH; ++i) {
      const int b = b0 + i * JOIN_WARPS;
      v[i] = b < nb && j < cols ? part[(size_t)b * cols + j] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < JOIN_BATCH; ++i) s += v[i];
  }
  sm[w][lane] = s;
  __syncthreads();
  if (w == 0 && j < cols) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < JOIN_WARPS; ++i) t += sm[i][lane];
    store_any(out, (size_t)j, dtype, t);
  }
}

}  // namespace emp
