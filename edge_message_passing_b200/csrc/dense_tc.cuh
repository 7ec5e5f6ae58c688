// The dense layer's products on the tensor cores (tcgen05, sm_100a):
//
//   out[m][n] = sum_k A(m, k) B(n, k),
//
// with A and B each stored with k contiguous ("k-major": x, W, and g in g_x = gz W) or with the other
// index contiguous ("mn-major": W in g_x, both operands of g_W = gz^T x), and the dense layer's epilogue.
//
// Persistent kernel, one CTA per SM, 128 x bn tiles (bn = 64, 128 or 256) taken round-robin with n
// fastest, so that neighbouring CTAs share an A tile in L2.  A long k axis with few tiles is split:
// each split leaves a partial product, and k_join adds them in order.  Warps: one issues TMA loads, one
// the MMAs, eight drain the accumulators (two per TMEM lane quarter, every other 32 columns each) and
// write the rows.
//
// bf16, fp16 and e4m3 operands go from TMA straight to the MMA: a ring of stages of 128 bytes of k
// (128-byte swizzle), two accumulators of bn columns, so the epilogue of a tile overlaps the next
// tile's products.
//
// FP32 operands are split a = hi + lo (hi = RN_tf32(a), lo = RN_tf32(a - hi)) inside the kernel, by two
// groups of four warps that take the 32-wide k stages in turn, so neither operand needs a pass of its
// own over memory: A's split goes to TMEM (the MMA's A operand may live there, and a thread's TMEM
// lane is its row, whichever way A is stored), B's to shared memory.  The tensor cores add into their
// FP32 accumulator by truncation, which shrinks a sum by about 2e-8 of itself per MMA (measured on the
// SO(2) products: 7e-9 K).  So an accumulator takes K_CHUNK = 64 of k only and is then added, rounded
// to nearest, to sums in the epilogue warps' registers, and within each stage the small products
// lo.hi and hi.lo come before hi.hi.
//
// Every mbarrier wait is bounded; the producer waits out its own copies before exit.
#pragma once
#include <atomic>
#include "so2_tc.cuh"
#include "dense.cuh"

namespace emp {
namespace dtc {

constexpr int BM = 128;
constexpr int EPI_WARPS = 8;
constexpr int SPLIT_GROUPS = 2, SPLIT_WARPS = 4 * SPLIT_GROUPS;
constexpr int A_BYTES = BM * 128;                       // one stage of A
constexpr int MAX_STAGES = 8;
constexpr int RING_BYTES = 4 * (A_BYTES + 256 * 128);   // 192 KB: four stages of 128 x 256 tiles
constexpr int LAND = 3;                                 // FP32: stages as they land ...
constexpr int LAND_BYTES = 2 * A_BYTES;
constexpr int HL_BYTES = 2 * A_BYTES;                   // ... and B's hi and lo, a slot per split group
static_assert(LAND * LAND_BYTES + SPLIT_GROUPS * HL_BYTES <= RING_BYTES, "FP32 rings");
constexpr int STAGING = EPI_WARPS * 32 * 32 * 4;        // a 32 x 32 tile per epilogue warp
constexpr int BAR_BYTES = 512;
constexpr int SMEM = 1024 + RING_BYTES + STAGING + BAR_BYTES;
static_assert(SMEM <= 232448, "shared memory of a CTA");
constexpr int CHUNK_STAGES = 2;                         // FP32: K_CHUNK = 64
constexpr int A_COL = 256;                              // FP32: TMEM columns of A's slots (64 each: hi, lo)

__host__ __device__ constexpr int threads(bool split) { return 32 * (2 + EPI_WARPS + (split ? SPLIT_WARPS : 0)); }

struct Plan {
  long long M, items;
  int N, nk, per, bn, mtiles, ntiles, splits;    // nk k-stages, `per` of them per split
  int a_mn, b_mn, stages;
  int kind;                                      // 0: f16 / bf16, 1: e4m3
  uint32_t idesc;
  float* part;                                   // [splits][M][N] or null
  int vec;                                       // rows of y, z and residual allow 16-byte accesses
};

__device__ __forceinline__ uint64_t sdesc_mn(uint32_t addr, uint32_t chunk_bytes) {
  // mn-major, 128-byte swizzle: 64-element runs of mn chunk_bytes apart, 8-k groups 1024 B apart
  return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(chunk_bytes >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(acc));
}
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d), "l"(a), "l"(b), "r"(id), "r"(acc));
}
// A in TMEM (128 lanes = rows, one 32-bit column per k)
__device__ __forceinline__ void mma_tf32_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::tf32 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d), "r"(a), "l"(b), "r"(id), "r"(acc));
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
      ::"r"(taddr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
        "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]),
        "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]),
        "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]), "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31])
      : "memory");
}

// 32 k of row r of a landed FP32 stage: k-major rows of 128 bytes (128-byte swizzle), or mn-major,
// [32 k][width] without a swizzle (a warp then reads 32 neighbouring floats at a time)
__device__ __forceinline__ void read_row(const unsigned char* src, int r, int mn, int width, float (&v)[32]) {
  if (!mn) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float4 a = *reinterpret_cast<const float4*>(src + r * 128 + ((j ^ (r & 7)) << 4));
      v[4 * j] = a.x; v[4 * j + 1] = a.y; v[4 * j + 2] = a.z; v[4 * j + 3] = a.w;
    }
  } else {
    const float* f = reinterpret_cast<const float*>(src) + r;
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = f[k * width];
  }
}

// ------------------------------------------------------------------ rows of a 32 x 32 tile
// v: the accumulator's row m0 + lane, columns n0 .. n0 + 31.  The tile is turned through the warp's staging
// (16-byte chunks XORed with the row) so that a row's lanes access whole segments of memory.
template <typename T>
__device__ __forceinline__ void out_vec(const dense::Epi& e, long long M, int N, long long m0, int n0, const float* stg, int lane) {
  constexpr int V = 16 / sizeof(T), L = 32 / V;          // elements and lanes of a row segment
  const int c = (lane % L) * V, n = n0 + c;
  if (n >= N) return;                                    // N is a multiple of V
  float b[V], ws[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    b[i] = e.bias ? load_any(e.bias, n + i, e.bias_dtype) : 0.f;
    ws[i] = e.w_scale ? e.w_scale[n + i] : 1.f;
  }
#pragma unroll
  for (int k = 0; k < 32; k += 32 / L) {
    const int r = k + lane / L;
    const long long m = m0 + r;
    if (m >= M) break;
    float v[V];
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 a = *reinterpret_cast<const float4*>(stg + r * 32 + (((c + i) / 4) ^ (r & 7)) * 4);
      v[i] = a.x; v[i + 1] = a.y; v[i + 2] = a.z; v[i + 3] = a.w;
    }
    if (e.x_scale) {
      const float xs = e.x_scale[m];
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] *= xs * ws[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += b[i];
    if (e.z) store_v<T, V>(static_cast<T*>(e.z) + m * e.ldz + n, v);
    if (e.act == EMP_ACT_SILU) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = silu_fast(v[i]);
    } else if (e.act == EMP_ACT_GELU) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = act_f(EMP_ACT_GELU, v[i]);
    }
    if (e.residual) {
      float a[V];
      load_v<T, V>(static_cast<const T*>(e.residual) + m * e.ldr + n, a);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] += a[i];
    }
    store_v<T, V>(static_cast<T*>(e.y) + m * e.ldy + n, v);
  }
}

__device__ __forceinline__ void out_tile(const Plan& p, const dense::Epi& e, int split, long long m0, int n0, const float (&v)[32],
                                         float* stg, int lane) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<float4*>(stg + lane * 32 + ((j ^ (lane & 7)) << 2)) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  __syncwarp();
  if (p.part) {
    float* o = p.part + (size_t)split * p.M * p.N;
    const int n = n0 + lane;
    if (n < p.N)
      for (int r = 0; r < 32 && m0 + r < p.M; ++r) o[(size_t)(m0 + r) * p.N + n] = stg[r * 32 + (((lane >> 2) ^ (r & 7)) << 2) + (lane & 3)];
  } else if (p.vec) {
    if (e.y_dtype == EMP_F32) out_vec<float>(e, p.M, p.N, m0, n0, stg, lane);
    else if (e.y_dtype == EMP_BF16) out_vec<__nv_bfloat16>(e, p.M, p.N, m0, n0, stg, lane);
    else out_vec<__half>(e, p.M, p.N, m0, n0, stg, lane);
  } else {
    const int n = n0 + lane;
    if (n < p.N)
      for (int r = 0; r < 32 && m0 + r < p.M; ++r) dense::put_one(e, m0 + r, n, stg[r * 32 + (((lane >> 2) ^ (r & 7)) << 2) + (lane & 3)]);
  }
  __syncwarp();
}

struct Item {
  int split, k_first, k_n, n0;
  long long m0;
};
__device__ __forceinline__ Item item_at(const Plan& p, long long w) {
  Item t;
  const int nt = (int)(w % p.ntiles);
  const long long q = w / p.ntiles;
  t.n0 = nt * p.bn;
  t.m0 = (q % p.mtiles) * BM;
  t.split = (int)(q / p.mtiles);
  t.k_first = t.split * p.per;
  t.k_n = min(p.per, p.nk - t.k_first);
  return t;
}

template <bool SPLIT>
__global__ void __launch_bounds__(threads(SPLIT), 1)
    k_dense_tc(const Plan p, const dense::Epi e, const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb) {
  extern __shared__ __align__(1024) unsigned char dtc_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(dtc_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* hl = sm + LAND * LAND_BYTES;                           // FP32: B's hi and lo
  float* staging = reinterpret_cast<float*>(sm + RING_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + RING_BYTES + STAGING);   // [MAX_STAGES] landed
  uint64_t* empty = full + MAX_STAGES;                                  // [MAX_STAGES] read
  uint64_t* sfull = empty + MAX_STAGES;                                 // [SPLIT_GROUPS] hi and lo written
  uint64_t* sempty = sfull + SPLIT_GROUPS;                              // [SPLIT_GROUPS] MMAs done with them
  uint64_t* acc_full = sempty + SPLIT_GROUPS;                           // [2]
  uint64_t* acc_empty = acc_full + 2;                                   // [2]
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = SPLIT ? LAND : p.stages;
  const int stage_bytes = SPLIT ? LAND_BYTES : A_BYTES + p.bn * 128;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], SPLIT ? 4 : 1);
    }
    for (int s = 0; s < SPLIT_GROUPS; ++s) {
      tc::mbar_init(&sfull[s], 4);
      tc::mbar_init(&sempty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&acc_full[b], 1);
      tc::mbar_init(&acc_empty[b], EPI_WARPS);
    }
    tc::mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_u32(tmem_slot)), "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0 && lane == 0) {
    // ---------------------------------------------------------------- TMA producer
    long long it = 0;
    bool ok = true;
    const int kw = SPLIT ? 32 : p.kind ? 128 : 64;                       // k of a stage
    for (long long w = blockIdx.x; w < p.items && ok; w += gridDim.x) {
      const Item t = item_at(p, w);
      for (int k = 0; k < t.k_n; ++k, ++it) {
        const int s = (int)(it % stages);
        if (it >= stages && !tc::mbar_wait(&empty[s], (uint32_t)(((it / stages) - 1) & 1))) { ok = false; break; }
        unsigned char* a = sm + s * stage_bytes;
        unsigned char* b = a + A_BYTES;
        const int k0 = (t.k_first + k) * kw;
        tc::mbar_expect_tx(&full[s], A_BYTES + p.bn * 128);
        if (SPLIT || !p.a_mn) {
          tc::tma_load(a, &ma, &full[s], p.a_mn ? (int)t.m0 : k0, p.a_mn ? k0 : (int)t.m0);
        } else {
          tc::tma_load(a, &ma, &full[s], (int)t.m0, k0);
          tc::tma_load(a + 8192, &ma, &full[s], (int)t.m0 + 64, k0);
        }
        if (SPLIT || !p.b_mn) {
          tc::tma_load(b, &mb, &full[s], p.b_mn ? t.n0 : k0, p.b_mn ? k0 : t.n0);
        } else {
          for (int c = 0; c < p.bn; c += 64) tc::tma_load(b + c * 128, &mb, &full[s], t.n0 + c, k0);
        }
      }
    }
    // copies in flight can only be among the last `stages`
    for (long long j = it > stages ? it - stages : 0; j < it; ++j) tc::mbar_wait(&full[j % stages], (uint32_t)((j / stages) & 1));
  } else if (warp == 1 && lane == 0) {
    // ---------------------------------------------------------------- MMA issuer
    long long it = 0, ch = 0;
    bool ok = true;
    for (long long w = blockIdx.x; w < p.items && ok; w += gridDim.x) {
      const Item t = item_at(p, w);
      uint32_t d = 0;
      for (int k = 0; k < t.k_n; ++k, ++it) {
        const bool first = SPLIT ? k % CHUNK_STAGES == 0 : k == 0;
        const bool last = k == t.k_n - 1 || (SPLIT && k % CHUNK_STAGES == CHUNK_STAGES - 1);
        const int buf = (int)(ch & 1);
        if (first) {
          if (ch >= 2 && !tc::mbar_wait(&acc_empty[buf], (uint32_t)(((ch >> 1) - 1) & 1))) { ok = false; break; }
          d = tmem + (uint32_t)(buf * (SPLIT ? 128 : 256));
        }
        if (SPLIT) {
          const int g = (int)(it % SPLIT_GROUPS);
          if (!tc::mbar_wait(&sfull[g], (uint32_t)((it / SPLIT_GROUPS) & 1))) { ok = false; break; }
          tc::fence_after();
          const uint32_t ahi = tmem + A_COL + g * 64, alo = ahi + 32;
          const uint32_t bhi = tc::smem_u32(hl + g * HL_BYTES), blo = bhi + A_BYTES;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            mma_tf32_ts(d, alo + kk * 8, tc::sdesc128(bhi + kk * 32), p.idesc, !(first && kk == 0));
            mma_tf32_ts(d, ahi + kk * 8, tc::sdesc128(blo + kk * 32), p.idesc, 1u);
          }
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma_tf32_ts(d, ahi + kk * 8, tc::sdesc128(bhi + kk * 32), p.idesc, 1u);
          commit(&sempty[g]);
        } else {
          const int s = (int)(it % stages);
          if (!tc::mbar_wait(&full[s], (uint32_t)((it / stages) & 1))) { ok = false; break; }
          tc::fence_after();
          const uint32_t a = tc::smem_u32(sm + s * stage_bytes), b = a + A_BYTES;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {             // 32 bytes of k each (mn-major: 16 k rows of 128 bytes)
            const uint64_t da = p.a_mn ? sdesc_mn(a + kk * 2048, 8192) : tc::sdesc128(a + kk * 32);
            const uint64_t db = p.b_mn ? sdesc_mn(b + kk * 2048, 8192) : tc::sdesc128(b + kk * 32);
            if (p.kind) mma_f8(d, da, db, p.idesc, !(first && kk == 0));
            else mma_f16(d, da, db, p.idesc, !(first && kk == 0));
          }
          commit(&empty[s]);
        }
        if (last) {
          commit(&acc_full[buf]);
          ++ch;
        }
      }
    }
    commit(drain);
    tc::mbar_wait(drain, 0);
  } else if (warp >= 2 && warp < 2 + EPI_WARPS) {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3, half = (warp - 2) >> 2;          // TMEM lanes q * 32 ..; chunks half, half + 2, ...
    float* stg = staging + (warp - 2) * 32 * 32;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
    const int nch = p.bn / 32;
    long long ch = 0;
    bool ok = true;
    for (long long w = blockIdx.x; w < p.items && ok; w += gridDim.x) {
      const Item t = item_at(p, w);
      const long long m0 = t.m0 + q * 32;
      if (SPLIT) {
        float acc[2][32];
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[0][i] = acc[1][i] = 0.f;
        for (int k = 0; k < t.k_n; k += CHUNK_STAGES, ++ch) {
          const int buf = (int)(ch & 1);
          if (!__all_sync(0xffffffffu, tc::mbar_wait(&acc_full[buf], (uint32_t)((ch >> 1) & 1)))) { ok = false; break; }
          tc::fence_after();
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (half + 2 * c < nch) {
              float v[32];
              tc::tmem_ld32(lanes + (uint32_t)(buf * 128 + (half + 2 * c) * 32), v);
#pragma unroll
              for (int i = 0; i < 32; ++i) acc[c][i] += v[i];
            }
          }
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&acc_empty[buf]);
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (half + 2 * c < nch) out_tile(p, e, t.split, m0, t.n0 + (half + 2 * c) * 32, acc[c], stg, lane);
      } else {
        const int buf = (int)(ch & 1);
        if (!__all_sync(0xffffffffu, tc::mbar_wait(&acc_full[buf], (uint32_t)((ch >> 1) & 1)))) break;
        tc::fence_after();
#pragma unroll 1
        for (int c = half; c < nch; c += 2) {
          float v[32];
          tc::tmem_ld32(lanes + (uint32_t)(buf * 256 + c * 32), v);
          if (c + 2 >= nch) {                                // the last read of this accumulator
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&acc_empty[buf]);
          }
          out_tile(p, e, t.split, m0, t.n0 + c * 32, v, stg, lane);
        }
        ++ch;
      }
    }
  } else if (SPLIT && warp >= 2 + EPI_WARPS) {
    // ---------------------------------------------------------------- split warps: group g takes stages g, g + 2, ...
    const int sw = warp - (2 + EPI_WARPS), g = sw >> 2, q = warp & 3;
    const int r = q * 32 + lane;                             // row of A (its TMEM lane) and of B
    const uint32_t ta = tmem + ((uint32_t)(q * 32) << 16) + A_COL + g * 64;
    unsigned char* bhi = hl + g * HL_BYTES;
    long long it = 0;
    bool ok = true;
    for (long long w = blockIdx.x; w < p.items && ok; w += gridDim.x) {
      const Item t = item_at(p, w);
      for (int k = 0; k < t.k_n; ++k, ++it) {
        if (it % SPLIT_GROUPS != g) continue;
        const int s = (int)(it % LAND);
        const long long u = it / SPLIT_GROUPS;
        // first this group's slot (its stage it - 2 multiplied, hence every stage up to it - 2 read), then the
        // landing: stage it - 3, the one before in the same place, has then landed, and the parity is unambiguous
        if (u >= 1 && !__all_sync(0xffffffffu, tc::mbar_wait(&sempty[g], (uint32_t)((u - 1) & 1)))) { ok = false; break; }
        if (!__all_sync(0xffffffffu, tc::mbar_wait(&full[s], (uint32_t)((it / LAND) & 1)))) { ok = false; break; }
        tc::fence_after();
        const unsigned char* land = sm + s * LAND_BYTES;
        float v[32], h[32];
        read_row(land, r, p.a_mn, BM, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) h[i] = tf32_rna(v[i]);
        tmem_st32(ta, h);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = tf32_rna(v[i] - h[i]);
        tmem_st32(ta + 32, v);
        if (r < p.bn) {
          read_row(land + A_BYTES, r, p.b_mn, p.bn, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float4 hi, lo;
            hi.x = tf32_rna(v[4 * j]);     lo.x = tf32_rna(v[4 * j] - hi.x);
            hi.y = tf32_rna(v[4 * j + 1]); lo.y = tf32_rna(v[4 * j + 1] - hi.y);
            hi.z = tf32_rna(v[4 * j + 2]); lo.z = tf32_rna(v[4 * j + 2] - hi.z);
            hi.w = tf32_rna(v[4 * j + 3]); lo.w = tf32_rna(v[4 * j + 3] - hi.w);
            const int o = r * 128 + ((j ^ (r & 7)) << 4);
            *reinterpret_cast<float4*>(bhi + o) = hi;
            *reinterpret_cast<float4*>(bhi + A_BYTES + o) = lo;
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&empty[s]);
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sfull[g]);
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
  }
}

// ------------------------------------------------------------------ host side
inline CUtensorMapDataType map_type(int t) {
  return t == EMP_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
       : t == EMP_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
       : t == EMP_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
}
// rows of `cols` contiguous elements; a box of [rows_box][cols_box]
inline bool make_map(CUtensorMap* m, const void* base, int t, long long cols, long long rows, long long ld, int cols_box,
                     int rows_box, bool swizzle) {
  auto fn = tc::encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld * dtype_size(t)};
  cuuint32_t box[2] = {(cuuint32_t)cols_box, (cuuint32_t)rows_box};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, map_type(t), 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// TMA reads rows whose start and pitch are multiples of 16 bytes
inline bool tma_ok(const void* p, long long ld, int t) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * dtype_size(t) % 16 == 0;
}

// Tile width and splits of the k axis of an M x N product with K summed.
struct Shape {
  int bn, splits, per, nk, mtiles, ntiles;
};
inline Shape shape_for(long long M, int N, long long K, int t) {
  Shape s;
  const int kw = 128 / dtype_size(t);
  s.nk = (int)((K + kw - 1) / kw);
  s.mtiles = (int)((M + BM - 1) / BM);
  const int sms = tc::num_sms();
  s.bn = N <= 64 ? 64 : N <= 128 || t == EMP_F32 ? 128 : 256;
  // too few tiles for the SMs: a short k axis gets narrower tiles, a long one is split
  auto tiles = [&] { return (long long)s.mtiles * ((N + s.bn - 1) / s.bn); };
  while (s.nk < 64 && s.bn > 64 && tiles() < sms) s.bn /= 2;
  s.ntiles = (N + s.bn - 1) / s.bn;
  // enough items for every SM, each at least eight stages long
  long long want = tiles() >= sms ? 1 : (sms + tiles() - 1) / tiles();
  want = std::max<long long>(1, std::min<long long>(want, s.nk / 8));
  s.per = (int)((s.nk + want - 1) / want);
  s.splits = (s.nk + s.per - 1) / s.per;
  return s;
}

// A k-major: rows [M][K] with pitch lda; mn-major: [K][M].  B likewise with N.  Both TMA-readable.
struct Operand {
  const void* p;
  long long ld;
  int mn;
};
inline int launch(long long M, int N, long long K, int t, const Operand& a, const Operand& b, const dense::Epi& e, const Shape& h,
                  float* part, bool vec, cudaStream_t st) {
  const int es = dtype_size(t), kw = 128 / es;
  const bool split = t == EMP_F32;
  Plan p{};
  p.M = M; p.N = N; p.nk = h.nk; p.per = h.per; p.bn = h.bn; p.mtiles = h.mtiles; p.ntiles = h.ntiles; p.splits = h.splits;
  p.items = (long long)h.mtiles * h.ntiles * h.splits;
  p.a_mn = a.mn; p.b_mn = b.mn;
  p.stages = std::min(MAX_STAGES, RING_BYTES / (A_BYTES + h.bn * 128));
  p.kind = t == EMP_E4M3;
  const uint32_t fmt = t == EMP_F32 ? 2 : t == EMP_BF16 ? 1 : 0;
  p.idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)(h.bn >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
  if (!split) p.idesc |= ((uint32_t)a.mn << 15) | ((uint32_t)b.mn << 16);
  p.part = part;
  p.vec = vec;
  CUtensorMap ma, mb;
  const bool ok_a = a.mn ? make_map(&ma, a.p, t, M, K, a.ld, split ? BM : 64, kw, !split) : make_map(&ma, a.p, t, K, M, a.ld, kw, BM, true);
  const bool ok_b = b.mn ? make_map(&mb, b.p, t, N, K, b.ld, split ? h.bn : 64, kw, !split) : make_map(&mb, b.p, t, K, N, b.ld, kw, h.bn, true);
  if (!ok_a || !ok_b) return EMP_ERR_CUDA;
  const unsigned grid = (unsigned)std::min<long long>(p.items, tc::num_sms());
  if (split) k_dense_tc<true><<<grid, threads(true), SMEM, st>>>(p, e, ma, mb);
  else k_dense_tc<false><<<grid, threads(false), SMEM, st>>>(p, e, ma, mb);
  return cudaGetLastError() == cudaSuccess ? EMP_OK : EMP_ERR_CUDA;
}

// once per device
inline int init() {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || !tc::encode_fn()) return EMP_ERR_UNSUPPORTED;
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load() & bit)) return EMP_OK;
  EMP_CUDA_TRY(cudaFuncSetAttribute(k_dense_tc<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM));
  EMP_CUDA_TRY(cudaFuncSetAttribute(k_dense_tc<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM));
  done.fetch_or(bit);
  return EMP_OK;
}

}  // namespace dtc
}  // namespace emp
