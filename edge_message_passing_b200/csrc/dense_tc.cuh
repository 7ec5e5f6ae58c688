// The dense layer's products on the tensor cores (tcgen05, sm_100a):
//
//   out[m][n] = sum_k A(m, k) B(n, k),
//
// with A and B each stored with k contiguous ("k-major": x, W, and g in g_x = gz W) or with the other
// index contiguous ("mn-major": W in g_x, both operands of g_W = gz^T x), and the dense layer's epilogue.
//
// Persistent kernel, one CTA per SM, 128 x bn tiles (bn a multiple of 32, up to 256 or in FP32 128) taken round-robin with n
// fastest, so that neighbouring CTAs share an A tile in L2.  A long k axis with few tiles is split:
// each split leaves a partial product, and k_join adds them in order.  Warps: one issues TMA loads, one
// the MMAs, 8 or 16 drain the accumulators (two or four per TMEM lane quarter) and write the rows.
//
// bf16, fp16 and e4m3 operands go from TMA straight to the MMA: a ring of stages of 128 bytes of k
// (128-byte swizzle), two accumulators of bn columns, so the epilogue of a tile overlaps the next
// tile's products.  Bound by shared memory, which takes every operand byte in and gives it out once: 16384 x 2048 -> 2048 in bf16
// 98 us, 1400 TFLOP/s (85 % of the measured rate; 106 us on rotating inputs; the tensor pipe is active 70 % of the time); 65536 x 2048
// -> 512 in e4m3 with SiLU and residual 94 us among other calls, 1460 TFLOP/s (the kernel alone 75), with half of its time per tile
// in the epilogue's exchange with memory.
//
// FP32 operands are split a = hi + lo (hi = RN_tf32(a), lo = RN_tf32(a - hi)) inside the kernel, by two
// groups of four warps that take the 32-wide k stages in turn, so neither operand needs a pass of its
// own over memory: A's split goes to TMEM (the MMA's A operand may live there, and a thread's TMEM
// lane is its row, whichever way A is stored), B's to shared memory.  The tensor cores add into their
// FP32 accumulator by truncation, which shrinks a sum by about 2e-8 of itself per MMA (measured on the
// SO(2) products: 7e-9 K).  So an accumulator takes K_CHUNK = 96 of k only and is then added, rounded
// to nearest, to sums in the epilogue warps' registers, and within each stage the small products
// lo.hi and hi.lo come before hi.hi.  Bound by the split (16 instructions per 4 elements and lane) and the epilogue's
// additions: 161792 x 512 -> 512 takes 408 us, 208 TFLOP/s of products (two thirds of what three TF32 products
// allow), 429 us on rotating inputs.  Spills 12 bytes with TMA rows, 112 without.
//
// FP32 with k of one chunk (SHORT) needs no sums in registers.  A CTA stays on one column of tiles, so that B is split
// once and kept, and the two halves of the epilogue's warps take every other tile each: a warp's way through a
// tile is latency (TMEM, staging, the store's read) as much as instructions (647168 x 64 -> 512 with SiLU on one buffer 340 us
// with all warps on each tile, 322 us thus; among other calls 389 us, 3.8 TB/s; 16-bit operands, whose epilogue overlaps more stages, gain nothing
// and 8-bit ones lose: 77 and 87 us at 65536 x 2048 -> 512).  Bound by the instructions of split and epilogue together.
//
// Every mbarrier wait is bounded; the producer waits out its own copies before exit.
#pragma once
#include <atomic>
#include <type_traits>
#include "so2_tc.cuh"
#include "dense.cuh"
#include "steps.cuh"

namespace emp {
namespace dtc {

constexpr int BM = 128;
constexpr int SPLIT_GROUPS = 2, SPLIT_WARPS = 4 * SPLIT_GROUPS;
constexpr int A_BYTES = BM * 128;                       // one stage of A
constexpr int MAX_STAGES = 8, MAX_EPI = 16;
constexpr int HL_BYTES = 2 * A_BYTES;                   // hi and lo of a stage of B
constexpr int CHUNK_STAGES = 3;                         // FP32: K_CHUNK = 96
constexpr int A_COL = 256;                              // FP32: TMEM columns of A's slots (64 each: hi, lo)

// The kernel's forms: 16- and 8-bit operands; FP32; FP32 with k of one chunk at most.  SHORT keeps no sums in
// registers, and each of its CTAs stays on one column of tiles, whose B is split once and kept.
enum Path { DIRECT, SPLIT, SHORT };

// T: the type of y, z and residual; ROWS: their rows by TMA; SCALED: 8-bit operands with scales.
// Epilogue warps: an epilogue warp issues an instruction every nine cycles or so, so short k is bound by how
// many there are: 16 where registers (65536 over the CTA) and staging (a tile of 32 x 32 each) allow, else 8.
template <Path PATH, typename T, bool ROWS, bool SCALED>
struct Cfg {
  static constexpr bool FP32 = PATH != DIRECT;
  static constexpr int EPI = PATH == SHORT || (ROWS && !SCALED) ? 16 : 8;
  static constexpr int SETS = PATH == SHORT ? 2 : 1;    // of epilogue warps, which take the tiles in turn
  static constexpr int W = PATH == SPLIT && ROWS ? 16 : 32;                   // columns put out at once (staging)
  static constexpr int LAND = 3, SLOTS = 3;             // FP32: stages as they land (A and B; A alone in SHORT) and split
  static constexpr int LAND_BYTES = PATH == SHORT ? A_BYTES : 2 * A_BYTES;
  // A's split is in TMEM, B's hi and lo in shared memory: a place per slot, or per stage of the whole k in SHORT
  static constexpr int RING_BYTES = FP32 ? LAND * LAND_BYTES + (PATH == SHORT ? CHUNK_STAGES : SLOTS) * HL_BYTES : 4 * (A_BYTES + 256 * 128);
  static constexpr int PLACE_BYTES = ROWS ? 32 * W * (int)sizeof(T) : 4096;
  static constexpr int PLACES = EPI == 8 && PLACE_BYTES == 2048 ? 2 : 1;      // of a warp
  static constexpr int STAGING = EPI * PLACES * PLACE_BYTES;
  static constexpr int BIAS = EPI * W * (SCALED ? 4 : (int)sizeof(T));
  static constexpr int BARS = 640;
  static constexpr int SMEM = 1024 + RING_BYTES + STAGING + BIAS + BARS;
  static constexpr int THREADS = 32 * (2 + EPI + (FP32 ? SPLIT_WARPS : 0));
  static_assert(SMEM <= 232448, "shared memory of a CTA");
  static_assert(A_COL + SLOTS * 64 <= 512, "TMEM columns");
  static_assert(LAND >= SLOTS, "order of the split warps' two waits");
};

struct Plan {
  long long M, items;
  int N, nk, per, bn, mtiles, ntiles, splits;    // nk k-stages, `per` of them per split
  int step_n, step_m, step_s;                    // the grid's size in tiles of n, m and splits
  int a_mn, b_mn, stages;
  uint32_t idesc;
  float* part;                                   // [splits][M][N] or null
};

// Shared-memory matrix descriptors, 128-byte swizzle.  k-major: rows of 128 bytes of k, 8-row groups 1024 B
// apart; mn-major: 64-element runs of mn 8192 B apart, 8-k groups 1024 B apart.  The upper word is the same;
// the lower one is the address / 16 and the distance of the runs, and moves by a constant per MMA of
// 32 bytes of k (k-major) or 16 k rows (mn-major).  The issuing warp only adds: it is alone on its critical path.
constexpr uint32_t DESC_HI = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, int mn) {
  return ((addr >> 4) & 0x3FFF) | ((mn ? 8192u >> 4 : 1u) << 16);
}
__device__ __forceinline__ uint64_t desc(uint32_t lo) { return ((uint64_t)DESC_HI << 32) | lo; }
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
  return p != 0;
}
template <bool F8>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t id, uint32_t acc) {
  if constexpr (F8)
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d), "l"(desc(a_lo)), "l"(desc(b_lo)), "r"(id), "r"(acc));
  else
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d), "l"(desc(a_lo)), "l"(desc(b_lo)), "r"(id), "r"(acc));
}
// A in TMEM (128 lanes = rows, one 32-bit column per k)
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t id, uint32_t acc) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
               "tcgen05.mma.cta_group::1.kind::tf32 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d), "r"(a), "l"(desc(b_lo)), "r"(id), "r"(acc));
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}
// Bounded wait.  A waiting warp is put to sleep by the hardware until the phase completes or WAIT_NS have
// passed: eighteen warps polling would take issue slots from the ones at work.
constexpr uint32_t WAIT_NS = 20000;
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  do {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}\n"
                 : "=r"(ok) : "r"(tc::smem_u32(bar)), "r"(parity), "r"(WAIT_NS) : "memory");
    if (ok) return true;
  } while (clock64() - t0 <= tc::g_wait_cycles);
  set_device_error(DEV_ERR_TIMEOUT);
  return false;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      ::"r"(taddr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
        "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr) : "memory");
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
// The accumulator comes a row per lane.  Where TMA can write the rows of y, a lane finishes its row's 32
// columns, packs them into the warp's staging (swizzled) and one TMA store writes the tile; the residual
// comes into the same place by a TMA load beforehand (one chunk ahead of its use for 16-bit types, which
// have two places), so the epilogue waits for no load and issues no addresses.
__device__ __forceinline__ void tma_store(const CUtensorMap* map, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];\n\t"
               "cp.async.bulk.commit_group;"
               ::"l"(reinterpret_cast<uint64_t>(map)), "r"(tc::smem_u32(src)), "r"(x), "r"(y) : "memory");
}
template <int N>
__device__ __forceinline__ void stores_read() {            // all but the N latest stores have read their place
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// 16-byte chunk j of row r of a staged tile: rows of 64 or 128 bytes, with the swizzle of that width
template <int ROW_BYTES>
__device__ __forceinline__ uint4* staged(unsigned char* place, int r, int j) {
  return reinterpret_cast<uint4*>(ROW_BYTES == 128 ? place + r * 128 + ((j ^ (r & 7)) << 4) : place + r * 64 + (((j ^ (r >> 1)) & 3) << 4));
}

// Where it cannot (rows off 16-byte boundaries), the tile is turned through the staging (16-byte chunks XORed
// with the row) and a lane takes one column, R rows at a time: their residuals are loaded together, for R = 32 a chunk
// ahead of their use.
template <typename T, int R>
__device__ __forceinline__ void load_column(float (&res)[R], const dense::Epi& e, int rows, long long m0, int n, int N, int k0) {
  if (!e.residual || n >= N) return;
  const T* rp = static_cast<const T*>(e.residual) + (m0 + k0) * e.ldr + n;
#pragma unroll
  for (int k = 0; k < R; ++k, rp += e.ldr)
    if (k0 + k < rows) res[k] = to_f(*rp);
}
// v: rows k0 .. k0 + R of column n, scaled sums; v becomes y
template <typename T, int R>
__device__ __forceinline__ void finish_column(float (&v)[R], const float (&res)[R], const dense::Epi& e, int rows, long long m0, int n,
                                              int N, int k0) {
  if (e.z && n < N) {
    T* z = static_cast<T*>(e.z) + (m0 + k0) * e.ldz + n;
#pragma unroll
    for (int k = 0; k < R; ++k, z += e.ldz)
      if (k0 + k < rows) *z = from_f<T>(v[k]);
  }
  if (e.act == EMP_ACT_SILU) {
#pragma unroll
    for (int k = 0; k < R; ++k) v[k] = act<EMP_ACT_SILU, T>(v[k]);
  } else if (e.act == EMP_ACT_GELU) {
#pragma unroll
    for (int k = 0; k < R; ++k) v[k] = act<EMP_ACT_GELU, T>(v[k]);
  }
  if (e.residual) {
#pragma unroll
    for (int k = 0; k < R; ++k) v[k] += res[k];
  }
}
template <typename T, int R>
__device__ __forceinline__ void store_column(const float (&v)[R], const dense::Epi& e, int rows, long long m0, int n, int N, int k0) {
  if (n >= N) return;
  T* y = static_cast<T*>(e.y) + (m0 + k0) * e.ldy + n;
#pragma unroll
  for (int k = 0; k < R; ++k, y += e.ldy)
    if (k0 + k < rows) *y = from_f<T>(v[k]);
}

// a row per lane (v) into the warp's staging
__device__ __forceinline__ void stage_rows(const float (&v)[32], float* stg, int lane) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<float4*>(stg + lane * 32 + ((j ^ (lane & 7)) << 2)) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  __syncwarp();
}
__device__ __forceinline__ void store_part(float* o, long long M, int N, long long m0, int n0, const float* stg, int lane) {
  const int n = n0 + lane, rows = (int)(M - m0 < 32 ? M - m0 : 32);
  if (n >= N) return;
  o += m0 * N + n;
#pragma unroll 8
  for (int r = 0; r < rows; ++r, o += N) *o = stg[r * 32 + (((lane >> 2) ^ (r & 7)) << 2) + (lane & 3)];
}

// A CTA's items are blockIdx.x, blockIdx.x + gridDim.x, ...; the tile advances by the grid's own (n, m, split)
// digits with carries, without divisions.
// Position in a ring of n places: the place and the parity of its current use.
struct Ring {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void advance(int n) {
    if (++at == n) { at = 0; phase ^= 1; }
  }
};

struct Item {
  int nt, mt, split, k_first, k_n, n0;
  long long m0;
  __device__ __forceinline__ void set(const Plan& p) {
    n0 = nt * p.bn;
    m0 = (long long)mt * BM;
    k_first = split * p.per;
    k_n = min(p.per, p.nk - k_first);
  }
  __device__ __forceinline__ Item next(const Plan& p) const {
    Item t;
    t.nt = nt + p.step_n;
    t.mt = mt + p.step_m;
    t.split = split + p.step_s;
    if (t.nt >= p.ntiles) { t.nt -= p.ntiles; ++t.mt; }
    if (t.mt >= p.mtiles) { t.mt -= p.mtiles; ++t.split; }
    t.set(p);
    return t;
  }
};
__device__ __forceinline__ Item first_item(const Plan& p) {
  Item t;
  t.nt = (int)blockIdx.x % p.ntiles;
  const int q = (int)blockIdx.x / p.ntiles;
  t.mt = q % p.mtiles;
  t.split = q / p.mtiles;
  t.set(p);
  return t;
}

struct Maps {
  CUtensorMap a, b, y, z, res;
};

template <Path PATH, typename T, bool ROWS, bool SCALED>
__global__ void __launch_bounds__(Cfg<PATH, T, ROWS, SCALED>::THREADS, 1)
    k_dense_tc(const Plan p, const dense::Epi e, const __grid_constant__ Maps maps) {
  using C = Cfg<PATH, T, ROWS, SCALED>;
  constexpr bool FP32 = C::FP32;
  constexpr int EPI_WARPS = C::EPI, PER_QUARTER = EPI_WARPS / 4, LAND = C::LAND, SLOTS = C::SLOTS, LAND_BYTES = C::LAND_BYTES;
  extern __shared__ __align__(1024) unsigned char dtc_raw[];
  unsigned char* sm = dtc_raw + (1024 - (tc::smem_u32(dtc_raw) & 1023)) % 1024;
  unsigned char* hl = sm + LAND * LAND_BYTES;                           // FP32: B's hi and lo
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::RING_BYTES + C::STAGING + C::BIAS);   // [MAX_STAGES] landed
  uint64_t* empty = full + MAX_STAGES;                                  // [MAX_STAGES] read
  uint64_t* sfull = empty + MAX_STAGES;                                 // [SLOTS] hi and lo written
  uint64_t* sempty = sfull + SLOTS;                                     // [SLOTS] MMAs done with them
  uint64_t* acc_full = sempty + SLOTS;                                  // [2]
  uint64_t* acc_empty = acc_full + 2;                                   // [2]
  uint64_t* res_full = acc_empty + 2;                                   // [MAX_EPI][2] residual chunks landed
  uint64_t* b_full = res_full + 2 * MAX_EPI;                             // [CHUNK_STAGES] SHORT: B landed ...
  uint64_t* b_split = b_full + CHUNK_STAGES;                            // [CHUNK_STAGES] ... and split
  uint64_t* drain = b_split + CHUNK_STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stages = FP32 ? LAND : p.stages;
  const int stage_bytes = FP32 ? LAND_BYTES : A_BYTES + p.bn * 128;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], FP32 ? 4 : 1);
    }
    for (int i = 0; i < 2 * MAX_EPI; ++i) tc::mbar_init(&res_full[i], 1);
    for (int s = 0; s < SLOTS; ++s) {
      tc::mbar_init(&sfull[s], 4);
      tc::mbar_init(&sempty[s], 1);
    }
    for (int k = 0; k < CHUNK_STAGES; ++k) {
      tc::mbar_init(&b_full[k], 1);
      tc::mbar_init(&b_split[k], 4);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&acc_full[b], 1);
      tc::mbar_init(&acc_empty[b], EPI_WARPS / C::SETS);
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

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer (one elected lane issues)
    Ring ring;
    uint32_t it = 0;
    bool ok = true;
    const int kw = FP32 ? 32 : SCALED ? 128 : 64;                       // k of a stage
    const uint32_t bytes = A_BYTES + (PATH == SHORT ? 0 : p.bn * 128);
    Item t = first_item(p);
    if (PATH == SHORT && elect_one()) {
      for (int k = 0; k < p.nk; ++k) {                                   // B of this CTA's column of tiles
        tc::mbar_expect_tx(&b_full[k], p.bn * 128);
        tc::tma_load(hl + k * HL_BYTES, &maps.b, &b_full[k], p.b_mn ? t.n0 : k * kw, p.b_mn ? k * kw : t.n0);
      }
    }
    __syncwarp();
    for (long long w = blockIdx.x; w < p.items && ok; w += gridDim.x, t = t.next(p)) {
      int k0 = t.k_first * kw;
      const int m0 = (int)t.m0, n0 = t.n0;
      for (int k = 0; k < t.k_n; ++k, ++it, k0 += kw, ring.advance(stages)) {
        const int s = ring.at;
        if (it >= (uint32_t)stages && !__all_sync(0xffffffffu, wait(&empty[s], ring.phase ^ 1))) { ok = false; break; }
        if (elect_one()) {
          unsigned char* a = sm + s * stage_bytes;
          unsigned char* b = a + A_BYTES;
          uint64_t* bar = &full[s];
          tc::mbar_expect_tx(bar, bytes);
          if (!p.a_mn) {
            tc::tma_load(a, &maps.a, bar, k0, m0);
          } else {
            tc::tma_load(a, &maps.a, bar, m0, k0);
            if (!FP32) tc::tma_load(a + 8192, &maps.a, bar, m0 + 64, k0);
          }
          if (PATH == SHORT) {
          } else if (!p.b_mn) {
            tc::tma_load(b, &maps.b, bar, k0, n0);
          } else if (FP32) {
            tc::tma_load(b, &maps.b, bar, n0, k0);
          } else {
            for (int c = 0; c < p.bn; c += 64) tc::tma_load(b + c * 128, &maps.b, bar, n0 + c, k0);
          }
        }
        __syncwarp();
      }
    }
    if (PATH == SHORT)
      for (int k = 0; k < p.nk; ++k) wait(&b_full[k], 0);
    // copies in flight can only be among the last `stages`
    for (uint32_t j = it > (uint32_t)stages ? it - stages : 0; j < it; ++j) wait(&full[j % stages], (j / stages) & 1);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (one elected lane issues)
    Ring ring, acc;
    uint32_t ch = 0;
    bool ok = true;
    const int ring_n = FP32 ? SLOTS : stages;
    const uint32_t step16 = FP32 ? HL_BYTES >> 4 : stage_bytes >> 4;
    const uint32_t a0 = FP32 ? tmem + A_COL : desc_lo(tc::smem_u32(sm), p.a_mn);
    const uint32_t b0 = FP32 ? desc_lo(tc::smem_u32(hl), 0) : desc_lo(tc::smem_u32(sm + A_BYTES), p.b_mn);
    const uint32_t sa = p.a_mn ? 2048 >> 4 : 32 >> 4, sb = p.b_mn ? 2048 >> 4 : 32 >> 4;
    uint64_t* in = FP32 ? sfull : full;
    uint64_t* out = FP32 ? sempty : empty;
    const uint32_t id = p.idesc;
    Item t = first_item(p);
    for (long long w = blockIdx.x; w < p.items && ok; w += gridDim.x, t = t.next(p)) {
      uint32_t d = 0;
      for (int k = 0; k < t.k_n; ++k, ring.advance(ring_n)) {
        const bool first = FP32 ? k % CHUNK_STAGES == 0 : k == 0;
        const bool last = k == t.k_n - 1 || (FP32 && k % CHUNK_STAGES == CHUNK_STAGES - 1);
        if (first) {
          if (ch >= 2 && !__all_sync(0xffffffffu, wait(&acc_empty[acc.at], acc.phase ^ 1))) { ok = false; break; }
          d = tmem + (uint32_t)(acc.at * (FP32 ? 128 : 256));
        }
        const int s = ring.at;
        if (!__all_sync(0xffffffffu, wait(&in[s], ring.phase))) { ok = false; break; }
        if (PATH == SHORT && w == blockIdx.x && !__all_sync(0xffffffffu, wait(&b_split[k], 0))) { ok = false; break; }
        tc::fence_after();
        if (elect_one()) {
          const uint32_t b = b0 + (PATH == SHORT ? k : s) * step16;
          if (FP32) {
            const uint32_t hi = a0 + s * 64, lo = hi + 32, bl = b + (A_BYTES >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              mma_ts(d, lo + kk * 8, b + kk * 2, id, kk || !first);
              mma_ts(d, hi + kk * 8, bl + kk * 2, id, 1u);
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_ts(d, hi + kk * 8, b + kk * 2, id, 1u);
          } else {
            const uint32_t a = a0 + s * step16;
            mma_ss<SCALED>(d, a, b, id, !first);
            mma_ss<SCALED>(d, a + sa, b + sb, id, 1u);
            mma_ss<SCALED>(d, a + 2 * sa, b + 2 * sb, id, 1u);
            mma_ss<SCALED>(d, a + 3 * sa, b + 3 * sb, id, 1u);
          }
          commit(&out[s]);
          if (last) commit(&acc_full[acc.at]);
        }
        __syncwarp();
        if (last) {
          acc.advance(2);
          ++ch;
        }
      }
    }
    if (elect_one()) commit(drain);
    __syncwarp();
    wait(drain, 0);
  } else if (warp >= 2 && warp < 2 + EPI_WARPS) {
    // ---------------------------------------------------------------- epilogue
    constexpr int V = 16 / sizeof(T), W = C::W, ROW_BYTES = W * sizeof(T), PLACE_BYTES = C::PLACE_BYTES, PLACES = C::PLACES;
    using B = std::conditional_t<SCALED, float, T>;          // the bias's type
    constexpr int SETS = C::SETS, per = PER_QUARTER / SETS;
    const int set = ((warp - 2) >> 2) / per;
    const int q = warp & 3, sub = ((warp - 2) >> 2) % per;   // TMEM lanes q * 32 ..; chunks sub, sub + per, ...
    unsigned char* place = sm + C::RING_BYTES + (warp - 2) * PLACES * PLACE_BYTES;
    B* bsm = reinterpret_cast<B*>(sm + C::RING_BYTES + C::STAGING) + (warp - 2) * W;
    uint64_t* rbar = res_full + (warp - 2) * 2;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
    const int nch = p.bn / 32;
    uint32_t done = 0;                                       // pieces of W columns put through the places
    bool ok = true, asked = false;                           // asked: what the next chunk reads is on its way
    bool coming = false;                                     // a residual's TMA load, into place done % PLACES
    B bias_l = from_f<B>(0.f);
    float ws_l = 0.f, xs_l = 0.f;                            // of the next chunk: column lane's bias and scale, row lane's scale
    auto here = [&](const Item& t, int c) { return t.m0 + q * 32 < p.M && t.n0 + c * 32 < p.N; };
    constexpr int R = PATH == DIRECT ? 32 : 8;               // rows of a column at a time, without TMA
    float res[ROWS ? 2 : R];
    auto ask_residual = [&](const Item& t, int c, int h) {   // of piece h of the chunk; its place must be free
      if constexpr (!ROWS) {
        if (R == 32) load_column<T, R>(res, e, (int)min((long long)32, p.M - t.m0 - q * 32), t.m0 + q * 32, t.n0 + c * 32 + lane, p.N, 0);
      } else {
        coming = true;
        if (lane == 0) {
          const int pl = done % PLACES;
          tc::mbar_expect_tx(&rbar[pl], PLACE_BYTES);
          tc::tma_load(place + pl * PLACE_BYTES, &maps.res, &rbar[pl], t.n0 + c * 32 + h * W, (int)(t.m0 + q * 32));
        }
      }
    };
    // ask for what chunk c of an item needs
    auto ask = [&](const Item& t, int c) {
      const int n = t.n0 + c * 32 + lane;
      const long long m = t.m0 + q * 32 + lane;
      ws_l = xs_l = 0.f;
      bias_l = from_f<B>(0.f);
      if (n < p.N) {
        if (e.bias) bias_l = static_cast<const B*>(e.bias)[n];
        if (SCALED) ws_l = e.w_scale[n];
      }
      if (SCALED && m < p.M) xs_l = e.x_scale[m];
      if (e.residual && (!ROWS || !e.z)) ask_residual(t, c, 0);
      asked = true;
    };
    // piece h of the warp's rows, packed, into a place, and ready for a TMA store
    auto stage = [&](unsigned char* pp, const float (&v)[32], int h) {
#pragma unroll
      for (int j = 0; j < W / V; ++j) {
        float y[V];
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] = v[h * W + j * V + i];
        store_v<T, V>(reinterpret_cast<T*>(staged<ROW_BYTES>(pp, lane, j)), y);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
    };
    // chunk c of an item, a row per lane in v; `next` (chunk of item tn, or -1) is asked for on the way
    auto put = [&](const Item& t, int c, float (&v)[32], const Item& tn, int next) {
      const long long m0 = t.m0 + q * 32;
      const int n0 = t.n0 + c * 32;
      if (!ok || !here(t, c)) return;                        // (after a wait that ran out no further load is asked for)
      if constexpr (!ROWS) {
        float* stg = reinterpret_cast<float*>(place);
        stage_rows(v, stg, lane);
        if (p.part) {
          store_part(p.part + (size_t)t.split * p.M * p.N, p.M, p.N, m0, n0, stg, lane);
        } else {
          const int rows = (int)min((long long)32, p.M - m0), n = n0 + lane;
          if (!asked) ask(t, c);
          const float b = to_f(bias_l), ws = ws_l;
          asked = false;
#pragma unroll 1
          for (int k0 = 0; k0 < 32; k0 += R) {
            float u[R];
#pragma unroll
            for (int k = 0; k < R; ++k) {
              const int r = k0 + k;
              u[k] = stg[r * 32 + (((lane >> 2) ^ (r & 7)) << 2) + (lane & 3)];
              u[k] = SCALED ? fmaf(u[k], __shfl_sync(0xffffffffu, xs_l, r) * ws, b) : u[k] + b;
            }
            if (R < 32) load_column<T, R>(res, e, rows, m0, n, p.N, k0);
            finish_column<T, R>(u, res, e, rows, m0, n, p.N, k0);
            if (R == 32 && next >= 0 && here(tn, next)) ask(tn, next);
            store_column<T, R>(u, e, rows, m0, n, p.N, k0);
          }
        }
        __syncwarp();
        return;
      }
      // the place's last store has to have read it before it is written: before a residual comes (here or in the
      // prefetch below), else only before the finished rows go in
      const bool res_now = e.residual && !e.z;
      if (res_now && !asked && lane == 0) stores_read<PLACES - 1>();
      if (!asked) ask(t, c);
      const B bias = bias_l;
      const float ws = ws_l, xs = xs_l;
#pragma unroll
      for (int h = 0; h < 32 / W; ++h) {
        const int nh = n0 + h * W;
        if (h && nh >= p.N) break;
        const int pl = done % PLACES;
        unsigned char* pp = place + pl * PLACE_BYTES;
        if (h && res_now) {
          if (lane == 0) stores_read<PLACES - 1>();
          ask_residual(t, c, h);
        }
        if (SCALED || PATH == SPLIT || e.bias) {             // (SPLIT: a branch here costs spills)
          constexpr int VB = 16 / sizeof(B);
          if (W == 32 || lane / W == h) bsm[lane % W] = bias;
          __syncwarp();
#pragma unroll
          for (int j = 0; j < W; j += VB) {
            float b[VB];
            unpack16<B, VB>(*reinterpret_cast<const uint4*>(bsm + j), b);
#pragma unroll
            for (int i = 0; i < VB; ++i) {
              float& u = v[h * W + j + i];
              u = SCALED ? fmaf(u, xs * __shfl_sync(0xffffffffu, ws, h * W + j + i), b[i]) : u + b[i];
            }
          }
        }
        if (e.z) {                                           // z takes the place first, the residual after it
          if (lane == 0) stores_read<PLACES - 1>();
          __syncwarp();
          stage(pp, v, h);
          if (lane == 0) {
            tma_store(&maps.z, pp, nh, (int)m0);
            stores_read<0>();
          }
          __syncwarp();
          if (e.residual) ask_residual(t, c, h);
        }
        // each step for the whole piece: a branch per element would jump over the other activations' code every time
        if (e.act == EMP_ACT_SILU) {
#pragma unroll
          for (int i = 0; i < W; ++i) v[h * W + i] = act<EMP_ACT_SILU, T>(v[h * W + i]);
        } else if (e.act == EMP_ACT_GELU) {
#pragma unroll
          for (int i = 0; i < W; ++i) v[h * W + i] = act<EMP_ACT_GELU, T>(v[h * W + i]);
        }
        if (e.residual) {
          if (!__all_sync(0xffffffffu, wait(&rbar[pl], (uint32_t)((done / PLACES) & 1)))) { ok = false; return; }
          coming = false;
#pragma unroll
          for (int j = 0; j < W / V; ++j) {
            float a[V];
            unpack16<T, V>(*staged<ROW_BYTES>(pp, lane, j), a);
#pragma unroll
            for (int i = 0; i < V; ++i) v[h * W + j * V + i] += a[i];
          }
        }
        if (!res_now && !e.z) {
          if (lane == 0) stores_read<PLACES - 1>();
          __syncwarp();
        }
        stage(pp, v, h);
        if (lane == 0) tma_store(&maps.y, pp, nh, (int)m0);
        ++done;
      }
      asked = false;
      if (next >= 0 && here(tn, next)) {
        if (e.residual && !e.z && lane == 0) stores_read<PLACES - 1>();
        ask(tn, next);
      }
    };
    uint32_t ch = set;                                       // accumulators before the warp's next one
    const long long step = (long long)SETS * gridDim.x;
    Item t = first_item(p);
    if (set) t = t.next(p);
    const long long w0 = blockIdx.x + (long long)set * gridDim.x;
    if (!p.part && w0 < p.items && sub < nch && here(t, sub)) ask(t, sub);
    Item tn;
    for (long long w = w0; w < p.items && ok; w += step, t = tn) {
      const bool more = w + step < p.items;
      tn = t.next(p);
      if (SETS == 2) tn = tn.next(p);
      if constexpr (PATH == SPLIT) {
        constexpr int HELD = 4 / PER_QUARTER;                // chunks of a warp (bn is 128 at most)
        float acc[HELD][32];
#pragma unroll
        for (int c = 0; c < HELD; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[c][i] = 0.f;
        for (int k = 0; k < t.k_n; k += CHUNK_STAGES, ++ch) {
          const int buf = (int)(ch & 1);
          if (!__all_sync(0xffffffffu, wait(&acc_full[buf], (uint32_t)((ch >> 1) & 1)))) { ok = false; break; }
          tc::fence_after();
#pragma unroll
          for (int c = 0; c < HELD; ++c) {
            if (sub + PER_QUARTER * c < nch) {
#pragma unroll
              for (int j = 0; j < 32; j += 16) {
                float v[16];
                tmem_ld16(lanes + (uint32_t)(buf * 128 + (sub + PER_QUARTER * c) * 32 + j), v);
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[c][j + i] += v[i];
              }
            }
          }
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&acc_empty[buf]);
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < HELD; ++c) {
          const int at = sub + PER_QUARTER * c;
          if (at < nch) {
            const bool last = at + PER_QUARTER >= nch;
            put(t, at, acc[c], last ? tn : t, last ? (more ? sub : -1) : at + PER_QUARTER);
          }
        }
      } else {
        const int buf = (int)(ch & 1);
        if (!__all_sync(0xffffffffu, wait(&acc_full[buf], (uint32_t)((ch >> 1) & 1)))) break;
        tc::fence_after();
#pragma unroll 1
        for (int c = sub; c < nch; c += per) {
          float v[32];
          tc::tmem_ld32(lanes + (uint32_t)(buf * (FP32 ? 128 : 256) + c * 32), v);
          const bool last = c + per >= nch;
          if (last) {                                        // the last read of this accumulator
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&acc_empty[buf]);
          }
          put(t, c, v, last ? tn : t, last ? (more ? sub : -1) : c + per);
        }
        if (sub >= nch && lane == 0) tc::mbar_arrive(&acc_empty[buf]);   // a narrow tile has no chunk for this warp
        ch += SETS;
      }
    }
    if (ROWS) {
      if (coming) wait(&rbar[done % PLACES], (uint32_t)((done / PLACES) & 1));   // a load in flight (after a timeout)
      if (lane == 0) stores_read<0>();                       // the places outlive the stores' reads
    }
  } else if (FP32 && warp >= 2 + EPI_WARPS) {
    // ---------------------------------------------------------------- split warps: group g takes stages g, g + 2, ...
    const int sw = warp - (2 + EPI_WARPS), g = sw >> 2, q = warp & 3;
    const int r = q * 32 + lane;                             // row of A (its TMEM lane) and of B
    uint32_t it = 0;
    bool ok = true;
    Item t = first_item(p);
    // x (32 k of B's row r) as hi and lo, k-major, 128-byte swizzle
    auto split_b = [&](unsigned char* bhi, const float (&x)[32]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float4 hi, lo;
        hi.x = tf32_rna(x[4 * j]);     lo.x = tf32_rna(x[4 * j] - hi.x);
        hi.y = tf32_rna(x[4 * j + 1]); lo.y = tf32_rna(x[4 * j + 1] - hi.y);
        hi.z = tf32_rna(x[4 * j + 2]); lo.z = tf32_rna(x[4 * j + 2] - hi.z);
        hi.w = tf32_rna(x[4 * j + 3]); lo.w = tf32_rna(x[4 * j + 3] - hi.w);
        const int o = r * 128 + ((j ^ (r & 7)) << 4);
        *reinterpret_cast<float4*>(bhi + o) = hi;
        *reinterpret_cast<float4*>(bhi + A_BYTES + o) = lo;
      }
    };
    if constexpr (PATH == SHORT) {
      float x[32];                                          // B, in place: the whole stage is read before hi is written over it
      ok = in_place_stages(g, SPLIT_GROUPS, p.nk,
          [&](int k) { return __all_sync(0xffffffffu, wait(&b_full[k], 0)) != 0; },
          [&](int k) { if (r < p.bn) read_row(hl + k * HL_BYTES, r, p.b_mn, p.bn, x); },
          [&] { asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory"); },
          [&](int k) {
            if (r < p.bn) split_b(hl + k * HL_BYTES, x);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&b_split[k]);
          });
    }
    for (long long w = blockIdx.x; w < p.items && ok; w += gridDim.x, t = t.next(p)) {
      for (int k = 0; k < t.k_n; ++k, ++it) {
        if (it % SPLIT_GROUPS != g) continue;
        const int s = (int)(it % LAND), slot = (int)(it % SLOTS);
        const uint32_t ta = tmem + ((uint32_t)(q * 32) << 16) + A_COL + slot * 64;
        // first the slot (stage it - SLOTS multiplied, hence every stage before it landed), then the landing:
        // the stage before in the same place, it - LAND, has landed, so its phase's parity is unambiguous
        if (it >= SLOTS && !__all_sync(0xffffffffu, wait(&sempty[slot], (uint32_t)(((it / SLOTS) - 1) & 1)))) { ok = false; break; }
        if (!__all_sync(0xffffffffu, wait(&full[s], (uint32_t)((it / LAND) & 1)))) { ok = false; break; }
        tc::fence_after();
        const unsigned char* land = sm + s * LAND_BYTES;
        float v[32];
        read_row(land, r, p.a_mn, BM, v);
#pragma unroll
        for (int j = 0; j < 32; j += 16) {
          float h[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) h[i] = tf32_rna(v[j + i]);
          tmem_st16(ta + j, h);
#pragma unroll
          for (int i = 0; i < 16; ++i) h[i] = tf32_rna(v[j + i] - h[i]);
          tmem_st16(ta + 32 + j, h);
        }
        if (PATH == SPLIT && r < p.bn) {
          float x[32];
          read_row(land + A_BYTES, r, p.b_mn, p.bn, x);
          split_b(hl + slot * HL_BYTES, x);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        if (PATH == SPLIT) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc::fence_before();
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(&empty[s]);
          tc::mbar_arrive(&sfull[slot]);
        }
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
                     int rows_box, int swizzle_bytes) {
  auto fn = tc::encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld * dtype_size(t)};
  cuuint32_t box[2] = {(cuuint32_t)cols_box, (cuuint32_t)rows_box};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, map_type(t), 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : swizzle_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// TMA reads rows whose start and pitch are multiples of 16 bytes
inline bool tma_ok(const void* p, long long ld, int t) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * dtype_size(t) % 16 == 0;
}

// Tile width and splits of the k axis of an M x N product with K summed (each at least 1): those of the least estimated time (a width
// that divides N well against one that uses each operand byte more often).  A CTA's
// tile takes the longer of its k stages and its epilogue (which runs beside the next tile's stages), the CTAs work in
// waves, and splits pay for their partial products.  Microseconds as measured for the 16-bit and the FP32 kernel: a
// stage with the operands in L2, the epilogue of a tile with one stage.
constexpr int MAX_CHAIN = 1024;   // 4096 MMAs: a sum shrinks by 9e-5 of itself at most, a fortieth of a bf16 step
struct Shape {
  int bn, splits, per, nk, mtiles, ntiles;
};
inline Shape shape_for(long long M, int N, long long K, int t, int b_mn) {
  const int kw = 128 / dtype_size(t), sms = tc::num_sms();
  const bool fp32 = t == EMP_F32;
  Shape best{};
  double best_us = 0;
  const int unit = b_mn && !fp32 ? 64 : 32;              // columns come in chunks of 32, in mn-major runs of 64
  for (int bn = unit; bn <= (fp32 ? 128 : 256); bn += unit) {
    if (bn > unit && bn >= N + unit) break;
    const double stage = fp32 ? 0.30 + 0.0016 * bn : 0.095 + 0.00104 * bn, epi = fp32 ? 0.3 + 0.015 * bn : 0.7 + 0.0045 * bn;
    Shape s;
    s.bn = bn;
    s.nk = (int)((K + kw - 1) / kw);
    s.mtiles = (int)((M + BM - 1) / BM);
    s.ntiles = (N + bn - 1) / bn;
    const long long tiles = (long long)s.mtiles * s.ntiles;
    // one split, or as many as fill one to three waves of CTAs, of at least four stages each; in any case so many that
    // the 16-bit kernel's sums, which stay in the truncating accumulator, end after MAX_CHAIN stages
    const int least = fp32 ? 1 : (s.nk + MAX_CHAIN - 1) / MAX_CHAIN;
    for (int waves = 0; waves <= (tiles < 3 * sms ? 3 : 0); ++waves) {
      const long long want = waves == 0 ? least : std::min<long long>(waves * (long long)sms / tiles, s.nk / 4);
      if (want < least || (waves && want < 2)) continue;
      s.per = (int)((s.nk + want - 1) / want);
      s.splits = (s.nk + s.per - 1) / s.per;
      const long long items = tiles * s.splits;
      const double work = std::max(s.per * stage, epi);
      double us = (double)((items + sms - 1) / sms) * work + epi;
      if (s.splits > 1) us += 4.0 + 2.0 * 4e-6 * (double)s.splits * (double)M * (double)N / 5.0;   // the join, at 5 TB/s
      if (best_us == 0 || us < best_us) {
        best_us = us;
        best = s;
      }
    }
  }
  return best;
}

// A k-major: rows [M][K] with pitch lda; mn-major: [K][M].  B likewise with N.  Both TMA-readable.
struct Operand {
  const void* p;
  long long ld;
  int mn;
};
struct Launch {
  const Plan& p;
  const dense::Epi& e;
  const Maps& maps;
  unsigned grid;
  cudaStream_t st;
  template <Path PATH, typename T, bool ROWS, bool SCALED>
  int go() const {
    using C = Cfg<PATH, T, ROWS, SCALED>;
    auto k = k_dense_tc<PATH, T, ROWS, SCALED>;
    // the shared-memory limit is set once per device and kernel
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    EMP_CUDA_TRY(cudaGetDevice(&dev));
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev > 63 || !(done.load() & bit)) {
      EMP_CUDA_TRY(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM));
      done.fetch_or(bit);
    }
    k<<<grid, C::THREADS, C::SMEM, st>>>(p, e, maps);
    return cudaGetLastError() == cudaSuccess ? EMP_OK : EMP_ERR_CUDA;
  }
  template <Path PATH, typename T, bool SCALED>
  int rows(bool by_tma) const { return by_tma ? go<PATH, T, true, SCALED>() : go<PATH, T, false, SCALED>(); }
};
inline int launch(long long M, int N, long long K, int t, const Operand& a, const Operand& b, const dense::Epi& e, const Shape& h,
                  float* part, cudaStream_t st) {
  const int es = dtype_size(t), kw = 128 / es;
  const bool split = t == EMP_F32;
  Plan p{};
  p.M = M; p.N = N; p.nk = h.nk; p.per = h.per; p.bn = h.bn; p.mtiles = h.mtiles; p.ntiles = h.ntiles; p.splits = h.splits;
  p.items = (long long)h.mtiles * h.ntiles * h.splits;
  p.a_mn = a.mn; p.b_mn = b.mn;
  p.stages = std::min(MAX_STAGES, Cfg<DIRECT, float, true, true>::RING_BYTES / (A_BYTES + h.bn * 128));
  const uint32_t fmt = t == EMP_F32 ? 2 : t == EMP_BF16 ? 1 : 0;
  p.idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)(h.bn >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
  if (!split) p.idesc |= ((uint32_t)a.mn << 15) | ((uint32_t)b.mn << 16);
  p.part = part;
  Maps maps{};
  const bool ok_a = a.mn ? make_map(&maps.a, a.p, t, M, K, a.ld, split ? BM : 64, kw, 128 * !split) : make_map(&maps.a, a.p, t, K, M, a.ld, kw, BM, 128);
  const bool ok_b = b.mn ? make_map(&maps.b, b.p, t, N, K, b.ld, split ? h.bn : 64, kw, 128 * !split) : make_map(&maps.b, b.p, t, K, N, b.ld, kw, h.bn, 128);
  if (!ok_a || !ok_b) return EMP_ERR_CUDA;
  // SHORT: a whole number of CTAs per column of tiles, so that a CTA's column does not change
  const bool one_chunk = split && h.splits == 1 && h.nk <= CHUNK_STAGES && h.ntiles <= tc::num_sms();
  // rows of y, z and residual in boxes of 32 rows
  const int cols = split && !one_chunk ? Cfg<SPLIT, float, true, false>::W : 32;
  // A TMA store fills its last 16 bytes of a row with zeros where the tensor ends inside them, so rows have to be whole 16 bytes.
  const int ys = dtype_size(e.y_dtype);
  auto fits = [&](const void* q, long long ld) { return !q || tma_ok(q, M == 1 ? N : ld, e.y_dtype); };      // (one row: any pitch)
  const bool rows = !part && N * ys % 16 == 0 && fits(e.y, e.ldy) && fits(e.z, e.ldz) && fits(e.residual, e.ldr);
  if (rows) {
    auto map = [&](CUtensorMap* m, const void* q, long long ld) {
      return !q || make_map(m, q, e.y_dtype, N, M, M == 1 ? N : ld, cols, 32, cols * ys);
    };
    if (!map(&maps.y, e.y, e.ldy) || !map(&maps.z, e.z, e.ldz) || !map(&maps.res, e.residual, e.ldr)) return EMP_ERR_CUDA;
  }
  const int sms = tc::num_sms();
  const unsigned grid = (unsigned)std::min<long long>(p.items, one_chunk ? sms / h.ntiles * h.ntiles : sms);
  p.step_n = (int)(grid % p.ntiles);
  p.step_m = (int)(grid / p.ntiles % p.mtiles);
  p.step_s = (int)(grid / p.ntiles / p.mtiles);
  Launch l{p, e, maps, grid, st};
  if (split) return one_chunk ? l.rows<SHORT, float, false>(rows) : l.rows<SPLIT, float, false>(rows);
  const bool sc = t == EMP_E4M3;
  switch (e.y_dtype) {
    case EMP_F32: return l.rows<DIRECT, float, true>(rows);                         // of 8-bit inputs only
    case EMP_BF16: return sc ? l.rows<DIRECT, __nv_bfloat16, true>(rows) : l.rows<DIRECT, __nv_bfloat16, false>(rows);
    default: return sc ? l.rows<DIRECT, __half, true>(rows) : l.rows<DIRECT, __half, false>(rows);
  }
}

}  // namespace dtc
}  // namespace emp
