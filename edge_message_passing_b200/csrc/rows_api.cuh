// Entry points of the row-wise operators (norm.cuh, dense.cuh): argument checks, workspace, launches.
// Included by emp_lib.cu.
#pragma once

namespace {

bool row_dtype(int t) { return t == EMP_F32 || t == EMP_BF16 || t == EMP_F16; }
bool on_element(const void* p, int t) { return reinterpret_cast<uintptr_t>(p) % dtype_size(t) == 0; }
// a row operand: present (if it must be), on its element, rows not overlapping
bool rows_ok(const void* p, long long ld, long long cols, long long rows, int t) {
  return p && on_element(p, t) && (rows <= 1 || ld >= cols) && ld >= 0 && ld < (1ll << 40);
}
bool rows_ok_or_null(const void* p, long long ld, long long cols, long long rows, int t) {
  return !p || rows_ok(p, ld, cols, rows, t);
}

// ------------------------------------------------------------------ norm
size_t norm_grad_bytes(const emp_rms_norm_grad& a) {
  if (!a.g_weight) return 0;
  return align_up((size_t)std::min<long long>(std::max<long long>(a.rows, 0), 4 * 148) * a.cols * 4);
}
bool norm_sizes_ok(long long rows, int cols, int dtype, int degrees, float eps) {
  return rows >= 0 && rows < (1ll << 31) && cols >= 1 && row_dtype(dtype) && (degrees == 0 || degrees == 1) &&
         (!degrees || cols % NCOMP == 0) && eps > 0.f && std::isfinite(eps);
}

// ------------------------------------------------------------------ dense
// An operand of the tensor-core products: as it is if TMA can read it, else its packed copy at ws + off.
struct Packed {
  bool copy = false;
  size_t off = 0;
  long long ld = 0;
};
template <typename Take>
Packed packed(const void* p, long long ld, long long rows, int cols, int t, Take& take) {
  Packed k;
  k.ld = ld;
  if (rows == 1) k.ld = ld = (cols * dtype_size(t) + 15) / 16 * 16 / dtype_size(t);    // one row: any pitch will do
  if (dtc::tma_ok(p, ld, t)) return k;
  const int es = dtype_size(t);
  k.copy = true;
  k.ld = (cols * es + 15) / 16 * 16 / es;
  k.off = take((size_t)rows * k.ld * es);
  return k;
}
// where an operand is read, and its copy noted in `all` if it takes one
const void* pack(dense::Pack& all, const Packed& k, const void* p, long long ld, long long rows, int cols, int t, void* ws) {
  if (!k.copy) return p;
  const int es = dtype_size(t), q = all.n++;
  all.rows[q] = rows;
  all.row_bytes[q] = cols * es;
  all.src[q] = static_cast<const unsigned char*>(p);
  all.pitch[q] = ld * es;
  all.dst[q] = at<unsigned char>(ws, k.off);
  all.pitch_d[q] = k.ld * es;
  return all.dst[q];
}
void pack_all(const dense::Pack& all, cudaStream_t s) {
  if (!all.n) return;
  long long rows = all.rows[0];
  int bytes = all.row_bytes[0];
  for (int q = 1; q < all.n; ++q) {
    rows = std::max(rows, all.rows[q]);
    bytes = std::max(bytes, all.row_bytes[q]);
  }
  const int chunks = (bytes + 15) / 16, bx = std::min(256, chunks), by = 256 / bx;
  const long long blocks = (rows + by * dense::PACK_ROWS - 1) / (by * dense::PACK_ROWS);
  const dim3 grid((chunks + bx - 1) / bx, (unsigned)std::min<long long>(blocks, 32 * tc::num_sms()), all.n);
  Scope sc_("dense_pack", s);
  dense::k_pack<<<grid, dim3(bx, by), 0, s>>>(all);
}

struct DenseLayout {
  bool few = false;
  Packed x, w;
  dtc::Shape h{};
  size_t part = 0, total = 0;
};
DenseLayout dense_layout(const emp_dense& a) {
  DenseLayout L;
  if (a.rows == 0) return L;                             // nothing to launch; shape_for wants a tile at least
  L.few = dense::few_rows(a.rows, a.fan_out, a.fan_in);
  if (L.few) return L;
  auto take = [&](size_t bytes) { size_t r = L.total; L.total = align_up(L.total + bytes); return r; };
  L.x = packed(a.x, a.ldx, a.rows, a.fan_in, a.dtype, take);
  L.w = packed(a.weight, a.ldw, a.fan_out, a.fan_in, a.dtype, take);
  L.h = dtc::shape_for(a.rows, a.fan_out, a.fan_in, a.dtype, 0);
  L.part = take(L.h.splits > 1 ? (size_t)L.h.splits * a.rows * a.fan_out * 4 : 0);
  return L;
}

struct DenseGradLayout {
  size_t gz = 0, colsum = 0, part_x = 0, part_w = 0, total = 0;
  long long ldgz = 0;
  int gz_v = 1;                  // elements of g and z (and gz) read at once
  bool prep = false;             // gz is written (an activation, or g that TMA cannot read)
  int gz_blocks = 0;
  Packed x, w;
  dtc::Shape hx{}, hw{};
};
// elements that g and z allow to be read at once: 16 bytes, a 32-bit word, or one
int gz_vec(const emp_dense_grad& a) {
  const int es = dtype_size(a.dtype);
  for (int bytes = 16; bytes > es; bytes = 4) {
    auto ok = [&](const void* p, long long ld) { return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (a.rows == 1 || ld * es % bytes == 0); };
    if (a.fan_out * es % bytes == 0 && ok(a.g, a.ldg) && ok(a.z, a.ldz)) return bytes / es;
    if (bytes == 4) break;
  }
  return 1;
}
template <typename T, int V>
void dense_gz_v(const dense::GzArgs& z, int blocks, cudaStream_t s) {
  const dim3 grid(blocks, (z.cols + 32 * V - 1) / (32 * V));
  Scope sc_("dense_gz", s);
  dense::k_dense_gz<T, V><<<grid, 32 * dense::GZ_WARPS, 0, s>>>(z);
}
template <typename T>
void dense_gz(const dense::GzArgs& z, int blocks, int V, cudaStream_t s) {
  if (V == 1) return dense_gz_v<T, 1>(z, blocks, s);
  if constexpr (sizeof(T) == 2) {
    if (V == 2) return dense_gz_v<T, 2>(z, blocks, s);
  }
  dense_gz_v<T, 16 / sizeof(T)>(z, blocks, s);
}
DenseGradLayout dense_grad_layout(const emp_dense_grad& a) {
  DenseGradLayout L{};
  const int es = dtype_size(a.dtype);
  auto take = [&](size_t bytes) { size_t r = L.total; L.total = align_up(L.total + bytes); return r; };
  const bool products = a.g_x || a.g_weight;
  L.ldgz = (a.fan_out * es + 15) / 16 * 16 / es;
  L.prep = products && (a.activation != EMP_ACT_NONE || !dtc::tma_ok(a.g, a.rows == 1 ? 0 : a.ldg, a.dtype));
  L.gz = take(L.prep ? (size_t)a.rows * L.ldgz * es : 0);
  if (!L.prep && a.rows > 1) L.ldgz = a.ldg;
  L.gz_v = gz_vec(a);
  const int per = 32 * L.gz_v;        // columns of a block; one wave of blocks
  // up to 256 rows one block per columns' block, which then needs no join (a launch less)
  L.gz_blocks = a.rows <= 256 ? 1 : (int)std::max<long long>(1, std::min<long long>((a.rows + 31) / 32, std::max(1, tc::num_sms() * dense::GZ_PER_SM / ((a.fan_out + per - 1) / per))));
  L.colsum = take(a.g_bias && L.gz_blocks > 1 ? (size_t)L.gz_blocks * a.fan_out * 4 : 0);
  if (a.g_x) {
    L.w = packed(a.weight, a.ldw, a.fan_out, a.fan_in, a.dtype, take);
    L.hx = dtc::shape_for(a.rows, a.fan_in, a.fan_out, a.dtype, 1);
    L.part_x = take(L.hx.splits > 1 ? (size_t)L.hx.splits * a.rows * a.fan_in * 4 : 0);
  }
  if (a.g_weight) {
    L.x = packed(a.x, a.ldx, a.rows, a.fan_in, a.dtype, take);
    L.hw = dtc::shape_for(a.fan_out, a.fan_in, a.rows, a.dtype, 1);
    L.part_w = take(L.hw.splits > 1 ? (size_t)L.hw.splits * a.fan_out * a.fan_in * 4 : 0);
  }
  return L;
}
bool dense_sizes_ok(long long rows, int fan_in, int fan_out, int act) {
  return rows >= 0 && rows < (1ll << 31) - 256 && fan_in >= 1 && fan_in <= 65536 && fan_out >= 1 && fan_out <= 65536 &&
         act >= EMP_ACT_NONE && act <= EMP_ACT_GELU;
}
bool dense_args_ok(const emp_dense& a) {
  const bool q = a.dtype == EMP_E4M3;
  if (!dense_sizes_ok(a.rows, a.fan_in, a.fan_out, a.activation) || (!q && !row_dtype(a.dtype)) || !row_dtype(a.y_dtype) ||
      (!q && a.y_dtype != a.dtype))
    return false;
  if (a.rows == 0) return true;
  return rows_ok(a.x, a.ldx, a.fan_in, a.rows, a.dtype) && rows_ok(a.weight, a.ldw, a.fan_in, a.fan_out, a.dtype) &&
         q == (a.x_scale != nullptr) && q == (a.w_scale != nullptr) && on_element(a.x_scale, EMP_F32) &&
         on_element(a.w_scale, EMP_F32) && on_element(a.bias, q ? EMP_F32 : a.dtype) &&
         rows_ok_or_null(a.residual, a.ldr, a.fan_out, a.rows, a.y_dtype) &&
         rows_ok(a.y, a.ldy, a.fan_out, a.rows, a.y_dtype) && rows_ok_or_null(a.z, a.ldz, a.fan_out, a.rows, a.y_dtype);
}
bool dense_grad_args_ok(const emp_dense_grad& a) {
  if (!dense_sizes_ok(a.rows, a.fan_in, a.fan_out, a.activation) || !row_dtype(a.dtype) || !on_element(a.g_weight, a.dtype) ||
      !on_element(a.g_bias, a.dtype))
    return false;
  if (a.rows == 0) return true;
  return rows_ok(a.g, a.ldg, a.fan_out, a.rows, a.dtype) && (a.z != nullptr) == (a.activation != EMP_ACT_NONE) &&
         rows_ok_or_null(a.z, a.ldz, a.fan_out, a.rows, a.dtype) &&
         (!a.g_x || (rows_ok(a.g_x, a.ldgx, a.fan_in, a.rows, a.dtype) && rows_ok(a.weight, a.ldw, a.fan_in, a.fan_out, a.dtype))) &&
         (!a.g_weight || rows_ok(a.x, a.ldx, a.fan_in, a.rows, a.dtype));
}
int dense_product(long long M, int N, long long K, int t, const dtc::Operand& a, const dtc::Operand& b, const dense::Epi& e,
                  const dtc::Shape& h, float* part, cudaStream_t s) {
  int st;
  { Scope sc_("dense", s); st = dtc::launch(M, N, K, t, a, b, e, h, h.splits > 1 ? part : nullptr, s); }
  if (st != EMP_OK || h.splits == 1) return st;
  Scope sc_("dense_join", s);
  if (h.splits > JOIN_WARPS && M * N <= (1 << 14) && e.ldy == N && !e.x_scale && !e.z && !e.bias && !e.residual && e.act == EMP_ACT_NONE)
    // few outputs of many splits (a weight gradient): warps share an output's splits
    k_col_join<<<(unsigned)((M * N + 31) / 32), 32 * JOIN_WARPS, 0, s>>>(h.splits, (int)(M * N), part, e.y, e.y_dtype);
  else if (N % 4 == 0) dense::k_join<4><<<grid_for(M * N, 1024), 256, 0, s>>>(M, N, h.splits, part, e);
  else dense::k_join<1><<<grid_for(M * N, 256), 256, 0, s>>>(M, N, h.splits, part, e);
  return cudaGetLastError() == cudaSuccess ? EMP_OK : EMP_ERR_CUDA;
}
template <typename T>
void dense_few(const emp_dense& a, const dense::Epi& e, cudaStream_t s) {
  constexpr int V = sizeof(T) == 1 ? 8 : 16 / sizeof(T);
  const dense::Few p{(int)a.rows, a.fan_out, a.fan_in, a.x, a.weight, a.ldx, a.ldw};
  const dim3 grid((a.fan_out + dense::FEW_WARPS * dense::FEW_COLS - 1) / (dense::FEW_WARPS * dense::FEW_COLS),
                  ((int)a.rows + dense::FEW_M - 1) / dense::FEW_M);
  auto ok = [&](const void* q, long long ld, long long rows) {
    return reinterpret_cast<uintptr_t>(q) % (V * sizeof(T)) == 0 && (rows == 1 || ld % V == 0);
  };
  Scope sc_("dense_few", s);
  if (a.fan_in % V == 0 && ok(a.x, a.ldx, a.rows) && ok(a.weight, a.ldw, a.fan_out))
    dense::k_dense_few<T, V><<<grid, 32 * dense::FEW_WARPS, 0, s>>>(p, e);
  else
    dense::k_dense_few<T, 1><<<grid, 32 * dense::FEW_WARPS, 0, s>>>(p, e);
}

}  // namespace

extern "C" {

int mp_rms_norm(const emp_rms_norm* a, cudaStream_t stream) {
  if (!a || !norm_sizes_ok(a->rows, a->cols, a->dtype, a->degrees, a->eps)) return EMP_ERR_ARG;
  if (a->cols > EMP_NORM_MAX_COLS) return EMP_ERR_UNSUPPORTED;
  const bool quant = a->y_dtype == EMP_E4M3;
  if (!quant && a->y_dtype != a->dtype) return EMP_ERR_ARG;
  if (a->rows == 0) return EMP_OK;
  if (!rows_ok(a->x, a->ldx, a->cols, a->rows, a->dtype) || !rows_ok_or_null(a->residual, a->ldr, a->cols, a->rows, a->dtype) ||
      !rows_ok(a->y, a->ldy, a->cols, a->rows, a->y_dtype) || !rows_ok_or_null(a->s, a->lds, a->cols, a->rows, a->dtype) ||
      !on_element(a->weight, a->dtype) || !on_element(a->scale, EMP_F32) || quant != (a->scale != nullptr))
    return EMP_ERR_ARG;
  int st = check_device();
  if (st != EMP_OK) return st;
  norm::Args p{a->rows, a->cols, a->degrees, a->eps, a->x, a->residual, a->weight, a->y, a->s, a->scale, a->ldx, a->ldr, a->ldy, a->lds};
  Scope sc_("rms_norm", stream);
  const cudaError_t e = a->dtype == EMP_F32 ? norm::launch_fwd<float>(p, quant, stream)
                      : a->dtype == EMP_BF16 ? norm::launch_fwd<__nv_bfloat16>(p, quant, stream)
                                             : norm::launch_fwd<__half>(p, quant, stream);
  return e == cudaSuccess ? EMP_OK : EMP_ERR_CUDA;
}

size_t mp_rms_norm_grad_workspace_bytes(const emp_rms_norm_grad* a) {
  return a && a->rows >= 0 && a->cols >= 1 ? norm_grad_bytes(*a) : 0;
}

int mp_rms_norm_grad(const emp_rms_norm_grad* a, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (!a || !norm_sizes_ok(a->rows, a->cols, a->dtype, a->degrees, a->eps)) return EMP_ERR_ARG;
  if (a->cols > EMP_NORM_MAX_COLS) return EMP_ERR_UNSUPPORTED;
  if (!on_element(a->weight, a->dtype) || !on_element(a->g_weight, a->dtype)) return EMP_ERR_ARG;
  const int nout = a->degrees ? a->cols / NCOMP * 4 : a->cols;
  if (a->rows == 0) {
    if (a->g_weight) EMP_CUDA_TRY(cudaMemsetAsync(a->g_weight, 0, (size_t)nout * dtype_size(a->dtype), stream));
    return EMP_OK;
  }
  if (!rows_ok(a->g, a->ldg, a->cols, a->rows, a->dtype) || !rows_ok(a->s, a->lds, a->cols, a->rows, a->dtype) ||
      !rows_ok_or_null(a->g_s, a->ldgs, a->cols, a->rows, a->dtype) || !rows_ok(a->g_x, a->ldgx, a->cols, a->rows, a->dtype))
    return EMP_ERR_ARG;
  const size_t need = norm_grad_bytes(*a);
  if (ws_bytes < need) return EMP_ERR_WORKSPACE;
  if (need && (!ws || reinterpret_cast<uintptr_t>(ws) % 256)) return EMP_ERR_ARG;
  int st = check_device();
  if (st != EMP_OK) return st;
  norm::GradArgs p{a->rows, a->cols, a->degrees, a->eps, a->g, a->s, a->g_s, a->weight, a->g_x,
                   a->g_weight ? static_cast<float*>(ws) : nullptr, a->ldg, a->lds, a->ldgs, a->ldgx};
  int blocks = 0;
  cudaError_t e;
  {
    Scope sc_("rms_norm_grad", stream);
    e = a->dtype == EMP_F32 ? norm::launch_grad<float>(p, &blocks, stream)
      : a->dtype == EMP_BF16 ? norm::launch_grad<__nv_bfloat16>(p, &blocks, stream)
                             : norm::launch_grad<__half>(p, &blocks, stream);
  }
  if (e != cudaSuccess) return EMP_ERR_CUDA;
  if (a->g_weight) {
    Scope sc_("col_join", stream);
    k_col_join<<<(nout + 31) / 32, 32 * JOIN_WARPS, 0, stream>>>(blocks, nout, p.part, a->g_weight, a->dtype);
  }
  return cudaGetLastError() == cudaSuccess ? EMP_OK : EMP_ERR_CUDA;
}

size_t mp_dense_workspace_bytes(const emp_dense* a) {
  if (!a || !dense_args_ok(*a)) return 0;
  return dense_layout(*a).total;
}

int mp_dense(const emp_dense* a, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (!a || !dense_args_ok(*a)) return EMP_ERR_ARG;
  if (a->rows == 0) return EMP_OK;
  const DenseLayout L = dense_layout(*a);
  if (ws_bytes < L.total) return EMP_ERR_WORKSPACE;
  if (L.total && (!ws || reinterpret_cast<uintptr_t>(ws) % 256)) return EMP_ERR_ARG;
  int st = check_device();
  if (st != EMP_OK) return st;
  const int bt = a->dtype == EMP_E4M3 ? EMP_F32 : a->dtype;
  const dense::Epi e{a->activation, a->y_dtype, bt, a->x_scale, a->w_scale, a->bias, a->residual, a->ldr, a->y, a->z, a->ldy, a->ldz};
  if (L.few) {
    if (a->dtype == EMP_F32) dense_few<float>(*a, e, stream);
    else if (a->dtype == EMP_BF16) dense_few<__nv_bfloat16>(*a, e, stream);
    else if (a->dtype == EMP_F16) dense_few<__half>(*a, e, stream);
    else dense_few<__nv_fp8_e4m3>(*a, e, stream);
    return cudaGetLastError() == cudaSuccess ? EMP_OK : EMP_ERR_CUDA;
  }
  dense::Pack copies;
  const dtc::Operand x{pack(copies, L.x, a->x, a->ldx, a->rows, a->fan_in, a->dtype, ws), L.x.ld, 0};
  const dtc::Operand w{pack(copies, L.w, a->weight, a->ldw, a->fan_out, a->fan_in, a->dtype, ws), L.w.ld, 0};
  pack_all(copies, stream);
  return dense_product(a->rows, a->fan_out, a->fan_in, a->dtype, x, w, e, L.h, at<float>(ws, L.part), stream);
}

size_t mp_dense_grad_workspace_bytes(const emp_dense_grad* a) {
  if (!a || !dense_grad_args_ok(*a) || a->rows == 0) return 0;
  return dense_grad_layout(*a).total;
}

int mp_dense_grad(const emp_dense_grad* a, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (!a || !dense_grad_args_ok(*a)) return EMP_ERR_ARG;
  const int es = dtype_size(a->dtype);
  if (a->rows == 0) {
    if (a->g_weight) EMP_CUDA_TRY(cudaMemsetAsync(a->g_weight, 0, (size_t)a->fan_out * a->fan_in * es, stream));
    if (a->g_bias) EMP_CUDA_TRY(cudaMemsetAsync(a->g_bias, 0, (size_t)a->fan_out * es, stream));
    return EMP_OK;
  }
  const DenseGradLayout L = dense_grad_layout(*a);
  if (ws_bytes < L.total) return EMP_ERR_WORKSPACE;
  if (L.total && (!ws || reinterpret_cast<uintptr_t>(ws) % 256)) return EMP_ERR_ARG;
  int st = check_device();
  if (st != EMP_OK) return st;
  if (L.prep || a->g_bias) {
    const dense::GzArgs z{a->rows, a->fan_out, a->activation, a->g, a->z, a->ldg, a->ldz, L.ldgz,
                          L.prep ? at<char>(ws, L.gz) : nullptr, L.gz_blocks > 1 ? at<float>(ws, L.colsum) : nullptr, a->g_bias};
    if (a->dtype == EMP_F32) dense_gz<float>(z, L.gz_blocks, L.gz_v, stream);
    else if (a->dtype == EMP_BF16) dense_gz<__nv_bfloat16>(z, L.gz_blocks, L.gz_v, stream);
    else dense_gz<__half>(z, L.gz_blocks, L.gz_v, stream);
    if (a->g_bias && L.gz_blocks > 1) {
      Scope sc_("col_join", stream);
      k_col_join<<<(a->fan_out + 31) / 32, 32 * JOIN_WARPS, 0, stream>>>(L.gz_blocks, a->fan_out, z.part, a->g_bias, a->dtype);
    }
  }
  const void* gz = L.prep ? at<char>(ws, L.gz) : static_cast<const char*>(a->g);
  dense::Pack copies;
  const dtc::Operand w{a->g_x ? pack(copies, L.w, a->weight, a->ldw, a->fan_out, a->fan_in, a->dtype, ws) : nullptr, L.w.ld, 1};
  const dtc::Operand x{a->g_weight ? pack(copies, L.x, a->x, a->ldx, a->rows, a->fan_in, a->dtype, ws) : nullptr, L.x.ld, 1};
  pack_all(copies, stream);
  if (a->g_x) {
    const dense::Epi e{EMP_ACT_NONE, a->dtype, 0, nullptr, nullptr, nullptr, nullptr, 0, a->g_x, nullptr, a->ldgx, 0};
    st = dense_product(a->rows, a->fan_in, a->fan_out, a->dtype, {gz, L.ldgz, 0}, w, e, L.hx, at<float>(ws, L.part_x), stream);
    if (st != EMP_OK) return st;
  }
  if (a->g_weight) {
    const dense::Epi e{EMP_ACT_NONE, a->dtype, 0, nullptr, nullptr, nullptr, nullptr, 0, a->g_weight, nullptr, a->fan_in, 0};
    st = dense_product(a->fan_out, a->fan_in, a->rows, a->dtype, {gz, L.ldgz, 1}, x, e, L.hw, at<float>(ws, L.part_w), stream);
  }
  return st != EMP_OK ? st : cudaGetLastError() == cudaSuccess ? EMP_OK : EMP_ERR_CUDA;
}

}  // extern "C"
