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
// splits of a product's k axis: enough tiles for every SM, at least 256 of k each
int simt_splits(long long M, long long N, long long K) {
  const long long tiles = ((M + dense::T_M - 1) / dense::T_M) * ((N + dense::T_M - 1) / dense::T_M);
  return (int)std::max<long long>(1, std::min<long long>((296 + tiles - 1) / tiles, K / 256));
}
struct DenseGradLayout {
  size_t gz, colsum, part, total;
  long long ldgz;
  int gz_blocks, splits;
};
DenseGradLayout dense_grad_layout(const emp_dense_grad& a) {
  DenseGradLayout L{};
  const int es = dtype_size(a.dtype);
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t r = o; o = align_up(o + bytes); return r; };
  L.ldgz = (a.fan_out * es + 15) / 16 * 16 / es;
  L.gz = take(a.activation != EMP_ACT_NONE && (a.g_x || a.g_weight) ? (size_t)a.rows * L.ldgz * es : 0);
  L.gz_blocks = (int)std::max<long long>(1, std::min<long long>((a.rows + 63) / 64, std::max(1, 592 * 32 / a.fan_out)));
  L.colsum = take(a.g_bias ? (size_t)L.gz_blocks * a.fan_out * 4 : 0);
  L.splits = simt_splits(a.fan_out, a.fan_in, a.rows);
  L.part = take(a.g_weight && L.splits > 1 ? (size_t)L.splits * a.fan_out * a.fan_in * 4 : 0);
  L.total = o;
  return L;
}
bool dense_sizes_ok(long long rows, int fan_in, int fan_out, int act) {
  return rows >= 0 && rows < (1ll << 31) - 256 && fan_in >= 1 && fan_in <= 65536 && fan_out >= 1 && fan_out <= 65536 &&
         act >= EMP_ACT_NONE && act <= EMP_ACT_GELU;
}
void dense_product(const dense::Prod& p, const dense::Epi& e, int splits, cudaStream_t s) {
  const dim3 grid((unsigned)((p.M + dense::T_M - 1) / dense::T_M), (unsigned)((p.N + dense::T_M - 1) / dense::T_M), splits);
  { Scope sc_("dense", s); dense::k_dense_simt<<<grid, 256, 0, s>>>(p, e); }
  if (p.part) {
    Scope sc_("dense_join", s);
    dense::k_join<<<grid_for((long long)p.M * p.N, 256), 256, 0, s>>>(p.M, p.N, splits, p.part, e);
  }
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
  if (a->dtype == EMP_F32) norm::launch_fwd<float>(p, quant, stream);
  else if (a->dtype == EMP_BF16) norm::launch_fwd<__nv_bfloat16>(p, quant, stream);
  else norm::launch_fwd<__half>(p, quant, stream);
  return cudaGetLastError() == cudaSuccess ? EMP_OK : EMP_ERR_CUDA;
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
  if (need && (!ws || reinterpret_cast<uintptr_t>(ws) % 16)) return EMP_ERR_ARG;
  if (ws_bytes < need) return EMP_ERR_WORKSPACE;
  int st = check_device();
  if (st != EMP_OK) return st;
  norm::GradArgs p{a->rows, a->cols, a->degrees, a->eps, a->g, a->s, a->g_s, a->weight, a->g_x,
                   a->g_weight ? static_cast<float*>(ws) : nullptr, a->ldg, a->lds, a->ldgs, a->ldgx};
  int blocks;
  {
    Scope sc_("rms_norm_grad", stream);
    if (a->dtype == EMP_F32) blocks = norm::launch_grad<float>(p, stream);
    else if (a->dtype == EMP_BF16) blocks = norm::launch_grad<__nv_bfloat16>(p, stream);
    else blocks = norm::launch_grad<__half>(p, stream);
  }
  if (a->g_weight) {
    Scope sc_("col_join", stream);
    k_col_join<<<(nout + 31) / 32, 32 * JOIN_WARPS, 0, stream>>>(blocks, a->cols, nout, a->degrees, p.part, a->g_weight, a->dtype);
  }
  return cudaGetLastError() == cudaSuccess ? EMP_OK : EMP_ERR_CUDA;
}

size_t mp_dense_workspace_bytes(const emp_dense* a) {
  (void)a;
  return 0;
}

int mp_dense(const emp_dense* a, void* ws, size_t ws_bytes, cudaStream_t stream) {
  (void)ws; (void)ws_bytes;
  if (!a || !dense_sizes_ok(a->rows, a->fan_in, a->fan_out, a->activation)) return EMP_ERR_ARG;
  const bool q = a->dtype == EMP_E4M3;
  if ((!q && !row_dtype(a->dtype)) || !row_dtype(a->y_dtype) || (!q && a->y_dtype != a->dtype)) return EMP_ERR_ARG;
  if (a->rows == 0) return EMP_OK;
  const int bt = q ? EMP_F32 : a->dtype;
  if (!rows_ok(a->x, a->ldx, a->fan_in, a->rows, a->dtype) || !rows_ok(a->weight, a->ldw, a->fan_in, a->fan_out, a->dtype) ||
      q != (a->x_scale != nullptr) || q != (a->w_scale != nullptr) || !on_element(a->x_scale, EMP_F32) ||
      !on_element(a->w_scale, EMP_F32) || !on_element(a->bias, bt) ||
      !rows_ok_or_null(a->residual, a->ldr, a->fan_out, a->rows, a->y_dtype) ||
      !rows_ok(a->y, a->ldy, a->fan_out, a->rows, a->y_dtype) || !rows_ok_or_null(a->z, a->ldz, a->fan_out, a->rows, a->y_dtype))
    return EMP_ERR_ARG;
  int st = check_device();
  if (st != EMP_OK) return st;
  const dense::Epi e{a->activation, a->y_dtype, bt, a->x_scale, a->w_scale, a->bias, a->residual, a->ldr, a->y, a->z, a->ldy, a->ldz};
  const dense::Prod p{a->rows, a->fan_in, a->fan_out, a->dtype, a->x, a->weight, a->ldx, 1, a->ldw, 1, nullptr};
  dense_product(p, e, 1, stream);
  return cudaGetLastError() == cudaSuccess ? EMP_OK : EMP_ERR_CUDA;
}

size_t mp_dense_grad_workspace_bytes(const emp_dense_grad* a) {
  return a && row_dtype(a->dtype) && dense_sizes_ok(a->rows, a->fan_in, a->fan_out, a->activation) ? dense_grad_layout(*a).total : 0;
}

int mp_dense_grad(const emp_dense_grad* a, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (!a || !dense_sizes_ok(a->rows, a->fan_in, a->fan_out, a->activation) || !row_dtype(a->dtype)) return EMP_ERR_ARG;
  const int es = dtype_size(a->dtype);
  if (!on_element(a->g_weight, a->dtype) || !on_element(a->g_bias, a->dtype)) return EMP_ERR_ARG;
  if (a->rows == 0) {
    if (a->g_weight) EMP_CUDA_TRY(cudaMemsetAsync(a->g_weight, 0, (size_t)a->fan_out * a->fan_in * es, stream));
    if (a->g_bias) EMP_CUDA_TRY(cudaMemsetAsync(a->g_bias, 0, (size_t)a->fan_out * es, stream));
    return EMP_OK;
  }
  if (!rows_ok(a->g, a->ldg, a->fan_out, a->rows, a->dtype) || (a->z != nullptr) != (a->activation != EMP_ACT_NONE) ||
      !rows_ok_or_null(a->z, a->ldz, a->fan_out, a->rows, a->dtype))
    return EMP_ERR_ARG;
  if (a->g_x && (!rows_ok(a->g_x, a->ldgx, a->fan_in, a->rows, a->dtype) || !rows_ok(a->weight, a->ldw, a->fan_in, a->fan_out, a->dtype)))
    return EMP_ERR_ARG;
  if (a->g_weight && !rows_ok(a->x, a->ldx, a->fan_in, a->rows, a->dtype)) return EMP_ERR_ARG;
  const DenseGradLayout L = dense_grad_layout(*a);
  if (L.total && (!ws || reinterpret_cast<uintptr_t>(ws) % 256)) return EMP_ERR_ARG;
  if (ws_bytes < L.total) return EMP_ERR_WORKSPACE;
  int st = check_device();
  if (st != EMP_OK) return st;
  const bool prep = a->activation != EMP_ACT_NONE && (a->g_x || a->g_weight);
  const void* gz = prep ? at<char>(ws, L.gz) : static_cast<const char*>(a->g);
  const long long ldgz = prep ? L.ldgz : a->ldg;
  if (prep || a->g_bias) {
    const dense::GzArgs z{a->rows, a->fan_out, a->dtype, a->activation, a->g, a->z, a->ldg, a->ldz, L.ldgz,
                          prep ? at<char>(ws, L.gz) : nullptr, a->g_bias ? at<float>(ws, L.colsum) : nullptr};
    { Scope sc_("dense_gz", stream);
      dense::k_dense_gz<<<dim3(L.gz_blocks, (a->fan_out + 31) / 32), 32 * dense::GZ_ROWS, 0, stream>>>(z); }
    if (a->g_bias) {
      Scope sc_("col_join", stream);
      k_col_join<<<(a->fan_out + 31) / 32, 32 * JOIN_WARPS, 0, stream>>>(L.gz_blocks, a->fan_out, a->fan_out, 0, z.part, a->g_bias, a->dtype);
    }
  }
  if (a->g_x) {
    const dense::Epi e{EMP_ACT_NONE, a->dtype, 0, nullptr, nullptr, nullptr, nullptr, 0, a->g_x, nullptr, a->ldgx, 0};
    const dense::Prod p{a->rows, a->fan_out, a->fan_in, a->dtype, gz, a->weight, ldgz, 1, 1, a->ldw, nullptr};
    dense_product(p, e, 1, stream);
  }
  if (a->g_weight) {
    const dense::Epi e{EMP_ACT_NONE, a->dtype, 0, nullptr, nullptr, nullptr, nullptr, 0, a->g_weight, nullptr, a->fan_in, 0};
    const dense::Prod p{a->fan_out, a->rows, a->fan_in, a->dtype, gz, a->x, 1, ldgz, 1, a->ldx,
                        L.splits > 1 ? at<float>(ws, L.part) : nullptr};
    dense_product(p, e, L.splits, stream);
  }
  return cudaGetLastError() == cudaSuccess ? EMP_OK : EMP_ERR_CUDA;
}

}  // extern "C"
