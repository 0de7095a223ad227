// extern "C" entry points of attention over a paged cache and of range-masked attention (mesh_attn.h): argument checks,
// workspace layout and the choice of kernels.  (mesh_attn_paged_append is beside its kernel.)
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "abi_util.h"
#include "internal.h"
#include "paged.h"
#include "score_bwd.h"
#include "score_fwd.h"

namespace mesh {

// Whether a batch of at most so many rows a sequence (new tokens times query heads of a KV head) goes to the few-rows kernel, which
// shares out the cached tokens evenly, rather than to those for chunks, a sequence and KV head or a part of it at a time: one
// sequence of 131,072 tokens, 16 heads on 4, bf16, 50 us where tiles of 256 rows take 98; 64 of up to 8,192, 32 heads on 8, 169
// (184); fp32, 16 of up to 2,048, 32 heads on 8, 63 (213); only tiny batches are the same or a little slower (4 of up to 300,
// bf16, 12.7 and 10.9).
static bool few_rows(bool bf16, int64_t rows) { return rows <= (bf16 ? PAGED_FEW_BF16 : PAGED_FEW_F32); }

static size_t paged_workspace(bool bf16, int64_t N, int32_t B, int32_t Hq, int32_t Hkv, int32_t d, int64_t max_new) {
  size_t need = paged_rows_slots();
  if (!few_rows(bf16, max_new * (Hq / Hkv)))
    need = std::max(need, bf16 ? score_fwd_paged_workspace(N, B, Hq, Hkv, d) : score_simt_workspace(d));
  return PAGED_WS_HEAD + need;
}

// Workspace of the range-masked calls, of one direction after the other.
static size_t range_workspace(bool bf16, int32_t B, int32_t Hq, int32_t Hkv, int64_t S, int32_t d, bool backward, int sms) {
  if (backward) return range_bwd_shape(bf16, S, B, Hq, Hkv, d, sms).total;
  return bf16 ? score_fwd_shape(false, S, 0, B, Hq, Hkv, d, sms).total : score_simt_workspace(d);
}

}  // namespace mesh

using mesh::is_aligned;
using mesh::launch_status;
using mesh::set_last_error;

namespace {

int check_heads(mesh_attn_dtype dt, int32_t Hq, int32_t Hkv, int32_t d) {
  if (dt != MESH_ATTN_F32 && dt != MESH_ATTN_BF16)
    return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "dtype must be MESH_ATTN_F32 or MESH_ATTN_BF16");
  if (Hq < 0) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "Hq must be >= 0");
  if (Hkv < 1 || Hq % Hkv != 0) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "need Hkv >= 1 and Hq % Hkv == 0");
  if (d != 64 && d != 128) return set_last_error(MESH_ATTN_ERR_UNSUPPORTED, "d must be 64 or 128");
  return MESH_ATTN_OK;
}
int check_score(float scale, float cap) {
  if (!(scale > 0.f) || !std::isfinite(scale)) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "scale must be finite and > 0");
  if (!(cap >= 0.f) || !std::isfinite(cap))
    return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "cap must be finite and >= 0 (0: scores are not capped)");
  // squares of both are taken in fp32
  if (cap > 0.f && !(cap >= 1e-18f && cap <= 1e18f && scale / cap >= 1e-18f && scale / cap <= 1e18f))
    return set_last_error(MESH_ATTN_ERR_UNSUPPORTED, "a cap, and scale / cap, must be within 1e-18 and 1e18");
  return MESH_ATTN_OK;
}
int sm_count(int* sms) {
  const cudaError_t e = mesh::current_sms(sms);
  if (e != cudaSuccess) return set_last_error(MESH_ATTN_ERR_CUDA, std::string("device query: ") + cudaGetErrorString(e));
  *sms = std::min(*sms, mesh::MAX_SMS);
  return MESH_ATTN_OK;
}
int check_paged_sizes(mesh_attn_dtype dt, int64_t N, int32_t B, int32_t Hq, int32_t Hkv, int32_t d, int64_t T, int64_t max_new) {
  if (const int rc = check_heads(dt, Hq, Hkv, d)) return rc;
  if (N < 0 || B < 0 || T < 0 || max_new < 0) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "N, B, T and max_new must be >= 0");
  if (B > mesh::PAGED_MAX_B) return set_last_error(MESH_ATTN_ERR_UNSUPPORTED, "B must be at most 4096");
  if (T > (1 << 30)) return set_last_error(MESH_ATTN_ERR_UNSUPPORTED, "a table's pages must hold at most 2^30 tokens");
  if (N > (1 << 24) || Hq > 65535 || N * Hq > 0x3fffffff)
    return set_last_error(MESH_ATTN_ERR_UNSUPPORTED, "need N <= 2^24, Hq <= 65535 and N * Hq < 2^30");
  return MESH_ATTN_OK;
}
int check_range_sizes(mesh_attn_dtype dt, int32_t B, int32_t Hq, int32_t Hkv, int64_t S, int32_t d) {
  if (const int rc = check_heads(dt, Hq, Hkv, d)) return rc;
  if (B < 0 || S < 0) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "B and S must be >= 0");
  if (S > (1 << 24) || B > 65535 || Hq > 65535 || (int64_t)B * Hq * std::max<int64_t>(S, 1) > 0x3fffffff)
    return set_last_error(MESH_ATTN_ERR_UNSUPPORTED, "need S <= 2^24, B and Hq <= 65535 and B * Hq * S < 2^30");
  return MESH_ATTN_OK;
}

}  // namespace

extern "C" int mesh_attn_paged_workspace_size(mesh_attn_dtype dtype, int64_t N, int32_t B, int32_t Hq, int32_t Hkv, int32_t d,
                                              int64_t max_new, size_t* bytes) {
  return mesh::guarded_call([&]() -> int {
    if (!bytes) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "bytes is NULL");
    if (const int rc = check_paged_sizes(dtype, N, B, Hq, Hkv, d, 0, max_new)) return rc;
    *bytes = mesh::paged_workspace(dtype == MESH_ATTN_BF16, N, B, Hq, Hkv, d, std::min(max_new, N));
    return (int)MESH_ATTN_OK;
  });
}

extern "C" int mesh_attn_paged_attn(mesh_attn_dtype dtype, int64_t N, int32_t B, int32_t Hq, int32_t Hkv, int32_t d, const void* q,
                                    const int64_t* q_strides, int32_t n_pages, int32_t page, const void* k_pages,
                                    const int64_t* k_strides, const void* v_pages, const int64_t* v_strides, const int32_t* table,
                                    int32_t max_pages, int64_t table_stride, const int32_t* offsets, const int32_t* lens,
                                    int64_t max_new, float scale, float cap, const float* slopes, int64_t window, void* O, float* LSE,
                                    void* workspace, size_t workspace_bytes, int32_t* d_status, void* stream) {
  return mesh::guarded_call([&]() -> int {
    if (page < 16 || page % 16 != 0) return set_last_error(MESH_ATTN_ERR_UNSUPPORTED, "page must be a multiple of 16");
    if (n_pages < 0 || max_pages < 0) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "n_pages and max_pages must be >= 0");
    const int64_t T = (int64_t)max_pages * page;
    if (const int rc = check_paged_sizes(dtype, N, B, Hq, Hkv, d, T, max_new)) return rc;
    if (const int rc = check_score(scale, cap)) return rc;
    if (window < 0) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "window must be >= 0 (0: all keys before a token)");
    if (N == 0 || B == 0 || Hq == 0) return (int)MESH_ATTN_OK;
    if (max_new < 1) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "max_new must be >= 1");
    max_new = std::min(max_new, N);
    if (!q || !q_strides || !k_pages || !k_strides || !v_pages || !v_strides || !table || !offsets || !lens || !O || !LSE || !workspace ||
        !d_status)
      return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "a tensor, its strides, workspace or status pointer is NULL");
    if (n_pages < 1 || max_pages < 1) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "there are tokens but no pages");
    const bool bf16 = dtype == MESH_ATTN_BF16;
    const int64_t es = bf16 ? 2 : 4;
    for (const void* x : {q, k_pages, v_pages, (const void*)O, (const void*)workspace})
      if (!is_aligned(x, 16))
        return set_last_error(MESH_ATTN_ERR_MISALIGNED, "q, the pages, O and workspace must be 16-byte aligned");
    for (const void* x : {(const void*)table, (const void*)offsets, (const void*)lens, (const void*)slopes, (const void*)LSE,
                          (const void*)d_status})
      if (!is_aligned(x, 4))
        return set_last_error(MESH_ATTN_ERR_MISALIGNED, "table, offsets, lens, slopes, LSE and status must be 4-byte aligned");
    const int64_t qd[2] = {N, Hq}, kd[3] = {n_pages, Hkv, page};
    auto stride_ok = [&](int64_t dim, int64_t s) { return dim <= 1 || (s > 0 && s * es % 16 == 0 && s < ((int64_t)1 << 37)); };
    for (int i = 0; i < 2; ++i)
      if (!stride_ok(qd[i], q_strides[i]))
        return set_last_error(MESH_ATTN_ERR_MISALIGNED, "strides of q must be positive multiples of 16 bytes");
    for (int i = 0; i < 3; ++i)
      if (!stride_ok(kd[i], k_strides[i]) || !stride_ok(kd[i], v_strides[i]))
        return set_last_error(MESH_ATTN_ERR_MISALIGNED, "strides of the pages must be positive multiples of 16 bytes");
    const size_t need = mesh::paged_workspace(bf16, N, B, Hq, Hkv, d, max_new);
    if (workspace_bytes < need)
      return set_last_error(MESH_ATTN_ERR_WORKSPACE, "workspace needs " + std::to_string(need) + " bytes");
    int sms = 0;
    if (const int rc = sm_count(&sms)) return rc;
    mesh::PagedArgs a{};
    a.bf16 = bf16;
    a.q = q;
    a.k = k_pages;
    a.v = v_pages;
    for (int i = 0; i < 2; ++i) a.qs[i] = qd[i] > 1 ? q_strides[i] : d;
    for (int i = 0; i < 3; ++i) a.ks[i] = kd[i] > 1 ? k_strides[i] : d, a.vs[i] = kd[i] > 1 ? v_strides[i] : d;
    a.table = table;
    a.table_s = table_stride;
    a.offsets = offsets;
    a.lens = lens;
    a.slopes = slopes;
    a.o = O;
    a.lse = LSE;
    a.ws = static_cast<char*>(workspace);
    a.status = d_status;
    a.N = (int32_t)N;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.d = d;
    a.n_pages = n_pages;
    a.page = page;
    a.max_pages = max_pages;
    a.max_new = (int32_t)max_new;
    a.window = (int32_t)std::min<int64_t>(window, (int64_t)1 << 30);
    a.scale = scale;
    a.cap = cap;
    a.wait_limit_ns = mesh::current_wait_limit_ns();
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    std::string err;
    if (mesh::few_rows(bf16, max_new * (Hq / Hkv))) return launch_status(mesh::launch_paged_rows(a, sms, st, &err), err);
    if (!bf16) return launch_status(mesh::launch_paged_simt(a, sms, st, &err), err);
    mesh::ScoreFwdArgs f{};
    f.paged = true;
    f.q = q;
    f.k = k_pages;
    f.v = v_pages;
    for (int i = 0; i < 2; ++i) f.qs[i] = a.qs[i];
    for (int i = 0; i < 3; ++i) f.ks[i] = a.ks[i], f.vs[i] = a.vs[i];
    f.slopes = slopes;
    f.o = O;
    f.lse = LSE;
    f.status = d_status;
    f.ws = a.ws + mesh::PAGED_WS_HEAD;
    f.S = T;
    f.N = a.N;
    f.B = B;
    f.Hq = Hq;
    f.Hkv = Hkv;
    f.d = d;
    f.offsets = offsets;
    f.lens = lens;
    f.table = table;
    f.table_s = table_stride;
    f.n_pages = n_pages;
    f.page = page;
    f.max_pages = max_pages;
    f.max_new = a.max_new;
    f.window = a.window;
    f.scale = scale;
    f.cap = cap;
    f.wait_limit_ns = a.wait_limit_ns;
    return launch_status(mesh::launch_score_fwd(f, sms, st, &err), err);
  });
}

extern "C" int mesh_attn_range_workspace_size(mesh_attn_dtype dtype, int32_t B, int32_t Hq, int32_t Hkv, int64_t S, int32_t d,
                                              int32_t backward, size_t* bytes) {
  return mesh::guarded_call([&]() -> int {
    if (!bytes) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "bytes is NULL");
    if (backward != 0 && backward != 1) return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "backward must be 0 or 1");
    if (const int rc = check_range_sizes(dtype, B, Hq, Hkv, S, d)) return rc;
    size_t most = 256;
    if (B > 0 && Hq > 0 && S > 0)
      for (int sms = 1; sms <= mesh::MAX_SMS; ++sms)
        for (int dir = 0; dir <= backward; ++dir)
          most = std::max(most, mesh::range_workspace(dtype == MESH_ATTN_BF16, B, Hq, Hkv, S, d, dir != 0, sms));
    *bytes = most;
    return (int)MESH_ATTN_OK;
  });
}

static int check_range_args(const mesh::RangeArgs& a, const void* workspace, size_t workspace_bytes, bool backward, int* sms) {
  if (const int rc = check_score(a.scale, a.cap)) return rc;
  if (!a.q || !a.k || !a.v || !a.lo || !a.hi || !a.o || !a.lse || !workspace || !a.status ||
      (backward && (!a.go || !a.dq || !a.dk || !a.dv)))
    return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "a tensor, workspace or status pointer is NULL");
  for (const void* x : {a.q, a.k, a.v, (const void*)a.o, a.go, (const void*)a.dq, (const void*)a.dk, (const void*)a.dv, workspace})
    if (!is_aligned(x, 16)) return set_last_error(MESH_ATTN_ERR_MISALIGNED, "tensors and workspace must be 16-byte aligned");
  for (const void* x : {(const void*)a.lo, (const void*)a.hi, (const void*)a.slopes, (const void*)a.lse, (const void*)a.status})
    if (!is_aligned(x, 4)) return set_last_error(MESH_ATTN_ERR_MISALIGNED, "lo, hi, slopes, LSE and status must be 4-byte aligned");
  if (a.mask_bs != 0 && a.mask_bs < a.S && a.B > 1)
    return set_last_error(MESH_ATTN_ERR_INVALID_ARG, "mask_stride must be 0 (one mask for all) or at least S");
  if (workspace_bytes < 256) return set_last_error(MESH_ATTN_ERR_WORKSPACE, "workspace needs 256 bytes or more");
  if (const int rc = sm_count(sms)) return rc;
  const size_t need = mesh::range_workspace(a.bf16, a.B, a.Hq, a.Hkv, a.S, a.d, backward, *sms);
  if (workspace_bytes < need)
    return set_last_error(MESH_ATTN_ERR_WORKSPACE, "workspace needs " + std::to_string(need) + " bytes");
  return MESH_ATTN_OK;
}

extern "C" int mesh_attn_range_fwd(mesh_attn_dtype dtype, int32_t B, int32_t Hq, int32_t Hkv, int64_t S, int32_t d, const void* Q,
                                   const void* K, const void* V, const int32_t* lo, const int32_t* hi, int64_t mask_stride,
                                   const float* slopes, float scale, float cap, void* O, float* LSE, void* workspace,
                                   size_t workspace_bytes, int32_t* d_status, void* stream) {
  return mesh::guarded_call([&]() -> int {
    if (const int rc = check_range_sizes(dtype, B, Hq, Hkv, S, d)) return rc;
    if (B == 0 || Hq == 0 || S == 0) return check_score(scale, cap);
    mesh::RangeArgs a{};
    a.bf16 = dtype == MESH_ATTN_BF16;
    a.q = Q, a.k = K, a.v = V, a.lo = lo, a.hi = hi, a.mask_bs = mask_stride, a.slopes = slopes, a.o = O, a.lse = LSE;
    a.ws = static_cast<char*>(workspace), a.status = d_status;
    a.S = S, a.B = B, a.Hq = Hq, a.Hkv = Hkv, a.d = d, a.scale = scale, a.cap = cap;
    a.wait_limit_ns = mesh::current_wait_limit_ns();
    int sms = 0;
    if (const int rc = check_range_args(a, workspace, workspace_bytes, false, &sms)) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    std::string err;
    if (!a.bf16) return launch_status(mesh::launch_range_fwd_simt(a, sms, st, &err), err);
    mesh::ScoreFwdArgs f{};
    f.q = Q, f.k = K, f.v = V, f.slopes = slopes, f.o = O, f.lse = LSE, f.status = d_status, f.ws = a.ws;
    f.S = S, f.B = B, f.Hq = Hq, f.Hkv = Hkv, f.d = d, f.lo = lo, f.hi = hi, f.mask_bs = mask_stride;
    f.scale = scale, f.cap = cap, f.wait_limit_ns = a.wait_limit_ns;
    return launch_status(mesh::launch_score_fwd(f, sms, st, &err), err);
  });
}

extern "C" int mesh_attn_range_bwd(mesh_attn_dtype dtype, int32_t B, int32_t Hq, int32_t Hkv, int64_t S, int32_t d, const void* Q,
                                   const void* K, const void* V, const int32_t* lo, const int32_t* hi, int64_t mask_stride,
                                   const float* slopes, const void* O, const float* LSE, const void* dO, float scale, float cap,
                                   void* dQ, void* dK, void* dV, void* workspace, size_t workspace_bytes, int32_t* d_status,
                                   void* stream) {
  return mesh::guarded_call([&]() -> int {
    if (const int rc = check_range_sizes(dtype, B, Hq, Hkv, S, d)) return rc;
    if (B == 0 || Hq == 0 || S == 0) return check_score(scale, cap);
    mesh::RangeArgs a{};
    a.bf16 = dtype == MESH_ATTN_BF16;
    a.q = Q, a.k = K, a.v = V, a.lo = lo, a.hi = hi, a.mask_bs = mask_stride, a.slopes = slopes;
    a.o = const_cast<void*>(O), a.lse = const_cast<float*>(LSE), a.go = dO, a.dq = dQ, a.dk = dK, a.dv = dV;
    a.ws = static_cast<char*>(workspace), a.status = d_status;
    a.S = S, a.B = B, a.Hq = Hq, a.Hkv = Hkv, a.d = d, a.scale = scale, a.cap = cap;
    a.wait_limit_ns = mesh::current_wait_limit_ns();
    int sms = 0;
    if (const int rc = check_range_args(a, workspace, workspace_bytes, true, &sms)) return rc;
    const mesh::RangeBwdShape z = mesh::range_bwd_shape(a.bf16, S, B, Hq, Hkv, d, sms);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    std::string err;
    if (!a.bf16) return launch_status(mesh::launch_range_bwd_simt(a, z, st, &err), err);
    return launch_status(d == 128 ? mesh::launch_range_bwd_128(a, z, sms, st, &err) : mesh::launch_range_bwd_64(a, z, sms, st, &err),
                         err);
  });
}
