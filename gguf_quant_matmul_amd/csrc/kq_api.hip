// C ABI of libkq: argument validation and kernel dispatch.
//
// Every entry point validates on the host and returns before any HIP call
// when an argument is wrong (outputs untouched); otherwise it enqueues the
// kernels on the caller's stream and returns without synchronizing.  The
// error style mirrors the "[module.op] message" invalid-argument text of the
// mlx-kquant bindings.cpp page and the "op: msg" errors of nuvec-core's
// quantized.rs page.
#include <ctype.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <cmath>
#include <string>

#include "kq_internal.h"
#include "../../include/kq.h"

namespace {

thread_local std::string g_err;

int fail(int status, const char* op, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_err = std::string("[") + op + "] " + buf;
  return status;
}

const char* codec_name(int c) {
  switch (c) {
    case KQ_Q4_0: return "q4_0";
    case KQ_Q8_0: return "q8_0";
    case KQ_Q4_K: return "q4_k";
    case KQ_Q5_K: return "q5_k";
    case KQ_Q2_K: return "q2_k";
    case KQ_Q3_K: return "q3_k";
    case KQ_Q4_1: return "q4_1";
    case KQ_Q5_0: return "q5_0";
    case KQ_Q5_1: return "q5_1";
    case KQ_Q6_K: return "q6_k";
    default: return "?";
  }
}

bool geometry(int c, int* bv, int* bb) {
  switch (c) {
    case KQ_Q4_0: *bv = 32; *bb = 18; return true;
    case KQ_Q8_0: *bv = 32; *bb = 34; return true;
    case KQ_Q4_K: *bv = 256; *bb = 144; return true;
    case KQ_Q5_K: *bv = 256; *bb = 176; return true;
    case KQ_Q2_K: *bv = 256; *bb = 84; return true;
    case KQ_Q3_K: *bv = 256; *bb = 110; return true;
    case KQ_Q4_1: *bv = 32; *bb = 20; return true;
    case KQ_Q5_0: *bv = 32; *bb = 22; return true;
    case KQ_Q5_1: *bv = 32; *bb = 24; return true;
    case KQ_Q6_K: *bv = 256; *bb = 210; return true;
    default: return false;
  }
}

constexpr int64_t kMaxDim = (int64_t)1 << 31;
constexpr int64_t kMaxElems = (int64_t)1 << 40;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Shared checks: codec, K, row bytes.  Returns KQ_OK and fills row_bytes.
int check_codec_k(const char* op, int codec, int64_t k, int64_t* row_bytes) {
  int bv, bb;
  if (!geometry(codec, &bv, &bb)) return fail(KQ_ERR_CODEC, op, "unknown codec id %d", codec);
  if (k <= 0 || k >= kMaxDim) return fail(KQ_ERR_SHAPE, op, "K=%lld out of range", (long long)k);
  if (k % bv)
    return fail(KQ_ERR_SHAPE, op, "K=%lld is not a multiple of %d for %s", (long long)k, bv, codec_name(codec));
  *row_bytes = k / bv * bb;
  return KQ_OK;
}

int check_dtype(const char* op, int dt, bool bf16 = false) {
  if (bf16 && dt == KQ_BF16) return KQ_OK;
  if (dt != KQ_F32 && dt != KQ_F16)
    return fail(KQ_ERR_ARG, op, "output dtype %d is not KQ_F32 or KQ_F16%s", dt, bf16 ? " or KQ_BF16" : "");
  return KQ_OK;
}

int hip_status(const char* op, hipError_t e) {
  if (e != hipSuccess) return fail(KQ_ERR_HIP, op, "HIP launch failed: %s", hipGetErrorString(e));
  g_err.clear();
  return KQ_OK;
}

int check_matmul(const char* op, int codec, const void* w, int64_t n, int64_t k, const void* x, int64_t m,
                 const void* y, int y_dtype, int64_t* rb, bool bf16 = false) {
  int st = check_codec_k(op, codec, k, rb);
  if (st) return st;
  if ((st = check_dtype(op, y_dtype, bf16))) return st;
  if (n < 0 || n >= kMaxDim) return fail(KQ_ERR_ARG, op, "N=%lld out of range", (long long)n);
  if (m < 0 || m >= kMaxDim) return fail(KQ_ERR_ARG, op, "M=%lld out of range", (long long)m);
  if (n * k >= kMaxElems || m * k >= kMaxElems || m * n >= kMaxElems)
    return fail(KQ_ERR_ARG, op, "tensor too large (M=%lld N=%lld K=%lld)", (long long)m, (long long)n, (long long)k);
  if (n == 0 || m == 0) return KQ_OK;
  if (!w || !x || !y) return fail(KQ_ERR_ARG, op, "null pointer (w=%p x=%p y=%p)", w, x, y);
  if (!aligned(w, 16)) return fail(KQ_ERR_ALIGN, op, "w=%p is not 16-byte aligned", w);
  if (!aligned(x, 16)) return fail(KQ_ERR_ALIGN, op, "x=%p is not 16-byte aligned", x);
  if (!aligned(y, y_dtype == KQ_F32 ? 4 : 2)) return fail(KQ_ERR_ALIGN, op, "y=%p is not element aligned", y);
  return KQ_OK;
}

}  // namespace

extern "C" {

const char* kq_last_error(void) { return g_err.c_str(); }

const char* kq_version(void) { return "kq 0.1 (gfx950)"; }

int kq_codec_from_name(const char* name, int* codec) {
  if (!name || !codec) return fail(KQ_ERR_ARG, "kq_codec_from_name", "null argument");
  char low[16];
  size_t i = 0;
  for (; name[i] && i + 1 < sizeof low; ++i) low[i] = (char)tolower((unsigned char)name[i]);
  low[i] = 0;
  static const struct { const char* n; int c; } table[] = {
      {"q4_0", KQ_Q4_0}, {"q8_0", KQ_Q8_0}, {"q4_k", KQ_Q4_K}, {"q5_k", KQ_Q5_K}, {"q6_k", KQ_Q6_K},
      {"q4_1", KQ_Q4_1}, {"q5_0", KQ_Q5_0}, {"q5_1", KQ_Q5_1}, {"q2_k", KQ_Q2_K}, {"q3_k", KQ_Q3_K}};
  for (const auto& t : table)
    if (!name[i] && strcmp(low, t.n) == 0) {
      *codec = t.c;
      return KQ_OK;
    }
  return fail(KQ_ERR_CODEC, "kq_codec_from_name", "unknown codec '%s' (known: q4_0, q4_1, q5_0, q5_1, q8_0, q2_k, q3_k, q4_k, q5_k, q6_k)", name);
}

int kq_codec_info(int codec, int* block_values, int* block_bytes) {
  int bv, bb;
  if (!geometry(codec, &bv, &bb)) return fail(KQ_ERR_CODEC, "kq_codec_info", "unknown codec id %d", codec);
  if (block_values) *block_values = bv;
  if (block_bytes) *block_bytes = bb;
  return KQ_OK;
}

int kq_row_bytes(int codec, int64_t k, int64_t* row_bytes) {
  int64_t rb;
  int st = check_codec_k("kq_row_bytes", codec, k, &rb);
  if (st) return st;
  if (!row_bytes) return fail(KQ_ERR_ARG, "kq_row_bytes", "null output");
  *row_bytes = rb;
  return KQ_OK;
}

int kq_dequantize(int codec, const void* w, int64_t rows, int64_t k, void* out, int out_dtype, void* stream) {
  const char* op = "kq_dequantize";
  int64_t rb;
  int st = check_codec_k(op, codec, k, &rb);
  if (st) return st;
  if ((st = check_dtype(op, out_dtype))) return st;
  if (rows < 0 || rows >= kMaxDim || rows * k >= kMaxElems)
    return fail(KQ_ERR_ARG, op, "rows=%lld out of range", (long long)rows);
  if (rows == 0) return KQ_OK;
  if (!w || !out) return fail(KQ_ERR_ARG, op, "null pointer (w=%p out=%p)", w, out);
  if (!aligned(w, 16)) return fail(KQ_ERR_ALIGN, op, "w=%p is not 16-byte aligned", w);
  if (!aligned(out, 16)) return fail(KQ_ERR_ALIGN, op, "out=%p is not 16-byte aligned", out);
  return hip_status(op, kq::launch_dequantize(codec, (const uint8_t*)w, rows, k, rb, out, out_dtype == KQ_F16,
                                              (hipStream_t)stream));
}

int kq_qmv(int codec, const void* w, int64_t n, int64_t k, const void* x, int64_t m, void* y, int y_dtype,
           void* stream) {
  const char* op = "kq_qmv";
  int64_t rb;
  int st = check_matmul(op, codec, w, n, k, x, m, y, y_dtype, &rb);
  if (st) return st;
  if (m > kq::QMV_MAX_M)
    return fail(KQ_ERR_SHAPE, op, "M=%lld rows; the GEMV takes 1..%d (use kq_qmm)", (long long)m, kq::QMV_MAX_M);
  if (n == 0 || m == 0) return KQ_OK;
  return hip_status(op, kq::launch_qmv(codec, (const uint8_t*)w, n, k, rb, (const kq::half_t*)x, (int)m, y,
                                       y_dtype == KQ_F16, (hipStream_t)stream));
}

int kq_qmm(int codec, const void* w, int64_t n, int64_t k, const void* x, int64_t m, void* y, int y_dtype,
           void* stream) {
  const char* op = "kq_qmm";
  int64_t rb;
  int st = check_matmul(op, codec, w, n, k, x, m, y, y_dtype, &rb);
  if (st) return st;
  if (n == 0 || m == 0) return KQ_OK;
  return hip_status(op, kq::launch_qmm(codec, (const uint8_t*)w, n, k, rb, (const kq::half_t*)x, m, y,
                                       y_dtype == KQ_F16, (hipStream_t)stream));
}

int kq_quantized_matmul(int codec, const void* w, int64_t n, int64_t k, const void* x, int64_t m, void* y,
                        int y_dtype, void* stream) {
  // 17..64 rows: the wide matrix-core GEMV (kq_qmv takes it from 9 rows)
  if (m >= 0 && m <= kq::QMV_MAX_M) return kq_qmv(codec, w, n, k, x, m, y, y_dtype, stream);
  if (m <= kq::QMV_WIDE_MAX_M && k % 64 == 0) {
    const char* op = "kq_quantized_matmul";
    int64_t rb;
    int st = check_matmul(op, codec, w, n, k, x, m, y, y_dtype, &rb);
    if (st) return st;
    if (n == 0) return KQ_OK;
    return hip_status(op, kq::launch_qmv_wide(codec, (const uint8_t*)w, n, k, rb, (const kq::half_t*)x, (int)m, y,
                                              y_dtype == KQ_F16, (hipStream_t)stream));
  }
  return kq_qmm(codec, w, n, k, x, m, y, y_dtype, stream);
}

// [a, a + na) and [b, b + nb) share a byte
static bool overlaps(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t pa = (uintptr_t)a, pb = (uintptr_t)b;
  return pa < pb + (uintptr_t)nb && pb < pa + (uintptr_t)na;
}

int kq_quantized_matmul_residual(int codec, const void* w, int64_t n, int64_t k, const void* x, int64_t m,
                                 const void* residual, const void* gate, int64_t gate_rows, void* y, int y_dtype,
                                 void* stream) {
  const char* op = "kq_quantized_matmul_residual";
  int64_t rb;
  int st = check_matmul(op, codec, w, n, k, x, m, y, y_dtype, &rb);
  if (st) return st;
  if (gate && (gate_rows <= 0 || gate_rows > m || (m > 0 && m % gate_rows != 0)))
    return fail(KQ_ERR_SHAPE, op, "gate_rows=%lld must divide M=%lld", (long long)gate_rows, (long long)m);
  if (n == 0 || m == 0) return KQ_OK;
  if (!residual) return fail(KQ_ERR_ARG, op, "null residual");
  const int64_t es = y_dtype == KQ_F32 ? 4 : 2;
  if (!aligned(residual, es) || (gate && !aligned(gate, es)))
    return fail(KQ_ERR_ALIGN, op, "residual/gate must be element aligned");
  const int64_t ybytes = m * n * es;
  if (residual != y && overlaps(residual, ybytes, y, ybytes))
    return fail(KQ_ERR_ARG, op, "residual overlaps y without being y");
  if (gate && overlaps(gate, gate_rows * n * es, y, ybytes)) return fail(KQ_ERR_ARG, op, "gate overlaps y");
  const kq::Epi epi{residual, gate, nullptr, gate ? (int)(m / gate_rows) : 1};
  const bool f16 = y_dtype == KQ_F16;
  const kq::half_t* xh = (const kq::half_t*)x;
  hipError_t e;
  // the dot2 GEMV body (its cost grows with M); q8_0 keeps it to 4 rows, as
  // kq_qmv does, because its decode costs the matrix-core GEMV more per byte
  const int64_t dot2_max_m = codec == KQ_Q8_0 ? 4 : 2;
  if (m <= dot2_max_m || (m <= 8 && k % 64 != 0))
    e = kq::launch_qmv_epi(codec, (const uint8_t*)w, n, k, rb, xh, (int)m, epi, y, f16, (hipStream_t)stream);
  else if (m <= kq::QMV_WIDE_MAX_M && k % 64 == 0)  // small batches: the wide matrix-core GEMV
    e = kq::launch_qmv_wide_epi(codec, (const uint8_t*)w, n, k, rb, xh, (int)m, epi, y, f16, (hipStream_t)stream);
  else
    e = kq::launch_qmm_epi(codec, (const uint8_t*)w, n, k, rb, xh, m, epi, y, f16, (hipStream_t)stream);
  return hip_status(op, e);
}

int kq_quantized_matmul_qmv_bias(int codec, const void* w, int64_t n, int64_t k, const void* x, int64_t m,
                                 const void* bias, void* y, int y_dtype, void* stream) {
  const char* op = "kq_quantized_matmul_qmv_bias";
  int64_t rb;
  int st = check_matmul(op, codec, w, n, k, x, m, y, y_dtype, &rb);
  if (st) return st;
  if (m != 1) return fail(KQ_ERR_SHAPE, op, "M=%lld rows; the bias-fused GEMV takes exactly one", (long long)m);
  if (n == 0) return KQ_OK;
  if (!bias) return fail(KQ_ERR_ARG, op, "null bias");
  const int64_t es = y_dtype == KQ_F32 ? 4 : 2;
  if (!aligned(bias, es)) return fail(KQ_ERR_ALIGN, op, "bias must be element aligned");
  if (overlaps(bias, n * es, y, n * es)) return fail(KQ_ERR_ARG, op, "bias overlaps y");
  const kq::Epi epi{nullptr, nullptr, bias, 1};
  return hip_status(op, kq::launch_qmv_epi(codec, (const uint8_t*)w, n, k, rb, (const kq::half_t*)x, 1, epi, y,
                                           y_dtype == KQ_F16, (hipStream_t)stream));
}

int kq_quantized_matmul_glu(int codec, const void* w_gate, const void* w_up, int64_t n, int64_t k, const void* x,
                            int64_t m, int act, void* y, int y_dtype, void* stream) {
  const char* op = "kq_quantized_matmul_glu";
  int64_t rb;
  int st = check_matmul(op, codec, w_gate, n, k, x, m, y, y_dtype, &rb);
  if (st) return st;
  if (act != KQ_GLU_SILU && act != KQ_GLU_GELU_TANH)
    return fail(KQ_ERR_ARG, op, "act=%d is not KQ_GLU_SILU or KQ_GLU_GELU_TANH", act);
  if (n == 0 || m == 0) return KQ_OK;
  if (!w_up) return fail(KQ_ERR_ARG, op, "null w_up");
  if (!aligned(w_up, 16)) return fail(KQ_ERR_ALIGN, op, "w_up=%p is not 16-byte aligned", w_up);
  const bool f16 = y_dtype == KQ_F16;
  const kq::half_t* xh = (const kq::half_t*)x;
  hipError_t e;
  if (m <= kq::qmv_glu_max_m(codec)) {  // one GEMV pass over both weights
    e = kq::launch_qmv_glu(codec, (const uint8_t*)w_gate, (const uint8_t*)w_up, n, k, rb, xh, (int)m, act, y, f16,
                           (hipStream_t)stream);
  } else if (m <= kq::QMV_WIDE_MAX_M && k % 64 == 0) {  // two wide matrix-core GEMV passes
    e = kq::launch_qmv_wide_glu_act(codec, (const uint8_t*)w_gate, n, k, rb, xh, (int)m, act, y, f16,
                                    (hipStream_t)stream);
    if (e == hipSuccess)
      e = kq::launch_qmv_wide_glu_mul(codec, (const uint8_t*)w_up, n, k, rb, xh, (int)m, y, f16, (hipStream_t)stream);
  } else {  // two GEMM passes
    e = kq::launch_qmm_glu(codec, (const uint8_t*)w_gate, (const uint8_t*)w_up, n, k, rb, xh, m, act, y, f16,
                           (hipStream_t)stream);
  }
  return hip_status(op, e);
}

int64_t kq_expert_tile_map_capacity(int64_t rows, int64_t n_experts) {
  if (rows < 0 || n_experts < 0) return -1;
  return (rows + 63) / 64 + (n_experts < rows ? n_experts : rows);
}

int kq_expert_tile_map(const uint32_t* ids, int64_t rows, int64_t n_experts, uint32_t* map, uint32_t* counts,
                       int64_t cap, uint32_t* status, void* stream) {
  const char* op = "kq_expert_tile_map";
  if (rows < 0 || rows >= kMaxDim) return fail(KQ_ERR_ARG, op, "rows=%lld out of range", (long long)rows);
  if (n_experts <= 0 || n_experts >= kMaxDim)
    return fail(KQ_ERR_ARG, op, "n_experts=%lld out of range", (long long)n_experts);
  const int64_t need = kq_expert_tile_map_capacity(rows, n_experts);
  if (cap < need || cap >= kMaxDim)
    return fail(KQ_ERR_CAPACITY, op, "cap=%lld is below the bound %lld for rows=%lld, n_experts=%lld",
                (long long)cap, (long long)need, (long long)rows, (long long)n_experts);
  if (!counts || (rows > 0 && (!ids || !map))) return fail(KQ_ERR_ARG, op, "null pointer");
  if (!aligned(counts, 4) || (ids && !aligned(ids, 4)) || (map && !aligned(map, 4)) || (status && !aligned(status, 4)))
    return fail(KQ_ERR_ALIGN, op, "ids/map/counts/status must be 4-byte aligned");
  return hip_status(op, kq::launch_tile_map(ids, rows, n_experts, map, counts, cap, status, (hipStream_t)stream));
}

int kq_gather_qmm_seg(int codec, const void* w, int64_t n_experts, int64_t n, int64_t k, const void* x,
                      int64_t rows, const uint32_t* map, const uint32_t* counts, int64_t cap, void* y, int y_dtype,
                      void* stream) {
  const char* op = "kq_gather_qmm_seg";
  int64_t rb;
  int st = check_matmul(op, codec, w, n, k, x, rows, y, y_dtype, &rb);
  if (st) return st;
  if (n_experts <= 0 || n_experts >= kMaxDim || n_experts * n >= kMaxDim * 64)
    return fail(KQ_ERR_ARG, op, "n_experts=%lld out of range", (long long)n_experts);
  if (cap < 0 || cap >= kMaxDim) return fail(KQ_ERR_ARG, op, "cap=%lld out of range", (long long)cap);
  if (n == 0 || rows == 0 || cap == 0) return KQ_OK;
  if (!map || !counts) return fail(KQ_ERR_ARG, op, "null map or counts");
  if (!aligned(map, 4) || !aligned(counts, 4)) return fail(KQ_ERR_ALIGN, op, "map/counts must be 4-byte aligned");
  return hip_status(op, kq::launch_gather_qmm_seg(codec, (const uint8_t*)w, n_experts, n, k, rb,
                                                  (const kq::half_t*)x, rows, map, counts, cap, y,
                                                  y_dtype == KQ_F16, (hipStream_t)stream));
}

int kq_gather_mix(const void* y, int64_t rows, int64_t n, const uint32_t* inv_order, const float* scores,
                  int64_t tokens, int64_t top_k, void* out, int dtype, void* stream) {
  const char* op = "kq_gather_mix";
  int st = check_dtype(op, dtype);
  if (st) return st;
  if (rows < 0 || rows >= kMaxDim) return fail(KQ_ERR_ARG, op, "rows=%lld out of range", (long long)rows);
  if (n < 0 || n >= kMaxDim) return fail(KQ_ERR_ARG, op, "N=%lld out of range", (long long)n);
  if (tokens < 0 || tokens >= kMaxDim) return fail(KQ_ERR_ARG, op, "tokens=%lld out of range", (long long)tokens);
  if (top_k < 0 || top_k >= kMaxDim || (top_k && tokens >= kMaxDim / top_k))
    return fail(KQ_ERR_ARG, op, "top_k=%lld out of range", (long long)top_k);
  if (n % 4) return fail(KQ_ERR_SHAPE, op, "N=%lld is not a multiple of 4", (long long)n);
  if (rows * n >= kMaxElems || tokens * n >= kMaxElems)
    return fail(KQ_ERR_ARG, op, "tensor too large (rows=%lld tokens=%lld N=%lld)", (long long)rows, (long long)tokens,
                (long long)n);
  if (n == 0 || tokens == 0) return KQ_OK;
  const int vec = 4 * (dtype == KQ_F16 ? 2 : 4);
  if (!out) return fail(KQ_ERR_ARG, op, "null out");
  if (!aligned(out, vec)) return fail(KQ_ERR_ALIGN, op, "out=%p is not aligned to 4 elements", out);
  if (top_k > 0) {
    if (!inv_order || !scores || (rows > 0 && !y)) return fail(KQ_ERR_ARG, op, "null y, inv_order or scores");
    if (y && !aligned(y, vec)) return fail(KQ_ERR_ALIGN, op, "y=%p is not aligned to 4 elements", y);
    if (!aligned(inv_order, 4) || !aligned(scores, 4))
      return fail(KQ_ERR_ALIGN, op, "inv_order/scores must be 4-byte aligned");
  }
  return hip_status(op, kq::launch_gather_mix(y, rows, n, inv_order, scores, tokens, top_k, out, dtype == KQ_F16,
                                              (hipStream_t)stream));
}

int kq_gather_qmv(int codec, const void* w, int64_t n_experts, int64_t n, int64_t k, const void* x,
                  const uint32_t* ids, int64_t rows, void* y, int y_dtype, void* stream) {
  const char* op = "kq_gather_qmv";
  int64_t rb;
  int st = check_matmul(op, codec, w, n, k, x, rows, y, y_dtype, &rb);
  if (st) return st;
  if (k % 256)
    return fail(KQ_ERR_SHAPE, op, "K=%lld is not a multiple of 256 (one activation row per slot)", (long long)k);
  if (n_experts <= 0 || n_experts >= kMaxDim || n_experts * n >= kMaxDim * 64)
    return fail(KQ_ERR_ARG, op, "n_experts=%lld out of range", (long long)n_experts);
  if (n == 0 || rows == 0) return KQ_OK;
  if (!ids) return fail(KQ_ERR_ARG, op, "null ids");
  if (!aligned(ids, 4)) return fail(KQ_ERR_ALIGN, op, "ids=%p is not 4-byte aligned", (const void*)ids);
  return hip_status(op, kq::launch_gather_qmv(codec, (const uint8_t*)w, n_experts, n, k, rb, (const kq::half_t*)x,
                                              ids, rows, y, y_dtype == KQ_F16, (hipStream_t)stream));
}

int kq_moe_glu_gather(int codec, const void* gate_w, const void* up_w, int64_t n_experts, int64_t n, int64_t k,
                      const void* x, int64_t tokens, const uint32_t* ids, int64_t top_k, int act, float limit,
                      void* y, int y_dtype, void* stream) {
  const char* op = "kq_moe_glu_gather";
  if (tokens < 0 || tokens >= kMaxDim) return fail(KQ_ERR_ARG, op, "tokens=%lld out of range", (long long)tokens);
  if (top_k < 0 || top_k >= kMaxDim || (top_k && tokens >= kMaxDim / top_k))
    return fail(KQ_ERR_ARG, op, "top_k=%lld out of range", (long long)top_k);
  const int64_t rows = tokens * top_k;
  int64_t rb;
  int st = check_matmul(op, codec, gate_w, n, k, x, rows, y, y_dtype, &rb);
  if (st) return st;
  if (k % 256)
    return fail(KQ_ERR_SHAPE, op, "K=%lld is not a multiple of 256 (one activation row per token)", (long long)k);
  if (n_experts <= 0 || n_experts >= kMaxDim || n_experts * n >= kMaxDim * 64)
    return fail(KQ_ERR_ARG, op, "n_experts=%lld out of range", (long long)n_experts);
  if (act != KQ_GLU_SILU && act != KQ_GLU_GELU_TANH && act != KQ_GLU_SILU_LIMIT)
    return fail(KQ_ERR_ARG, op, "act=%d is not a kq_glu_act", act);
  if (act == KQ_GLU_SILU_LIMIT && !(limit > 0.f && limit <= 3.0e38f))
    return fail(KQ_ERR_ARG, op, "limit=%g must be finite and > 0 for KQ_GLU_SILU_LIMIT", (double)limit);
  if (n == 0 || rows == 0) return KQ_OK;
  if (!up_w) return fail(KQ_ERR_ARG, op, "null up_w");
  if (!aligned(up_w, 16)) return fail(KQ_ERR_ALIGN, op, "up_w=%p is not 16-byte aligned", up_w);
  if (!ids) return fail(KQ_ERR_ARG, op, "null ids");
  if (!aligned(ids, 4)) return fail(KQ_ERR_ALIGN, op, "ids=%p is not 4-byte aligned", (const void*)ids);
  return hip_status(op, kq::launch_moe_glu_gather(codec, (const uint8_t*)gate_w, (const uint8_t*)up_w, n_experts, n,
                                                  k, rb, (const kq::half_t*)x, ids, rows, top_k, act, limit, y,
                                                  y_dtype == KQ_F16, (hipStream_t)stream));
}

int kq_quantize(int codec, const float* w, int64_t rows, int64_t k, void* out, void* stream) {
  const char* op = "kq_quantize";
  int64_t rb;
  int st = check_codec_k(op, codec, k, &rb);
  if (st) return st;
  if (rows < 0 || rows >= kMaxDim || rows * k >= kMaxElems)
    return fail(KQ_ERR_ARG, op, "rows=%lld out of range", (long long)rows);
  if (rows == 0) return KQ_OK;
  if (!w || !out) return fail(KQ_ERR_ARG, op, "null pointer (w=%p out=%p)", (const void*)w, out);
  if (!aligned(w, 16) || !aligned(out, 16)) return fail(KQ_ERR_ALIGN, op, "w and out must be 16-byte aligned");
  return hip_status(op, kq::launch_quantize(codec, w, rows, k, rb, (uint8_t*)out, (hipStream_t)stream));
}

int kq_stream_read(const void* src, int64_t bytes, uint32_t* out, int64_t groups, void* stream) {
  const char* op = "kq_stream_read";
  if (bytes < 0 || bytes % 16 != 0 || bytes >= kMaxElems)
    return fail(KQ_ERR_ARG, op, "bytes=%lld must be a non-negative multiple of 16", (long long)bytes);
  if (groups < 1 || groups > (1 << 20)) return fail(KQ_ERR_ARG, op, "groups=%lld out of 1..2^20", (long long)groups);
  // out holds 4 * groups words (one per wave)
  if (!src || !out) return fail(KQ_ERR_ARG, op, "null pointer (src=%p out=%p)", src, (void*)out);
  if (!aligned(src, 16) || !aligned(out, 4)) return fail(KQ_ERR_ALIGN, op, "src must be 16-byte, out 4-byte aligned");
  return hip_status(op, kq::launch_stream_read(src, bytes, out, groups, (hipStream_t)stream));
}

// ---- bfloat16 activations ----
// y dtype: KQ_F32, KQ_F16 or KQ_BF16 (2)
static int bf16_out(int y_dtype) { return y_dtype == KQ_BF16 ? 2 : y_dtype == KQ_F16 ? 1 : 0; }

int kq_qmv_bf16(int codec, const void* w, int64_t n, int64_t k, const void* x, int64_t m, void* y, int y_dtype,
                void* stream) {
  const char* op = "kq_qmv_bf16";
  int64_t rb;
  int st = check_matmul(op, codec, w, n, k, x, m, y, y_dtype, &rb, true);
  if (st) return st;
  if (m > kq::QMV_MAX_M)
    return fail(KQ_ERR_SHAPE, op, "M=%lld rows; the GEMV takes 1..%d (use kq_qmm_bf16)", (long long)m, kq::QMV_MAX_M);
  if (n == 0 || m == 0) return KQ_OK;
  return hip_status(op, kq::launch_mm_bf16(codec, (const uint8_t*)w, n, k, rb, x, m, y, bf16_out(y_dtype),
                                           (hipStream_t)stream));
}

int kq_qmm_bf16(int codec, const void* w, int64_t n, int64_t k, const void* x, int64_t m, void* y, int y_dtype,
                void* stream) {
  const char* op = "kq_qmm_bf16";
  int64_t rb;
  int st = check_matmul(op, codec, w, n, k, x, m, y, y_dtype, &rb, true);
  if (st) return st;
  if (n == 0 || m == 0) return KQ_OK;
  return hip_status(op, kq::launch_mm_bf16(codec, (const uint8_t*)w, n, k, rb, x, m, y, bf16_out(y_dtype),
                                           (hipStream_t)stream));
}

int kq_gather_qmm_seg_bf16(int codec, const void* w, int64_t n_experts, int64_t n, int64_t k, const void* x,
                           int64_t rows, const uint32_t* map, const uint32_t* counts, int64_t cap, void* y,
                           int y_dtype, void* stream) {
  const char* op = "kq_gather_qmm_seg_bf16";
  int64_t rb;
  int st = check_matmul(op, codec, w, n, k, x, rows, y, y_dtype, &rb, true);
  if (st) return st;
  if (n_experts <= 0 || n_experts >= kMaxDim || n_experts * n >= kMaxDim * 64)
    return fail(KQ_ERR_ARG, op, "n_experts=%lld out of range", (long long)n_experts);
  if (cap < 0 || cap >= kMaxDim) return fail(KQ_ERR_ARG, op, "cap=%lld out of range", (long long)cap);
  if (n == 0 || rows == 0 || cap == 0) return KQ_OK;
  if (!map || !counts) return fail(KQ_ERR_ARG, op, "null map or counts");
  if (!aligned(map, 4) || !aligned(counts, 4)) return fail(KQ_ERR_ALIGN, op, "map/counts must be 4-byte aligned");
  return hip_status(op, kq::launch_seg_bf16(codec, (const uint8_t*)w, n_experts, n, k, rb, x, rows, map, counts, cap,
                                            y, bf16_out(y_dtype), (hipStream_t)stream));
}

// ---- key/value cache in 4 bits ----
namespace {

constexpr int64_t kMaxSeqs = 65536;

// codec, page, row size and kv heads of a cache; fills log2(page)
int check_cache(const char* op, int codec, int64_t page, int64_t d, int64_t heads, int* shift) {
  if (codec != KQ_Q4_0) return fail(KQ_ERR_CODEC, op, "codec id %d: the cache holds q4_0 blocks", codec);
  if (page < 16 || page > 4096 || (page & (page - 1)))
    return fail(KQ_ERR_SHAPE, op, "page=%lld is not a power of two in 16..4096", (long long)page);
  if (d < 32 || d > 256 || d % 32)
    return fail(KQ_ERR_SHAPE, op, "d=%lld is not a multiple of 32 in 32..256", (long long)d);
  if (heads < 1 || heads > 4096) return fail(KQ_ERR_ARG, op, "kv_heads=%lld out of 1..4096", (long long)heads);
  *shift = __builtin_ctzll((unsigned long long)page);
  return KQ_OK;
}

// the two caches: page count and pointers
int check_pages(const char* op, const void* kc, const void* vc, int64_t pages, int64_t page) {
  if (pages < 1 || pages * page >= kMaxDim || pages >= kMaxDim)
    return fail(KQ_ERR_ARG, op, "pages=%lld out of range", (long long)pages);
  if (!kc || !vc) return fail(KQ_ERR_ARG, op, "null cache (k_cache=%p v_cache=%p)", kc, vc);
  if (!aligned(kc, 16) || !aligned(vc, 16)) return fail(KQ_ERR_ALIGN, op, "caches must be 16-byte aligned");
  return KQ_OK;
}

int elem_bytes(int dt) { return dt == KQ_F32 ? 4 : 2; }
int elem_id(int dt) { return dt == KQ_F32 ? 0 : dt == KQ_F16 ? 1 : 2; }

int check_any_dtype(const char* op, const char* what, int dt) {
  if (dt != KQ_F32 && dt != KQ_F16 && dt != KQ_BF16)
    return fail(KQ_ERR_ARG, op, "%s dtype %d is not KQ_F32, KQ_F16 or KQ_BF16", what, dt);
  return KQ_OK;
}

int check_rows(const char* op, int64_t tokens, int64_t heads, int64_t d) {
  if (tokens < 0 || tokens >= kMaxDim || tokens * heads * d >= (int64_t)1 << 34)
    return fail(KQ_ERR_ARG, op, "tokens=%lld out of range", (long long)tokens);
  return KQ_OK;
}

int check_attn_sizes(const char* op, int64_t tokens, int64_t n_seqs, int64_t q_heads, int64_t kv_heads, int64_t d,
                     int64_t max_new, int64_t max_kv) {
  if (d < 32 || d > 256 || d % 32)
    return fail(KQ_ERR_SHAPE, op, "d=%lld is not a multiple of 32 in 32..256", (long long)d);
  if (kv_heads < 1 || kv_heads > 4096) return fail(KQ_ERR_ARG, op, "kv_heads=%lld out of 1..4096", (long long)kv_heads);
  if (q_heads < 1 || q_heads > 4096 || q_heads % kv_heads)
    return fail(KQ_ERR_SHAPE, op, "q_heads=%lld is not a multiple of kv_heads=%lld (at most 4096)", (long long)q_heads,
                (long long)kv_heads);
  if (tokens < 0 || tokens >= kMaxDim || tokens * q_heads >= (int64_t)1 << 25)
    return fail(KQ_ERR_ARG, op, "tokens=%lld out of range (tokens * q_heads below 2^25)", (long long)tokens);
  if (n_seqs < 0 || n_seqs > kMaxSeqs || n_seqs * kv_heads >= (int64_t)1 << 22)
    return fail(KQ_ERR_ARG, op, "n_seqs=%lld out of range (n_seqs * kv_heads below 2^22)", (long long)n_seqs);
  if (max_new < 1 || max_new >= kMaxDim) return fail(KQ_ERR_ARG, op, "max_new=%lld out of range", (long long)max_new);
  if (max_kv < 1 || max_kv >= kMaxDim) return fail(KQ_ERR_ARG, op, "max_kv=%lld out of range", (long long)max_kv);
  return KQ_OK;
}

}  // namespace

int kq_kv_page_bytes(int codec, int64_t page, int64_t d, int64_t* page_bytes) {
  const char* op = "kq_kv_page_bytes";
  int shift;
  const int st = check_cache(op, codec, page, d, 1, &shift);
  if (st) return st;
  if (!page_bytes) return fail(KQ_ERR_ARG, op, "null output");
  *page_bytes = page * (d / 2 + d / 16);
  return KQ_OK;
}

int kq_block_tables(const int32_t* ctx_lens, const int32_t* new_lens, int64_t n_seqs, int64_t page,
                    const int32_t* free_pages, int64_t n_free, const int32_t* free_head, int32_t* table,
                    int64_t width, int32_t* slots, int64_t tokens, int32_t* cu_new, int32_t* seq_lens,
                    int32_t* free_head_out, uint32_t* status, void* stream) {
  const char* op = "kq_block_tables";
  int shift;
  const int st = check_cache(op, KQ_Q4_0, page, 32, 1, &shift);
  if (st) return st;
  if (n_seqs < 0 || n_seqs > kMaxSeqs) return fail(KQ_ERR_ARG, op, "n_seqs=%lld out of range", (long long)n_seqs);
  if (n_free < 0 || n_free >= kMaxDim) return fail(KQ_ERR_ARG, op, "n_free=%lld out of range", (long long)n_free);
  if (width < 0 || width >= kMaxDim || n_seqs * width >= kMaxElems)
    return fail(KQ_ERR_ARG, op, "width=%lld out of range", (long long)width);
  if (tokens < 0 || tokens >= kMaxDim) return fail(KQ_ERR_ARG, op, "tokens=%lld out of range", (long long)tokens);
  if (!free_head || !free_head_out || !cu_new) return fail(KQ_ERR_ARG, op, "null free_head, free_head_out or cu_new");
  if (n_seqs > 0 && (!ctx_lens || !new_lens || !seq_lens || (width > 0 && !table)))
    return fail(KQ_ERR_ARG, op, "null ctx_lens, new_lens, table or seq_lens");
  if ((n_free > 0 && !free_pages) || (tokens > 0 && !slots)) return fail(KQ_ERR_ARG, op, "null free_pages or slots");
  const void* in[] = {ctx_lens, new_lens, free_pages, free_head};
  const int64_t in_n[] = {n_seqs, n_seqs, n_free, 1};
  const void* out[] = {table, slots, cu_new, seq_lens, free_head_out, status};
  const int64_t out_n[] = {n_seqs * width, tokens, n_seqs + 1, n_seqs, 1, 1};
  for (int i = 0; i < 6; ++i) {
    if (!out[i] || out_n[i] == 0) continue;
    if (!aligned(out[i], 4)) return fail(KQ_ERR_ALIGN, op, "arrays must be 4-byte aligned");
    for (int j = 0; j < 4; ++j)
      if (in[j] && overlaps(in[j], 4 * in_n[j], out[i], 4 * out_n[i]))
        return fail(KQ_ERR_ARG, op, "an output overlaps an input");
    for (int j = 0; j < i; ++j)
      if (out[j] && overlaps(out[j], 4 * out_n[j], out[i], 4 * out_n[i]))
        return fail(KQ_ERR_ARG, op, "two outputs overlap");
  }
  for (const void* p : in)
    if (p && !aligned(p, 4)) return fail(KQ_ERR_ALIGN, op, "arrays must be 4-byte aligned");
  return hip_status(op, kq::launch_block_tables(ctx_lens, new_lens, n_seqs, shift, free_pages, n_free, free_head,
                                                table, width, slots, tokens, cu_new, seq_lens, free_head_out, status,
                                                (hipStream_t)stream));
}

int kq_kv_store(int codec, const void* k, const void* v, int x_dtype, int64_t tokens, int64_t kv_heads, int64_t d,
                int64_t k_stride, int64_t v_stride, const int32_t* slots, void* k_cache, void* v_cache,
                int64_t pages, int64_t page, void* stream) {
  const char* op = "kq_kv_store";
  int shift;
  int st = check_cache(op, codec, page, d, kv_heads, &shift);
  if (st) return st;
  if ((st = check_any_dtype(op, "row", x_dtype))) return st;
  if ((st = check_rows(op, tokens, kv_heads, d))) return st;
  if (k_stride < kv_heads * d || v_stride < kv_heads * d || k_stride >= kMaxDim || v_stride >= kMaxDim)
    return fail(KQ_ERR_SHAPE, op, "row strides k=%lld v=%lld out of range (kv_heads * d = %lld)", (long long)k_stride,
                (long long)v_stride, (long long)(kv_heads * d));
  if (k_stride % 8 || v_stride % 8)
    return fail(KQ_ERR_ALIGN, op, "row strides k=%lld v=%lld are not multiples of 8", (long long)k_stride,
                (long long)v_stride);
  if ((st = check_pages(op, k_cache, v_cache, pages, page))) return st;
  const int64_t cache = pages * kv_heads * page * (d / 2 + d / 16);
  if (overlaps(k_cache, cache, v_cache, cache)) return fail(KQ_ERR_ARG, op, "k_cache and v_cache overlap");
  if (tokens == 0) return KQ_OK;
  if (!k || !v || !slots) return fail(KQ_ERR_ARG, op, "null pointer (k=%p v=%p slots=%p)", k, v, (const void*)slots);
  if (!aligned(k, 16) || !aligned(v, 16)) return fail(KQ_ERR_ALIGN, op, "k=%p, v=%p are not 16-byte aligned", k, v);
  if (!aligned(slots, 4)) return fail(KQ_ERR_ALIGN, op, "slots=%p is not 4-byte aligned", (const void*)slots);
  const int64_t es = elem_bytes(x_dtype), row = kv_heads * d;
  for (const void* c : {k_cache, v_cache})
    if (overlaps(k, ((tokens - 1) * k_stride + row) * es, c, cache) ||
        overlaps(v, ((tokens - 1) * v_stride + row) * es, c, cache) || overlaps(slots, 4 * tokens, c, cache))
      return fail(KQ_ERR_ARG, op, "k, v or slots overlap a cache");
  return hip_status(op, kq::launch_kv_store(k, v, elem_id(x_dtype), tokens, kv_heads, d, k_stride, v_stride, slots,
                                            (uint8_t*)k_cache, (uint8_t*)v_cache, pages, shift, (hipStream_t)stream));
}

int kq_kv_load(int codec, const void* k_cache, const void* v_cache, int64_t pages, int64_t page, int64_t kv_heads,
               int64_t d, const int32_t* slots, int64_t tokens, void* k, void* v, int out_dtype, void* stream) {
  const char* op = "kq_kv_load";
  int shift;
  int st = check_cache(op, codec, page, d, kv_heads, &shift);
  if (st) return st;
  if ((st = check_any_dtype(op, "output", out_dtype))) return st;
  if ((st = check_rows(op, tokens, kv_heads, d))) return st;
  if ((st = check_pages(op, k_cache, v_cache, pages, page))) return st;
  if (tokens == 0) return KQ_OK;
  if (!k || !v || !slots) return fail(KQ_ERR_ARG, op, "null pointer (k=%p v=%p slots=%p)", k, v, (const void*)slots);
  if (!aligned(k, 16) || !aligned(v, 16)) return fail(KQ_ERR_ALIGN, op, "k=%p, v=%p are not 16-byte aligned", k, v);
  if (!aligned(slots, 4)) return fail(KQ_ERR_ALIGN, op, "slots=%p is not 4-byte aligned", (const void*)slots);
  const int64_t bytes = tokens * kv_heads * d * elem_bytes(out_dtype);
  if (overlaps(k, bytes, v, bytes)) return fail(KQ_ERR_ARG, op, "k and v overlap");
  const int64_t cache = pages * kv_heads * page * (d / 2 + d / 16);
  for (const void* o : {k, v})
    if (overlaps(o, bytes, k_cache, cache) || overlaps(o, bytes, v_cache, cache) || overlaps(o, bytes, slots, 4 * tokens))
      return fail(KQ_ERR_ARG, op, "k or v overlaps a cache or slots");
  return hip_status(op, kq::launch_kv_load((const uint8_t*)k_cache, (const uint8_t*)v_cache, pages, shift, kv_heads, d,
                                           slots, tokens, k, v, elem_id(out_dtype), (hipStream_t)stream));
}

int kq_kv_attention_workspace(int64_t tokens, int64_t n_seqs, int64_t q_heads, int64_t kv_heads, int64_t d,
                              int64_t max_new, int64_t max_kv, int64_t* bytes) {
  const char* op = "kq_kv_attention_workspace";
  const int st = check_attn_sizes(op, tokens, n_seqs, q_heads, kv_heads, d, max_new, max_kv);
  if (st) return st;
  if (!bytes) return fail(KQ_ERR_ARG, op, "null output");
  *bytes = tokens == 0 || n_seqs == 0 ? 0 : kq::attn_plan(tokens, n_seqs, q_heads, kv_heads, d, max_new, max_kv, 0).bytes;
  return KQ_OK;
}

namespace {

// What kq_kv_attention, kq_kv_attention_sinks and kq_kv_attention_prefix are
// called with; the latter two's own are 0 and null elsewhere.
struct AttnCall {
  int codec;
  const void* q;
  int q_dtype;
  int64_t tokens, q_heads, kv_heads, d, q_stride;
  const int32_t *cu_new, *seq_lens;
  int64_t n_seqs;
  const int32_t* table;
  int64_t width;
  const void *k_cache, *v_cache;
  int64_t pages, page;
  float scale;
  int64_t window, sinks;
  const int32_t* prefix;
  int64_t n_prefix, max_new, max_kv;
  void* out;
  int out_dtype;
  void* workspace;
  int64_t workspace_bytes;
  hipStream_t stream;
};

// A prefix of n_prefix pages: its keys, and the plan of the keys behind it.
kq::AttnPlan tail_plan(int64_t tokens, int64_t n_seqs, int64_t q_heads, int64_t kv_heads, int64_t d, int64_t max_new,
                       int64_t max_kv, int64_t prefix_len) {
  const int64_t own = max_kv > prefix_len ? max_kv - prefix_len : 1;
  kq::AttnPlan p = kq::attn_plan(tokens, n_seqs, q_heads, kv_heads, d, max_new, own, 0);
  kq::plan_tiles(p, tokens, q_heads, kv_heads, d, own);
  return p;
}

int check_prefix(const char* op, int64_t prefix_len) {
  if (prefix_len < 1 || prefix_len >= (int64_t)1 << 30)
    return fail(KQ_ERR_ARG, op, "a prefix of %lld keys is out of range (1 .. 2^30 - 1)", (long long)prefix_len);
  return KQ_OK;
}

int attention(const char* op, const AttnCall& c) {
  int shift;
  int st = check_cache(op, c.codec, c.page, c.d, c.kv_heads, &shift);
  if (st) return st;
  if ((st = check_attn_sizes(op, c.tokens, c.n_seqs, c.q_heads, c.kv_heads, c.d, c.max_new, c.max_kv))) return st;
  if (c.q_dtype != KQ_F16 && c.q_dtype != KQ_BF16)
    return fail(KQ_ERR_ARG, op, "query dtype %d is not KQ_F16 or KQ_BF16", c.q_dtype);
  if ((st = check_any_dtype(op, "output", c.out_dtype))) return st;
  if (c.q_stride < c.q_heads * c.d || c.q_stride >= kMaxDim)
    return fail(KQ_ERR_SHAPE, op, "row stride %lld out of range (q_heads * d = %lld)", (long long)c.q_stride,
                (long long)(c.q_heads * c.d));
  if (c.q_stride % 8) return fail(KQ_ERR_ALIGN, op, "row stride %lld is not a multiple of 8", (long long)c.q_stride);
  if (c.width < 0 || c.width * c.page >= (int64_t)1 << 30 || c.width >= (int64_t)1 << 30)
    return fail(KQ_ERR_ARG, op, "width=%lld out of range (width * page below 2^30)", (long long)c.width);
  if (!(c.scale >= -3.0e38f && c.scale <= 3.0e38f))
    return fail(KQ_ERR_ARG, op, "scale=%g is not finite", (double)c.scale);
  if (c.window < 0) return fail(KQ_ERR_ARG, op, "window=%lld is negative", (long long)c.window);
  if (c.sinks < 0) return fail(KQ_ERR_ARG, op, "sinks=%lld is negative", (long long)c.sinks);
  // no request is that long
  const int64_t window = c.window >= (int64_t)1 << 30 || c.sinks >= (int64_t)1 << 30 ? 0 : c.window;
  const int64_t sinks = window > 0 ? c.sinks : 0;
  int64_t prefix_len = 0;
  if (c.prefix) {
    if (c.n_prefix < 1 || c.n_prefix >= (int64_t)1 << 30)
      return fail(KQ_ERR_ARG, op, "n_prefix=%lld out of range", (long long)c.n_prefix);
    prefix_len = c.n_prefix * c.page;
    if ((st = check_prefix(op, prefix_len))) return st;
  }
  if ((st = check_pages(op, c.k_cache, c.v_cache, c.pages, c.page))) return st;
  if (c.tokens == 0 || c.n_seqs == 0) return KQ_OK;
  if (!c.q || !c.out || !c.cu_new || !c.seq_lens || (c.width > 0 && !c.table))
    return fail(KQ_ERR_ARG, op, "null pointer (q=%p out=%p cu_new=%p seq_lens=%p table=%p)", c.q, c.out,
                (const void*)c.cu_new, (const void*)c.seq_lens, (const void*)c.table);
  if (!aligned(c.q, 16) || !aligned(c.out, 16))
    return fail(KQ_ERR_ALIGN, op, "q=%p, out=%p are not 16-byte aligned", c.q, c.out);
  if (!aligned(c.cu_new, 4) || !aligned(c.seq_lens, 4) || !aligned(c.table, 4) || !aligned(c.prefix, 4))
    return fail(KQ_ERR_ALIGN, op, "cu_new, seq_lens and table must be 4-byte aligned");
  const int64_t out_bytes = c.tokens * c.q_heads * c.d * elem_bytes(c.out_dtype);
  // what the call reads, against what it writes
  const int64_t cache = c.pages * c.kv_heads * c.page * (c.d / 2 + c.d / 16);
  const struct { const char* name; const void* p; int64_t bytes; } in[] = {
      {"q", c.q, ((c.tokens - 1) * c.q_stride + c.q_heads * c.d) * 2}, {"cu_new", c.cu_new, 4 * (c.n_seqs + 1)},
      {"seq_lens", c.seq_lens, 4 * c.n_seqs}, {"table", c.table, 4 * c.n_seqs * c.width}, {"k_cache", c.k_cache, cache},
      {"v_cache", c.v_cache, cache}, {"prefix", c.prefix, 4 * c.n_prefix}};
  for (const auto& r : in)
    if (r.bytes > 0 && overlaps(r.p, r.bytes, c.out, out_bytes)) return fail(KQ_ERR_ARG, op, "out overlaps %s", r.name);
  const kq::AttnPlan plan =
      c.prefix ? tail_plan(c.tokens, c.n_seqs, c.q_heads, c.kv_heads, c.d, c.max_new, c.max_kv, prefix_len)
      : sinks > 0
          ? kq::sinks_plan(c.tokens, c.n_seqs, c.q_heads, c.kv_heads, c.d, c.max_new, c.max_kv, window, sinks)
          : kq::attn_plan(c.tokens, c.n_seqs, c.q_heads, c.kv_heads, c.d, c.max_new, c.max_kv, window);
  kq::PrefixPlan flat = {0, 0, 0, 0};
  if (c.prefix) flat = kq::prefix_plan(c.tokens, c.q_heads, c.kv_heads, c.d, prefix_len);
  // (a prefix: the bytes of all smaller calls, what this one takes among them)
  const int64_t need =
      c.prefix ? kq::prefix_need(c.tokens, c.q_heads, c.kv_heads, c.d, prefix_len, c.max_new, c.max_kv) : plan.bytes;
  if (need > 0) {
    if (!c.workspace || c.workspace_bytes < need)
      return fail(KQ_ERR_CAPACITY, op, "workspace of %lld bytes is below the %lld these sizes need",
                  (long long)(c.workspace ? c.workspace_bytes : 0), (long long)need);
    if (!aligned(c.workspace, 16)) return fail(KQ_ERR_ALIGN, op, "workspace=%p is not 16-byte aligned", c.workspace);
    if (overlaps(c.workspace, need, c.out, out_bytes)) return fail(KQ_ERR_ARG, op, "workspace overlaps out");
    for (const auto& r : in)
      if (r.bytes > 0 && overlaps(r.p, r.bytes, c.workspace, need))
        return fail(KQ_ERR_ARG, op, "workspace overlaps %s", r.name);
  }
  uint8_t* ws = (uint8_t*)c.workspace;
  kq::AttnArgs a;
  a.q = c.q;
  a.cu = c.cu_new;
  a.lens = c.seq_lens;
  a.table = c.table;
  a.kc = (const uint8_t*)c.k_cache;
  a.vc = (const uint8_t*)c.v_cache;
  a.out = c.out;
  a.many = (float*)(ws + flat.bytes);
  a.few = (float*)(ws + flat.bytes + plan.few_at);
  a.where = plan.bytes > 0 ? (int32_t*)(ws + flat.bytes + plan.where_at) : nullptr;
  a.q_stride = c.q_stride;
  a.width = c.width;
  a.page_head_bytes = c.page * (c.d / 2 + c.d / 16);
  a.tokens = (int)c.tokens;
  a.n_seqs = (int)c.n_seqs;
  a.hq = (int)c.q_heads;
  a.hkv = (int)c.kv_heads;
  a.group = (int)(c.q_heads / c.kv_heads);
  a.group_shift = (a.group & (a.group - 1)) ? -1 : __builtin_ctz((unsigned)a.group);
  a.d = (int)c.d;
  a.pages = (int)c.pages;
  a.page_shift = shift;
  a.window = (int)window;
  a.scale = c.scale;
  a.q_bf16 = c.q_dtype == KQ_BF16;
  a.out_type = elem_id(c.out_dtype);
  a.few_rows = plan.few_rows;
  a.one_tile = plan.one_tile;
  a.few_wgs = plan.few_wgs;
  a.many_wgs = plan.many_wgs;
  a.many_shift = __builtin_ctz((unsigned)kq::attn_prompt_rows(c.d));
  a.sinks = (int)sinks;
  a.prefix = c.prefix;
  a.prefix_len = (int)prefix_len;
  a.splits = flat.splits;
  a.prefix_sums = (float*)ws;
  if (c.prefix) return hip_status(op, kq::launch_kv_attention_prefix(a, plan, flat, c.stream));
  if (sinks > 0) return hip_status(op, kq::launch_kv_attention_sinks(a, plan, c.stream));
  return hip_status(op, kq::launch_kv_attention(a, plan, c.stream));
}

}  // namespace

int kq_kv_attention(int codec, const void* q, int q_dtype, int64_t tokens, int64_t q_heads, int64_t kv_heads,
                    int64_t d, int64_t q_stride, const int32_t* cu_new, const int32_t* seq_lens, int64_t n_seqs,
                    const int32_t* table, int64_t width, const void* k_cache, const void* v_cache, int64_t pages,
                    int64_t page, float scale, int64_t window, int64_t max_new, int64_t max_kv, void* out,
                    int out_dtype, void* workspace, int64_t workspace_bytes, void* stream) {
  return attention("kq_kv_attention",
                   AttnCall{codec, q, q_dtype, tokens, q_heads, kv_heads, d, q_stride, cu_new, seq_lens, n_seqs, table,
                            width, k_cache, v_cache, pages, page, scale, window, 0, nullptr, 0, max_new, max_kv, out,
                            out_dtype, workspace, workspace_bytes, (hipStream_t)stream});
}

int kq_kv_attention_sinks(int codec, const void* q, int q_dtype, int64_t tokens, int64_t q_heads, int64_t kv_heads,
                          int64_t d, int64_t q_stride, const int32_t* cu_new, const int32_t* seq_lens, int64_t n_seqs,
                          const int32_t* table, int64_t width, const void* k_cache, const void* v_cache, int64_t pages,
                          int64_t page, float scale, int64_t window, int64_t sinks, int64_t max_new, int64_t max_kv,
                          void* out, int out_dtype, void* workspace, int64_t workspace_bytes, void* stream) {
  return attention("kq_kv_attention_sinks",
                   AttnCall{codec, q, q_dtype, tokens, q_heads, kv_heads, d, q_stride, cu_new, seq_lens, n_seqs, table,
                            width, k_cache, v_cache, pages, page, scale, window, sinks, nullptr, 0, max_new, max_kv,
                            out, out_dtype, workspace, workspace_bytes, (hipStream_t)stream});
}

int kq_kv_attention_prefix_workspace(int64_t tokens, int64_t n_seqs, int64_t q_heads, int64_t kv_heads, int64_t d,
                                     int64_t prefix_len, int64_t max_new, int64_t max_kv, int64_t* bytes) {
  const char* op = "kq_kv_attention_prefix_workspace";
  int st = check_attn_sizes(op, tokens, n_seqs, q_heads, kv_heads, d, max_new, max_kv);
  if (st) return st;
  if ((st = check_prefix(op, prefix_len))) return st;
  if (!bytes) return fail(KQ_ERR_ARG, op, "null output");
  *bytes = tokens == 0 || n_seqs == 0
               ? 0
               : kq::prefix_need(tokens, q_heads, kv_heads, d, prefix_len, max_new, max_kv);
  return KQ_OK;
}

int kq_kv_attention_prefix(int codec, const void* q, int q_dtype, int64_t tokens, int64_t q_heads, int64_t kv_heads,
                           int64_t d, int64_t q_stride, const int32_t* cu_new, const int32_t* seq_lens, int64_t n_seqs,
                           const int32_t* table, int64_t width, const int32_t* prefix, int64_t n_prefix,
                           const void* k_cache, const void* v_cache, int64_t pages, int64_t page, float scale,
                           int64_t max_new, int64_t max_kv, void* out, int out_dtype, void* workspace,
                           int64_t workspace_bytes, void* stream) {
  if (!prefix) return fail(KQ_ERR_ARG, "kq_kv_attention_prefix", "null prefix");
  return attention("kq_kv_attention_prefix",
                   AttnCall{codec, q, q_dtype, tokens, q_heads, kv_heads, d, q_stride, cu_new, seq_lens, n_seqs, table,
                            width, k_cache, v_cache, pages, page, scale, 0, 0, prefix, n_prefix, max_new, max_kv, out,
                            out_dtype, workspace, workspace_bytes, (hipStream_t)stream});
}

// ---- pages of the cache ----

namespace {

// Device arrays of 32-bit integers of a call: alignment, and no output over an
// input or another output (`same` inputs may be the output of that index).
struct Ints {
  const char* name;
  const void* p;
  int64_t n;
  int out;       // 0 read, 1 written
  int in_place;  // 1 + index of the entry that this output may be
};
int check_ints(const char* op, const Ints* x, int n) {
  for (int i = 0; i < n; ++i) {
    if (x[i].n <= 0 || !x[i].p) continue;
    if (!aligned(x[i].p, 4)) return fail(KQ_ERR_ALIGN, op, "%s=%p is not 4-byte aligned", x[i].name, x[i].p);
    if (!x[i].out) continue;
    for (int j = 0; j < n; ++j) {
      if (j == i || x[j].n <= 0 || !x[j].p || (x[i].in_place == 1 + j && x[i].p == x[j].p)) continue;
      if (x[j].out && j > i) continue;  // seen from there
      if (overlaps(x[j].p, 4 * x[j].n, x[i].p, 4 * x[i].n))
        return fail(KQ_ERR_ARG, op, "%s overlaps %s", x[i].name, x[j].name);
    }
  }
  return KQ_OK;
}
int check_count(const char* op, const char* name, int64_t n, int64_t least, int64_t most) {
  if (n < least || n > most)
    return fail(KQ_ERR_ARG, op, "%s=%lld out of %lld..%lld", name, (long long)n, (long long)least, (long long)most);
  return KQ_OK;
}
int check_table(const char* op, int64_t n_seqs, int64_t width) {
  int st = check_count(op, "n_seqs", n_seqs, 0, kMaxSeqs);
  if (st || (st = check_count(op, "width", width, 0, kMaxDim - 1))) return st;
  return n_seqs * width >= kMaxElems ? fail(KQ_ERR_ARG, op, "width=%lld out of range", (long long)width) : KQ_OK;
}

}  // namespace

int kq_kv_fork(const int32_t* parents, const int32_t* children, const int32_t* lens, int64_t n, int64_t page,
               int32_t* table, int64_t n_seqs, int64_t width, int32_t* refs, int64_t pages, const int32_t* free_pages,
               int64_t n_free, const int32_t* free_head, int32_t* copy_src, int32_t* copy_dst, int32_t* free_head_out,
               uint32_t* status, void* stream) {
  const char* op = "kq_kv_fork";
  int shift;
  int st = check_cache(op, KQ_Q4_0, page, 32, 1, &shift);
  if (st || (st = check_count(op, "n", n, 0, kMaxSeqs)) || (st = check_table(op, n_seqs, width)) ||
      (st = check_count(op, "pages", pages, 1, kMaxDim - 1)) || (st = check_count(op, "n_free", n_free, 0, kMaxDim - 1)))
    return st;
  if (!free_head || !free_head_out) return fail(KQ_ERR_ARG, op, "null free_head or free_head_out");
  if (n > 0 && (!parents || !children || !lens || !copy_src || !copy_dst || !refs || (n_seqs * width > 0 && !table)))
    return fail(KQ_ERR_ARG, op, "null parents, children, lens, table, refs, copy_src or copy_dst");
  if (n_free > 0 && !free_pages) return fail(KQ_ERR_ARG, op, "null free_pages");
  const Ints x[] = {{"parents", parents, n, 0, 0}, {"children", children, n, 0, 0}, {"lens", lens, n, 0, 0},
                    {"free_pages", free_pages, n_free, 0, 0}, {"free_head", free_head, 1, 0, 0},
                    {"table", table, n_seqs * width, 1, 0}, {"refs", refs, pages, 1, 0}, {"copy_src", copy_src, n, 1, 0},
                    {"copy_dst", copy_dst, n, 1, 0}, {"free_head_out", free_head_out, 1, 1, 0}, {"status", status, 1, 1, 0}};
  if ((st = check_ints(op, x, 11))) return st;
  return hip_status(op, kq::launch_kv_fork(parents, children, lens, n, shift, table, n_seqs, width, refs, pages, free_pages,
                                           n_free, free_head, copy_src, copy_dst, free_head_out, status,
                                           (hipStream_t)stream));
}

int kq_kv_free(const int32_t* first, const int32_t* last, int64_t n_seqs, const int32_t* table, int64_t width,
               int32_t* refs, int64_t pages, int32_t* free_pages, int64_t n_free, const int32_t* free_head,
               int32_t* free_head_out, uint32_t* status, void* stream) {
  const char* op = "kq_kv_free";
  int st = check_table(op, n_seqs, width);
  if (st || (st = check_count(op, "pages", pages, 1, kMaxDim - 1)) || (st = check_count(op, "n_free", n_free, 0, kMaxDim - 1)))
    return st;
  if (!refs || !free_head || !free_head_out) return fail(KQ_ERR_ARG, op, "null refs, free_head or free_head_out");
  if (n_seqs > 0 && (!first || !last || (width > 0 && !table))) return fail(KQ_ERR_ARG, op, "null first, last or table");
  if (n_free > 0 && !free_pages) return fail(KQ_ERR_ARG, op, "null free_pages");
  const Ints x[] = {{"first", first, n_seqs, 0, 0}, {"last", last, n_seqs, 0, 0}, {"table", table, n_seqs * width, 0, 0},
                    {"free_head", free_head, 1, 0, 0}, {"refs", refs, pages, 1, 0}, {"free_pages", free_pages, n_free, 1, 0},
                    {"free_head_out", free_head_out, 1, 1, 0}, {"status", status, 1, 1, 0}};
  if ((st = check_ints(op, x, 8))) return st;
  return hip_status(op, kq::launch_kv_free(first, last, n_seqs, table, width, refs, pages, free_pages, n_free, free_head,
                                           free_head_out, status, (hipStream_t)stream));
}

int kq_kv_compact(const int32_t* free_pages, int64_t n_free, const int32_t* free_head, const int32_t* table,
                  int64_t n_entries, const int32_t* refs, int64_t pages, int32_t* table_out, int32_t* refs_out,
                  int32_t* free_out, int32_t* remap, int32_t* copy_src, int32_t* copy_dst, int64_t n_copy,
                  int32_t* free_head_out, uint32_t* status, void* stream) {
  const char* op = "kq_kv_compact";
  int st = check_count(op, "pages", pages, 1, kq::COMPACT_PAGES);
  if (st || (st = check_count(op, "n_free", n_free, 0, kMaxDim - 1)) ||
      (st = check_count(op, "n_entries", n_entries, 0, kMaxElems - 1)) ||
      (st = check_count(op, "n_copy", n_copy, 0, kMaxDim - 1)))
    return st;
  const int64_t most = pages / 2 < n_free ? pages / 2 : n_free;
  if (n_copy < most)
    return fail(KQ_ERR_CAPACITY, op, "n_copy=%lld is below the %lld pages that may move", (long long)n_copy, (long long)most);
  if (!free_head || !free_head_out || !remap || !refs || !refs_out)
    return fail(KQ_ERR_ARG, op, "null free_head, free_head_out, remap, refs or refs_out");
  if ((n_free > 0 && (!free_pages || !free_out)) || (n_entries > 0 && (!table || !table_out)) ||
      (n_copy > 0 && (!copy_src || !copy_dst)))
    return fail(KQ_ERR_ARG, op, "null free_pages, free_out, table, table_out, copy_src or copy_dst");
  const Ints x[] = {{"free_pages", free_pages, n_free, 0, 0}, {"free_head", free_head, 1, 0, 0},
                    {"table", table, n_entries, 0, 0}, {"refs", refs, pages, 0, 0}, {"table_out", table_out, n_entries, 1, 3},
                    {"refs_out", refs_out, pages, 1, 4}, {"free_out", free_out, n_free, 1, 1}, {"remap", remap, pages, 1, 0},
                    {"copy_src", copy_src, n_copy, 1, 0}, {"copy_dst", copy_dst, n_copy, 1, 0},
                    {"free_head_out", free_head_out, 1, 1, 2}, {"status", status, 1, 1, 0}};
  if ((st = check_ints(op, x, 12))) return st;
  return hip_status(op, kq::launch_kv_compact(free_pages, n_free, free_head, table, n_entries, refs, pages, table_out,
                                              refs_out, free_out, remap, copy_src, copy_dst, n_copy, free_head_out,
                                              status, (hipStream_t)stream));
}

int kq_kv_copy_pages(const int32_t* src, const int32_t* dst, int64_t n, void* k_cache, void* v_cache, int64_t pages,
                     int64_t bytes, void* stream) {
  const char* op = "kq_kv_copy_pages";
  int st = check_count(op, "n", n, 0, kMaxDim - 1);
  if (st || (st = check_count(op, "pages", pages, 1, kMaxDim - 1))) return st;
  if (bytes < 16 || bytes >= kMaxDim || bytes % 16)
    return fail(KQ_ERR_SHAPE, op, "bytes=%lld of a page is not a multiple of 16 below 2^31", (long long)bytes);
  if (!k_cache || !v_cache) return fail(KQ_ERR_ARG, op, "null cache (k_cache=%p v_cache=%p)", k_cache, v_cache);
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return fail(KQ_ERR_ALIGN, op, "caches must be 16-byte aligned");
  const int64_t cache = pages * bytes;
  if (overlaps(k_cache, cache, v_cache, cache)) return fail(KQ_ERR_ARG, op, "k_cache and v_cache overlap");
  if (n == 0) return KQ_OK;
  if (!src || !dst) return fail(KQ_ERR_ARG, op, "null src or dst");
  if (!aligned(src, 4) || !aligned(dst, 4)) return fail(KQ_ERR_ALIGN, op, "src and dst must be 4-byte aligned");
  for (const void* c : {k_cache, v_cache})
    if (overlaps(src, 4 * n, c, cache) || overlaps(dst, 4 * n, c, cache))
      return fail(KQ_ERR_ARG, op, "src or dst overlaps a cache");
  return hip_status(op, kq::launch_kv_copy_pages(src, dst, n, (uint8_t*)k_cache, (uint8_t*)v_cache, pages, bytes,
                                                 (hipStream_t)stream));
}

// ---- rotary positions ----

int kq_rope_freqs(int64_t rot, double base, int scaling, double factor, int64_t original, double fast, double slow,
                  const float* factors, float* inv_freq, float* mscale) {
  const char* op = "kq_rope_freqs";
  if (rot < 2 || rot > 4096 || rot % 2) return fail(KQ_ERR_SHAPE, op, "rot=%lld is not even in 2..4096", (long long)rot);
  if (!(base > 1. && base <= 1e30)) return fail(KQ_ERR_ARG, op, "base=%g is not above 1 (at most 1e30)", base);
  if (scaling < KQ_ROPE_NONE || scaling > KQ_ROPE_YARN) return fail(KQ_ERR_ARG, op, "scaling=%d is unknown", scaling);
  if (scaling != KQ_ROPE_NONE && !(factor >= 1. && factor <= 1e6))
    return fail(KQ_ERR_ARG, op, "factor=%g out of 1..1e6", factor);
  if (scaling == KQ_ROPE_NTK && rot < 4) return fail(KQ_ERR_SHAPE, op, "rot=%lld is below 4", (long long)rot);
  if (scaling == KQ_ROPE_YARN && (original < 1 || !(fast > slow && slow > 0. && fast <= 1e9)))
    return fail(KQ_ERR_ARG, op, "original=%lld, fast=%g, slow=%g: wanted are original >= 1 and fast > slow > 0",
                (long long)original, fast, slow);
  if (!inv_freq || !mscale) return fail(KQ_ERR_ARG, op, "null output");
  const int64_t pairs = rot / 2;
  if (factors)
    for (int64_t i = 0; i < pairs; ++i)
      if (!(factors[i] >= 1e-30f && factors[i] <= 1e30f))
        return fail(KQ_ERR_ARG, op, "factors[%lld]=%g out of 1e-30..1e30", (long long)i, factors[i]);
  // NTK: the lowest frequency is divided by `factor`, the highest stays
  if (scaling == KQ_ROPE_NTK) base *= std::pow(factor, (double)rot / (double)(rot - 2));
  double lo = 0., hi = 1.;
  if (scaling == KQ_ROPE_YARN) {
    // the pair that makes `turns` turns over the original length
    const auto at = [&](double turns) {
      return (double)rot * std::log((double)original / (turns * 2. * M_PI)) / (2. * std::log(base));
    };
    lo = std::floor(at(fast));
    hi = std::ceil(at(slow));
    lo = lo < 0. ? 0. : lo;
    hi = hi > (double)(rot - 1) ? (double)(rot - 1) : hi;
  }
  for (int64_t i = 0; i < pairs; ++i) {
    double f = std::pow(base, -2. * (double)i / (double)rot);
    if (factors) f /= (double)factors[i];
    if (scaling == KQ_ROPE_LINEAR) f /= factor;
    if (scaling == KQ_ROPE_YARN) {
      const double span = hi - lo > 0.001 ? hi - lo : 0.001;
      double r = ((double)i - lo) / span;
      r = r < 0. ? 0. : r > 1. ? 1. : r;
      f = f / factor * r + f * (1. - r);
    }
    inv_freq[i] = (float)f;
  }
  *mscale = scaling == KQ_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.) : 1.f;
  return KQ_OK;
}

namespace {

// Rows of heads * d elements, `stride` apart.
struct Rows {
  const void* p;
  int64_t stride, width;
};
// Whether rows of a and b (bytes) share any: rows of the same stride may lie
// side by side, as slices of one buffer do.
bool rows_overlap(const Rows& a, const Rows& b, int64_t tokens, int64_t es) {
  if (!a.p || !b.p || tokens == 0) return false;
  if (!overlaps(a.p, ((tokens - 1) * a.stride + a.width) * es, b.p, ((tokens - 1) * b.stride + b.width) * es)) return false;
  if (a.stride != b.stride) return true;
  const int64_t s = a.stride * es, at = (((intptr_t)b.p - (intptr_t)a.p) % s + s) % s;
  return at < a.width * es || at + b.width * es > s;
}

}  // namespace

int kq_rope(const void* q, int64_t q_heads, int64_t q_stride, const void* k, int64_t kv_heads, int64_t k_stride,
            int dtype, int64_t tokens, int64_t d, int64_t rot, int layout, const int32_t* cu_new,
            const int32_t* seq_lens, int64_t n_seqs, const float* inv_freq, float mscale, void* q_out,
            int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream) {
  const char* op = "kq_rope";
  int st = check_any_dtype(op, "row", dtype);
  if (st) return st;
  if (d < 32 || d > 256 || d % 32) return fail(KQ_ERR_SHAPE, op, "d=%lld is not a multiple of 32 in 32..256", (long long)d);
  if (rot < 8 || rot > d || rot % 8)
    return fail(KQ_ERR_SHAPE, op, "rot=%lld is not a multiple of 8 in 8..d=%lld", (long long)rot, (long long)d);
  if (layout != KQ_ROPE_HALF && layout != KQ_ROPE_PAIRS) return fail(KQ_ERR_ARG, op, "layout=%d is unknown", layout);
  if ((st = check_count(op, "q_heads", q_heads, 0, 4096)) || (st = check_count(op, "kv_heads", kv_heads, 0, 4096)) ||
      (st = check_count(op, "n_seqs", n_seqs, 0, kMaxSeqs)))
    return st;
  if (tokens < 0 || tokens >= kMaxDim || tokens * (q_heads + kv_heads) * d >= (int64_t)1 << 34)
    return fail(KQ_ERR_ARG, op, "tokens=%lld out of range", (long long)tokens);
  if (!(mscale >= -3.0e38f && mscale <= 3.0e38f)) return fail(KQ_ERR_ARG, op, "mscale=%g is not finite", (double)mscale);
  const struct { const char* name; int64_t stride, heads; } strides[] = {
      {"q", q_stride, q_heads}, {"k", k_stride, kv_heads}, {"q_out", q_out_stride, q_heads}, {"k_out", k_out_stride, kv_heads}};
  for (const auto& r : strides) {
    if (r.heads == 0) continue;
    if (r.stride < r.heads * d || r.stride >= kMaxDim)
      return fail(KQ_ERR_SHAPE, op, "%s's row stride %lld out of range (heads * d = %lld)", r.name, (long long)r.stride,
                  (long long)(r.heads * d));
    if (r.stride % 8) return fail(KQ_ERR_ALIGN, op, "%s's row stride %lld is not a multiple of 8", r.name, (long long)r.stride);
  }
  if (tokens == 0 || n_seqs == 0 || q_heads + kv_heads == 0) return KQ_OK;
  if ((q_heads > 0 && (!q || !q_out)) || (kv_heads > 0 && (!k || !k_out)) || !cu_new || !seq_lens || !inv_freq)
    return fail(KQ_ERR_ARG, op, "null pointer (q=%p k=%p cu_new=%p seq_lens=%p inv_freq=%p q_out=%p k_out=%p)", q, k,
                (const void*)cu_new, (const void*)seq_lens, (const void*)inv_freq, q_out, k_out);
  if (q_heads == 0) q = q_out = nullptr;
  if (kv_heads == 0) k = k_out = nullptr;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16))
    return fail(KQ_ERR_ALIGN, op, "q=%p, k=%p, q_out=%p, k_out=%p are not 16-byte aligned", q, k, q_out, k_out);
  if (!aligned(cu_new, 4) || !aligned(seq_lens, 4) || !aligned(inv_freq, 4))
    return fail(KQ_ERR_ALIGN, op, "cu_new, seq_lens and inv_freq must be 4-byte aligned");
  const int64_t es = elem_bytes(dtype);
  const Rows in[] = {{q, q_stride, q_heads * d}, {k, k_stride, kv_heads * d}};
  const Rows out[] = {{q_out, q_out_stride, q_heads * d}, {k_out, k_out_stride, kv_heads * d}};
  const struct { const char* name; const void* p; int64_t bytes; } small[] = {
      {"cu_new", cu_new, 4 * (n_seqs + 1)}, {"seq_lens", seq_lens, 4 * n_seqs}, {"inv_freq", inv_freq, 2 * rot}};
  for (int i = 0; i < 2; ++i) {
    const bool in_place = out[i].p == in[i].p && out[i].stride == in[i].stride;
    for (int j = 0; j < 2; ++j)
      if (!(i == j && in_place) && rows_overlap(out[i], in[j], tokens, es))
        return fail(KQ_ERR_ARG, op, "%s overlaps %s", i ? "k_out" : "q_out", j ? "k" : "q");
    if (out[i].p)
      for (const auto& r : small)
        if (overlaps(r.p, r.bytes, out[i].p, ((tokens - 1) * out[i].stride + out[i].width) * es))
          return fail(KQ_ERR_ARG, op, "%s overlaps %s", i ? "k_out" : "q_out", r.name);
  }
  if (rows_overlap(out[0], out[1], tokens, es)) return fail(KQ_ERR_ARG, op, "q_out and k_out overlap");
  kq::RopeArgs a;
  a.q = q;
  a.k = k;
  a.q_out = q_out;
  a.k_out = k_out;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.q_out_stride = q_out_stride;
  a.k_out_stride = k_out_stride;
  a.cu = cu_new;
  a.lens = seq_lens;
  a.inv_freq = inv_freq;
  a.mscale = mscale;
  a.tokens = (int)tokens;
  a.n_seqs = (int)n_seqs;
  a.hq = (int)q_heads;
  a.hkv = (int)kv_heads;
  a.d = (int)d;
  a.rot = (int)rot;
  a.copy_q = q_out != q || q_out_stride != q_stride;
  a.copy_k = k_out != k || k_out_stride != k_stride;
  return hip_status(op, kq::launch_rope(a, elem_id(dtype), layout == KQ_ROPE_PAIRS, (hipStream_t)stream));
}

}  // extern "C"
