// api.hip -- the C ABI of libconvrot.so (declared and documented in include/convrot.h).
//
// Host side only: argument validation (a pure function of the arguments, no HIP call),
// workspace carving, and the launches of the two kernels on the caller's stream. Nothing is
// allocated. The only state is rq_rotq_linear_noalloc's static device scratch and the per-device
// cache of its address.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdarg.h>
#include <stdio.h>

#include <mutex>
#include <string>

#include "convrot.h"
#include "internal.h"

namespace {

thread_local std::string g_detail;

constexpr int64_t kMaxK = 131072;          // int32 accumulators: 127^2 * K and 256 * 7^2 * K < 2^31
constexpr int64_t kMaxRowsOrCols = (int64_t(1) << 31) - 1;

rq_status fail(rq_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
rq_status fail(rq_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_detail = buf;
  return s;
}

rq_status ok() { return RQ_OK; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int64_t elem_size(int32_t dt) { return dt == RQ_F32 ? 4 : 2; }

int64_t code_bytes(int64_t rows, int64_t K, int bits) { return bits == 8 ? rows * K : rows * K / 2; }

// FP6 tiles: 48 bytes per 64 codes, rows padded to whole panels.
int64_t fp6_bytes(int64_t rows, int64_t K, int64_t panel) { return (rows + panel - 1) / panel * panel * (K / 64) * 48; }

// Activation codes in a layout: the tiled layouts pad the rows to whole 256-row panels.
int64_t x_code_bytes(int64_t rows, int64_t K, int bits, int32_t layout) {
  if (layout == RQ_X_FP6) return fp6_bytes(rows, K, 256);
  const int64_t r = layout == RQ_X_TILED ? (rows + 255) / 256 * 256 : rows;
  return code_bytes(r, K, bits);
}

// Weight codes in a layout: FP6 tiles pad the rows to whole 128-row panels.
int64_t w_code_bytes(int64_t rows, int64_t K, int bits, int32_t layout) {
  return layout == RQ_W_FP6 ? fp6_bytes(rows, K, 128) : code_bytes(rows, K, bits);
}

// The activation layout the fused call uses inside its workspace: FP6 tiles to match FP6
// weights, else the tiled int layout.
int32_t fused_x_layout(const rq_qconfig* cfg) { return cfg->w_layout == RQ_W_FP6 ? RQ_X_FP6 : RQ_X_TILED; }

int code_layout(int32_t x_layout) {
  return x_layout == RQ_X_FP6 ? convrot::kCodeFp6X : x_layout == RQ_X_TILED ? convrot::kCodeTiled : convrot::kCodeRows;
}

int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }

bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  if (!a || !b || na <= 0 || nb <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

rq_status check_cfg(const rq_qconfig* cfg) {
  if (!cfg) return fail(RQ_EINVAL, "cfg is NULL");
  if (cfg->bits != 8 && cfg->bits != 4)
    return fail(RQ_EUNSUPPORTED, "bits = %d (supported: 8, 4)", cfg->bits);
  if (cfg->rot_kind != RQ_ROT_WHT)
    return fail(RQ_EUNSUPPORTED, "rot_kind = %d (supported: RQ_ROT_WHT)", cfg->rot_kind);
  if (cfg->rot_block != 128)
    return fail(RQ_EUNSUPPORTED, "rot_block = %d (supported: 128)", cfg->rot_block);
  if (cfg->x_layout != RQ_X_ROWS && cfg->x_layout != RQ_X_TILED && cfg->x_layout != RQ_X_FP6)
    return fail(RQ_EINVAL, "x_layout = %d (RQ_X_ROWS, RQ_X_TILED or RQ_X_FP6)", cfg->x_layout);
  if (cfg->w_layout != RQ_W_ROWS && cfg->w_layout != RQ_W_FP6)
    return fail(RQ_EINVAL, "w_layout = %d (RQ_W_ROWS or RQ_W_FP6)", cfg->w_layout);
  if ((cfg->x_layout == RQ_X_FP6 || cfg->w_layout == RQ_W_FP6) && cfg->bits != 4)
    return fail(RQ_EUNSUPPORTED, "FP6 code layouts hold 4-bit codes only (bits = %d)", cfg->bits);
  if (cfg->w_scale_mode != RQ_W_ABSMAX && cfg->w_scale_mode != RQ_W_MSE &&
      cfg->w_scale_mode != RQ_W_TENSOR)
    return fail(RQ_EINVAL, "w_scale_mode = %d (RQ_W_ABSMAX, RQ_W_MSE or RQ_W_TENSOR)",
                cfg->w_scale_mode);
  if (cfg->act != RQ_ACT_NONE && cfg->act != RQ_ACT_GELU_ERF && cfg->act != RQ_ACT_GELU_TANH)
    return fail(RQ_EINVAL, "act = %d (RQ_ACT_NONE, RQ_ACT_GELU_ERF or RQ_ACT_GELU_TANH)", cfg->act);
  return ok();
}

rq_status check_rows_k(int64_t rows, int64_t K, const char* what) {
  if (rows < 0) return fail(RQ_EINVAL, "%s rows = %lld < 0", what, (long long)rows);
  if (rows > kMaxRowsOrCols) return fail(RQ_EUNSUPPORTED, "%s rows = %lld >= 2^31", what, (long long)rows);
  if (K < 128 || K % 128 != 0 || K > kMaxK)
    return fail(RQ_EUNSUPPORTED, "K = %lld (need a multiple of 128 in [128, %lld])", (long long)K,
                (long long)kMaxK);
  return ok();
}

rq_status check_gemm_shape(int64_t M, int64_t N, int64_t K) {
  rq_status s = check_rows_k(M, K, "M");
  if (s) return s;
  if (N <= 0 || N % 16 != 0 || N > kMaxRowsOrCols)
    return fail(RQ_EUNSUPPORTED, "N = %lld (need a positive multiple of 16 below 2^31)", (long long)N);
  return ok();
}

rq_status check_ptr(const void* p, const char* name, bool required = true) {
  if (!p) return required ? fail(RQ_EINVAL, "%s is NULL", name) : ok();
  if (!aligned16(p)) return fail(RQ_EINVAL, "%s is not 16-byte aligned", name);
  return ok();
}

rq_status from_hip(hipError_t e, const char* where) {
  if (e == hipSuccess) return RQ_OK;
  return fail(RQ_EHIP, "%s: %s", where, hipGetErrorString(e));
}

rq_status check_rotate_args(const void* X, int32_t dt, int64_t rows, int64_t K, const rq_qconfig* cfg,
                            const void* Q, const float* S, const char* xname, bool activations) {
  rq_status s = check_cfg(cfg);
  if (s) return s;
  if (dt != RQ_F32 && dt != RQ_F16 && dt != RQ_BF16) return fail(RQ_EINVAL, "bad %s dtype %d", xname, dt);
  if ((s = check_rows_k(rows, K, xname))) return s;
  if (rows == 0) return ok();
  if ((s = check_ptr(X, xname))) return s;
  if ((s = check_ptr(Q, "codes output"))) return s;
  if (!S) return fail(RQ_EINVAL, "scale output is NULL");
  if ((reinterpret_cast<uintptr_t>(S) & 3u) != 0) return fail(RQ_EINVAL, "scale output is not 4-byte aligned");
  const int64_t xb = rows * K * elem_size(dt);
  const int64_t qb = activations ? x_code_bytes(rows, K, cfg->bits, cfg->x_layout)
                                 : w_code_bytes(rows, K, cfg->bits, cfg->w_layout);
  if (overlap(X, xb, Q, qb) || overlap(X, xb, S, rows * 4) || overlap(Q, qb, S, rows * 4))
    return fail(RQ_EINVAL, "input, codes and scales must not overlap");
  return ok();
}

// Everything of rq_rotq_linear's arguments but the workspace (M == 0 passes here).
rq_status check_linear_core(const void* X, int32_t x_dtype, int64_t M, int64_t K, const void* Wq,
                            const float* w_scale, int64_t N, const float* bias,
                            const rq_qconfig* cfg, const void* Y) {
  rq_status s = check_cfg(cfg);
  if (s) return s;
  if (x_dtype != RQ_F16 && x_dtype != RQ_BF16)
    return fail(x_dtype == RQ_F32 ? RQ_EUNSUPPORTED : RQ_EINVAL,
                "X dtype %d (supported: RQ_F16, RQ_BF16; Y has X's dtype)", x_dtype);
  if ((s = check_gemm_shape(M, N, K))) return s;
  if (M == 0) return ok();
  if ((s = check_ptr(X, "X"))) return s;
  if ((s = check_ptr(Wq, "Wq"))) return s;
  if ((s = check_ptr(w_scale, "w_scale"))) return s;
  if ((s = check_ptr(bias, "bias", false))) return s;
  if ((s = check_ptr(Y, "Y"))) return s;
  const int64_t xb = M * K * 2, wb = w_code_bytes(N, K, cfg->bits, cfg->w_layout), yb = M * N * 2;
  if (overlap(Y, yb, X, xb) || overlap(Y, yb, Wq, wb) || overlap(Y, yb, w_scale, N * 4) ||
      overlap(Y, yb, bias, N * 4))
    return fail(RQ_EINVAL, "Y overlaps an input");
  return ok();
}

// The workspace part: size, alignment and no overlap with the other buffers (M > 0).
rq_status check_linear_ws(const void* X, int64_t M, int64_t K, const void* Wq, const float* w_scale,
                          int64_t N, const float* bias, const rq_qconfig* cfg, const void* Y,
                          const void* ws, size_t ws_bytes) {
  rq_status s = check_ptr(ws, "workspace");
  if (s) return s;
  const size_t need = rq_rotq_linear_workspace_size(M, K, cfg);
  if (ws_bytes < need)
    return fail(RQ_EWORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
  const int64_t xb = M * K * 2, wb = w_code_bytes(N, K, cfg->bits, cfg->w_layout), yb = M * N * 2;
  if (overlap(Y, yb, ws, (int64_t)need))
    return fail(RQ_EINVAL, "Y overlaps the workspace");
  if (overlap(ws, (int64_t)need, X, xb) || overlap(ws, (int64_t)need, Wq, wb) ||
      overlap(ws, (int64_t)need, w_scale, N * 4) || overlap(ws, (int64_t)need, bias, N * 4))
    return fail(RQ_EINVAL, "workspace overlaps an input");
  return ok();
}

rq_status check_linear(const void* X, int32_t x_dtype, int64_t M, int64_t K, const void* Wq,
                       const float* w_scale, int64_t N, const float* bias, const rq_qconfig* cfg,
                       const void* Y, const void* ws, size_t ws_bytes) {
  rq_status s = check_linear_core(X, x_dtype, M, K, Wq, w_scale, N, bias, cfg, Y);
  if (s || M == 0) return s;
  return check_linear_ws(X, M, K, Wq, w_scale, N, bias, cfg, Y, ws, ws_bytes);
}

// The two kernels of the quantized linear on an already validated call; `workspace` holds at
// least rq_rotq_linear_workspace_size(M, K, cfg) bytes.
rq_status launch_linear(const void* X, int32_t x_dtype, int64_t M, int64_t K, const void* Wq,
                        const float* w_scale, int64_t N, const float* bias, const rq_qconfig* cfg,
                        void* Y, void* workspace, hipStream_t st) {
  // The workspace holds the codes in the tiled layout (FP6 tiles with FP6 weights), then x_scale.
  const int32_t xl = fused_x_layout(cfg);
  uint8_t* Xq = static_cast<uint8_t*>(workspace);
  float* sx = reinterpret_cast<float*>(Xq + round256(x_code_bytes(M, K, cfg->bits, xl)));
  rq_status s;
  if ((s = from_hip(convrot::launch_rotate_quant(X, x_dtype, M, K, cfg->bits, code_layout(xl), Xq, sx, st),
                    "rotate_quant launch")))
    return s;
  if (xl == RQ_X_FP6)
    return from_hip(convrot::launch_gemm_fp6(Xq, sx, Wq, w_scale, bias, M, N, K, Y, x_dtype, nullptr,
                                             cfg->act, st),
                    "gemm launch");
  return from_hip(convrot::launch_gemm(Xq, sx, Wq, w_scale, bias, M, N, K, cfg->bits, true, Y,
                                       x_dtype, nullptr, cfg->act, st),
                  "gemm launch");
}

// ---- The entry point that allocates nothing: its workspace is `scratch`, a file-scope device
// array (one copy per GPU, held until the process ends). Host code never passes the array's
// name to a kernel: it is a host-side stand-in there. Its device address is looked up once per
// device with hipGetSymbolAddress, with that device current, and cached here.
__device__ __align__(256) uint8_t scratch[RQ_NOALLOC_SCRATCH_BYTES];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices];

rq_status scratch_of_current_device(void** out) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return from_hip(e, "hipGetDevice");
  if (dev < 0 || dev >= kMaxDevices)
    return fail(RQ_EUNSUPPORTED, "device %d (the static scratch serves devices 0..%d)", dev, kMaxDevices - 1);
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess) return from_hip(e, "hipGetSymbolAddress(scratch)");
    if (!p) return fail(RQ_EHIP, "hipGetSymbolAddress(scratch) returned NULL");
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return ok();
}

rq_status check_gemm(const void* Xq, const float* x_scale, const void* Wq, const float* w_scale,
                     const float* bias, int64_t M, int64_t N, int64_t K, const rq_qconfig* cfg,
                     const void* out, int64_t out_elem) {
  rq_status s = check_cfg(cfg);
  if (s) return s;
  if ((s = check_gemm_shape(M, N, K))) return s;
  if (M == 0) return ok();
  if ((s = check_ptr(Xq, "Xq"))) return s;
  if ((s = check_ptr(Wq, "Wq"))) return s;
  if ((s = check_ptr(out, "output"))) return s;
  if (x_scale && (reinterpret_cast<uintptr_t>(x_scale) & 3u)) return fail(RQ_EINVAL, "x_scale misaligned");
  if ((s = check_ptr(w_scale, "w_scale", out_elem != 4))) return s;
  if ((s = check_ptr(bias, "bias", false))) return s;
  if (out_elem != 4 && !x_scale) return fail(RQ_EINVAL, "x_scale is NULL");
  if ((cfg->x_layout == RQ_X_FP6) != (cfg->w_layout == RQ_W_FP6))
    return fail(RQ_EINVAL, "FP6 activation codes go with FP6 weight codes (x_layout %d, w_layout %d)",
                cfg->x_layout, cfg->w_layout);
  const int64_t ob = M * N * out_elem;
  if (overlap(out, ob, Xq, x_code_bytes(M, K, cfg->bits, cfg->x_layout)) ||
      overlap(out, ob, Wq, w_code_bytes(N, K, cfg->bits, cfg->w_layout)) ||
      overlap(out, ob, x_scale, M * 4) || overlap(out, ob, w_scale, N * 4) || overlap(out, ob, bias, N * 4))
    return fail(RQ_EINVAL, "output overlaps an input");
  return ok();
}

// ---- the cache operators
constexpr int64_t kMaxKvTokens = int64_t(1) << 30;   // of a sequence's page table
constexpr int64_t kMaxKvBytes = int64_t(1) << 46;    // of a cache, and of what strided rows span
constexpr int64_t kMaxKvRows = int64_t(1) << 30;     // query rows times heads

int log2_of(int32_t n) {
  int l = 0;
  while ((1 << l) < n) l++;
  return l;
}

rq_status check_kv_cfg(const rq_kv_config* cfg) {
  if (!cfg) return fail(RQ_EINVAL, "cfg is NULL");
  if (cfg->bits != 8 && cfg->bits != 4) return fail(RQ_EUNSUPPORTED, "bits = %d (supported: 8, 4)", cfg->bits);
  if (cfg->head_dim != 64 && cfg->head_dim != 128 && cfg->head_dim != 256)
    return fail(RQ_EUNSUPPORTED, "head_dim = %d (supported: 64, 128, 256)", cfg->head_dim);
  if (cfg->kv_heads < 1 || cfg->kv_heads > 65535)
    return fail(RQ_EUNSUPPORTED, "kv_heads = %d (supported: 1 .. 65535)", cfg->kv_heads);
  const int32_t ps = cfg->page_size;
  if (ps < 16 || ps > 1024 || (ps & (ps - 1)) != 0)
    return fail(RQ_EUNSUPPORTED, "page_size = %d (supported: powers of two in 16 .. 1024)", ps);
  return ok();
}

int64_t kv_head_bytes(const rq_kv_config* cfg) {
  return (int64_t)cfg->page_size * (2 * (cfg->head_dim * cfg->bits / 8) + 8);
}

rq_status check_kv_cache(const void* cache, int64_t num_pages, const rq_kv_config* cfg) {
  rq_status s = check_ptr(cache, "cache");
  if (s) return s;
  if (num_pages < 1 || num_pages > kMaxRowsOrCols)
    return fail(num_pages < 1 ? RQ_EINVAL : RQ_EUNSUPPORTED, "num_pages = %lld (need 1 .. 2^31 - 1)", (long long)num_pages);
  if (num_pages > kMaxKvBytes / (kv_head_bytes(cfg) * cfg->kv_heads))
    return fail(RQ_EUNSUPPORTED, "the cache has over 2^46 bytes (%lld pages)", (long long)num_pages);
  return ok();
}

// Rows [tokens, heads, dim] at p with strides in elements of `es` bytes; returns their extent in
// bytes. Output rows must not overlap one another.
rq_status check_kv_rows(const void* p, const char* name, int64_t tokens, int64_t heads, int64_t dim, int64_t es,
                        int64_t token_stride, int64_t head_stride, bool out, int64_t* bytes) {
  rq_status s = check_ptr(p, name);
  if (s) return s;
  constexpr int64_t kMost = int64_t(1) << 40;
  if (tokens == 1) token_stride = 0;   // a single one's stride is never taken
  if (heads == 1) head_stride = 0;
  if (token_stride < 0 || head_stride < 0 || token_stride > kMost || head_stride > kMost)
    return fail(RQ_EINVAL, "%s strides (%lld, %lld) out of range", name, (long long)token_stride, (long long)head_stride);
  if (token_stride * es % 16 != 0 || head_stride * es % 16 != 0)
    return fail(RQ_EINVAL, "%s strides (%lld, %lld) are not multiples of 16 bytes", name, (long long)token_stride,
                (long long)head_stride);
  if (out) {
    // Heads within a token, or tokens within a head: one lies inside the other's stride. In
    // 128 bits: 2^31 rows at strides up to 2^40 elements pass 64.
    typedef __int128 wide;
    const wide over_heads = (wide)(heads - 1) * head_stride + dim, over_tokens = (wide)(tokens - 1) * token_stride + dim;
    const bool h_in_t = (heads == 1 || head_stride >= dim) && (tokens == 1 || token_stride >= over_heads);
    const bool t_in_h = (tokens == 1 || token_stride >= dim) && (heads == 1 || head_stride >= over_tokens);
    if (!h_in_t && !t_in_h)
      return fail(RQ_EINVAL, "%s strides (%lld, %lld): rows overlap", name, (long long)token_stride, (long long)head_stride);
  }
  const __int128 extent = ((__int128)(tokens - 1) * token_stride + (__int128)(heads - 1) * head_stride + dim) * es;
  if (extent > kMaxKvBytes) return fail(RQ_EUNSUPPORTED, "%s spans over 2^46 bytes", name);
  *bytes = (int64_t)extent;
  return ok();
}

// Two sets of rows of `dim` elements in one buffer, each set's rows apart from one another: 1 if a row of one
// meets a row of the other, 0 if none does, -1 if that is not worked out.
// `n` rows at 0, ks, 2 ks, .. and at r, r + vs, ...
int rows_meet(int64_t n, int64_t dim, int64_t ks, int64_t vs, int64_t r) {
  if (n == 1) return r > -dim && r < dim;
  if (ks == vs) {   // r plus a multiple of the stride, next to 0 on either side
    int64_t j = r >= 0 ? -(r / ks) - 1 : -r / ks;
    for (const int64_t last = j + 1; j <= last; j++)
      if (j > -n && j < n && r + j * ks > -dim && r + j * ks < dim) return 1;
    return 0;
  }
  if (n > 65536) return -1;
  for (int64_t i = 0, j = 0; i < n && j < n;) {
    const int64_t d = r + j * vs - i * ks;
    if (d > -dim && d < dim) return 1;
    if (d < 0)
      j++;
    else
      i++;
  }
  return 0;
}
// `outer` groups of `inner` rows, the groups `stride` apart in both sets and each as long as that at most.
int groups_meet(int64_t outer, int64_t stride, int64_t inner, int64_t dim, int64_t ks, int64_t vs, int64_t r) {
  if (outer == 1) return rows_meet(inner, dim, ks, vs, r);
  const int64_t k_len = (inner - 1) * ks + dim, v_len = (inner - 1) * vs + dim;
  int64_t i = (-v_len - r) / stride - 1;   // the groups that may meet begin between -v_len and k_len
  for (; r + i * stride < k_len; i++) {
    if (i <= -outer || i >= outer) continue;
    const int m = rows_meet(inner, dim, ks, vs, r + i * stride);
    if (m) return m;
  }
  return 0;
}

// K and V as outputs: no row of one on a row of the other. (K's rows are apart already, V's too.)
rq_status check_kv_apart(const void* K, int64_t kb, const void* V, int64_t vb, int64_t es, int64_t tokens, int64_t heads,
                         int64_t dim, int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head) {
  if (!overlap(K, kb, V, vb)) return ok();
  const int64_t r = (int64_t)(reinterpret_cast<intptr_t>(V) - reinterpret_cast<intptr_t>(K)) / es;   // both 16-byte aligned
  // Groups of one axis inside the other's stride, in both sets.
  auto inside = [&](int64_t inner, int64_t s, int64_t outer, int64_t stride) {
    return outer == 1 || (inner == 1 ? stride >= dim : stride >= (inner - 1) * s + dim);
  };
  int m = -1;
  if ((tokens == 1 || k_token == v_token) && inside(heads, k_head, tokens, k_token) && inside(heads, v_head, tokens, v_token))
    m = groups_meet(tokens, k_token, heads, dim, heads == 1 ? 0 : k_head, heads == 1 ? 0 : v_head, r);
  else if ((heads == 1 || k_head == v_head) && inside(tokens, k_token, heads, k_head) && inside(tokens, v_token, heads, v_head))
    m = groups_meet(heads, k_head, tokens, dim, tokens == 1 ? 0 : k_token, tokens == 1 ? 0 : v_token, r);
  if (m == 1) return fail(RQ_EINVAL, "K and V overlap");
  if (m < 0) return fail(RQ_EUNSUPPORTED, "K and V lie in each other with strides (%lld, %lld) and (%lld, %lld)",
                         (long long)k_token, (long long)k_head, (long long)v_token, (long long)v_head);
  return ok();
}

rq_status check_kv_rw(const void* K, const void* V, int32_t dtype, int64_t tokens, int64_t k_token, int64_t k_head,
                      int64_t v_token, int64_t v_head, const int64_t* slots, const rq_kv_config* cfg, const void* cache,
                      int64_t num_pages, bool out) {
  rq_status s = check_kv_cfg(cfg);
  if (s) return s;
  if (dtype != RQ_F32 && dtype != RQ_F16 && dtype != RQ_BF16) return fail(RQ_EINVAL, "bad K / V dtype %d", dtype);
  if (tokens < 0) return fail(RQ_EINVAL, "tokens = %lld < 0", (long long)tokens);
  if (tokens > kMaxRowsOrCols) return fail(RQ_EUNSUPPORTED, "tokens = %lld >= 2^31", (long long)tokens);
  if ((s = check_kv_cache(cache, num_pages, cfg))) return s;
  if (tokens == 0) return ok();
  const int64_t es = elem_size(dtype);
  int64_t kb = 0, vb = 0;
  if ((s = check_kv_rows(K, "K", tokens, cfg->kv_heads, cfg->head_dim, es, k_token, k_head, out, &kb))) return s;
  if ((s = check_kv_rows(V, "V", tokens, cfg->kv_heads, cfg->head_dim, es, v_token, v_head, out, &vb))) return s;
  if (out && (s = check_kv_apart(K, kb, V, vb, es, tokens, cfg->kv_heads, cfg->head_dim, k_token, k_head, v_token, v_head)))
    return s;
  if (!slots) return fail(RQ_EINVAL, "slots is NULL");
  if ((reinterpret_cast<uintptr_t>(slots) & 7u) != 0) return fail(RQ_EINVAL, "slots is not 8-byte aligned");
  const int64_t cb = num_pages * kv_head_bytes(cfg) * cfg->kv_heads;
  if (overlap(cache, cb, K, kb) || overlap(cache, cb, V, vb) || overlap(cache, cb, slots, tokens * 8))
    return fail(RQ_EINVAL, "the cache overlaps K, V or slots");
  if (out && (overlap(K, kb, slots, tokens * 8) || overlap(V, vb, slots, tokens * 8)))
    return fail(RQ_EINVAL, "K or V overlaps slots");
  return ok();
}

convrot::KvCacheArgs kv_cache_args(int32_t dtype, int64_t tokens, int64_t k_token, int64_t k_head, int64_t v_token,
                                   int64_t v_head, const int64_t* slots, const rq_kv_config* cfg, const void* cache,
                                   int64_t num_pages) {
  convrot::KvCacheArgs a = {};
  a.cache = static_cast<uint8_t*>(const_cast<void*>(cache));
  a.slots = slots;
  a.k_token = k_token;
  a.k_head = k_head;
  a.v_token = v_token;
  a.v_head = v_head;
  a.tokens = tokens;
  a.num_pages = num_pages;
  a.head_bytes = kv_head_bytes(cfg);
  a.heads = cfg->kv_heads;
  a.lps = log2_of(cfg->page_size);
  a.dt = dtype;
  return a;
}

// Everything the sizes of an attention call are taken from; the lengths that choose the split.
rq_status check_kv_shape(const rq_kv_attention_params* p, const rq_kv_config* cfg, int64_t* max_q, int64_t* max_kv) {
  rq_status s = check_kv_cfg(cfg);
  if (s) return s;
  if (!p) return fail(RQ_EINVAL, "params is NULL");
  if (p->dtype != RQ_F16 && p->dtype != RQ_BF16)
    return fail(p->dtype == RQ_F32 ? RQ_EUNSUPPORTED : RQ_EINVAL, "Q dtype %d (supported: RQ_F16, RQ_BF16)", p->dtype);
  if (p->seqs < 0 || p->total_q < 0 || p->max_pages < 0 || p->window < 0)
    return fail(RQ_EINVAL, "seqs = %d, total_q = %lld, max_pages = %d, window = %d: none may be negative", p->seqs,
                (long long)p->total_q, p->max_pages, p->window);
  if (p->seqs > 65535) return fail(RQ_EUNSUPPORTED, "seqs = %d > 65535", p->seqs);
  if (p->q_heads < 1 || p->q_heads % cfg->kv_heads != 0)
    return fail(RQ_EINVAL, "q_heads = %d is not a positive multiple of kv_heads = %d", p->q_heads, cfg->kv_heads);
  if (p->total_q > kMaxKvRows || p->total_q * p->q_heads > kMaxKvRows)
    return fail(RQ_EUNSUPPORTED, "total_q * q_heads = %lld * %d > 2^30", (long long)p->total_q, p->q_heads);
  if ((int64_t)p->max_pages * cfg->page_size > kMaxKvTokens)
    return fail(RQ_EUNSUPPORTED, "max_pages * page_size = %d * %d > 2^30", p->max_pages, cfg->page_size);
  if (p->window > 0 && !p->causal) return fail(RQ_EINVAL, "window needs causal");
  if (!(p->softmax_scale > 0.0f) || p->softmax_scale > 3.4028234e38f)
    return fail(RQ_EINVAL, "softmax_scale = %g (need a finite value > 0)", (double)p->softmax_scale);
  if (p->total_q > 0 && p->seqs == 0) return fail(RQ_EINVAL, "seqs = 0 with total_q = %lld", (long long)p->total_q);
  if (!p->q_start && p->seqs > 0 && p->total_q % p->seqs != 0)
    return fail(RQ_EINVAL, "total_q = %lld is not a multiple of seqs = %d, and q_start is NULL", (long long)p->total_q, p->seqs);
  const int64_t kv = (int64_t)p->max_pages * cfg->page_size;
  *max_q = p->max_q_len < 1 || p->max_q_len > p->total_q ? p->total_q : p->max_q_len;
  if (!p->q_start && p->seqs > 0) *max_q = p->total_q / p->seqs;
  *max_kv = p->max_kv_len < 1 || p->max_kv_len > kv ? kv : p->max_kv_len;
  return ok();
}

rq_status check_kv_attention(const rq_kv_attention_params* p, const rq_kv_config* cfg, const void* cache,
                             int64_t num_pages, const void* ws, size_t ws_bytes, convrot::KvAttentionPlan* plan,
                             int64_t* max_q_len) {
  int64_t max_q = 0, max_kv = 0;
  rq_status s = check_kv_shape(p, cfg, &max_q, &max_kv);
  if (s) return s;
  if ((s = check_kv_cache(cache, num_pages, cfg))) return s;
  if (p->total_q == 0) return ok();
  int64_t qb = 0, ob = 0;
  if ((s = check_kv_rows(p->Q, "Q", p->total_q, p->q_heads, cfg->head_dim, 2, p->q_token_stride, p->q_head_stride, false, &qb)))
    return s;
  if ((s = check_kv_rows(p->O, "O", p->total_q, p->q_heads, cfg->head_dim, 2, p->o_token_stride, p->o_head_stride, true, &ob)))
    return s;
  if (!p->kv_len || (!p->pages && p->max_pages > 0)) return fail(RQ_EINVAL, "kv_len or pages is NULL");
  const void* words[4] = {p->kv_len, p->pages, p->q_start, p->lse};
  for (const void* w : words)
    if ((reinterpret_cast<uintptr_t>(w) & 3u) != 0)
      return fail(RQ_EINVAL, "kv_len, pages, q_start or lse is not 4-byte aligned");
  *max_q_len = max_q;
  *plan = convrot::plan_kv_attention(p->total_q, p->seqs, p->q_heads, cfg->kv_heads, cfg->head_dim, max_q, max_kv, p->window);
  // A grid has fewer than 2^32 threads, 256 a workgroup. (Splits come with few rows: the join's fits.)
  if (((int64_t)p->seqs * plan->splits + 8) * cfg->kv_heads >= ((int64_t)1 << 24) / plan->row_tiles)
    return fail(RQ_EUNSUPPORTED, "%d sequences of up to %lld query rows: too many workgroups (give max_q_len)", p->seqs,
                (long long)max_q);
  const int64_t need = (int64_t)plan->workspace_bytes;
  if (need > 0) {
    if (ws_bytes < plan->workspace_bytes)
      return fail(RQ_EWORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, plan->workspace_bytes);
    if ((s = check_ptr(ws, "workspace"))) return s;
  }
  const struct { const void* at; int64_t bytes; } outs[3] = {{p->O, ob}, {p->lse, p->total_q * p->q_heads * 4}, {ws, need}},
                                                 ins[5] = {{p->Q, qb},
                                                           {cache, num_pages * kv_head_bytes(cfg) * cfg->kv_heads},
                                                           {p->kv_len, (int64_t)p->seqs * 4},
                                                           {p->q_start, (int64_t)(p->seqs + 1) * 4},
                                                           {p->pages, (int64_t)p->seqs * p->max_pages * 4}};
  for (int i = 0; i < 3; i++) {
    for (const auto& in : ins)
      if (overlap(outs[i].at, outs[i].bytes, in.at, in.bytes)) return fail(RQ_EINVAL, "O, lse or the workspace overlaps an input");
    for (int j = 0; j < i; j++)
      if (overlap(outs[i].at, outs[i].bytes, outs[j].at, outs[j].bytes))
        return fail(RQ_EINVAL, "O, lse and the workspace must not overlap");
  }
  return ok();
}

}  // namespace

extern "C" {

const char* rq_status_string(rq_status s) {
  switch (s) {
    case RQ_OK: return "RQ_OK: success";
    case RQ_EINVAL: return "RQ_EINVAL: invalid argument (NULL, misaligned, negative size, bad dtype, overlap)";
    case RQ_EUNSUPPORTED: return "RQ_EUNSUPPORTED: shape or configuration outside the supported limits";
    case RQ_EWORKSPACE: return "RQ_EWORKSPACE: workspace too small";
    case RQ_EHIP: return "RQ_EHIP: HIP runtime error";
  }
  return "unknown rq_status";
}

const char* rq_last_error_detail(void) { return g_detail.c_str(); }

const char* rq_version(void) { return "0.1.0"; }

size_t rq_rotq_linear_workspace_size(int64_t M, int64_t K, const rq_qconfig* cfg) {
  if (check_cfg(cfg) != RQ_OK || M < 0 || K <= 0) return 0;
  return (size_t)(round256(x_code_bytes(M, K, cfg->bits, fused_x_layout(cfg))) + round256(M * 4));
}

size_t rq_weight_bytes(int64_t N, int64_t K, const rq_qconfig* cfg) {
  if (check_cfg(cfg) != RQ_OK || N < 0 || N > kMaxRowsOrCols || K <= 0 || K > kMaxK || K % 128)
    return 0;
  return (size_t)w_code_bytes(N, K, cfg->bits, cfg->w_layout);
}

size_t rq_codes_bytes(int64_t rows, int64_t K, const rq_qconfig* cfg) {
  if (check_cfg(cfg) != RQ_OK || rows < 0 || rows > kMaxRowsOrCols || K <= 0 || K > kMaxK || K % 128)
    return 0;
  return (size_t)x_code_bytes(rows, K, cfg->bits, cfg->x_layout);
}

rq_status rq_quantize_weights(const void* W, int32_t w_dtype, int64_t N, int64_t K,
                              const rq_qconfig* cfg, void* Wq, float* w_scale, void* stream) {
  rq_status s = check_rotate_args(W, w_dtype, N, K, cfg, Wq, w_scale, "W", false);
  if (s) return s;
  const bool fp6 = cfg->w_layout == RQ_W_FP6;
  if (cfg->w_scale_mode != RQ_W_ABSMAX)
    return from_hip(convrot::launch_weight_quant(cfg->w_scale_mode == RQ_W_MSE ? convrot::kWScaleMse
                                                                                : convrot::kWScaleTensor,
                                                 W, w_dtype, N, K, cfg->bits, fp6, Wq, w_scale,
                                                 static_cast<hipStream_t>(stream)),
                    "weight_quant launch");
  return from_hip(convrot::launch_rotate_quant(W, w_dtype, N, K, cfg->bits,
                                               fp6 ? convrot::kCodeFp6W : convrot::kCodeRows, Wq, w_scale,
                                               static_cast<hipStream_t>(stream)),
                  "rotate_quant launch");
}

rq_status rq_rotate_quantize(const void* X, int32_t x_dtype, int64_t M, int64_t K,
                             const rq_qconfig* cfg, void* Xq, float* x_scale, void* stream) {
  rq_status s = check_rotate_args(X, x_dtype, M, K, cfg, Xq, x_scale, "X", true);
  if (s) return s;
  return from_hip(convrot::launch_rotate_quant(X, x_dtype, M, K, cfg->bits, code_layout(cfg->x_layout),
                                               Xq, x_scale, static_cast<hipStream_t>(stream)),
                  "rotate_quant launch");
}

rq_status rq_check_rotq_linear_args(const void* X, int32_t x_dtype, int64_t M, int64_t K,
                                    const void* Wq, const float* w_scale, int64_t N,
                                    const float* bias, const rq_qconfig* cfg, const void* Y,
                                    const void* workspace, size_t ws_bytes) {
  return check_linear(X, x_dtype, M, K, Wq, w_scale, N, bias, cfg, Y, workspace, ws_bytes);
}

rq_status rq_rotq_linear(const void* X, int32_t x_dtype, int64_t M, int64_t K, const void* Wq,
                         const float* w_scale, int64_t N, const float* bias,
                         const rq_qconfig* cfg, void* Y, void* workspace, size_t ws_bytes,
                         void* stream) {
  rq_status s = check_linear(X, x_dtype, M, K, Wq, w_scale, N, bias, cfg, Y, workspace, ws_bytes);
  if (s || M == 0) return s;
  return launch_linear(X, x_dtype, M, K, Wq, w_scale, N, bias, cfg, Y, workspace,
                       static_cast<hipStream_t>(stream));
}

rq_status rq_rotq_linear_noalloc(const void* X, int32_t x_dtype, int64_t M, int64_t K,
                                 const void* Wq, const float* w_scale, int64_t N, const float* bias,
                                 const rq_qconfig* cfg, void* Y, void* stream) {
  // The size limit first, so that an oversized call gets this status whatever its pointers.
  rq_status s = check_cfg(cfg);
  if (s) return s;
  if ((s = check_gemm_shape(M, N, K))) return s;
  const size_t need = rq_rotq_linear_workspace_size(M, K, cfg);
  if (need > (size_t)RQ_NOALLOC_SCRATCH_BYTES)
    return fail(RQ_EWORKSPACE, "the call needs %zu bytes of workspace; the static scratch holds %zu "
                               "(use rq_rotq_linear with a caller workspace)",
                need, (size_t)RQ_NOALLOC_SCRATCH_BYTES);
  if ((s = check_linear_core(X, x_dtype, M, K, Wq, w_scale, N, bias, cfg, Y)) || M == 0) return s;
  void* ws = nullptr;
  if ((s = scratch_of_current_device(&ws))) return s;
  if ((s = check_linear_ws(X, M, K, Wq, w_scale, N, bias, cfg, Y, ws, RQ_NOALLOC_SCRATCH_BYTES))) return s;
  return launch_linear(X, x_dtype, M, K, Wq, w_scale, N, bias, cfg, Y, ws, static_cast<hipStream_t>(stream));
}

rq_status rq_gemm_dequant(const void* Xq, const float* x_scale, const void* Wq,
                          const float* w_scale, const float* bias, int64_t M, int64_t N,
                          int64_t K, const rq_qconfig* cfg, void* Y, int32_t y_dtype,
                          void* stream) {
  if (y_dtype != RQ_F16 && y_dtype != RQ_BF16)
    return fail(y_dtype == RQ_F32 ? RQ_EUNSUPPORTED : RQ_EINVAL, "Y dtype %d (supported: RQ_F16, RQ_BF16)", y_dtype);
  rq_status s = check_gemm(Xq, x_scale, Wq, w_scale, bias, M, N, K, cfg, Y, 2);
  if (s || M == 0) return s;
  if (cfg->x_layout == RQ_X_FP6)
    return from_hip(convrot::launch_gemm_fp6(Xq, x_scale, Wq, w_scale, bias, M, N, K, Y, y_dtype, nullptr,
                                             cfg->act, static_cast<hipStream_t>(stream)),
                    "gemm launch");
  return from_hip(convrot::launch_gemm(Xq, x_scale, Wq, w_scale, bias, M, N, K, cfg->bits,
                                       cfg->x_layout == RQ_X_TILED, Y, y_dtype, nullptr, cfg->act,
                                       static_cast<hipStream_t>(stream)),
                  "gemm launch");
}

rq_status rq_gemm_s32(const void* Xq, const void* Wq, int64_t M, int64_t N, int64_t K,
                      const rq_qconfig* cfg, int32_t* acc, void* stream) {
  rq_status s = check_gemm(Xq, nullptr, Wq, nullptr, nullptr, M, N, K, cfg, acc, 4);
  if (s || M == 0) return s;
  if (cfg->x_layout == RQ_X_FP6)
    return from_hip(convrot::launch_gemm_fp6(Xq, nullptr, Wq, nullptr, nullptr, M, N, K, acc, RQ_F16, acc,
                                             RQ_ACT_NONE, static_cast<hipStream_t>(stream)),
                    "gemm launch");
  return from_hip(convrot::launch_gemm(Xq, nullptr, Wq, nullptr, nullptr, M, N, K, cfg->bits,
                                       cfg->x_layout == RQ_X_TILED, acc, RQ_F16, acc, RQ_ACT_NONE,
                                       static_cast<hipStream_t>(stream)),
                  "gemm launch");
}

size_t rq_kv_page_bytes(const rq_kv_config* cfg) {
  if (check_kv_cfg(cfg) != RQ_OK) return 0;
  return (size_t)(kv_head_bytes(cfg) * cfg->kv_heads);
}

rq_status rq_kv_cache_write(const void* K, const void* V, int32_t dtype, int64_t tokens, int64_t k_token_stride,
                            int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride, const int64_t* slots,
                            const rq_kv_config* cfg, void* cache, int64_t num_pages, void* stream) {
  rq_status s = check_kv_rw(K, V, dtype, tokens, k_token_stride, k_head_stride, v_token_stride, v_head_stride, slots, cfg,
                            cache, num_pages, false);
  if (s || tokens == 0) return s;
  convrot::KvCacheArgs a = kv_cache_args(dtype, tokens, k_token_stride, k_head_stride, v_token_stride, v_head_stride, slots,
                                         cfg, cache, num_pages);
  a.k = static_cast<const uint8_t*>(K);
  a.v = static_cast<const uint8_t*>(V);
  return from_hip(convrot::launch_kv_cache(a, cfg->head_dim, cfg->bits, true, static_cast<hipStream_t>(stream)),
                  "kv_write launch");
}

rq_status rq_kv_cache_read(const void* cache, int64_t num_pages, const int64_t* slots, int64_t tokens,
                           const rq_kv_config* cfg, void* K, void* V, int32_t dtype, int64_t k_token_stride,
                           int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride, void* stream) {
  rq_status s = check_kv_rw(K, V, dtype, tokens, k_token_stride, k_head_stride, v_token_stride, v_head_stride, slots, cfg,
                            cache, num_pages, true);
  if (s || tokens == 0) return s;
  convrot::KvCacheArgs a = kv_cache_args(dtype, tokens, k_token_stride, k_head_stride, v_token_stride, v_head_stride, slots,
                                         cfg, cache, num_pages);
  a.k_out = static_cast<uint8_t*>(K);
  a.v_out = static_cast<uint8_t*>(V);
  return from_hip(convrot::launch_kv_cache(a, cfg->head_dim, cfg->bits, false, static_cast<hipStream_t>(stream)),
                  "kv_read launch");
}

size_t rq_kv_attention_workspace_size(const rq_kv_attention_params* p, const rq_kv_config* cfg) {
  int64_t max_q = 0, max_kv = 0;
  if (check_kv_shape(p, cfg, &max_q, &max_kv) != RQ_OK || p->total_q == 0) return 0;
  return convrot::plan_kv_attention(p->total_q, p->seqs, p->q_heads, cfg->kv_heads, cfg->head_dim, max_q, max_kv, p->window)
      .workspace_bytes;
}

rq_status rq_kv_attention(const rq_kv_attention_params* p, const rq_kv_config* cfg, const void* cache, int64_t num_pages,
                          void* workspace, size_t ws_bytes, void* stream) {
  convrot::KvAttentionPlan plan = {};
  int64_t max_q = 0;
  rq_status s = check_kv_attention(p, cfg, cache, num_pages, workspace, ws_bytes, &plan, &max_q);
  if (s || p->total_q == 0) return s;
  convrot::KvAttentionArgs a = {};
  a.cache = static_cast<const uint8_t*>(cache);
  a.q = static_cast<const uint8_t*>(p->Q);
  a.out = static_cast<uint8_t*>(p->O);
  a.lse = p->lse;
  a.q_start = p->q_start;
  a.kv_len = p->kv_len;
  a.pages = p->pages;
  a.part_out = static_cast<float*>(workspace);
  if (plan.splits > 1) a.part_stat = a.part_out + p->total_q * p->q_heads * plan.splits * cfg->head_dim;
  a.q_token = p->q_token_stride;
  a.q_head = p->q_head_stride;
  a.out_token = p->o_token_stride;
  a.out_head = p->o_head_stride;
  a.total_q = p->total_q;
  a.num_pages = num_pages;
  a.head_bytes = kv_head_bytes(cfg);
  a.seqs = p->seqs;
  a.q_heads = p->q_heads;
  a.heads = cfg->kv_heads;
  a.group = p->q_heads / cfg->kv_heads;
  a.even_q = p->q_start ? 0 : static_cast<int>(p->total_q / p->seqs);
  a.group_shift = log2_of(a.group);
  a.group_mul = static_cast<uint32_t>((((uint64_t)1 << 32) * (((uint64_t)1 << a.group_shift) - a.group)) / a.group + 1);
  a.max_pages = p->max_pages;
  a.lps = log2_of(cfg->page_size);
  a.dt = p->dtype;
  a.causal = p->causal;
  // Positions are below 2^30: a wider window is no other, and the kernels' differences stay in 32 bits.
  a.window = p->window < kMaxKvTokens ? p->window : static_cast<int>(kMaxKvTokens);
  a.splits = plan.splits;
  a.row_tiles = plan.row_tiles;
  a.chunk = plan.chunk;
  a.block = plan.block;
  a.max_q = static_cast<int>(max_q);
  a.scale = p->softmax_scale;
  return from_hip(convrot::launch_kv_attention(a, cfg->head_dim, cfg->bits, static_cast<hipStream_t>(stream)),
                  "kv_attention launch");
}

}  // extern "C"
