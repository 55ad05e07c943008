// C ABI entry points: argument checks, workspace sizing, dispatch.
#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "common.h"

namespace {

thread_local char g_last_error[512] = "";

gptq_status fail(gptq_status st, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
    va_end(ap);
    return st;
}

gptq_status hip_status(hipError_t e, const char *what) {
    if (e == hipSuccess) return GPTQ_OK;
    return fail(GPTQ_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool aligned(const void *p, size_t a = 16) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

gptq_status check_cfg(const gptq_config *c, int64_t d_in, const char *fn) {
    if (!c) return fail(GPTQ_ERR_INVALID_ARG, "%s: cfg is NULL", fn);
    if (c->bits < 2 || c->bits > 8) return fail(GPTQ_ERR_INVALID_ARG, "%s: bits=%d outside 2..8", fn, c->bits);
    if (c->group_size < 0 || (c->group_size > 0 && d_in % c->group_size != 0))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: group_size=%d does not divide d_in=%lld", fn, c->group_size, (long long)d_in);
    if (!(c->damp_rel >= 0.0f)) return fail(GPTQ_ERR_INVALID_ARG, "%s: damp_rel must be >= 0", fn);
    if (c->grid != GPTQ_GRID_DYNAMIC && c->grid != GPTQ_GRID_STATIC && c->grid != GPTQ_GRID_TENSOR)
        return fail(GPTQ_ERR_INVALID_ARG, "%s: unknown grid %d", fn, c->grid);
    if (c->super_cols < 0) return fail(GPTQ_ERR_INVALID_ARG, "%s: super_cols must be >= 0", fn);
    if (c->grid == GPTQ_GRID_TENSOR && c->group_size != 0)
        return fail(GPTQ_ERR_INVALID_ARG, "%s: a per-tensor grid needs group_size 0", fn);
    return GPTQ_OK;
}

gptq_status check_quantize(float *W, int64_t d_out, int64_t d_in, const float *U, const int32_t *perm,
                           const gptq_config *cfg, uint8_t *codes, float *scales, float *zeros, int32_t *g_idx,
                           const char *fn) {
    if (d_out <= 0 || d_in <= 0) return fail(GPTQ_ERR_INVALID_ARG, "%s: sizes must be > 0", fn);
    gptq_status st = check_cfg(cfg, d_in, fn);
    if (st != GPTQ_OK) return st;
    if (!W || !U || !codes || !scales || !zeros) return fail(GPTQ_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (cfg->act_order && !perm) return fail(GPTQ_ERR_INVALID_ARG, "%s: act_order needs perm", fn);
    if (!aligned(W) || !aligned(U) || !aligned(scales, 4) || !aligned(zeros, 4) || (perm && !aligned(perm, 4)) ||
        (g_idx && !aligned(g_idx, 4)))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    if (!gptq::quantize_supported(*cfg, d_in))
        return fail(GPTQ_ERR_UNSUPPORTED, "%s: block_size=%d group_size=%d not supported", fn, cfg->block_size, cfg->group_size);
    if (d_out > ((int64_t)1 << 21)) return fail(GPTQ_ERR_UNSUPPORTED, "%s: d_out above 2^21", fn);  // 64-row tiles on grid y
    return GPTQ_OK;
}

bool few_dtype(gptq_dtype t) { return t == GPTQ_DT_BF16 || t == GPTQ_DT_F16; }
bool out_dtype(gptq_dtype t) { return few_dtype(t) || t == GPTQ_DT_F32; }

// A packed layer, or a stack of them, for the few-token products.
gptq_status check_packed(const gptq_packed *w, const char *fn, const char *name) {
    if (!w) return fail(GPTQ_ERR_INVALID_ARG, "%s: %s is NULL", fn, name);
    if (w->d_out <= 0 || w->d_in <= 0) return fail(GPTQ_ERR_INVALID_ARG, "%s: %s: sizes must be > 0", fn, name);
    if (w->bits < 2 || w->bits > 8) return fail(GPTQ_ERR_INVALID_ARG, "%s: %s: bits=%d outside 2..8", fn, name, w->bits);
    if (w->group_size < 0 || (w->group_size > 0 && w->d_in % w->group_size != 0))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: %s: group_size does not divide d_in", fn, name);
    if (w->bits != 2 && w->bits != 3 && w->bits != 4 && w->bits != 8)
        return fail(GPTQ_ERR_UNSUPPORTED, "%s: %s: bits must be 2, 3, 4 or 8", fn, name);
    if (w->d_in % 32 != 0 || w->group_size % 32 != 0)
        return fail(GPTQ_ERR_UNSUPPORTED, "%s: %s: d_in and group_size must be multiples of 32", fn, name);
    if (w->d_in > ((int64_t)1 << 20) || w->d_out > ((int64_t)1 << 28))  // 2^28 rows: 2^31 threads of one launch
        return fail(GPTQ_ERR_UNSUPPORTED, "%s: %s: d_in above 2^20 or d_out above 2^28", fn, name);
    if (!w->packed || !w->scales || !w->zeros) return fail(GPTQ_ERR_INVALID_ARG, "%s: %s: NULL pointer", fn, name);
    if (!aligned(w->packed) || !aligned(w->scales, 4) || !aligned(w->zeros, 4) || (w->kperm && !aligned(w->kperm, 4)))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: %s: packed must be 16-byte aligned, the other pointers 4-byte aligned", fn, name);
    return GPTQ_OK;
}

gptq_status check_pair(const gptq_packed *gate, const gptq_packed *up, const char *fn) {
    gptq_status st = check_packed(gate, fn, "gate");
    if (st == GPTQ_OK) st = check_packed(up, fn, "up");
    if (st != GPTQ_OK) return st;
    if (gate->d_out != up->d_out || gate->d_in != up->d_in || gate->bits != up->bits || gate->group_size != up->group_size ||
        gate->kperm != up->kperm)
        return fail(GPTQ_ERR_INVALID_ARG, "%s: gate and up must agree in sizes, bits, group_size and kperm", fn);
    return GPTQ_OK;
}

// Activations and results of a few-token product.
gptq_status check_few(const void *X, gptq_dtype x_dt, int64_t M, int64_t ldx, int64_t d_in, const void *Y, gptq_dtype y_dt,
                      int64_t ldy, int64_t d_out, const char *fn) {
    if (!few_dtype(x_dt) || !out_dtype(y_dt))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: activations must be fp16 or bf16, results fp16, bf16 or fp32", fn);
    if (M > 0 && (!X || !Y)) return fail(GPTQ_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (ldx < d_in || ldy < d_out) return fail(GPTQ_ERR_INVALID_ARG, "%s: leading dimension too small", fn);
    if (!aligned(X) || ldx % 8 != 0 || !aligned(Y, y_dt == GPTQ_DT_F32 ? 4 : 2))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: X must be 16-byte aligned with ldx a multiple of 8, Y aligned to its type", fn);
    return GPTQ_OK;
}

// Whether any two of n rows of bytes, at a and at b, share one.
bool rows_overlap(const void *a, int64_t a_pitch, int64_t a_row, const void *b, int64_t b_pitch, int64_t b_row, int64_t n) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    if (a0 + (n - 1) * a_pitch + a_row <= b0 || b0 + (n - 1) * b_pitch + b_row <= a0) return false;
    for (int64_t i = 0; i < n; ++i)
        for (int64_t j = 0; j < n; ++j) {
            const uintptr_t r = a0 + i * a_pitch, t = b0 + j * b_pitch;
            if (r < t + b_row && t < r + a_row) return true;
        }
    return false;
}

// The workgroups read X while others write Y.
gptq_status check_apart(const void *X, int64_t M, int64_t ldx, int64_t d_in, const void *Y, gptq_dtype y_dt, int64_t ldy,
                        int64_t d_out, const char *fn) {
    const int64_t y = y_dt == GPTQ_DT_F32 ? 4 : 2;
    if (rows_overlap(X, 2 * ldx, 2 * d_in, Y, y * ldy, y * d_out, M)) return fail(GPTQ_ERR_INVALID_ARG, "%s: X and the result overlap", fn);
    return GPTQ_OK;
}

// The same for many rows of one kind: rows next to each other (or columns of one tensor) take no loop.
bool many_overlap(const void *a, int64_t a_pitch, int64_t a_row, const void *b, int64_t b_pitch, int64_t b_row, int64_t n) {
    const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
    if ((n - 1) * a_pitch + a_row <= d || (n - 1) * b_pitch + b_row <= -d) return false;
    // row i of a and row j of b share a byte where -b_row < d + j b_pitch - i a_pitch < a_row
    for (int64_t i = 0; i < n; ++i) {
        const int64_t at = i * a_pitch - d;  // the first j with at - b_row < j b_pitch
        const int64_t j = at - b_row < 0 ? 0 : (at - b_row) / b_pitch + 1;
        if (j < n && j * b_pitch < at + a_row) return true;
        if (a_pitch == b_pitch && j > 0) return false;  // a later row lies to its neighbours as this one does
    }
    return false;
}

constexpr int64_t kKvTokens = (int64_t)1 << 30;  // of a table

gptq_status check_kv(const gptq_kv_cache *c, const char *fn) {
    if (!c) return fail(GPTQ_ERR_INVALID_ARG, "%s: cache is NULL", fn);
    if (c->n_pages <= 0 || c->n_heads <= 0 || c->head_dim <= 0 || c->page <= 0)
        return fail(GPTQ_ERR_INVALID_ARG, "%s: cache: sizes must be > 0", fn);
    if (c->group_size < 0 || (c->group_size > 0 && c->head_dim % c->group_size != 0))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: cache: group_size does not divide head_dim", fn);
    if (c->symmetric != 0 && c->symmetric != 1) return fail(GPTQ_ERR_INVALID_ARG, "%s: cache: symmetric must be 0 or 1", fn);
    if (c->head_dim % 64 != 0 || c->head_dim > 256) return fail(GPTQ_ERR_UNSUPPORTED, "%s: cache: head_dim must be 64, 128, 192 or 256", fn);
    if (c->group_size != 0 && c->group_size != c->head_dim && c->group_size != 32 && c->group_size != 64 && c->group_size != 128)
        return fail(GPTQ_ERR_UNSUPPORTED, "%s: cache: group_size must be 32, 64, 128 or head_dim", fn);
    if ((c->page & (c->page - 1)) != 0 || c->page < 16 || c->page > (1 << 20))
        return fail(GPTQ_ERR_UNSUPPORTED, "%s: cache: page must be a power of two, 16 .. 2^20", fn);
    if (c->n_pages > 0x7FFFFFFF || c->n_heads > 65535) return fail(GPTQ_ERR_UNSUPPORTED, "%s: cache: too many pages or heads", fn);
    if (!c->k || !c->v || !c->k_grid || !c->v_grid) return fail(GPTQ_ERR_INVALID_ARG, "%s: cache: NULL pointer", fn);
    if (!aligned(c->k) || !aligned(c->v) || !aligned(c->k_grid) || !aligned(c->v_grid) || !aligned(c->weight))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: cache: pointers must be 16-byte aligned", fn);
    return GPTQ_OK;
}

// The sequences of a call, and the longest length that counts.
gptq_status check_seqs(const gptq_kv_cache *c, const int32_t *table, int64_t width, const int32_t *lens, int64_t n_seq, int64_t max_len,
                       const char *fn) {
    if (n_seq < 0 || width <= 0 || max_len < 0) return fail(GPTQ_ERR_INVALID_ARG, "%s: bad sizes", fn);
    if (n_seq > 65535 || width > kKvTokens / c->page) return fail(GPTQ_ERR_UNSUPPORTED, "%s: more than 65535 sequences or 2^30 tokens of one", fn);
    if (max_len > width * c->page) return fail(GPTQ_ERR_INVALID_ARG, "%s: max_len is more than the table holds", fn);
    if (n_seq > 0 && (!table || !lens)) return fail(GPTQ_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (!aligned(table, 4) || !aligned(lens, 4)) return fail(GPTQ_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    return GPTQ_OK;
}

gptq_status check_kv_queries(const gptq_kv_cache *c, int64_t n_seq, int64_t n, int64_t q_heads, int64_t max_len, const char *fn) {
    if (n_seq < 0 || max_len < 0 || n <= 0 || q_heads <= 0 || q_heads % c->n_heads != 0)
        return fail(GPTQ_ERR_INVALID_ARG, "%s: bad sizes (q_heads must be a multiple of n_heads)", fn);
    if (n > 16 || q_heads / c->n_heads > 256) return fail(GPTQ_ERR_UNSUPPORTED, "%s: at most 16 tokens, and 256 query heads on one", fn);
    const int64_t tiles = gptq::ceil_div(n * (q_heads / c->n_heads), 16);
    if (n_seq > 65535 || max_len > kKvTokens || n_seq * c->n_heads * tiles > ((int64_t)1 << 19) ||
        n_seq * gptq::ceil_div(max_len, 32) > ((int64_t)1 << 30))
        return fail(GPTQ_ERR_UNSUPPORTED, "%s: too many sequences, heads and queries at once", fn);
    return GPTQ_OK;
}

gptq_status check_kv_budget(const gptq_kv_cache *c, int64_t n_seq, int64_t max_len, int64_t budget, const char *fn) {
    if (n_seq < 0 || max_len < 0 || budget < 1) return fail(GPTQ_ERR_INVALID_ARG, "%s: bad sizes", fn);
    if (n_seq > 65535 || max_len > kKvTokens || budget > kKvTokens || n_seq * c->n_heads > ((int64_t)1 << 20) ||
        n_seq * c->n_heads * budget > ((int64_t)1 << 27))
        return fail(GPTQ_ERR_UNSUPPORTED, "%s: too many sequences, heads and kept tokens at once", fn);
    return GPTQ_OK;
}

gptq_status run_gemv_checked(const void *X, gptq_dtype x_dt, int64_t M, int64_t ldx, const gptq_packed *w,
                             const gptq_packed *up, const float *bias, void *Y, gptq_dtype y_dt, int64_t ldy, void *ws,
                             size_t ws_bytes, hipStream_t stream, const char *fn) {
    if (M < 0) return fail(GPTQ_ERR_INVALID_ARG, "%s: M must be >= 0", fn);
    if (M > 16) return fail(GPTQ_ERR_UNSUPPORTED, "%s: at most 16 tokens", fn);
    gptq_status st = check_few(X, x_dt, M, ldx, w->d_in, Y, y_dt, ldy, w->d_out, fn);
    if (st != GPTQ_OK) return st;
    if (bias && !aligned(bias, 4)) return fail(GPTQ_ERR_INVALID_ARG, "%s: misaligned bias", fn);
    if (M == 0) return GPTQ_OK;
    const size_t need = w->kperm ? gptq::gemv_ws_bytes(M, w->d_in) : 0;
    if (need > 0 && (!ws || ws_bytes < need))
        return fail(GPTQ_ERR_WORKSPACE, "%s: need %zu workspace bytes, got %zu", fn, need, ws ? ws_bytes : (size_t)0);
    if (need > 0 && !aligned(ws)) return fail(GPTQ_ERR_INVALID_ARG, "%s: misaligned workspace", fn);
    st = check_apart(X, M, ldx, w->d_in, Y, y_dt, ldy, w->d_out, fn);
    if (st != GPTQ_OK) return st;
    return hip_status(gptq::run_gemv(X, x_dt, M, ldx, *w, up, bias, Y, y_dt, ldy, ws, stream), fn);
}

gptq_status check_moe_sizes(int64_t T, int64_t d, int64_t d_ff, int32_t n_experts, int32_t top_k, const char *fn) {
    if (T < 0 || d <= 0 || d_ff <= 0 || n_experts <= 0 || top_k <= 0 || top_k > n_experts)
        return fail(GPTQ_ERR_INVALID_ARG, "%s: bad sizes (1 <= top_k <= n_experts)", fn);
    if (T > gptq::kMoeMaxTokens || n_experts > gptq::kMoeMaxExperts || top_k > gptq::kMoeMaxTopK)
        return fail(GPTQ_ERR_UNSUPPORTED, "%s: at most %d tokens, %d experts and %d of them per token", fn,
                    gptq::kMoeMaxTokens, gptq::kMoeMaxExperts, gptq::kMoeMaxTopK);
    if (d > ((int64_t)1 << 20) || d_ff > ((int64_t)1 << 20))
        return fail(GPTQ_ERR_UNSUPPORTED, "%s: d or d_ff above 2^20", fn);
    return GPTQ_OK;
}

// Scratch memory of gptq_quantize_layer_noalloc: one fixed array per device,
// part of the library's device image (the runtime places it on each device
// the library runs on, for the life of the process).  In host code `scratch`
// names a host-side stand-in: the device copy's address comes from
// hipGetSymbolAddress, looked up once per device with that device current.
static __device__ __align__(256) unsigned char scratch[GPTQ_NOALLOC_SCRATCH_BYTES];

hipError_t scratch_address(void **out) {
    constexpr int kMaxDevices = 64;
    static void *addr[kMaxDevices] = {};
    static std::mutex mu;
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!addr[dev]) {
        void *p = nullptr;
        e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (e != hipSuccess) return e;
        if (!p) return hipErrorInvalidSymbol;
        addr[dev] = p;
    }
    *out = addr[dev];
    return hipSuccess;
}

}  // namespace

extern "C" {

const char *gptq_status_string(gptq_status st) {
    switch (st) {
    case GPTQ_OK: return "ok";
    case GPTQ_ERR_INVALID_ARG: return "invalid argument";
    case GPTQ_ERR_UNSUPPORTED: return "unsupported configuration";
    case GPTQ_ERR_WORKSPACE: return "workspace missing or too small";
    case GPTQ_ERR_HIP: return "HIP runtime error";
    }
    return "unknown status";
}

const char *gptq_last_error(void) { return g_last_error; }

gptq_status gptq_timing_enable(int32_t on) {
    gptq::timing_set(on != 0);
    return GPTQ_OK;
}

gptq_status gptq_timing_read(int32_t op, double *ms, int64_t *count, double *flops) {
    const char *fn = "gptq_timing_read";
    if (op < 0 || op >= gptq::kTimedOps) return fail(GPTQ_ERR_INVALID_ARG, "%s: unknown op %d", fn, op);
    if (!ms || !count) return fail(GPTQ_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    double w = 0.0;
    const hipError_t e = gptq::timing_read(static_cast<gptq::TimedOp>(op), ms, count, &w);
    if (flops) *flops = w;
    return hip_status(e, fn);
}

gptq_status gptq_workspace_bytes(int op, int64_t d_out, int64_t d_in, int64_t n_tok, const gptq_config *cfg, size_t *out) {
    if (!out) return fail(GPTQ_ERR_INVALID_ARG, "gptq_workspace_bytes: out is NULL");
    if (d_in <= 0 || d_out < 0 || n_tok < 0) return fail(GPTQ_ERR_INVALID_ARG, "gptq_workspace_bytes: bad sizes");
    switch (op) {
    case GPTQ_OP_HESSIAN:
        *out = gptq::hessian_ws_bytes(d_in, n_tok, GPTQ_DT_BF16);
        return GPTQ_OK;
    case GPTQ_OP_PREPARE:
        *out = gptq::prepare_ws_bytes(d_in);
        return GPTQ_OK;
    case GPTQ_OP_QUANTIZE: {
        if (!cfg) return fail(GPTQ_ERR_INVALID_ARG, "gptq_workspace_bytes: quantize needs cfg");
        if (cfg->block_size <= 0) return fail(GPTQ_ERR_INVALID_ARG, "gptq_workspace_bytes: block_size must be > 0");
        if (cfg->super_cols < 0) return fail(GPTQ_ERR_INVALID_ARG, "gptq_workspace_bytes: super_cols must be >= 0");
        *out = gptq::quantize_ws_bytes(d_out, d_in, *cfg);
        return GPTQ_OK;
    }
    case GPTQ_OP_LOSS:
        *out = gptq::loss_ws_bytes(d_out, d_in);
        return GPTQ_OK;
    case GPTQ_OP_HESSIAN_TOKENS:
        *out = gptq::hessian_ws_bytes(d_in, n_tok, GPTQ_DT_BF16);
        return GPTQ_OK;
    case GPTQ_OP_CALIBRATE:
        *out = gptq::calibrate_ws_bytes(d_in, n_tok);
        return GPTQ_OK;
    case GPTQ_OP_SMOOTH:
        *out = gptq::smooth_ws_bytes(d_out, d_in);
        return GPTQ_OK;
    case GPTQ_OP_AWQ: {
        if (!cfg) return fail(GPTQ_ERR_INVALID_ARG, "gptq_workspace_bytes: the AWQ search needs cfg");
        gptq_status st = check_cfg(cfg, d_in, "gptq_workspace_bytes");
        if (st != GPTQ_OK) return st;
        *out = gptq::awq_ws_bytes(d_out, d_in, *cfg);
        return GPTQ_OK;
    }
    case GPTQ_OP_GEMV:
        *out = gptq::gemv_ws_bytes(n_tok, d_in);
        return GPTQ_OK;
    case GPTQ_OP_W4A16:  // the largest plan over the group sizes (the plan depends on g only through 32, 64, 128 | g)
        *out = std::max(gptq::w4a16_ws_bytes(n_tok, d_in, d_out, 32),
                        std::max(gptq::w4a16_ws_bytes(n_tok, d_in, d_out, 64), gptq::w4a16_ws_bytes(n_tok, d_in, d_out, 128)));
        return GPTQ_OK;
    }
    return fail(GPTQ_ERR_INVALID_ARG, "gptq_workspace_bytes: unknown op %d", op);
}

gptq_status gptq_hessian_accumulate(float *H, double *hdiag, const void *X, gptq_dtype x_dtype, int64_t d_in,
                                    int64_t n_tok, int64_t ldx, void *ws, size_t ws_bytes, hipStream_t stream) {
    const char *fn = "gptq_hessian_accumulate";
    if (d_in <= 0 || n_tok < 0) return fail(GPTQ_ERR_INVALID_ARG, "%s: d_in must be > 0 and n_tok >= 0", fn);
    if (x_dtype != GPTQ_DT_F32 && x_dtype != GPTQ_DT_BF16) return fail(GPTQ_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (ldx < n_tok) return fail(GPTQ_ERR_INVALID_ARG, "%s: ldx < n_tok", fn);
    const int64_t esz = x_dtype == GPTQ_DT_BF16 ? 2 : 4;
    if (!H || (n_tok > 0 && !X)) return fail(GPTQ_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (!aligned(H) || (X && !aligned(X)) || (hdiag && !aligned(hdiag, 8)) || (ldx * esz) % 16 != 0)
        return fail(GPTQ_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned and ldx*elem a multiple of 16", fn);
    if (n_tok == 0) return GPTQ_OK;
    const size_t need = gptq::hessian_ws_bytes(d_in, n_tok, x_dtype);
    if (need > 0 && (!ws || ws_bytes < need))
        return fail(GPTQ_ERR_WORKSPACE, "%s: need %zu workspace bytes, got %zu", fn, need, ws ? ws_bytes : (size_t)0);
    return hip_status(gptq::run_hessian(H, hdiag, X, x_dtype, d_in, n_tok, ldx, false, ws, stream), fn);
}

gptq_status gptq_hessian_accumulate_tokens(float *H, double *hdiag, const void *X, gptq_dtype x_dtype, int64_t d_in,
                                           int64_t n_tok, int64_t ldx, void *ws, size_t ws_bytes, hipStream_t stream) {
    const char *fn = "gptq_hessian_accumulate_tokens";
    if (d_in <= 0 || n_tok < 0) return fail(GPTQ_ERR_INVALID_ARG, "%s: d_in must be > 0 and n_tok >= 0", fn);
    if (x_dtype != GPTQ_DT_F32 && x_dtype != GPTQ_DT_BF16) return fail(GPTQ_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if (ldx < d_in) return fail(GPTQ_ERR_INVALID_ARG, "%s: ldx < d_in", fn);
    if (!H || (n_tok > 0 && !X)) return fail(GPTQ_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (!aligned(H) || (hdiag && !aligned(hdiag, 8)))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    // bf16: each lane loads 4 channels of a token as one 8-byte word
    if (x_dtype == GPTQ_DT_BF16 && ((X && !aligned(X, 8)) || ldx % 4 != 0))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: bf16 X must be 8-byte aligned with ldx a multiple of 4", fn);
    if (x_dtype == GPTQ_DT_F32 && X && !aligned(X, 4)) return fail(GPTQ_ERR_INVALID_ARG, "%s: misaligned X", fn);
    if (n_tok == 0) return GPTQ_OK;
    const size_t need = gptq::hessian_ws_bytes(d_in, n_tok, x_dtype);
    if (need > 0 && (!ws || ws_bytes < need))
        return fail(GPTQ_ERR_WORKSPACE, "%s: need %zu workspace bytes, got %zu", fn, need, ws ? ws_bytes : (size_t)0);
    return hip_status(gptq::run_hessian(H, hdiag, X, x_dtype, d_in, n_tok, ldx, true, ws, stream), fn);
}

gptq_status gptq_linear_forward(void *Y, int64_t ldy, const void *X, int64_t ldx, const void *W, int64_t ldw,
                                int64_t n_tok, int64_t d_prev, int64_t d_out, hipStream_t stream) {
    const char *fn = "gptq_linear_forward";
    if (n_tok < 0 || d_out < 0 || d_prev <= 0) return fail(GPTQ_ERR_INVALID_ARG, "%s: bad sizes", fn);
    if (n_tok == 0 || d_out == 0) return GPTQ_OK;
    if (!Y || !X || !W) return fail(GPTQ_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (ldx < d_prev || ldw < d_prev || ldy < d_out) return fail(GPTQ_ERR_INVALID_ARG, "%s: leading dimension too small", fn);
    if (!aligned(X) || !aligned(W) || ldx % 8 != 0 || ldw % 8 != 0 || !aligned(Y, 2))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: X and W must be 16-byte aligned with ldx, ldw multiples of 8", fn);
    return hip_status(gptq::run_linear_forward(static_cast<uint16_t *>(Y), ldy, static_cast<const uint16_t *>(X), ldx,
                                               static_cast<const uint16_t *>(W), ldw, n_tok, d_prev, d_out, stream),
                      fn);
}

gptq_status gptq_calibrate_hessian(float *H, double *hdiag, const void *X, int64_t ldx, const void *W, int64_t ldw,
                                   int64_t n_tok, int64_t d_prev, int64_t d_in, void *ws, size_t ws_bytes,
                                   hipStream_t stream) {
    const char *fn = "gptq_calibrate_hessian";
    if (n_tok < 0 || d_in <= 0 || d_prev <= 0) return fail(GPTQ_ERR_INVALID_ARG, "%s: bad sizes", fn);
    if (n_tok == 0) return GPTQ_OK;
    if (!H || !X || !W) return fail(GPTQ_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (ldx < d_prev || ldw < d_prev) return fail(GPTQ_ERR_INVALID_ARG, "%s: leading dimension too small", fn);
    if (!aligned(H) || (hdiag && !aligned(hdiag, 8)) || !aligned(X) || !aligned(W) || ldx % 8 != 0 || ldw % 8 != 0)
        return fail(GPTQ_ERR_INVALID_ARG, "%s: X and W must be 16-byte aligned with ldx, ldw multiples of 8", fn);
    const size_t need = gptq::calibrate_ws_bytes(d_in, n_tok);
    if (!ws || ws_bytes < need || !aligned(ws))
        return fail(GPTQ_ERR_WORKSPACE, "%s: need %zu workspace bytes, got %zu", fn, need, ws ? ws_bytes : (size_t)0);
    return hip_status(gptq::run_calibrate(H, hdiag, static_cast<const uint16_t *>(X), ldx,
                                          static_cast<const uint16_t *>(W), ldw, n_tok, d_prev, d_in, ws, stream),
                      fn);
}

int64_t gptq_calibrate_chunk_tokens(int64_t d_in) { return d_in > 0 ? gptq::calibrate_chunk_tokens(d_in) : 0; }

gptq_status gptq_prepare_hinv(const float *H, const double *hdiag, int64_t d_in, const gptq_config *cfg, float *U,
                              int32_t *perm, int32_t *info_dev, void *ws, size_t ws_bytes, hipStream_t stream) {
    const char *fn = "gptq_prepare_hinv";
    if (d_in <= 0) return fail(GPTQ_ERR_INVALID_ARG, "%s: d_in must be > 0", fn);
    if (!cfg) return fail(GPTQ_ERR_INVALID_ARG, "%s: cfg is NULL", fn);
    if (!(cfg->damp_rel >= 0.0f)) return fail(GPTQ_ERR_INVALID_ARG, "%s: damp_rel must be >= 0", fn);
    if (!H || !U || !info_dev) return fail(GPTQ_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (cfg->act_order && !perm) return fail(GPTQ_ERR_INVALID_ARG, "%s: act_order needs perm", fn);
    if (!aligned(H) || !aligned(U) || (perm && !aligned(perm, 4)) || !aligned(info_dev, 4) || (hdiag && !aligned(hdiag, 8)))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    if (d_in > (int64_t)1 << 20) return fail(GPTQ_ERR_UNSUPPORTED, "%s: d_in too large", fn);
    const size_t need = gptq::prepare_ws_bytes(d_in);
    if (!ws || ws_bytes < need) return fail(GPTQ_ERR_WORKSPACE, "%s: need %zu workspace bytes, got %zu", fn, need, ws ? ws_bytes : (size_t)0);
    if (!aligned(ws)) return fail(GPTQ_ERR_INVALID_ARG, "%s: misaligned workspace", fn);
    return hip_status(gptq::run_prepare(H, hdiag, d_in, cfg->damp_rel, cfg->act_order ? 1 : 0, U, perm, info_dev, ws, stream), fn);
}

gptq_status gptq_quantize_layer(float *W, int64_t d_out, int64_t d_in, const float *U, const int32_t *perm,
                                const gptq_config *cfg, uint8_t *codes, float *scales, float *zeros, int32_t *g_idx,
                                void *ws, size_t ws_bytes, hipStream_t stream) {
    const char *fn = "gptq_quantize_layer";
    gptq_status st = check_quantize(W, d_out, d_in, U, perm, cfg, codes, scales, zeros, g_idx, fn);
    if (st != GPTQ_OK) return st;
    const size_t need = gptq::quantize_ws_bytes(d_out, d_in, *cfg);
    if (!ws || ws_bytes < need) return fail(GPTQ_ERR_WORKSPACE, "%s: need %zu workspace bytes, got %zu", fn, need, ws ? ws_bytes : (size_t)0);
    if (need > 0 && !aligned(ws)) return fail(GPTQ_ERR_INVALID_ARG, "%s: misaligned workspace", fn);
    return hip_status(gptq::run_quantize(W, d_out, d_in, U, perm, *cfg, codes, scales, zeros, g_idx, ws, stream), fn);
}

gptq_status gptq_quantize_layer_noalloc(float *W, int64_t d_out, int64_t d_in, const float *U, const int32_t *perm,
                                        const gptq_config *cfg, uint8_t *codes, float *scales, float *zeros,
                                        int32_t *g_idx, hipStream_t stream) {
    const char *fn = "gptq_quantize_layer_noalloc";
    gptq_status st = check_quantize(W, d_out, d_in, U, perm, cfg, codes, scales, zeros, g_idx, fn);
    if (st != GPTQ_OK) return st;
    const size_t need = gptq::quantize_ws_bytes(d_out, d_in, *cfg);
    if (need > GPTQ_NOALLOC_SCRATCH_BYTES)
        return fail(GPTQ_ERR_WORKSPACE, "%s: this layer needs %zu scratch bytes, above the fixed %zu of the entry point",
                    fn, need, (size_t)GPTQ_NOALLOC_SCRATCH_BYTES);
    void *ws = nullptr;
    st = hip_status(scratch_address(&ws), fn);
    if (st != GPTQ_OK) return st;
    return hip_status(gptq::run_quantize(W, d_out, d_in, U, perm, *cfg, codes, scales, zeros, g_idx, ws, stream), fn);
}

gptq_status gptq_rtn_quantize(const float *W, int64_t d_out, int64_t d_in, const gptq_config *cfg, uint8_t *codes,
                              float *scales, float *zeros, hipStream_t stream) {
    const char *fn = "gptq_rtn_quantize";
    if (d_out <= 0 || d_in <= 0) return fail(GPTQ_ERR_INVALID_ARG, "%s: sizes must be > 0", fn);
    gptq_status st = check_cfg(cfg, d_in, fn);
    if (st != GPTQ_OK) return st;
    if (!W || !codes || !scales || !zeros) return fail(GPTQ_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (!aligned(W, 4) || !aligned(scales, 4) || !aligned(zeros, 4)) return fail(GPTQ_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    return hip_status(gptq::run_rtn(W, d_out, d_in, *cfg, codes, scales, zeros, stream), fn);
}

gptq_status gptq_layer_loss(const float *W, const uint8_t *codes, const float *scales, const float *zeros,
                            const int32_t *g_idx, const float *H, int64_t d_out, int64_t d_in, int32_t group_size,
                            double *loss_dev, void *ws, size_t ws_bytes, hipStream_t stream) {
    const char *fn = "gptq_layer_loss";
    if (d_out <= 0 || d_in <= 0) return fail(GPTQ_ERR_INVALID_ARG, "%s: sizes must be > 0", fn);
    if (group_size < 0 || (group_size > 0 && d_in % group_size != 0))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: group_size does not divide d_in", fn);
    if (!W || !codes || !scales || !zeros || !H || !loss_dev) return fail(GPTQ_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (!aligned(W, 4) || !aligned(H, 4) || !aligned(loss_dev, 8)) return fail(GPTQ_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    const size_t need = gptq::loss_ws_bytes(d_out, d_in);
    if (!ws || ws_bytes < need) return fail(GPTQ_ERR_WORKSPACE, "%s: need %zu workspace bytes, got %zu", fn, need, ws ? ws_bytes : (size_t)0);
    return hip_status(gptq::run_loss(W, codes, scales, zeros, g_idx, H, d_out, d_in, group_size, loss_dev, ws, stream), fn);
}

gptq_status gptq_channel_stats(const void *X, gptq_dtype x_dtype, int64_t d_in, int64_t n_tok, int64_t ldx, float *absmax,
                               double *abssum, hipStream_t stream) {
    const char *fn = "gptq_channel_stats";
    if (d_in <= 0 || n_tok < 0 || ldx < n_tok) return fail(GPTQ_ERR_INVALID_ARG, "%s: bad sizes", fn);
    if (x_dtype != GPTQ_DT_F32 && x_dtype != GPTQ_DT_BF16) return fail(GPTQ_ERR_INVALID_ARG, "%s: unknown dtype", fn);
    if ((n_tok > 0 && !X) || !absmax || !abssum) return fail(GPTQ_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if ((X && !aligned(X, 4)) || !aligned(absmax, 4) || !aligned(abssum, 8)) return fail(GPTQ_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    return hip_status(gptq::run_channel_stats(X, x_dtype, d_in, n_tok, ldx, absmax, abssum, stream), fn);
}

gptq_status gptq_smooth_scales(const float *act_absmax, const float *W, int64_t d_out, int64_t d_in, float alpha, float *s,
                               void *ws, size_t ws_bytes, hipStream_t stream) {
    const char *fn = "gptq_smooth_scales";
    if (d_out <= 0 || d_in <= 0) return fail(GPTQ_ERR_INVALID_ARG, "%s: sizes must be > 0", fn);
    if (!(alpha >= 0.0f && alpha <= 1.0f)) return fail(GPTQ_ERR_INVALID_ARG, "%s: alpha outside [0, 1]", fn);
    if (!act_absmax || !W || !s) return fail(GPTQ_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (!aligned(act_absmax, 4) || !aligned(W, 4) || !aligned(s, 4)) return fail(GPTQ_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    const size_t need = gptq::smooth_ws_bytes(d_out, d_in);
    if (!ws || ws_bytes < need) return fail(GPTQ_ERR_WORKSPACE, "%s: need %zu workspace bytes, got %zu", fn, need, ws ? ws_bytes : (size_t)0);
    return hip_status(gptq::run_smooth_scales(act_absmax, W, d_out, d_in, alpha, s, ws, stream), fn);
}

gptq_status gptq_awq_search(const float *W, int64_t d_out, int64_t d_in, const float *H, const double *act_abssum,
                            int64_t n_tok, const gptq_config *cfg, int32_t n_grid, float *s, double *losses,
                            int32_t *best, void *ws, size_t ws_bytes, hipStream_t stream) {
    const char *fn = "gptq_awq_search";
    if (d_out <= 0 || d_in <= 0 || n_tok <= 0) return fail(GPTQ_ERR_INVALID_ARG, "%s: sizes must be > 0", fn);
    gptq_status st = check_cfg(cfg, d_in, fn);
    if (st != GPTQ_OK) return st;
    if (n_grid < 1 || n_grid > 64) return fail(GPTQ_ERR_INVALID_ARG, "%s: n_grid outside 1..64", fn);
    if (!W || !H || !act_abssum || !s || !losses || !best) return fail(GPTQ_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (!aligned(W, 4) || !aligned(H, 4) || !aligned(act_abssum, 8) || !aligned(s, 4) || !aligned(losses, 8) || !aligned(best, 4))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    const size_t need = gptq::awq_ws_bytes(d_out, d_in, *cfg);
    if (!ws || ws_bytes < need) return fail(GPTQ_ERR_WORKSPACE, "%s: need %zu workspace bytes, got %zu", fn, need, ws ? ws_bytes : (size_t)0);
    return hip_status(gptq::run_awq_search(W, d_out, d_in, H, act_abssum, n_tok, *cfg, n_grid, s, losses, best, ws, stream), fn);
}

gptq_status gptq_scale_layer(float *W, int64_t d_out, int64_t d_in, float *H, double *hdiag, const float *s,
                             hipStream_t stream) {
    const char *fn = "gptq_scale_layer";
    if (d_in <= 0 || (W && d_out <= 0)) return fail(GPTQ_ERR_INVALID_ARG, "%s: sizes must be > 0", fn);
    if (!s) return fail(GPTQ_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if ((W && !aligned(W, 4)) || (H && !aligned(H, 4)) || (hdiag && !aligned(hdiag, 8)) || !aligned(s, 4))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    return hip_status(gptq::run_scale_layer(W, d_out, d_in, H, hdiag, s, stream), fn);
}

gptq_status gptq_pack_codes(const uint8_t *codes, int64_t d_out, int64_t d_in, int32_t bits, const int32_t *perm,
                            uint32_t *packed, hipStream_t stream) {
    const char *fn = "gptq_pack_codes";
    if (d_out <= 0 || d_in <= 0) return fail(GPTQ_ERR_INVALID_ARG, "%s: sizes must be > 0", fn);
    if (bits < 2 || bits > 8) return fail(GPTQ_ERR_INVALID_ARG, "%s: bits=%d outside 2..8", fn, bits);
    if (!codes || !packed) return fail(GPTQ_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (!aligned(packed, 4) || (perm && !aligned(perm, 4))) return fail(GPTQ_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    return hip_status(gptq::run_pack(codes, d_out, d_in, bits, perm, packed, stream), fn);
}

gptq_status gptq_w4a16_gemm(const void *X, gptq_dtype x_dtype, int64_t M, int64_t d_in, int64_t ldx,
                            const int32_t *kperm, const uint32_t *packed, const float *scales, const float *zeros,
                            int32_t group_size, int64_t d_out, float *Y, int64_t ldy, void *ws, size_t ws_bytes,
                            hipStream_t stream) {
    const char *fn = "gptq_w4a16_gemm";
    if (M <= 0 || d_in <= 0 || d_out <= 0) return fail(GPTQ_ERR_INVALID_ARG, "%s: sizes must be > 0", fn);
    if (x_dtype != GPTQ_DT_F16) return fail(GPTQ_ERR_UNSUPPORTED, "%s: activations must be fp16", fn);
    if (group_size < 0 || (group_size > 0 && d_in % group_size != 0))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: group_size does not divide d_in", fn);
    const int64_t g = group_size > 0 ? group_size : d_in;
    if (g % 32 != 0) return fail(GPTQ_ERR_UNSUPPORTED, "%s: group_size (or d_in when 0) must be a multiple of 32", fn);
    if (!X || !packed || !scales || !zeros || !Y) return fail(GPTQ_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (ldx < d_in || ldy < d_out) return fail(GPTQ_ERR_INVALID_ARG, "%s: ldx < d_in or ldy < d_out", fn);
    if (!aligned(X) || ldx % 8 != 0 || !aligned(packed) || !aligned(scales, 4) || !aligned(zeros, 4) || !aligned(Y, 4) ||
        (kperm && !aligned(kperm, 4)))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: X and packed must be 16-byte aligned, ldx a multiple of 8; other pointers 4-byte aligned", fn);
    const size_t need = gptq::w4a16_ws_bytes(M, d_in, d_out, g);
    if (!ws || ws_bytes < need) return fail(GPTQ_ERR_WORKSPACE, "%s: need %zu workspace bytes, got %zu", fn, need, ws ? ws_bytes : (size_t)0);
    return hip_status(gptq::run_w4a16(X, M, d_in, ldx, kperm, packed, scales, zeros, g, d_out, Y, ldy, ws, stream), fn);
}

gptq_status gptq_gemv(const void *X, gptq_dtype x_dtype, int64_t M, int64_t ldx, const gptq_packed *w, const float *bias,
                      void *Y, gptq_dtype y_dtype, int64_t ldy, void *ws, size_t ws_bytes, hipStream_t stream) {
    const char *fn = "gptq_gemv";
    const gptq_status st = check_packed(w, fn, "w");
    if (st != GPTQ_OK) return st;
    return run_gemv_checked(X, x_dtype, M, ldx, w, nullptr, bias, Y, y_dtype, ldy, ws, ws_bytes, stream, fn);
}

gptq_status gptq_gemv_gated(const void *X, gptq_dtype x_dtype, int64_t M, int64_t ldx, const gptq_packed *gate,
                            const gptq_packed *up, void *H, gptq_dtype h_dtype, int64_t ldh, void *ws, size_t ws_bytes,
                            hipStream_t stream) {
    const char *fn = "gptq_gemv_gated";
    const gptq_status st = check_pair(gate, up, fn);
    if (st != GPTQ_OK) return st;
    return run_gemv_checked(X, x_dtype, M, ldx, gate, up, nullptr, H, h_dtype, ldh, ws, ws_bytes, stream, fn);
}

gptq_status gptq_moe_workspace_bytes(int64_t T, int64_t d, int64_t d_ff, int32_t n_experts, int32_t top_k, size_t *out) {
    const char *fn = "gptq_moe_workspace_bytes";
    if (!out) return fail(GPTQ_ERR_INVALID_ARG, "%s: out is NULL", fn);
    const gptq_status st = check_moe_sizes(T, d, d_ff, n_experts, top_k, fn);
    if (st != GPTQ_OK) return st;
    *out = gptq::moe_ws_bytes(T, d, d_ff, n_experts, top_k);
    return GPTQ_OK;
}

gptq_status gptq_moe_layer(const void *X, gptq_dtype x_dtype, int64_t T, int64_t ldx, const void *router,
                           gptq_dtype router_dtype, int32_t n_experts, int32_t top_k, int32_t renormalize,
                           const gptq_packed *gate, const gptq_packed *up, const gptq_packed *down, int32_t *ids,
                           float *weights, void *Y, gptq_dtype y_dtype, int64_t ldy, void *ws, size_t ws_bytes,
                           hipStream_t stream) {
    const char *fn = "gptq_moe_layer";
    gptq_status st = check_pair(gate, up, fn);
    if (st == GPTQ_OK) st = check_packed(down, fn, "down");
    if (st == GPTQ_OK) st = check_moe_sizes(T, gate->d_in, gate->d_out, n_experts, top_k, fn);
    if (st != GPTQ_OK) return st;
    if (down->d_in != gate->d_out || down->d_out != gate->d_in || down->bits != gate->bits)
        return fail(GPTQ_ERR_INVALID_ARG, "%s: down must be [d][d_ff] with the bits of gate [d_ff][d]", fn);
    st = check_few(X, x_dtype, T, ldx, gate->d_in, Y, y_dtype, ldy, gate->d_in, fn);
    if (st != GPTQ_OK) return st;
    if (router && router_dtype != GPTQ_DT_F32 && router_dtype != x_dtype)
        return fail(GPTQ_ERR_INVALID_ARG, "%s: the router must be fp32 or of X's type", fn);
    if (T > 0 && !router && (!ids || !weights))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: without a router, ids and weights are inputs", fn);
    if ((router && !aligned(router)) || (ids && !aligned(ids, 4)) || (weights && !aligned(weights, 4)))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    if (T == 0) return GPTQ_OK;
    const size_t need = gptq::moe_ws_bytes(T, gate->d_in, gate->d_out, n_experts, top_k);
    if (!ws || ws_bytes < need)
        return fail(GPTQ_ERR_WORKSPACE, "%s: need %zu workspace bytes, got %zu", fn, need, ws ? ws_bytes : (size_t)0);
    if (!aligned(ws)) return fail(GPTQ_ERR_INVALID_ARG, "%s: misaligned workspace", fn);
    st = check_apart(X, T, ldx, gate->d_in, Y, y_dtype, ldy, gate->d_in, fn);
    if (st != GPTQ_OK) return st;
    return hip_status(gptq::run_moe(X, x_dtype, T, ldx, router, router_dtype, n_experts, top_k, renormalize ? 1 : 0, *gate,
                                    *up, *down, ids, weights, Y, y_dtype, ldy, ws, stream),
                      fn);
}

gptq_status gptq_kv_append(const void *K, int64_t ldk, const void *V, int64_t ldv, gptq_dtype dtype, int64_t T, const int32_t *offs,
                           const gptq_kv_cache *cache, const int32_t *table, int64_t width, const int32_t *lens, int64_t n_seq,
                           void *K_out, int64_t ldko, void *V_out, int64_t ldvo, hipStream_t stream) {
    const char *fn = "gptq_kv_append";
    gptq_status st = check_kv(cache, fn);
    if (st == GPTQ_OK) st = check_seqs(cache, table, width, lens, n_seq, 0, fn);
    if (st != GPTQ_OK) return st;
    const int64_t row = (int64_t)cache->n_heads * cache->head_dim;
    if (!few_dtype(dtype)) return fail(GPTQ_ERR_INVALID_ARG, "%s: keys and values must be fp16 or bf16", fn);
    if (T < 0 || (!offs && T > 0 && (n_seq == 0 || T % n_seq != 0)))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: T must be a multiple of n_seq where there are no offsets", fn);
    if (T > ((int64_t)1 << 26) / cache->n_heads) return fail(GPTQ_ERR_UNSUPPORTED, "%s: T * n_heads above 2^26", fn);
    if (T > 0 && (!K || !V)) return fail(GPTQ_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (ldk < row || ldv < row || (K_out && ldko < row) || (V_out && ldvo < row))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: leading dimension too small", fn);
    if (!aligned(K) || !aligned(V) || ldk % 8 != 0 || ldv % 8 != 0 || (K_out && (!aligned(K_out) || ldko % 8 != 0)) ||
        (V_out && (!aligned(V_out) || ldvo % 8 != 0)))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: K, V and the results must be 16-byte aligned, their pitches multiples of 8", fn);
    if (offs && !aligned(offs, 4)) return fail(GPTQ_ERR_INVALID_ARG, "%s: misaligned offsets", fn);
    if (T == 0 || n_seq == 0) return GPTQ_OK;
    // a thread writes the values that it read, after reading them
    const bool same_k = K_out == K && ldko == ldk, same_v = V_out == V && ldvo == ldv;
    if ((K_out && ((!same_k && many_overlap(K, 2 * ldk, 2 * row, K_out, 2 * ldko, 2 * row, T)) ||
                   many_overlap(V, 2 * ldv, 2 * row, K_out, 2 * ldko, 2 * row, T))) ||
        (V_out && ((!same_v && many_overlap(V, 2 * ldv, 2 * row, V_out, 2 * ldvo, 2 * row, T)) ||
                   many_overlap(K, 2 * ldk, 2 * row, V_out, 2 * ldvo, 2 * row, T))) ||
        (K_out && V_out && many_overlap(K_out, 2 * ldko, 2 * row, V_out, 2 * ldvo, 2 * row, T)))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: K, V and the results overlap", fn);
    return hip_status(gptq::run_kv_append(K, ldk, V, ldv, dtype, T, offs, *cache, table, width, lens, n_seq, K_out, ldko, V_out, ldvo, stream),
                      fn);
}

gptq_status gptq_kv_attention_workspace_bytes(const gptq_kv_cache *cache, int64_t n_seq, int64_t n, int64_t q_heads, int64_t max_len,
                                              size_t *out) {
    const char *fn = "gptq_kv_attention_workspace_bytes";
    if (!out) return fail(GPTQ_ERR_INVALID_ARG, "%s: out is NULL", fn);
    gptq_status st = check_kv(cache, fn);
    if (st == GPTQ_OK) st = check_kv_queries(cache, n_seq, n, q_heads, max_len, fn);
    if (st != GPTQ_OK) return st;
    *out = gptq::kv_attention_ws_bytes(*cache, n_seq, n, q_heads, max_len);
    return GPTQ_OK;
}

gptq_status gptq_kv_attention(const void *Q, gptq_dtype dtype, int64_t n_seq, int64_t n, int64_t q_heads, int64_t ldq,
                              const gptq_kv_cache *cache, const int32_t *table, int64_t width, const int32_t *lens, int64_t max_len,
                              float scale, int32_t accumulate, float decay, void *O, int64_t ldo, void *ws, size_t ws_bytes,
                              hipStream_t stream) {
    const char *fn = "gptq_kv_attention";
    gptq_status st = check_kv(cache, fn);
    if (st == GPTQ_OK) st = check_seqs(cache, table, width, lens, n_seq, max_len, fn);
    if (st == GPTQ_OK) st = check_kv_queries(cache, n_seq, n, q_heads, max_len, fn);
    if (st != GPTQ_OK) return st;
    const int64_t row = q_heads * cache->head_dim;
    if (!few_dtype(dtype)) return fail(GPTQ_ERR_INVALID_ARG, "%s: queries must be fp16 or bf16", fn);
    if (!(scale > 0.0f) || scale > 0x1p127f)  // (times log2 e it is finite)
        return fail(GPTQ_ERR_INVALID_ARG, "%s: scale must be > 0 and at most 2^127", fn);
    if (accumulate && !(decay >= 0.0f && decay <= 1.0f)) return fail(GPTQ_ERR_INVALID_ARG, "%s: decay outside [0, 1]", fn);
    if (accumulate && !cache->weight) return fail(GPTQ_ERR_INVALID_ARG, "%s: the cache keeps no weights", fn);
    if (n_seq > 0 && (!Q || !O)) return fail(GPTQ_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (ldq < row || ldo < row) return fail(GPTQ_ERR_INVALID_ARG, "%s: leading dimension too small", fn);
    if (!aligned(Q) || ldq % 8 != 0 || !aligned(O, 2))
        return fail(GPTQ_ERR_INVALID_ARG, "%s: Q must be 16-byte aligned with ldq a multiple of 8, O 2-byte aligned", fn);
    if (n_seq == 0) return GPTQ_OK;
    const size_t need = gptq::kv_attention_ws_bytes(*cache, n_seq, n, q_heads, max_len);
    if (!ws || ws_bytes < need) return fail(GPTQ_ERR_WORKSPACE, "%s: need %zu workspace bytes, got %zu", fn, need, ws ? ws_bytes : (size_t)0);
    if (!aligned(ws)) return fail(GPTQ_ERR_INVALID_ARG, "%s: misaligned workspace", fn);
    if (many_overlap(Q, 2 * ldq, 2 * row, O, 2 * ldo, 2 * row, n_seq * n)) return fail(GPTQ_ERR_INVALID_ARG, "%s: Q and the result overlap", fn);
    return hip_status(gptq::run_kv_attention(Q, dtype, n_seq, n, q_heads, ldq, *cache, table, width, lens, max_len, scale, accumulate != 0,
                                             decay, O, ldo, ws, stream),
                      fn);
}

gptq_status gptq_kv_evict_workspace_bytes(const gptq_kv_cache *cache, int64_t n_seq, int64_t max_len, int64_t budget, size_t *out) {
    const char *fn = "gptq_kv_evict_workspace_bytes";
    if (!out) return fail(GPTQ_ERR_INVALID_ARG, "%s: out is NULL", fn);
    gptq_status st = check_kv(cache, fn);
    if (st == GPTQ_OK) st = check_kv_budget(cache, n_seq, max_len, budget, fn);
    if (st != GPTQ_OK) return st;
    *out = gptq::kv_evict_ws_bytes(*cache, n_seq, max_len, budget);
    return GPTQ_OK;
}

gptq_status gptq_kv_evict(const gptq_kv_cache *cache, const int32_t *table, int64_t width, const int32_t *lens, int64_t n_seq,
                          int64_t max_len, const int32_t *to, int64_t to_width, int64_t budget, int64_t recent, int32_t *kept,
                          int32_t *new_lens, void *ws, size_t ws_bytes, hipStream_t stream) {
    const char *fn = "gptq_kv_evict";
    gptq_status st = check_kv(cache, fn);
    if (st == GPTQ_OK) st = check_seqs(cache, table, width, lens, n_seq, max_len, fn);
    if (st == GPTQ_OK) st = check_kv_budget(cache, n_seq, max_len, budget, fn);
    if (st != GPTQ_OK) return st;
    if (recent < 0 || recent > budget) return fail(GPTQ_ERR_INVALID_ARG, "%s: recent outside 0 .. budget", fn);
    if (to_width <= 0 || to_width > kKvTokens / cache->page || to_width * cache->page < budget)
        return fail(GPTQ_ERR_INVALID_ARG, "%s: the pages to fill do not hold the budget", fn);
    if (!cache->weight) return fail(GPTQ_ERR_INVALID_ARG, "%s: the cache keeps no weights", fn);
    if (n_seq > 0 && (!to || !kept)) return fail(GPTQ_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    if (!aligned(to, 4) || !aligned(kept, 4) || !aligned(new_lens, 4)) return fail(GPTQ_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    if (n_seq == 0) return GPTQ_OK;
    const size_t need = gptq::kv_evict_ws_bytes(*cache, n_seq, max_len, budget);
    if (need > 0 && (!ws || ws_bytes < need))
        return fail(GPTQ_ERR_WORKSPACE, "%s: need %zu workspace bytes, got %zu", fn, need, ws ? ws_bytes : (size_t)0);
    if (need > 0 && !aligned(ws)) return fail(GPTQ_ERR_INVALID_ARG, "%s: misaligned workspace", fn);
    // what a workgroup writes, others read: no result may lie in an input or in the other
    const int64_t kept_bytes = 4 * n_seq * cache->n_heads * budget, lens_bytes = 4 * n_seq;
    auto overlap = [](const void *a, int64_t na, const void *b, int64_t nb) { return a && many_overlap(a, na, na, b, nb, nb, 1); };
    const struct { const void *p; int64_t bytes; } in[] = {{table, 4 * n_seq * width}, {lens, lens_bytes}, {to, 4 * n_seq * to_width}};
    bool shared = overlap(new_lens, lens_bytes, kept, kept_bytes);
    for (const auto &x : in) shared |= overlap(kept, kept_bytes, x.p, x.bytes) || overlap(new_lens, lens_bytes, x.p, x.bytes);
    if (shared) return fail(GPTQ_ERR_INVALID_ARG, "%s: kept or new_lens overlaps table, lens, to or the other", fn);
    return hip_status(gptq::run_kv_evict(*cache, table, width, lens, n_seq, max_len, to, to_width, budget, recent, kept, new_lens, ws, stream),
                      fn);
}

}  // extern "C"
