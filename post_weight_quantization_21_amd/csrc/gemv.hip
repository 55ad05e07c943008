// Products of a few tokens with packed weights: Y = X' W^T (+ bias), and the
// first half of a gated MLP, H = silu(X' Wg^T) * (X' Wu^T).
//
// A workgroup of eight waves stages the activations in LDS and owns one to eight
// tiles of 16 weight rows; the waves of a tile share K and their sums meet in
// LDS, where they are added in wave order, so results do not depend on timing.
// Gated, half the tiles are the same rows of the other matrix.
#include <algorithm>

#include "few_core.h"

namespace gptq {
namespace {

struct GemvArgs {
    FewMat w[2];
    FewShape shape;
    int M;
    const uint16_t *x;
    int64_t ldx;
    const int32_t *order;
    const float *bias;
    void *y;
    int64_t ldy;
    gptq_dtype y_dt;
};

// Gated: the even tiles are the gate's rows, the odd ones up's.
// Cold weights, between calls.  Bound by the weights' bytes where they are many: one
// token of 28672 x 8192 in 4 bits (132 MB) takes 32.5 us, 4.1 TB/s; gated, eight
// tokens of 28672 x 8192 in groups of 64 (294 MB) 92-93 us, 3.2 TB/s, where
// unpacking, transposing and folding bind.  By start and staging where they are few:
// 6.1 us for 1024 x 4096, 23.9 us for sixteen tokens of 8192 x 8192 in 3 bits (256 KB
// of x per workgroup).
template <int b, typename T, bool kGated, bool kSplit, FewX kX>
__global__ __launch_bounds__(kFewThreads, kFewOccupancy) void gemv_kernel(GemvArgs a) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    constexpr int R = kGated ? 2 : 1, LR = kGated ? 1 : 0;
    const int wave = few_wave(), lg = a.shape.lg;
    const int lt = 3 - lg - LR;  // log2 of the row tiles
    const int64_t r0 = (int64_t)blockIdx.x * kTileRows << lt, d_out = a.shape.d_out;
    const XRows x = {a.x, a.ldx, false, 0, a.order, 0.0f};
    float *sums = reinterpret_cast<float *>(smem);
    const floatx4 acc = few_product<b, T, R, kSplit, kX>(a.w, a.shape, r0, (int)std::min<int64_t>(d_out - r0, kTileRows * kFewWaves), x,
                                                            a.M, wave, smem);
    few_share(sums, wave, acc, a.M);
    for (int n = threadIdx.x; n < a.M * kTileRows << lt; n += kFewThreads) {
        const int m = n >> (4 + lt), c = n & ((kTileRows << lt) - 1);
        if (r0 + c >= d_out) continue;
        const int w0 = (c >> 4) << (LR + lg);
        float y = few_sum(sums, w0, lg, a.M, m, c & 15);
        if constexpr (kGated)
            y = silu_mul(y, few_sum(sums, w0 + (1 << lg), lg, a.M, m, c & 15));
        else if (a.bias)
            y += a.bias[r0 + c];
        store_as(a.y, m * a.ldy + r0 + c, a.y_dt, y);
    }
}

// x prepared in memory, its columns in packed order: a thread per value (2.4 us
// for one token of 4096, a launch's least).
template <int b>
__global__ __launch_bounds__(256) void prepare_kernel(const uint16_t *__restrict__ X, int64_t ldx, int d_in,
                                                      const int32_t *__restrict__ kperm, uint16_t *__restrict__ out) {
    const int k = blockIdx.x * 256 + threadIdx.x, M = gridDim.y, m = blockIdx.y;  // k: column of whole quads
    if (k >= few_quads(d_in / kUnit) * kQuad) return;
    uint16_t v = 0;
    if (k < d_in) {
        int c = kperm[k];
        c = c < 0 ? 0 : (c >= d_in ? d_in - 1 : c);
        v = X[m * ldx + c];
    }
    out[prepared_at<b>(k, M, m)] = v;
}

template <int b, typename T, bool kGated, bool kSplit>
void launch_gemv(const GemvArgs &a, FewX x, hipStream_t s) {
    const dim3 grid((unsigned)ceil_div(a.shape.d_out, kTileRows * ((kFewWaves >> a.shape.lg) / (kGated ? 2 : 1))));
    auto kernel = x == kRawX ? gemv_kernel<b, T, kGated, kSplit, kRawX>
                             : (x == kOrderedX ? gemv_kernel<b, T, kGated, kSplit, kOrderedX> : gemv_kernel<b, T, kGated, kSplit, kPreparedX>);
    kernel<<<grid, kFewThreads, a.shape.lds, s>>>(a);
}

template <int b>
hipError_t launch_gemv_bits(GemvArgs a, gptq_dtype x_dt, const gptq_packed &w, bool gated, void *ws, hipStream_t s) {
    const FewX x = !w.kperm ? kRawX : (gemv_prepares(a.M, w.d_in) ? kPreparedX : kOrderedX);
    if (x == kPreparedX) {
        prepare_kernel<b><<<dim3((unsigned)(few_quads(a.shape.units) * kQuad / 256), (unsigned)a.M), 256, 0, s>>>(
            a.x, a.ldx, (int)w.d_in, w.kperm, static_cast<uint16_t *>(ws));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        a.x = static_cast<const uint16_t *>(ws);
    }
    const bool split = few_split(w);
    if (x_dt == GPTQ_DT_BF16) {
        if (gated)
            split ? launch_gemv<b, __bf16, true, true>(a, x, s) : launch_gemv<b, __bf16, true, false>(a, x, s);
        else
            split ? launch_gemv<b, __bf16, false, true>(a, x, s) : launch_gemv<b, __bf16, false, false>(a, x, s);
    } else {
        if (gated)
            split ? launch_gemv<b, _Float16, true, true>(a, x, s) : launch_gemv<b, _Float16, true, false>(a, x, s);
        else
            split ? launch_gemv<b, _Float16, false, true>(a, x, s) : launch_gemv<b, _Float16, false, false>(a, x, s);
    }
    return hipGetLastError();
}

}  // namespace

FewMat few_mat(const gptq_packed &w) { return {w.packed, w.scales, w.zeros}; }

bool few_split(const gptq_packed &w) { return w.group_size != 0 && w.group_size != w.d_in && w.group_size % kStep != 0; }

FewShape few_shape(const gptq_packed &w, double tiles, int most, int rows, int max_rows) {
    FewShape d;
    const int64_t g = w.group_size > 0 ? w.group_size : w.d_in;
    d.d_out = (int32_t)w.d_out;
    d.words = (int32_t)(w.d_in / kUnit * w.bits);
    d.groups = (int32_t)(w.d_in / g);
    d.units = (int32_t)(w.d_in / kUnit);
    // one group per row: any divisor above the number of steps
    d.by = small_div((uint32_t)(few_split(w) ? g / kUnit : (d.groups == 1 ? d.units + 1 : g / kStep)));
    // As many slices as leave the tiles room on the chip at once, and a phase of a quad each at least.
    const int quads = few_quads(d.units);
    d.lg = 0;
    while (2 << d.lg <= most && tiles * (2 << d.lg) <= kFewResident && 2 << d.lg <= quads) ++d.lg;
    auto plan = [&](int lg) {  // the phase of lg
        d.lg = lg;
        const int per_wg = (kFewWaves >> lg) * kTileRows;  // rows of weights
        const bool alone = tiles * (1 << lg) <= 256 * kFewWaves;
        d.quad_entries = (int32_t)ceil_div((int64_t)per_wg * kQuad * 8, g);
        if (d.groups == 1) d.quad_entries = 0;
        const int64_t all = few_fixed(lg) + (int64_t)quads * ((int64_t)max_rows * kQuad * 2 + d.quad_entries);
        d.lds = (int32_t)std::min<int64_t>(all, alone ? kLdsAlone : kLdsShared);
        return few_phase(d, rows);
    };
    int lg = d.lg, phase = plan(lg);
    while (lg > 0 && phase < 1 << lg) phase = plan(--lg);
    // Half the slices where that takes fewer phases (the workgroups, no more than compute units then, have the larger
    // LDS) and x fills most of a phase: 8 tokens of 8192 x 8192 in 17.2 us instead of 20.3, 16 of 28672 x 8192 in 50.4
    // instead of 55.2.  With x no more than twice the entries it loses: 4 of 28672 x 8192 39.9 us instead of 38.1,
    // 2 of 8192 x 28672 in groups of 32 75.6 instead of 63.9.
    if (lg > 0 && phase < quads) {
        const int lower = plan(lg - 1);
        if (ceil_div(quads, lower) >= ceil_div(quads, phase) || rows * kQuad * 2 < 3 * d.quad_entries) plan(lg);
    }
    return d;
}

// Up to eight values a thread the product's own gather costs less than a launch
// and a pass through memory: one token of 4096 x 4096 takes 6.9 us against 8.1,
// two of them 8.3 against 8.4, but four 11.6 against 8.6 and one token of 8192 x
// 8192 18.6 against 15.5, since every workgroup gathers all of x.
bool gemv_prepares(int64_t M, int64_t d_in) { return M * d_in > GPTQ_GEMV_GATHERS; }

size_t gemv_ws_bytes(int64_t M, int64_t d_in) {
    return gemv_prepares(M, d_in) ? align_up((size_t)prepared_values(M, (int)(d_in / kUnit)) * 2, 256) : 0;
}

hipError_t run_gemv(const void *X, gptq_dtype x_dt, int64_t M, int64_t ldx, const gptq_packed &w, const gptq_packed *up,
                    const float *bias, void *Y, gptq_dtype y_dt, int64_t ldy, void *ws, hipStream_t s) {
    GemvArgs a;
    a.w[0] = few_mat(w);
    a.w[1] = few_mat(up ? *up : w);
    const double tiles = (double)ceil_div(w.d_out, kTileRows);
    a.M = (int)M;
    a.shape = up ? few_shape(w, 2 * tiles, kFewWaves / 2, a.M, a.M) : few_shape(w, tiles, kFewWaves, a.M, a.M);
    a.x = static_cast<const uint16_t *>(X);
    a.ldx = ldx;
    a.order = w.kperm;
    a.bias = bias;
    a.y = Y;
    a.ldy = ldy;
    a.y_dt = y_dt;
    switch (w.bits) {
    case 2: return launch_gemv_bits<2>(a, x_dt, w, up, ws, s);
    case 3: return launch_gemv_bits<3>(a, x_dt, w, up, ws, s);
    case 4: return launch_gemv_bits<4>(a, x_dt, w, up, ws, s);
    default: return launch_gemv_bits<8>(a, x_dt, w, up, ws, s);
    }
}

}  // namespace gptq
