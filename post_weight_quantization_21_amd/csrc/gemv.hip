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
    PackedDev w[2];
    const uint16_t *x;
    int64_t ldx;
    int M, lg;
    const float *bias;
    void *y;
    int64_t ldy;
    gptq_dtype y_dt;
};

// Gated: waves of the even tiles take the gate's rows, those of the odd ones up's.
template <int b, typename T, bool kGated, bool kSplit>
__global__ __launch_bounds__(kFewThreads, kFewOccupancy) void gemv_kernel(GemvArgs a) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    constexpr int R = kGated ? 2 : 1, LR = kGated ? 1 : 0;
    const int wave = few_wave(), lg = a.lg;
    const int lt = 3 - lg - LR;  // log2 of the row tiles
    const int tile = wave >> lg;
    const int64_t r0 = (int64_t)blockIdx.x * kTileRows << lt, d_out = a.w[0].d_out;
    const int64_t rt = std::min(r0 + (tile >> LR) * kTileRows, d_out - 1);
    const XRows x = {a.x, a.ldx, 0, false, 0};
    const floatx4 acc = few_product<b, T, 1, kSplit>(kGated && (tile & 1) ? a.w[R - 1] : a.w[0], rt, (int)std::min<int64_t>(kTileRows, d_out - rt),
                                                     x, a.M, wave & ((1 << lg) - 1), lg, reinterpret_cast<uint16_t *>(smem));
    float *sums = reinterpret_cast<float *>(smem);
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

// The activations in packed column order: Xg[m][k] = X[m][kperm[k]].
__global__ __launch_bounds__(256) void gather_kernel(const uint16_t *__restrict__ X, int64_t ldx, int64_t d_in,
                                                     const int32_t *__restrict__ kperm, uint16_t *__restrict__ Xg) {
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k >= d_in) return;
    int64_t c = kperm[k];
    c = c < 0 ? 0 : (c >= d_in ? d_in - 1 : c);
    Xg[blockIdx.y * d_in + k] = X[blockIdx.y * ldx + c];
}

template <int b, typename T>
void launch_gemv(const GemvArgs &a, bool gated, hipStream_t s) {
    const dim3 grid((unsigned)ceil_div(a.w[0].d_out, kTileRows * ((kFewWaves >> a.lg) / (gated ? 2 : 1))));
    const size_t lds = few_lds_bytes(a.M, 1, a.w[0].units);
    if (gated) {
        if (a.w[0].split)
            gemv_kernel<b, T, true, true><<<grid, kFewThreads, lds, s>>>(a);
        else
            gemv_kernel<b, T, true, false><<<grid, kFewThreads, lds, s>>>(a);
    } else {
        if (a.w[0].split)
            gemv_kernel<b, T, false, true><<<grid, kFewThreads, lds, s>>>(a);
        else
            gemv_kernel<b, T, false, false><<<grid, kFewThreads, lds, s>>>(a);
    }
}

template <typename T>
void launch_gemv_bits(const GemvArgs &a, int bits, bool gated, hipStream_t s) {
    switch (bits) {
    case 2: return launch_gemv<2, T>(a, gated, s);
    case 3: return launch_gemv<3, T>(a, gated, s);
    case 4: return launch_gemv<4, T>(a, gated, s);
    default: return launch_gemv<8, T>(a, gated, s);
    }
}

}  // namespace

PackedDev packed_dev(const gptq_packed &w) {
    PackedDev d;
    d.packed = w.packed;
    d.scales = w.scales;
    d.zeros = w.zeros;
    d.d_out = (int32_t)w.d_out;
    d.words = (int32_t)(w.d_in / kUnit * w.bits);
    const int64_t g = w.group_size > 0 ? w.group_size : w.d_in;
    d.groups = (int32_t)(w.d_in / g);
    d.units = (int32_t)(w.d_in / kUnit);
    d.split = d.groups > 1 && g % kStep != 0;
    // one group per row: any divisor above the number of steps
    d.by = small_div((uint32_t)(d.groups == 1 ? d.units + 1 : (d.split ? g / kUnit : g / kStep)));
    return d;
}

int few_slices(int64_t tiles, int units, int most) {
    const int steps = (units + 3) / 4;
    int lg = 0;
    while (2 << lg <= most && (tiles << (lg + 1)) <= kFewResident && (4 << lg) < steps) ++lg;
    return lg;
}

size_t gemv_ws_bytes(int64_t M, int64_t d_in) { return align_up((size_t)M * (size_t)d_in * 2, 256); }

hipError_t run_gemv(const void *X, gptq_dtype x_dt, int64_t M, int64_t ldx, const gptq_packed &w, const gptq_packed *up,
                    const float *bias, void *Y, gptq_dtype y_dt, int64_t ldy, void *ws, hipStream_t s) {
    GemvArgs a;
    a.w[0] = packed_dev(w);
    a.w[1] = packed_dev(up ? *up : w);
    a.x = static_cast<const uint16_t *>(X);
    a.ldx = ldx;
    a.M = (int)M;
    a.lg = up ? few_slices(2 * ceil_div(w.d_out, kTileRows), a.w[0].units, kFewWaves / 2)
              : few_slices(ceil_div(w.d_out, kTileRows), a.w[0].units, kFewWaves);
    a.bias = bias;
    a.y = Y;
    a.ldy = ldy;
    a.y_dt = y_dt;
    if (w.kperm) {
        gather_kernel<<<dim3((unsigned)ceil_div(w.d_in, 256), (unsigned)M), 256, 0, s>>>(
            static_cast<const uint16_t *>(X), ldx, w.d_in, w.kperm, static_cast<uint16_t *>(ws));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        a.x = static_cast<const uint16_t *>(ws);
        a.ldx = w.d_in;
    }
    if (x_dt == GPTQ_DT_BF16)
        launch_gemv_bits<__bf16>(a, w.bits, up != nullptr, s);
    else
        launch_gemv_bits<_Float16>(a, w.bits, up != nullptr, s);
    return hipGetLastError();
}

}  // namespace gptq
