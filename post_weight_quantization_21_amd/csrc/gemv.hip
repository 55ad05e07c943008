// Products of a few tokens with packed weights: Y = X' W^T (+ bias), and the
// first half of a gated MLP, H = silu(X' Wg^T) * (X' Wu^T).
//
// A workgroup owns 16 weight rows (gated: the same 16 of both matrices, so the
// activations are read once and the pair meets in registers) and its waves
// share K; their sums meet in LDS and are added in wave order, so results do
// not depend on timing.
#include <algorithm>

#include "few_core.h"

namespace gptq {
namespace {

struct GemvArgs {
    PackedDev w[2];
    const void *x;
    int64_t ldx, M;
    const float *bias;
    void *y;
    int64_t ldy;
    gptq_dtype y_dt;
};

constexpr int kMaxWaves = 16;

template <int b, typename T, bool kGated, bool kSplit>
__global__ __launch_bounds__(1024) void gemv_kernel(GemvArgs a) {
    constexpr int R = kGated ? 2 : 1;
    __shared__ float red[kMaxWaves][R][kFewRows][kTileRows];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave, waves = blockDim.x / kWave;
    const int64_t r0 = (int64_t)blockIdx.x * kTileRows;
    const int64_t o = r0 + (lane & 15);
    const int64_t oc = o < a.w[0].d_out ? o : a.w[0].d_out - 1;
    const int64_t m = (lane & 15) < a.M ? (lane & 15) : a.M - 1;
    const int steps = (a.w[0].units + 3) / 4;
    floatx4 acc[R];
    int64_t row[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        acc[r] = (floatx4){0.0f, 0.0f, 0.0f, 0.0f};
        row[r] = oc;
    }
    few_product<b, T, R, kSplit>(a.w, row, static_cast<const T *>(a.x) + m * a.ldx, wave * steps / waves,
                                 (wave + 1) * steps / waves, acc);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) red[wave][r][4 * (lane >> 4) + j][lane & 15] = acc[r][j];
    __syncthreads();
    const int n = threadIdx.x;  // token n / 16, row n % 16
    if (n >= a.M * kTileRows) return;
    const int64_t out = r0 + (n & 15);
    if (out >= a.w[0].d_out) return;
    float v[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        v[r] = 0.0f;
        for (int w = 0; w < waves; ++w) v[r] += red[w][r][n >> 4][n & 15];
    }
    float y;
    if constexpr (kGated)
        y = silu_mul(v[0], v[R - 1]);
    else
        y = a.bias ? v[0] + a.bias[out] : v[0];
    store_as(a.y, (n >> 4) * a.ldy + out, a.y_dt, y);
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
    const int steps = (a.w[0].units + 3) / 4;
    // two steps per wave at least (below, the waves only add to the final sum), and 256 threads for the epilogue
    const int waves = std::clamp(steps / 2, 4, kMaxWaves);
    const dim3 grid((unsigned)ceil_div(a.w[0].d_out, kTileRows)), block(waves * kWave);
    if (gated) {
        if (a.w[0].split)
            gemv_kernel<b, T, true, true><<<grid, block, 0, s>>>(a);
        else
            gemv_kernel<b, T, true, false><<<grid, block, 0, s>>>(a);
    } else {
        if (a.w[0].split)
            gemv_kernel<b, T, false, true><<<grid, block, 0, s>>>(a);
        else
            gemv_kernel<b, T, false, false><<<grid, block, 0, s>>>(a);
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

size_t gemv_ws_bytes(int64_t M, int64_t d_in) { return align_up((size_t)M * (size_t)d_in * 2, 256); }

hipError_t run_gemv(const void *X, gptq_dtype x_dt, int64_t M, int64_t ldx, const gptq_packed &w, const gptq_packed *up,
                    const float *bias, void *Y, gptq_dtype y_dt, int64_t ldy, void *ws, hipStream_t s) {
    GemvArgs a;
    a.w[0] = packed_dev(w);
    a.w[1] = packed_dev(up ? *up : w);
    a.x = X;
    a.ldx = ldx;
    a.M = M;
    a.bias = bias;
    a.y = Y;
    a.ldy = ldy;
    a.y_dt = y_dt;
    if (w.kperm) {
        gather_kernel<<<dim3((unsigned)ceil_div(w.d_in, 256), (unsigned)M), 256, 0, s>>>(
            static_cast<const uint16_t *>(X), ldx, w.d_in, w.kperm, static_cast<uint16_t *>(ws));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        a.x = ws;
        a.ldx = w.d_in;
    }
    if (x_dt == GPTQ_DT_BF16)
        launch_gemv_bits<__bf16>(a, w.bits, up != nullptr, s);
    else
        launch_gemv_bits<_Float16>(a, w.bits, up != nullptr, s);
    return hipGetLastError();
}

}  // namespace gptq
