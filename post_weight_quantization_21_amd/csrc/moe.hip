// A mixture-of-experts layer for a few tokens, its experts packed.
//
//   router:  L = X R^T in fp64, one workgroup per expert and four tokens
//   choose:  one workgroup: a wave per token picks its top_k experts; then the
//            (token, expert) pairs are listed expert by expert
//   gate/up: a workgroup per listed expert and 16 rows of both matrices; its
//            pairs are the rows of one 16-row matrix operand (few_core.h), so an
//            expert's weights are read once however many tokens chose it
//   down:    a workgroup per 16 rows of the result; its waves share the listed
//            experts' K steps laid end to end, each adding weight * product to
//            its own sums per token; the waves' sums are added in wave order
#include <algorithm>

#include "few_core.h"

namespace gptq {
namespace {

constexpr int kMaxPairs = kMoeMaxTokens * kMoeMaxTopK;
constexpr int kMaxWaves = 16;

// The chosen (token, expert) pairs, expert by expert, tokens ascending.
struct Lists {
    int32_t n;                      // experts chosen by any token
    int32_t expert[kMaxPairs];      // ... in ascending order
    int32_t start[kMaxPairs + 1];   // their first pairs
    int32_t token[kMaxPairs];
    float weight[kMaxPairs];
};

template <typename T>
__device__ __forceinline__ void load8(const T *p, float v[8]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    typename Vec8<T>::V h = __builtin_bit_cast(typename Vec8<T>::V, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
}
template <>
__device__ __forceinline__ void load8<float>(const float *p, float v[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

constexpr int kRouterTokens = 4;  // per workgroup

template <typename T, typename TR>
__global__ __launch_bounds__(256) void router_kernel(const T *__restrict__ X, int64_t ldx, int n_tok,
                                                     const TR *__restrict__ R, int d, int n_experts,
                                                     double *__restrict__ logits) {
    const int e = blockIdx.x, t0 = blockIdx.y * kRouterTokens;
    __shared__ double part[4][kRouterTokens];
    double acc[kRouterTokens] = {};
    for (int c = 8 * threadIdx.x; c < d; c += 8 * 256) {
        float r[8], x[8];
        load8(R + (int64_t)e * d + c, r);
#pragma unroll
        for (int t = 0; t < kRouterTokens; ++t) {
            load8(X + std::min(t0 + t, n_tok - 1) * ldx + c, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[t] = fma((double)x[i], (double)r[i], acc[t]);
        }
    }
#pragma unroll
    for (int t = 0; t < kRouterTokens; ++t) {
        for (int o = 32; o > 0; o >>= 1) acc[t] += __shfl_xor(acc[t], o);
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6][t] = acc[t];
    }
    __syncthreads();
    const int t = threadIdx.x;
    if (t < kRouterTokens && t0 + t < n_tok)
        logits[(int64_t)(t0 + t) * n_experts + e] = part[0][t] + part[1][t] + part[2][t] + part[3][t];
}

__global__ __launch_bounds__(1024) void choose_kernel(const double *__restrict__ logits, int n_tok, int n_experts,
                                                      int top_k, int renormalize, int32_t *ids, float *weights,
                                                      Lists *lists) {
    __shared__ int32_t sel[kMoeMaxTokens][kMoeMaxTopK];
    __shared__ float wsel[kMoeMaxTokens][kMoeMaxTopK];
    __shared__ uint32_t tokens_of[kMoeMaxExperts];  // bit t: token t chose the expert
    __shared__ uint32_t wave_sum[kMaxWaves];
    const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
    constexpr int kPer = kMoeMaxExperts / kWave;
    if (tid < kMoeMaxExperts) tokens_of[tid] = 0;
    if (wave < n_tok) {
        if (!logits) {
            if (lane < top_k) {
                sel[wave][lane] = ids[wave * top_k + lane];
                wsel[wave][lane] = weights[wave * top_k + lane];
            }
        } else {
            double v[kPer];
            double top = -INFINITY;
            uint32_t left = 0;  // bit i: expert lane + 64 i not chosen yet
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int e = lane + kWave * i;
                v[i] = e < n_experts ? logits[(int64_t)wave * n_experts + e] : 0.0;
                if (e < n_experts) left |= 1u << i;
            }
            bool bad = false;  // a NaN logit makes every probability NaN, as the softmax's sum is
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (left >> i & 1) {
                    bad |= v[i] != v[i];
                    top = fmax(top, v[i]);
                }
            for (int o = 32; o > 0; o >>= 1) top = fmax(top, __shfl_xor(top, o));
            double sum = 0.0;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (left >> i & 1) sum += exp(v[i] - top);
            for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
            if (__any(bad)) sum = NAN;
            double chosen = 0.0, mine = 0.0;  // sum of the chosen probabilities; lane j: the j-th
            for (int j = 0; j < top_k; ++j) {
                double bv = -INFINITY;
                int be = INT32_MAX;  // none
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const double c = v[i] == v[i] ? v[i] : -INFINITY;  // NaN ranks below every number
                    if ((left >> i & 1) && (be == INT32_MAX || c > bv)) bv = c, be = lane + kWave * i;
                }
                for (int o = 32; o > 0; o >>= 1) {
                    const double ov = __shfl_xor(bv, o);
                    const int oe = __shfl_xor(be, o);
                    if (oe != INT32_MAX && (be == INT32_MAX || ov > bv || (ov == bv && oe < be))) bv = ov, be = oe;
                }
                if ((be & 63) == lane) left &= ~(1u << (be >> 6));
                const double p = exp(bv - top) / sum;
                chosen += p;
                if (lane == j) {
                    mine = p;
                    sel[wave][j] = be;
                }
            }
            if (lane < top_k) wsel[wave][lane] = (float)(renormalize ? mine / chosen : mine);
        }
    }
    __syncthreads();
    if (wave < n_tok && lane < top_k) {
        const int e = sel[wave][lane];
        if ((unsigned)e < (unsigned)n_experts) atomicOr(&tokens_of[e], 1u << wave);
        if (logits && ids) ids[wave * top_k + lane] = e;
        if (logits && weights) weights[wave * top_k + lane] = wsel[wave][lane];
    }
    __syncthreads();
    // positions by a prefix sum over the experts: chosen experts in the high half, pairs in the low one
    const uint32_t mask = tid < kMoeMaxExperts ? tokens_of[tid] : 0;
    const uint32_t own = (mask ? 0x10000u : 0u) + __popc(mask);
    uint32_t inc = own;
    for (int o = 1; o < kWave; o <<= 1) {
        const uint32_t up = __shfl_up(inc, o);
        if (lane >= o) inc += up;
    }
    if (lane == kWave - 1) wave_sum[wave] = inc;
    __syncthreads();
    uint32_t before = inc - own, total = 0;
    for (int w = 0; w < kMoeMaxExperts / kWave; ++w) {
        if (w < wave) before += wave_sum[w];
        total += wave_sum[w];
    }
    if (mask) {
        int p = before & 0xFFFF;
        lists->expert[before >> 16] = tid;
        lists->start[before >> 16] = p;
        for (uint32_t m = mask; m; m &= m - 1, ++p) {
            const int t = __ffs(m) - 1;
            float w = 0.0f;
            for (int j = 0; j < top_k; ++j)
                if (sel[t][j] == tid) w += wsel[t][j];
            lists->token[p] = t;
            lists->weight[p] = w;
        }
    }
    if (tid == 0) {
        lists->n = total >> 16;
        lists->start[total >> 16] = total & 0xFFFF;
    }
}

// Rows of activations in an expert's packed column order: out[p][k] =
// in[token of p or p][kperm[expert][k]], one workgroup row per pair.
__global__ __launch_bounds__(256) void gather_pairs_kernel(const uint16_t *__restrict__ in, int64_t ld, int by_token,
                                                           const Lists *__restrict__ lists, const int32_t *__restrict__ kperm,
                                                           int d, uint16_t *__restrict__ out) {
    const int a = blockIdx.y;
    if (a >= lists->n) return;
    const int k = blockIdx.x * 256 + threadIdx.x;
    if (k >= d) return;
    int c = kperm[(int64_t)lists->expert[a] * d + k];
    c = c < 0 ? 0 : (c >= d ? d - 1 : c);
    for (int p = lists->start[a]; p < lists->start[a + 1]; ++p)
        out[(int64_t)p * d + k] = in[(by_token ? lists->token[p] : p) * ld + c];
}

struct GateUpArgs {
    PackedDev w[2];
    const void *x;  // rows by token, or by pair (ldx = d) when gathered
    int64_t ldx;
    int by_pair;
    const Lists *lists;
    void *h;
};

template <int b, typename T, bool kSplit>
__global__ __launch_bounds__(1024) void gate_up_kernel(GateUpArgs a) {
    __shared__ float red[kMaxWaves][2][kFewRows][kTileRows];
    if ((int)blockIdx.y >= a.lists->n) return;
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave, waves = blockDim.x / kWave;
    const int start = a.lists->start[blockIdx.y], count = a.lists->start[blockIdx.y + 1] - start;
    const int ff = a.w[0].d_out;
    const int r0 = blockIdx.x * kTileRows;
    const int o = std::min(r0 + (lane & 15), ff - 1);
    const int p = start + std::min(lane & 15, count - 1);
    const int64_t xr = a.by_pair ? p : a.lists->token[p];
    const int steps = (a.w[0].units + 3) / 4;
    const int64_t at = (int64_t)a.lists->expert[blockIdx.y] * ff + o;
    const int64_t row[2] = {at, at};
    floatx4 acc[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
    few_product<b, T, 2, kSplit>(a.w, row, static_cast<const T *>(a.x) + xr * a.ldx, wave * steps / waves,
                                 (wave + 1) * steps / waves, acc);
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) red[wave][r][4 * (lane >> 4) + j][lane & 15] = acc[r][j];
    __syncthreads();
    const int n = threadIdx.x;
    if (n >= count * kTileRows || r0 + (n & 15) >= ff) return;
    float g = 0.0f, u = 0.0f;
    for (int w = 0; w < waves; ++w) {
        g += red[w][0][n >> 4][n & 15];
        u += red[w][1][n >> 4][n & 15];
    }
    static_cast<T *>(a.h)[(int64_t)(start + (n >> 4)) * ff + r0 + (n & 15)] = (T)silu_mul(g, u);
}

struct DownArgs {
    PackedDev w;
    const void *h;  // rows by pair
    const Lists *lists;
    int n_tok;
    void *y;
    int64_t ldy;
    gptq_dtype y_dt;
};

template <int b, typename T, bool kSplit>
__global__ __launch_bounds__(1024) void down_kernel(DownArgs a) {
    __shared__ float sums[kMaxWaves][kFewRows][kTileRows];
    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave, waves = blockDim.x / kWave;
    const int r0 = blockIdx.x * kTileRows, d = a.w.d_out, ff = a.w.units * kUnit;
    const int o = std::min(r0 + (lane & 15), d - 1);
    for (int i = lane; i < kFewRows * kTileRows; i += kWave) sums[wave][i / kTileRows][i % kTileRows] = 0.0f;
    const int steps = (a.w.units + 3) / 4;
    const int total = a.lists->n * steps;
    int s = (int)((int64_t)wave * total / waves);
    const int end = (int)((int64_t)(wave + 1) * total / waves);
    while (s < end) {
        const int i = s / steps, s0 = s - i * steps, s1 = std::min(steps, s0 + end - s);
        const int start = a.lists->start[i], count = a.lists->start[i + 1] - start;
        const int p = start + std::min(lane & 15, count - 1);
        const int64_t row[1] = {(int64_t)a.lists->expert[i] * d + o};
        floatx4 acc[1] = {{0.0f, 0.0f, 0.0f, 0.0f}};
        few_product<b, T, 1, kSplit>(&a.w, row, static_cast<const T *>(a.h) + (int64_t)p * ff, s0, s1, acc);
        // the wave's own sums: another lane may have written the element before, in order within the wave
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = 4 * (lane >> 4) + j;
            if (m < count) sums[wave][a.lists->token[start + m]][lane & 15] += a.lists->weight[start + m] * acc[0][j];
        }
        s += s1 - s0;
    }
    __syncthreads();
    const int n = threadIdx.x;
    if (n >= a.n_tok * kTileRows || r0 + (n & 15) >= d) return;
    float y = 0.0f;
    for (int w = 0; w < waves; ++w) y += sums[w][n >> 4][n & 15];
    store_as(a.y, (int64_t)(n >> 4) * a.ldy + r0 + (n & 15), a.y_dt, y);
}

struct Layout {
    size_t logits, lists, h, xg, hg, bytes;
};
Layout layout(int64_t T, int64_t d, int64_t d_ff, int n_experts, int top_k) {
    const size_t pairs = (size_t)T * top_k;
    Layout l;
    l.logits = 0;
    l.lists = align_up((size_t)T * n_experts * sizeof(double), 256);
    l.h = l.lists + align_up(sizeof(Lists), 256);
    l.xg = l.h + align_up(pairs * d_ff * 2, 256);
    l.hg = l.xg + align_up(pairs * d * 2, 256);
    l.bytes = l.hg + align_up(pairs * d_ff * 2, 256);
    return l;
}

struct MoeCall {
    const void *X;
    int64_t T, ldx;
    const void *router;
    gptq_dtype router_dt;
    int n_experts, top_k, renormalize;
    const gptq_packed *gate, *up, *down;
    int32_t *ids;
    float *weights;
    void *Y;
    gptq_dtype y_dt;
    int64_t ldy;
    char *ws;
};

template <int b, typename T>
void launch_experts(const MoeCall &c, const Layout &l, hipStream_t s) {
    const int64_t d = c.gate->d_in, ff = c.gate->d_out;
    Lists *lists = reinterpret_cast<Lists *>(c.ws + l.lists);
    const unsigned slots = (unsigned)std::min<int64_t>(c.n_experts, c.T * c.top_k);
    GateUpArgs g;
    g.w[0] = packed_dev(*c.gate);
    g.w[1] = packed_dev(*c.up);
    g.x = c.X;
    g.ldx = c.ldx;
    g.by_pair = 0;
    g.lists = lists;
    g.h = c.ws + l.h;
    if (c.gate->kperm) {
        gather_pairs_kernel<<<dim3((unsigned)ceil_div(d, 256), slots), 256, 0, s>>>(
            static_cast<const uint16_t *>(c.X), c.ldx, 1, lists, c.gate->kperm, (int)d, reinterpret_cast<uint16_t *>(c.ws + l.xg));
        g.x = c.ws + l.xg;
        g.ldx = d;
        g.by_pair = 1;
    }
    const dim3 grid((unsigned)ceil_div(ff, kTileRows), slots);
    const int waves = std::clamp((g.w[0].units + 3) / 4 / 2, 4, kMaxWaves);
    if (g.w[0].split)
        gate_up_kernel<b, T, true><<<grid, waves * kWave, 0, s>>>(g);
    else
        gate_up_kernel<b, T, false><<<grid, waves * kWave, 0, s>>>(g);
    DownArgs w;
    w.w = packed_dev(*c.down);
    w.h = g.h;
    w.lists = lists;
    w.n_tok = (int)c.T;
    w.y = c.Y;
    w.ldy = c.ldy;
    w.y_dt = c.y_dt;
    if (c.down->kperm) {
        gather_pairs_kernel<<<dim3((unsigned)ceil_div(ff, 256), slots), 256, 0, s>>>(
            reinterpret_cast<const uint16_t *>(c.ws + l.h), ff, 0, lists, c.down->kperm, (int)ff, reinterpret_cast<uint16_t *>(c.ws + l.hg));
        w.h = c.ws + l.hg;
    }
    if (w.w.split)
        down_kernel<b, T, true><<<(unsigned)ceil_div(d, kTileRows), 1024, 0, s>>>(w);
    else
        down_kernel<b, T, false><<<(unsigned)ceil_div(d, kTileRows), 1024, 0, s>>>(w);
}

template <typename T>
void launch_moe(const MoeCall &c, const Layout &l, hipStream_t s) {
    const int d = (int)c.gate->d_in;
    double *logits = c.router ? reinterpret_cast<double *>(c.ws + l.logits) : nullptr;
    if (logits) {
        const dim3 grid(c.n_experts, (unsigned)ceil_div(c.T, kRouterTokens));
        const T *x = static_cast<const T *>(c.X);
        if (c.router_dt == GPTQ_DT_F32)
            router_kernel<T, float><<<grid, 256, 0, s>>>(x, c.ldx, (int)c.T, static_cast<const float *>(c.router), d, c.n_experts, logits);
        else
            router_kernel<T, T><<<grid, 256, 0, s>>>(x, c.ldx, (int)c.T, static_cast<const T *>(c.router), d, c.n_experts, logits);
    }
    choose_kernel<<<1, 1024, 0, s>>>(logits, (int)c.T, c.n_experts, c.top_k, c.renormalize, c.ids, c.weights,
                                     reinterpret_cast<Lists *>(c.ws + l.lists));
    switch (c.gate->bits) {
    case 2: return launch_experts<2, T>(c, l, s);
    case 3: return launch_experts<3, T>(c, l, s);
    case 4: return launch_experts<4, T>(c, l, s);
    default: return launch_experts<8, T>(c, l, s);
    }
}

}  // namespace

size_t moe_ws_bytes(int64_t T, int64_t d, int64_t d_ff, int n_experts, int top_k) {
    return layout(T, d, d_ff, n_experts, top_k).bytes;
}

hipError_t run_moe(const void *X, gptq_dtype x_dt, int64_t T, int64_t ldx, const void *router, gptq_dtype router_dt,
                   int n_experts, int top_k, int renormalize, const gptq_packed &gate, const gptq_packed &up,
                   const gptq_packed &down, int32_t *ids, float *weights, void *Y, gptq_dtype y_dt, int64_t ldy,
                   void *ws, hipStream_t s) {
    const MoeCall c = {X, T, ldx, router, router_dt, n_experts, top_k, renormalize, &gate, &up, &down, ids, weights,
                       Y, y_dt, ldy, static_cast<char *>(ws)};
    const Layout l = layout(T, gate.d_in, gate.d_out, n_experts, top_k);
    if (x_dt == GPTQ_DT_BF16)
        launch_moe<__bf16>(c, l, s);
    else
        launch_moe<_Float16>(c, l, s);
    return hipGetLastError();
}

}  // namespace gptq
