// A mixture-of-experts layer for a few tokens, its experts packed.
//
//   router:  L = X R^T in fp64, one workgroup per expert and four tokens
//   choose:  one workgroup: a wave per token picks its top_k experts; then the
//            (token, expert) pairs are listed expert by expert
//   gate/up: workgroups per listed expert and tiles of 16 rows of both matrices;
//            the expert's pairs are the rows of one 16-row matrix operand
//            (few_core.h), so its weights are read once however many tokens chose
//            it
//   down:    the same for the second product, whose rows by pair are left in fp32
//   combine: Y[t] = the sum of the token's pairs, expert by expert, weighted
//
// h = silu(gate) * up between the products is a sum of bf16 values, two for a
// 16-bit result and three for an fp32 one (16 and 24 significant bits): each is
// an operand plane of the down product, whose weights are exact in bf16 up to a
// constant, so nothing of h is lost that the result could show.  One bf16 or fp16
// value per h costs 1.5 times the error of the final rounding.
#include <algorithm>
#include <cmath>

#include "few_core.h"

namespace gptq {
namespace {

constexpr int kMaxPairs = kMoeMaxTokens * kMoeMaxTopK;
constexpr int kChooseWaves = 16;

// The chosen (token, expert) pairs, expert by expert, tokens ascending.
struct Lists {
    int32_t n;                      // experts chosen by any token
    int32_t expert[kMaxPairs];      // ... in ascending order
    int32_t start[kMaxPairs + 1];   // their first pairs
    int32_t token[kMaxPairs];
    float weight[kMaxPairs];
    int32_t of_count[kMoeMaxTokens];               // a token's pairs ...
    int32_t of_token[kMoeMaxTokens][kMoeMaxTopK];  // ... in their order
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
    __shared__ uint32_t wave_sum[kChooseWaves];
    __shared__ uint8_t token_of[kMaxPairs];
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
            token_of[p] = (uint8_t)t;
            lists->token[p] = t;
            lists->weight[p] = w;
        }
    }
    if (tid == 0) {
        lists->n = total >> 16;
        lists->start[total >> 16] = total & 0xFFFF;
    }
    __syncthreads();
    if (wave < n_tok) {
        const int pairs = total & 0xFFFF;
        int n = 0;
        for (int p0 = 0; p0 < pairs; p0 += kWave) {
            const bool hit = p0 + lane < pairs && token_of[p0 + lane] == wave;
            const uint64_t hits = __ballot(hit);
            if (hit) lists->of_token[wave][n + __popcll(hits & ((1ull << lane) - 1))] = p0 + lane;
            n += __popcll(hits);
        }
        if (lane == 0) lists->of_count[wave] = n;
    }
}

// Rows of activations in an expert's packed column order: out[p][k] =
// in[token of p or p][kperm[expert][k]], plane by plane.
__global__ __launch_bounds__(256) void gather_pairs_kernel(const uint16_t *__restrict__ in, int64_t ld, int by_token,
                                                           int64_t plane, const Lists *__restrict__ lists, const int32_t *__restrict__ kperm,
                                                           int d, uint16_t *__restrict__ out) {
    const int a = blockIdx.y;
    if (a >= lists->n) return;
    const int k = blockIdx.x * 256 + threadIdx.x;
    if (k >= d) return;
    in += blockIdx.z * plane;
    out += blockIdx.z * plane;
    int c = kperm[(int64_t)lists->expert[a] * d + k];
    c = c < 0 ? 0 : (c >= d ? d - 1 : c);
    for (int p = lists->start[a]; p < lists->start[a + 1]; ++p)
        out[(int64_t)p * d + k] = in[(by_token ? lists->token[p] : p) * ld + c];
}

struct GateUpArgs {
    PackedDev w[2];
    const uint16_t *x;  // rows by token, or by pair (ldx = d) when gathered
    int64_t ldx;
    int by_pair, slices, planes;
    const Lists *lists;
    __bf16 *h;
    int64_t h_plane;
};

template <int b, typename T, bool kSplit>
__global__ __launch_bounds__(kFewThreads, 4) void gate_up_kernel(GateUpArgs a) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    if ((int)blockIdx.y >= a.lists->n) return;
    const int wave = few_wave(), lane = threadIdx.x % kWave;
    const int tiles = kFewWaves / a.slices / 2, tile = wave / a.slices;
    const int start = a.lists->start[blockIdx.y], count = a.lists->start[blockIdx.y + 1] - start;
    const int ff = a.w[0].d_out, r0 = blockIdx.x * tiles * kTileRows;
    const int64_t row = (int64_t)a.lists->expert[blockIdx.y] * ff + std::min(r0 + tile / 2 * kTileRows + (lane & 15), ff - 1);
    const XRows x = {a.by_pair ? a.x + start * a.ldx : a.x, a.ldx, 0, a.by_pair ? nullptr : a.lists->token + start};
    const floatx4 acc = few_product<b, T, 1, kSplit>(a.w[tile & 1], row, x, count, wave % a.slices, a.slices,
                                                     reinterpret_cast<uint16_t *>(smem));
    FewSums *sums = reinterpret_cast<FewSums *>(smem);
    few_share(sums, wave, acc, count);
    for (int n = threadIdx.x; n < count * tiles * kTileRows; n += kFewThreads) {
        const int m = n / (tiles * kTileRows), c = n % (tiles * kTileRows);
        if (r0 + c >= ff) continue;
        float v[2] = {0.0f, 0.0f};
#pragma unroll
        for (int r = 0; r < 2; ++r)
            for (int k = 0; k < a.slices; ++k) v[r] += sums[(c / kTileRows * 2 + r) * a.slices + k][m][c % kTileRows];
        float h = silu_mul(v[0], v[1]);
        __bf16 *dst = a.h + (int64_t)(start + m) * ff + r0 + c;
        for (int p = 0; p < a.planes; ++p) {
            const __bf16 t = (__bf16)h;
            dst[p * a.h_plane] = t;
            h -= (float)t;  // exact
        }
    }
}

struct DownArgs {
    PackedDev w;
    const uint16_t *h;  // planes of rows by pair
    int64_t h_plane;
    int slices;
    const Lists *lists;
    float *part;  // rows by pair
};

template <int b, int P, bool kSplit>
__global__ __launch_bounds__(kFewThreads, 4) void down_kernel(DownArgs a) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    if ((int)blockIdx.y >= a.lists->n) return;
    const int wave = few_wave(), lane = threadIdx.x % kWave;
    const int tiles = kFewWaves / a.slices, tile = wave / a.slices;
    const int start = a.lists->start[blockIdx.y], count = a.lists->start[blockIdx.y + 1] - start;
    const int d = a.w.d_out, r0 = blockIdx.x * tiles * kTileRows;
    const int64_t row = (int64_t)a.lists->expert[blockIdx.y] * d + std::min(r0 + tile * kTileRows + (lane & 15), d - 1);
    const int64_t ff = a.w.units * kUnit;
    const XRows x = {a.h + start * ff, ff, a.h_plane, nullptr};
    const floatx4 acc = few_product<b, __bf16, P, kSplit>(a.w, row, x, count, wave % a.slices, a.slices,
                                                          reinterpret_cast<uint16_t *>(smem));
    FewSums *sums = reinterpret_cast<FewSums *>(smem);
    few_share(sums, wave, acc, count);
    for (int n = threadIdx.x; n < count * tiles * kTileRows; n += kFewThreads) {
        const int m = n / (tiles * kTileRows), c = n % (tiles * kTileRows);
        if (r0 + c >= d) continue;
        float v = 0.0f;
        for (int k = 0; k < a.slices; ++k) v += sums[c / kTileRows * a.slices + k][m][c % kTileRows];
        a.part[(int64_t)(start + m) * d + r0 + c] = v;
    }
}

__global__ __launch_bounds__(256) void combine_kernel(const float *__restrict__ part, const Lists *__restrict__ lists, int d,
                                                      void *y, int64_t ldy, gptq_dtype y_dt) {
    const int c = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
    if (c >= d) return;
    float v = 0.0f;
    const int n = lists->of_count[t];
    for (int j = 0; j < n; ++j) {
        const int p = lists->of_token[t][j];
        v = fmaf(lists->weight[p], part[(int64_t)p * d + c], v);
    }
    store_as(y, t * ldy + c, y_dt, v);
}

constexpr int kMaxPlanes = 3;
struct Layout {
    size_t logits, lists, h, part, xg, hg, bytes;
};
Layout layout(int64_t T, int64_t d, int64_t d_ff, int n_experts, int top_k) {
    const size_t pairs = (size_t)T * top_k;
    Layout l;
    l.logits = 0;
    l.lists = align_up((size_t)T * n_experts * sizeof(double), 256);
    l.h = l.lists + align_up(sizeof(Lists), 256);
    l.part = l.h + align_up(kMaxPlanes * pairs * d_ff * 2, 256);
    l.xg = l.part + align_up(pairs * d * 4, 256);
    l.hg = l.xg + align_up(pairs * d * 2, 256);
    l.bytes = l.hg + align_up(kMaxPlanes * pairs * d_ff * 2, 256);
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

template <int b, int P>
void launch_down(const DownArgs &w, dim3 grid, size_t lds, hipStream_t s) {
    if (w.w.split)
        down_kernel<b, P, true><<<grid, kFewThreads, lds, s>>>(w);
    else
        down_kernel<b, P, false><<<grid, kFewThreads, lds, s>>>(w);
}

template <int b, typename T>
void launch_experts(const MoeCall &c, const Layout &l, hipStream_t s) {
    const int64_t d = c.gate->d_in, ff = c.gate->d_out, pairs = c.T * c.top_k;
    Lists *lists = reinterpret_cast<Lists *>(c.ws + l.lists);
    const unsigned slots = (unsigned)std::min<int64_t>(c.n_experts, pairs);
    // experts that `pairs` independent choices would hit, which the work is spread for
    const double busy = c.n_experts * (1.0 - std::pow(1.0 - 1.0 / c.n_experts, (double)pairs));
    GateUpArgs g;
    g.w[0] = packed_dev(*c.gate);
    g.w[1] = packed_dev(*c.up);
    g.x = static_cast<const uint16_t *>(c.X);
    g.ldx = c.ldx;
    g.by_pair = 0;
    g.lists = lists;
    g.h = reinterpret_cast<__bf16 *>(c.ws + l.h);
    g.h_plane = pairs * ff;
    g.planes = c.y_dt == GPTQ_DT_F32 ? 3 : 2;
    if (c.gate->kperm) {
        uint16_t *xg = reinterpret_cast<uint16_t *>(c.ws + l.xg);
        gather_pairs_kernel<<<dim3((unsigned)ceil_div(d, 256), slots), 256, 0, s>>>(g.x, c.ldx, 1, 0, lists, c.gate->kperm, (int)d, xg);
        g.x = xg;
        g.ldx = d;
        g.by_pair = 1;
    }
    const int64_t gu_tiles = ceil_div(ff, kTileRows);
    g.slices = few_slices((int64_t)(2 * busy * gu_tiles), g.w[0].units, kFewWaves / 2);
    const dim3 grid((unsigned)ceil_div(gu_tiles, kFewWaves / g.slices / 2), slots);
    const size_t lds = few_lds_bytes((int)c.T, 1, g.w[0].units);
    if (g.w[0].split)
        gate_up_kernel<b, T, true><<<grid, kFewThreads, lds, s>>>(g);
    else
        gate_up_kernel<b, T, false><<<grid, kFewThreads, lds, s>>>(g);
    DownArgs w;
    w.w = packed_dev(*c.down);
    w.h = reinterpret_cast<const uint16_t *>(g.h);
    w.h_plane = g.h_plane;
    w.lists = lists;
    w.part = reinterpret_cast<float *>(c.ws + l.part);
    if (c.down->kperm) {
        uint16_t *hg = reinterpret_cast<uint16_t *>(c.ws + l.hg);
        gather_pairs_kernel<<<dim3((unsigned)ceil_div(ff, 256), slots, g.planes), 256, 0, s>>>(w.h, ff, 0, w.h_plane, lists,
                                                                                               c.down->kperm, (int)ff, hg);
        w.h = hg;
    }
    const int64_t tiles = ceil_div(d, kTileRows);
    w.slices = few_slices((int64_t)(busy * tiles), w.w.units, kFewWaves);
    const dim3 dgrid((unsigned)ceil_div(tiles, kFewWaves / w.slices), slots);
    const size_t dlds = few_lds_bytes((int)c.T, g.planes, w.w.units);
    if (g.planes == 3)
        launch_down<b, 3>(w, dgrid, dlds, s);
    else
        launch_down<b, 2>(w, dgrid, dlds, s);
    combine_kernel<<<dim3((unsigned)ceil_div(d, 256), (unsigned)c.T), 256, 0, s>>>(w.part, lists, (int)d, c.Y, c.ldy, c.y_dt);
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
