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

// The chosen (token, expert) pairs, numbered expert by expert, tokens ascending.
struct Expert {  // the a-th expert chosen by any token; count 0 past the last
    int32_t expert, start, count, pad;  // its pairs
    int32_t token[kMoeMaxTokens];
};
struct Token {  // a token's pairs, ascending
    int32_t count, pad[3];
    int32_t pair[kMoeMaxTopK];
    float weight[kMoeMaxTopK];
};
struct Lists {
    Token token[kMoeMaxTokens];
    Expert expert[kMaxPairs];
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

// A logit's rank as an unsigned key: ascending with the logit to 43 significant
// bits, then descending with the expert's index; a NaN lies below every number.
__device__ __forceinline__ uint64_t rank_key(double v, int e) {
    uint64_t k = __builtin_bit_cast(uint64_t, v + 0.0);  // -0 is 0
    k = k >> 63 ? ~k : k | (1ull << 63);
    if (v != v) k = 1ull << 9;  // above "no candidate", which is 0
    return (k & ~511ull) | (511 - e);
}
template <int ctrl, int rows>
__device__ __forceinline__ uint64_t dpp_max(uint64_t v) {
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, ctrl, rows, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), ctrl, rows, 0xf, false);
    const uint64_t o = (uint64_t)hi << 32 | lo;
    return o > v ? o : v;
}
// The largest of the wave's values, in every lane: prefix maxima within rows of
// 16 lanes (row_shr), then across rows (row_bcast), and the last lane's value.
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
    v = dpp_max<0x111, 0xf>(v);
    v = dpp_max<0x112, 0xf>(v);
    v = dpp_max<0x114, 0xf>(v);
    v = dpp_max<0x118, 0xf>(v);
    v = dpp_max<0x142, 0xa>(v);
    v = dpp_max<0x143, 0xc>(v);
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), 63) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, 63);
}

__global__ __launch_bounds__(1024) void choose_kernel(const double *__restrict__ logits, int n_tok, int n_experts,
                                                      int top_k, int renormalize, int slots, int32_t *ids, float *weights,
                                                      Lists *lists) {
    __shared__ int32_t sel[kMoeMaxTokens][kMoeMaxTopK];
    __shared__ float wsel[kMoeMaxTokens][kMoeMaxTopK];
    __shared__ uint32_t tokens_of[kMoeMaxExperts];  // bit t: token t chose the expert
    __shared__ uint32_t wave_sum[kMoeMaxExperts / kWave];
    __shared__ uint8_t token_of[kMaxPairs];
    __shared__ float weight_of[kMaxPairs];
    const int tid = threadIdx.x, wave = few_wave(), lane = tid % kWave;
    constexpr int kPer = kMoeMaxExperts / kWave;
    if (tid < kMoeMaxExperts) tokens_of[tid] = 0;
    if (wave < n_tok) {
        int e = -1;
        float w = 0.0f;
        if (!logits) {
            if (lane < top_k) {
                e = ids[wave * top_k + lane];
                w = weights[wave * top_k + lane];
            }
        } else {
            double v[kPer];
            uint64_t key[kPer];  // 0: no candidate (any more)
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int c = lane + kWave * i;
                v[i] = 0.0;
                key[i] = 0;
                if (kWave * i < n_experts && c < n_experts) {
                    v[i] = logits[(int64_t)wave * n_experts + c];
                    key[i] = rank_key(v[i], c);
                }
            }
            uint64_t any_nan = 0;
            double top = -INFINITY;
            for (int j = 0; j < top_k; ++j) {
                uint64_t best = key[0];
#pragma unroll
                for (int i = 1; i < kPer; ++i)
                    if (kWave * i < n_experts) best = key[i] > best ? key[i] : best;
                best = wave_max(best);
                const int be = 511 - (int)(best & 511);
                if (lane == j) e = be;
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (key[i] == best) key[i] = 0;
            }
            // softmax: the first choice holds the largest logit
            const int e0 = __builtin_amdgcn_readfirstlane(e);
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (kWave * i < n_experts) {
                    if (e0 >> 6 == i) top = __shfl(v[i], e0 & 63);
                    any_nan |= __ballot(v[i] != v[i]);
                }
            double sum = 0.0, mine = 0.0;  // lane j < top_k: its chosen logit
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (kWave * i < n_experts) {
                    if (lane + kWave * i < n_experts) sum += exp(v[i] - top);
                    const double c = __shfl(v[i], e & 63);
                    if (e >> 6 == i) mine = c;
                }
            for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
            if (any_nan) sum = NAN;  // as the sum over the softmax would be
            double p = lane < top_k ? exp(mine - top) / sum : 0.0, chosen = p;
            if (renormalize) {
                for (int o = kMoeMaxTopK / 2; o > 0; o >>= 1) chosen += __shfl_xor(chosen, o);
                p /= chosen;
            }
            w = (float)p;
        }
        if (lane < top_k) {
            sel[wave][lane] = e;
            wsel[wave][lane] = w;
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
    if (tid < kMoeMaxExperts) {
        for (int o = 1; o < kWave; o <<= 1) {
            const uint32_t up = __shfl_up(inc, o);
            if (lane >= o) inc += up;
        }
        if (lane == kWave - 1) wave_sum[wave] = inc;
    }
    __syncthreads();
    uint32_t before = inc - own, total = 0;
    for (int w = 0; w < kMoeMaxExperts / kWave; ++w) {
        if (w < wave) before += wave_sum[w];
        total += wave_sum[w];
    }
    if (mask) {
        Expert &x = lists->expert[before >> 16];
        int p = before & 0xFFFF, n = 0;
        x.expert = tid;
        x.start = p;
        x.count = __popc(mask);
        for (uint32_t m = mask; m; m &= m - 1, ++p, ++n) {
            const int t = __ffs(m) - 1;
            float w = 0.0f;
            for (int j = 0; j < top_k; ++j)
                if (sel[t][j] == tid) w += wsel[t][j];
            x.token[n] = t;
            token_of[p] = (uint8_t)t;
            weight_of[p] = w;
        }
    }
    if (tid >= (int)(total >> 16) && tid < slots) lists->expert[tid].count = 0;
    __syncthreads();
    if (wave < n_tok) {
        const int pairs = total & 0xFFFF;
        Token &x = lists->token[wave];
        int n = 0;
        for (int p0 = 0; p0 < pairs; p0 += kWave) {
            const bool hit = p0 + lane < pairs && token_of[p0 + lane] == wave;
            const uint64_t hits = __ballot(hit);
            if (hit) {
                const int i = n + __popcll(hits & ((1ull << lane) - 1));
                x.pair[i] = p0 + lane;
                x.weight[i] = weight_of[p0 + lane];
            }
            n += __popcll(hits);
        }
        if (lane == 0) x.count = n;
    }
}

// Rows of activations in an expert's packed column order: out[p][k] =
// in[token of p or p][kperm[expert][k]], plane by plane.
__global__ __launch_bounds__(256) void gather_pairs_kernel(const uint16_t *__restrict__ in, int64_t ld, int by_token,
                                                           int64_t plane, const Lists *__restrict__ lists, const int32_t *__restrict__ kperm,
                                                           int d, uint16_t *__restrict__ out) {
    const Expert &e = lists->expert[blockIdx.y];
    const int k = blockIdx.x * 256 + threadIdx.x;
    if (k >= d) return;
    in += blockIdx.z * plane;
    out += blockIdx.z * plane;
    if (e.count == 0) return;
    int c = kperm[(int64_t)e.expert * d + k];
    c = c < 0 ? 0 : (c >= d ? d - 1 : c);
    for (int i = 0; i < e.count; ++i)
        out[(int64_t)(e.start + i) * d + k] = in[(by_token ? e.token[i] : e.start + i) * ld + c];
}

struct GateUpArgs {
    PackedDev w[2];
    const uint16_t *x;  // rows by token, or by pair (ldx = d) when gathered
    int64_t ldx;
    int by_pair, lg, planes;
    const Lists *lists;
    __bf16 *h;
    int64_t h_plane;
};

template <int b, typename T, bool kSplit>
__global__ __launch_bounds__(kFewThreads, kFewOccupancy) void gate_up_kernel(GateUpArgs a) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const Expert &e = a.lists->expert[blockIdx.y];
    const int token = e.token[threadIdx.x & (kMoeMaxTokens - 1)];
    const int start = e.start, count = e.count, wave = few_wave(), lg = a.lg;
    if (count == 0) return;
    const int lt = 2 - lg;  // log2 of the row tiles
    const int tile = wave >> lg;
    const int ff = a.w[0].d_out, r0 = blockIdx.x * kTileRows << lt, rt = std::min(r0 + (tile >> 1) * kTileRows, ff - 1);
    const XRows x = {a.by_pair ? a.x + start * a.ldx : a.x, a.ldx, 0, !a.by_pair, token};
    const floatx4 acc = few_product<b, T, 1, kSplit>(tile & 1 ? a.w[1] : a.w[0], (int64_t)e.expert * ff + rt, std::min(kTileRows, ff - rt), x,
                                                     count, wave & ((1 << lg) - 1), lg, reinterpret_cast<uint16_t *>(smem));
    float *sums = reinterpret_cast<float *>(smem);
    few_share(sums, wave, acc, count);
    for (int n = threadIdx.x; n < count * kTileRows << lt; n += kFewThreads) {
        const int m = n >> (4 + lt), c = n & ((kTileRows << lt) - 1);
        if (r0 + c >= ff) continue;
        const int w0 = (c >> 4) << (1 + lg);
        float h = silu_mul(few_sum(sums, w0, lg, count, m, c & 15), few_sum(sums, w0 + (1 << lg), lg, count, m, c & 15));
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
    int lg;
    const Lists *lists;
    float *part;  // rows by pair
};

template <int b, int P, bool kSplit>
__global__ __launch_bounds__(kFewThreads, kFewOccupancy) void down_kernel(DownArgs a) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const Expert &e = a.lists->expert[blockIdx.y];
    const int start = e.start, count = e.count, wave = few_wave(), lg = a.lg;
    if (count == 0) return;
    const int lt = 3 - lg, tile = wave >> lg;
    const int d = a.w.d_out, r0 = blockIdx.x * kTileRows << lt, rt = std::min(r0 + tile * kTileRows, d - 1);
    const int64_t ff = a.w.units * kUnit;
    const XRows x = {a.h + start * ff, ff, a.h_plane, false, 0};
    const floatx4 acc = few_product<b, __bf16, P, kSplit>(a.w, (int64_t)e.expert * d + rt, std::min(kTileRows, d - rt), x, count,
                                                          wave & ((1 << lg) - 1), lg, reinterpret_cast<uint16_t *>(smem));
    float *sums = reinterpret_cast<float *>(smem);
    few_share(sums, wave, acc, count);
    for (int n = threadIdx.x; n < count * kTileRows << lt; n += kFewThreads) {
        const int m = n >> (4 + lt), c = n & ((kTileRows << lt) - 1);
        if (r0 + c < d) a.part[(int64_t)(start + m) * d + r0 + c] = few_sum(sums, (c >> 4) << lg, lg, count, m, c & 15);
    }
}

__global__ __launch_bounds__(256) void combine_kernel(const float *__restrict__ part, const Lists *__restrict__ lists, int d,
                                                      void *y, int64_t ldy, gptq_dtype y_dt) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    const Token &t = lists->token[blockIdx.y];
    if (c >= d) return;
    const int n = t.count;
    float v[kMoeMaxTopK], y0 = 0.0f;
#pragma unroll
    for (int j = 0; j < kMoeMaxTopK; ++j)
        if (j < n) v[j] = part[(int64_t)t.pair[j] * d + c];
#pragma unroll
    for (int j = 0; j < kMoeMaxTopK; ++j)
        if (j < n) y0 = fmaf(t.weight[j], v[j], y0);
    store_as(y, blockIdx.y * ldy + c, y_dt, y0);
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
    g.lg = few_slices((int64_t)(2 * busy * gu_tiles), g.w[0].units, kFewWaves / 2);
    const dim3 grid((unsigned)ceil_div(gu_tiles, (kFewWaves >> g.lg) / 2), slots);
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
    w.lg = few_slices((int64_t)(busy * tiles), w.w.units, kFewWaves);
    const dim3 dgrid((unsigned)ceil_div(tiles, kFewWaves >> w.lg), slots);
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
    choose_kernel<<<1, 1024, 0, s>>>(logits, (int)c.T, c.n_experts, c.top_k, c.renormalize,
                                     (int)std::min<int64_t>(c.n_experts, c.T * c.top_k), c.ids, c.weights,
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
