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
// h = silu(gate) * up passes between the products in fp32.  The second one, whose
// weights q - z are exact in fp16, takes it as two fp16 values of 11 bits and a
// sign each, after a power of two per row has brought the row's largest to 2^14 ..
// 2^15: a value loses at most 2^-24 of itself, or 2^-39 of its row's largest.  (A
// sum of two bf16 values, 2^-17, was the same in error against 64 bits for 16-bit
// results, but twice as many of them fell to the other side of their rounding.)
#include <algorithm>
#include <cmath>

#include "expert_load.h"
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
    // of a pair's h: the largest magnitude, as fp32 bits; a line each, as the atomics on one line wait for each other (32
    // pairs of 14336 values side by side: 142 us instead of 115)
    uint32_t top[kMaxPairs][32];
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

// Bound by latency (two reads, then the reduction): 3.6 us for one token, 4.7 for
// 16 tokens of 128 experts x 2048.  Four tokens share a row of R in registers;
// fp64 multiply-adds run at half the fp32 rate and are not what it waits for.
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

// A logit's rank as an unsigned key, ascending with the logit; a NaN lies below
// every number, and above "no candidate", which is 0.
__device__ __forceinline__ uint64_t rank_key(double v) {
    const uint64_t k = __builtin_bit_cast(uint64_t, v + 0.0);  // -0 is 0
    return v != v ? 1 : (k >> 63 ? ~k : k | (1ull << 63));
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

template <int ctrl, int rows>
__device__ __forceinline__ double dpp_add(double v) {
    const uint64_t k = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)k, ctrl, rows, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(k >> 32), ctrl, rows, 0xf, false);
    return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum_d(double v) {  // as wave_max
    v = dpp_add<0x111, 0xf>(v);
    v = dpp_add<0x112, 0xf>(v);
    v = dpp_add<0x114, 0xf>(v);
    v = dpp_add<0x118, 0xf>(v);
    v = dpp_add<0x142, 0xa>(v);
    v = dpp_add<0x143, 0xc>(v);
    const uint64_t k = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(k >> 32), 63) << 32 |
                                          (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)k, 63));
}

// kPer: logits of a lane, n_experts <= 64 kPer.  One workgroup, since the numbering
// needs every token's choice: 4.1 us for one token's 6 of 64, 8.2 for 16 tokens' 8
// of 128 (its rounds of maxima are dependent, 18 steps each).
template <int kPer>
__global__ __launch_bounds__(1024) void choose_kernel(const double *__restrict__ logits, int n_tok, int n_experts,
                                                      int top_k, int renormalize, int slots, int32_t *ids, float *weights,
                                                      Lists *lists) {
    __shared__ float weight_in[kMoeMaxTokens][kMoeMaxExperts];  // of a token's chosen experts
    __shared__ uint32_t tokens_of[kMoeMaxExperts];  // bit t: token t chose the expert
    __shared__ uint32_t wave_sum[kMoeMaxExperts / kWave];
    __shared__ uint8_t token_of[kMaxPairs];
    __shared__ float weight_of[kMaxPairs];
    const int tid = threadIdx.x, wave = few_wave(), lane = tid % kWave;
    if (tid < kMoeMaxExperts) tokens_of[tid] = 0;
    if (tid < kMaxPairs) lists->top[tid][0] = 0;
    int e = -1;  // lane j < top_k: the token's j-th choice
    bool chosen = false;
    if (wave < n_tok) {
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
                v[i] = c < n_experts ? logits[(int64_t)wave * n_experts + c] : -INFINITY;
                key[i] = c < n_experts ? rank_key(v[i]) : 0;
            }
            for (int j = 0; j < top_k; ++j) {
                uint64_t best = key[0];
#pragma unroll
                for (int i = 1; i < kPer; ++i) best = key[i] > best ? key[i] : best;
                best = wave_max(best);
                int first = 0;  // the lowest index that holds it: registers go before lanes
#pragma unroll
                for (int i = kPer - 1; i >= 0; --i) {
                    const uint64_t at = __ballot(key[i] == best);
                    if (at) first = kWave * i + __builtin_ctzll(at);
                }
                if (lane == j) e = first;
#pragma unroll
                for (int i = 0; i < kPer; ++i) key[i] = lane + kWave * i == first ? 0 : key[i];
            }
            // softmax in fp64, each weight rounded once: the first choice holds the largest logit
            uint64_t any_nan = 0;
            double mine = 0.0;  // lane j < top_k: its chosen logit
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const double c = __shfl(v[i], e & 63);
                if (e >> 6 == i) mine = c;
                any_nan |= __ballot(v[i] != v[i]);
            }
            const double top = __shfl(mine, 0), p = lane < top_k ? exp(mine - top) : 0.0;
            double sum = p;
            if (!renormalize) {
                sum = 0.0;
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (lane + kWave * i < n_experts) sum += exp(v[i] - top);
            }
            w = (float)(p / wave_sum_d(sum));
            if (any_nan) w = NAN;  // as the softmax's sum is
        }
        float total_w = 0.0f;  // a caller may name an expert twice
        for (int j = 0; j < top_k; ++j) {
            const int ej = __builtin_amdgcn_readlane(e, j);
            const float wj = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), j));
            total_w += ej == e ? wj : 0.0f;
        }
        chosen = lane < top_k && (unsigned)e < (unsigned)n_experts;
        if (chosen) weight_in[wave][e] = total_w;
        if (logits && lane < top_k) {
            if (ids) ids[wave * top_k + lane] = e;
            if (weights) weights[wave * top_k + lane] = w;
        }
    }
    __syncthreads();
    if (chosen) atomicOr(&tokens_of[e], 1u << wave);
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
            x.token[n] = t;
            token_of[p] = (uint8_t)t;
            weight_of[p] = weight_in[t][tid];
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

// Prepared x of an expert's pairs starts at its first pair's row: value
// start * (whole quads of columns).  One workgroup row per expert.
template <int b>
__global__ __launch_bounds__(256) void prepare_pairs_kernel(const uint16_t *__restrict__ X, int64_t ldx, int d,
                                                            const Lists *__restrict__ lists, const int32_t *__restrict__ kperm,
                                                            uint16_t *__restrict__ out) {
    const Expert &e = lists->expert[blockIdx.y];
    const int k = blockIdx.x * 256 + threadIdx.x, n = e.count;
    if (n == 0) return;
    int c = k < d ? kperm[(int64_t)e.expert * d + k] : 0;
    c = c < 0 ? 0 : (c >= d ? d - 1 : c);
    out += prepared_values(e.start, d / kUnit);
    for (int m = 0; m < n; ++m) out[prepared_at<b>(k, n, m)] = k < d ? X[e.token[m] * ldx + c] : 0;
}

// h with its columns in the packed order of the down product.
__global__ __launch_bounds__(256) void permute_pairs_kernel(const float *__restrict__ h, int ff, const Lists *__restrict__ lists,
                                                            const int32_t *__restrict__ kperm, float *__restrict__ out) {
    const Expert &e = lists->expert[blockIdx.y];
    const int k = blockIdx.x * 256 + threadIdx.x, n = e.count;
    if (n == 0 || k >= ff) return;
    int c = kperm[(int64_t)e.expert * ff + k];
    c = c < 0 ? 0 : (c >= ff ? ff - 1 : c);
    for (int m = 0; m < n; ++m) out[(int64_t)(e.start + m) * ff + k] = h[(int64_t)(e.start + m) * ff + c];
}

struct GateUpArgs {
    FewMat w[2];
    FewShape shape;
    const uint16_t *x;  // rows by token, or prepared by pair
    int64_t ldx;
    const int32_t *order;  // ordered: of every expert
    Lists *lists;
    float *h;  // rows by pair
};

// Cold weights: 14 us for 6 experts of 1408 x 2048 in 4 bits (19 MB), 38 us for the
// ~82 that 16 tokens choose of 128 x 768 x 2048 (146 MB, 3.8 TB/s), 87 us for ~5.5 of
// 14336 x 4096 (361 MB, 4.1 TB/s): a workgroup's start and staging per 128 rows or
// fewer, then the bytes.
template <int b, typename T, bool kSplit, FewX kX>
__global__ __launch_bounds__(kFewThreads, kFewOccupancy) void gate_up_kernel(GateUpArgs a) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const Expert &e = a.lists->expert[blockIdx.y];
    const int token = e.token[threadIdx.x & (kMoeMaxTokens - 1)];
    const int start = e.start, count = e.count, wave = few_wave(), lg = a.shape.lg;
    if (count == 0) return;
    const int lt = 2 - lg;  // log2 of the row tiles
    const int ff = a.shape.d_out, r0 = blockIdx.x * kTileRows << lt;
    const int64_t row = (int64_t)e.expert * ff + r0;
    constexpr bool rows = kX != kPreparedX;
    const XRows x = {rows ? a.x : a.x + prepared_values(start, a.shape.units), a.ldx, rows, token,
                     kX == kOrderedX ? a.order + (int64_t)e.expert * a.shape.units * kUnit : nullptr, 0.0f};
    const floatx4 acc = few_product<b, T, 2, kSplit, kX>(a.w, a.shape, row, ff - r0, x, count, wave, smem);
    float *sums = reinterpret_cast<float *>(smem);
    few_share(sums, wave, acc, count);
    for (int n = threadIdx.x; n < count * kTileRows << lt; n += kFewThreads) {
        const int m = n >> (4 + lt), c = n & ((kTileRows << lt) - 1);  // (m is one in 16 << lt <= 64 lanes)
        const int w0 = (c >> 4) << (1 + lg);
        const float v = silu_mul(few_sum(sums, w0, lg, count, m, c & 15), few_sum(sums, w0 + (1 << lg), lg, count, m, c & 15));
        uint32_t most = 0;
        if (r0 + c < ff) {
            a.h[(int64_t)(start + m) * ff + r0 + c] = v;
            most = __float_as_uint(v) & 0x7FFFFFFFu;
        }
        for (int o = 8 << lt; o > 0; o >>= 1) most = std::max(most, (uint32_t)__shfl_xor((int)most, o));
        if (c == 0) atomicMax(a.lists->top[start + m], most);  // a maximum, whatever the order
    }
}

struct DownArgs {
    FewMat w;
    FewShape shape;
    const float *h;  // rows by pair
    const Lists *lists;
    float *part;  // rows by pair
};

// The exponent that brings a row's largest magnitude (fp32 bits) to 2^14 .. 2^15,
// or a smaller row up by as much as fp32 has.
__device__ __forceinline__ int row_exponent(uint32_t top) { return std::min(126, 127 + 14 - (int)(top >> 23)); }
__device__ __forceinline__ float power_of_2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// Two matrix instructions per fragment of weights, which are unpacked once for both
// planes of h.  8 us, 26 us and 62 us for the experts of gate_up_kernel's figures:
// half their bytes in 57-70% of the time, for h has two planes and K is d_ff.  Adding
// a token's pairs here, by the last workgroup to arrive, took 35 us instead of 8 and
// 200 instead of 28: the fence before its count.
template <int b, bool kSplit>
__global__ __launch_bounds__(kFewThreads, kFewOccupancy) void down_kernel(DownArgs a) {
    extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
    const Expert &e = a.lists->expert[blockIdx.y];
    const int start = e.start, count = e.count, wave = few_wave(), lg = a.shape.lg;
    if (count == 0) return;
    const int lt = 3 - lg;
    const int d = a.shape.d_out, ff = a.shape.units * kUnit, r0 = blockIdx.x * kTileRows << lt;
    const int64_t row = (int64_t)e.expert * d + r0;
    const float scale = power_of_2(row_exponent(a.lists->top[start + std::min((int)(threadIdx.x & (kMoeMaxTokens - 1)), count - 1)][0]));
    const XRows x = {a.h + (int64_t)start * ff, ff, false, 0, nullptr, scale};
    const floatx4 acc = few_product<b, _Float16, 1, kSplit, kFloatX>(&a.w, a.shape, row, d - r0, x, count, wave, smem);
    float *sums = reinterpret_cast<float *>(smem);
    few_share(sums, wave, acc, count);
    for (int n = threadIdx.x; n < count * kTileRows << lt; n += kFewThreads) {
        const int m = n >> (4 + lt), c = n & ((kTileRows << lt) - 1);
        const float back = power_of_2(-row_exponent(a.lists->top[start + m][0]));
        if (r0 + c < d) a.part[(int64_t)(start + m) * d + r0 + c] = few_sum(sums, (c >> 4) << lg, lg, count, m, c & 15) * back;
    }
}

// A thread per value of Y; all its loads before the sum.  3-5 us, a launch and two
// dependent reads.
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

struct Layout {
    size_t logits, lists, h, part, xg, hg, bytes;
};
Layout layout(int64_t T, int64_t d, int64_t d_ff, int n_experts, int top_k) {
    const size_t pairs = (size_t)T * top_k, hb = align_up(pairs * d_ff * 4, 256);
    Layout l;
    l.logits = 0;
    l.lists = align_up((size_t)T * n_experts * sizeof(double), 256);
    l.h = l.lists + align_up(sizeof(Lists), 256);
    l.part = l.h + hb;
    l.xg = l.part + align_up(pairs * d * 4, 256);
    l.hg = l.xg + align_up((size_t)prepared_values((int64_t)pairs, (int)(d / kUnit)) * 2, 256);
    l.bytes = l.hg + hb;
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

template <int b, typename T, bool kSplit>
void launch_gate_up(const GateUpArgs &g, FewX x, dim3 grid, hipStream_t s) {
    auto kernel = x == kRawX ? gate_up_kernel<b, T, kSplit, kRawX>
                             : (x == kOrderedX ? gate_up_kernel<b, T, kSplit, kOrderedX> : gate_up_kernel<b, T, kSplit, kPreparedX>);
    kernel<<<grid, kFewThreads, g.shape.lds, s>>>(g);
}
template <int b, typename T>
void launch_experts(const MoeCall &c, const Layout &l, hipStream_t s) {
    const int64_t d = c.gate->d_in, ff = c.gate->d_out, pairs = c.T * c.top_k;
    Lists *lists = reinterpret_cast<Lists *>(c.ws + l.lists);
    const unsigned slots = (unsigned)std::min<int64_t>(c.n_experts, pairs);
    const ExpertLoad load = expert_load(c.T, c.n_experts, c.top_k);
    GateUpArgs g;
    const int64_t pair_tiles = ceil_div(ff, kTileRows);
    g.w[0] = few_mat(*c.gate);
    g.w[1] = few_mat(*c.up);
    g.shape = few_shape(*c.gate, 2 * load.experts * pair_tiles, kFewWaves / 2, load.rows, (int)c.T);
    g.x = static_cast<const uint16_t *>(c.X);
    g.ldx = c.ldx;
    g.lists = lists;
    g.h = reinterpret_cast<float *>(c.ws + l.h);
    // gathered by the products up to the same size as in gemv.hip, with an expert's rows for M: one token of 64 experts x
    // 1408 x 2048 takes 30.4 us against 31.7 through a kernel of its own, of 1408 x 4096 39.4 against 39.8
    g.order = c.gate->kperm;
    const FewX x = !c.gate->kperm ? kRawX : (gemv_prepares(load.rows, d) ? kPreparedX : kOrderedX);
    if (x == kPreparedX) {
        uint16_t *xg = reinterpret_cast<uint16_t *>(c.ws + l.xg);
        prepare_pairs_kernel<b><<<dim3((unsigned)(few_quads(g.shape.units) * kQuad / 256), slots), 256, 0, s>>>(g.x, c.ldx, (int)d, lists,
                                                                                                               c.gate->kperm, xg);
        g.x = xg;
    }
    const dim3 grid((unsigned)ceil_div(pair_tiles, (kFewWaves >> g.shape.lg) / 2), slots);
    if (few_split(*c.gate))
        launch_gate_up<b, T, true>(g, x, grid, s);
    else
        launch_gate_up<b, T, false>(g, x, grid, s);
    DownArgs w;
    const int64_t tiles = ceil_div(d, kTileRows);
    w.w = few_mat(*c.down);
    w.shape = few_shape(*c.down, load.experts * tiles, kFewWaves, 2 * load.rows, 2 * (int)c.T);
    w.h = g.h;
    w.lists = lists;
    w.part = reinterpret_cast<float *>(c.ws + l.part);
    if (c.down->kperm) {
        float *hg = reinterpret_cast<float *>(c.ws + l.hg);
        permute_pairs_kernel<<<dim3((unsigned)ceil_div(ff, 256), slots), 256, 0, s>>>(g.h, (int)ff, lists, c.down->kperm, hg);
        w.h = hg;
    }
    auto down = few_split(*c.down) ? down_kernel<b, true> : down_kernel<b, false>;
    down<<<dim3((unsigned)ceil_div(tiles, kFewWaves >> w.shape.lg), slots), kFewThreads, w.shape.lds, s>>>(w);
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
    auto choose = c.n_experts <= 64 ? choose_kernel<1> : (c.n_experts <= 128 ? choose_kernel<2> : (c.n_experts <= 256 ? choose_kernel<4> : choose_kernel<8>));
    choose<<<1, 1024, 0, s>>>(logits, (int)c.T, c.n_experts, c.top_k, c.renormalize, (int)std::min<int64_t>(c.n_experts, c.T * c.top_k),
                              c.ids, c.weights, reinterpret_cast<Lists *>(c.ws + l.lists));
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
