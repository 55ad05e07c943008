// Attention of a few tokens over a 4-bit cache.
//
// The n G columns of a kv head (n tokens, G query heads each) are the B operand of
// v_mfma_f32_16x16x32_f16, sixteen at a time.  A wave takes tiles of 32 cached tokens:
//   S[token][column] = s_k (sum_d (q_k - 8) x + c_k X),   c = 8 - z,  X = sum_d x
// with the codes as exact fp16 integers in [-8, 7], so nothing but the fp32 sums rounds.
// The A operand's row r of half t is token 8 (r / 4) + 4 t + r % 4, so a lane ends up with
// S of eight tokens next to each other in one column, which is what the second product
//   O[dim][column] = sum_token (q_v - 8) (p s_v) + sum_token c_v (p s_v)
// wants of its B operand: p never leaves the lane.  It is held there as p s_v in fp16,
// scaled by a power of two that follows the largest s_v: a rounding of 2^-11 of each
// term at most, as that of an fp16 result, where bf16 would lose eight times that.
// Values s_v more than 2^29 below the largest lose bits, those more than 2^40 below it vanish.
//
// bf16 queries enter as fp16 times a power of two of their row, which takes no bit from
// a value above 2^-30 of the row's largest.
//
// One pass with a running maximum: the sums are rescaled only when a score passes the
// maximum they are held to by 2^6 (p may then be up to 64, which fp16 and fp32 hold).
#include <algorithm>

#include "kv_cache.h"

namespace gptq {
namespace {

constexpr int kKvTile = 32;   // tokens of a tile
constexpr int kKvWaves = 4;   // waves of a workgroup, each with tiles of its own
constexpr int kKvThreads = kKvWaves * kWave;
constexpr int kKvLeast = 8;   // tiles of a workgroup at least
constexpr float kSlack = 6.0f;
constexpr float kNegInf = -__builtin_inff();

struct AttnArgs {
    KvPool pool;
    KvSeqs seqs;
    const uint16_t *q;
    int64_t ldq;
    uint16_t *o;
    int64_t ldo;
    float *part;   // [item][head][column][D], unnormalized, relative to the item's maximum
    float2 *stat;  // [item][head][column]: maximum (of log2) and sum
    float scale;   // times log2 e
    float decay;
    int32_t n, group, cols;  // new tokens, query heads of a kv head, n * group
    int32_t target;  // items wanted over all sequences
    int32_t bf16, direct, keep_stat;
};

__device__ __forceinline__ float xor_max(float v, int o) { return fmaxf(v, __shfl_xor(v, o)); }
__device__ __forceinline__ float xor_add(float v, int o) { return v + __shfl_xor(v, o); }

// How the cached tokens are shared out: items of `chunk` tiles, sequence after sequence.
struct Share {
    int b, first, tiles, chunk;  // the item's sequence, its first tile and how many; tiles of a whole item
    int base, splits, len;       // the sequence's first item, and how many it has
};
__device__ __forceinline__ int tiles_of(const KvSeqs &s, int b) { return b < s.n ? (s.len(b) + kKvTile - 1) / kKvTile : 0; }
__device__ __forceinline__ int chunk_of(const AttnArgs &a) {
    const int lane = threadIdx.x & 63;
    int total = 0;
    for (int b0 = 0; b0 < a.seqs.n; b0 += kWave) total += tiles_of(a.seqs, b0 + lane);
    for (int o = 1; o < kWave; o *= 2) total += __shfl_xor(total, o);
    const int c = (total + a.target - 1) / a.target;
    return max(kKvLeast, (c + kKvWaves - 1) / kKvWaves * kKvWaves);
}
// The share of item x (b < 0: there is none), or with `seq` the items of sequence x.
__device__ __forceinline__ Share share_of(const AttnArgs &a, int x, bool seq) {
    const int lane = threadIdx.x & 63;
    Share s;
    s.b = -1;
    s.chunk = chunk_of(a);
    int base = 0;
    for (int b0 = 0; b0 < a.seqs.n; b0 += kWave) {
        const int tiles = tiles_of(a.seqs, b0 + lane), mine = (tiles + s.chunk - 1) / s.chunk;
        int sum = mine;
        for (int o = 1; o < kWave; o *= 2) {
            const int v = __shfl_up(sum, o);
            if (lane >= o) sum += v;
        }
        const int from = base + sum - mine;
        const uint64_t hit = __ballot(seq ? b0 + lane == x : from <= x && x < from + mine);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            s.b = b0 + l;
            s.base = __shfl(from, l);
            s.splits = __shfl(mine, l);
            s.first = (x - s.base) * s.chunk;
            s.tiles = min(s.chunk, __shfl(tiles, l) - s.first);
            s.len = a.seqs.len(s.b);
            return s;
        }
        base += __shfl(sum, kWave - 1);
    }
    return s;
}

// The share of this workgroup.
__device__ __forceinline__ Share my_share(const AttnArgs &a) {
    if (!a.direct) return share_of(a, blockIdx.x, false);
    const int b = blockIdx.x, tiles = tiles_of(a.seqs, b);
    return {b, 0, tiles, tiles, b, 1, a.seqs.len(b)};
}

template <int D64, int NG>
struct Tile {  // a lane's part of 32 cached tokens
    static constexpr int D = 64 * D64, KW = D / 32;
    uint32_t k[2][KW];
    u32x4 v[D64];
    u32x4 kg[NG][2], vg[NG][2];
    bool there;  // the page of this lane's eight tokens exists

    __device__ __forceinline__ void load(const KvPool &pool, const KvSeqs &seqs, const int32_t *row, int tile, int last_block, int h) {
        const int lane = threadIdx.x & 63, r = lane & 15, kb = lane >> 4, mask = pool.page() - 1;
        const int bk = min(4 * tile + (r >> 2), last_block), bv = min(4 * tile + kb, last_block);  // blocks of eight tokens
        const int pk = seqs.page_of(pool, row, 8 * bk), pv = seqs.page_of(pool, row, 8 * bv);
        there = pv >= 0;
        const int64_t fk = pool.first(max(pk, 0), h), fv = pool.first(max(pv, 0), h);
        const int ak = (8 * bk) & mask, av = (8 * bv) & mask;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t *p = pool.k + (fk + ak + 4 * t + (r & 3)) * (D / 8) + kb * KW;
            if constexpr (KW % 4 == 0) {
#pragma unroll
                for (int i = 0; i < KW; i += 4) {
                    const u32x4 w = *reinterpret_cast<const u32x4 *>(p + i);
                    k[t][i] = w[0], k[t][i + 1] = w[1], k[t][i + 2] = w[2], k[t][i + 3] = w[3];
                }
            } else {
#pragma unroll
                for (int i = 0; i < KW; i += 2) {
                    const u32x2 w = *reinterpret_cast<const u32x2 *>(p + i);
                    k[t][i] = w[0], k[t][i + 1] = w[1];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < D64; ++u)
            v[u] = *reinterpret_cast<const u32x4 *>(pool.v + (fv + av) * (D / 4) + (16 * u + r) * 8);
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int64_t at = fv * NG + (int64_t)g * (mask + 1) + av + 4 * t;
                kg[g][t] = *reinterpret_cast<const u32x4 *>(pool.k_grid + at);
                vg[g][t] = *reinterpret_cast<const u32x4 *>(pool.v_grid + at);
            }
    }
};

// Codes as fp16 q - 8: masked in place they make 1024 + q or, four bits up, 64 + q.
struct Unpack {
    uint32_t m0 = 0x64006400u, m1 = 0x54005400u;
    __device__ __forceinline__ Unpack() { asm volatile("" : "+v"(m0), "+v"(m1)); }  // registers: VOP3 takes no literal
    __device__ __forceinline__ uint32_t low(uint32_t w) const {
        const f16x2 h = __builtin_bit_cast(f16x2, (w & 0x000F000Fu) | m0) - (f16x2){(_Float16)1032.0f, (_Float16)1032.0f};
        return __builtin_bit_cast(uint32_t, h);
    }
    __device__ __forceinline__ uint32_t high(uint32_t w) const {
        const f16x2 h = __builtin_bit_cast(f16x2, (w & 0x00F000F0u) | m1) - (f16x2){(_Float16)72.0f, (_Float16)72.0f};
        return __builtin_bit_cast(uint32_t, h);
    }
    __device__ __forceinline__ f16x8 keys(uint32_t w) const {
        const u32x4 f = {low(w), high(w), low(w >> 8), high(w >> 8)};
        return __builtin_bit_cast(f16x8, f);
    }
    // Dim j of the four of each unit: eight tokens.
    __device__ __forceinline__ f16x8 values(const u32x4 &w, int j) const {
        u32x4 f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = j < 2 ? w[i] : w[i] >> 8;
            f[i] = j & 1 ? high(x) : low(x);
        }
        return __builtin_bit_cast(f16x8, f);
    }
};

__device__ __forceinline__ floatx4 mma(f16x8 a, f16x8 b, floatx4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

// Sixteen columns of queries as B operands, with their sums per group.
template <int D64, int NG>
struct Queries {
    static constexpr int KW = 2 * D64;
    f16x8 x[KW];
    float sum[NG];  // of the group's x: what c_k multiplies
    float scale;    // of S, to log2
    int sees;       // slots below this are visible

    __device__ __forceinline__ void load(const AttnArgs &a, int b, int h, int len, int col) {
        const int lane = threadIdx.x & 63, kb = lane >> 4;
        const bool real = col < a.cols;
        const int i = real ? col / a.group : 0, hq = h * a.group + (real ? col - i * a.group : 0);
        sees = real ? len - a.n + 1 + i : 0;
        const uint16_t *q = a.q + ((int64_t)b * a.n + i) * a.ldq + (int64_t)hq * (64 * D64) + 8 * kb;
        u32x4 w[KW];
        float top = 0.0f;
#pragma unroll
        for (int t = 0; t < KW; ++t) {
            w[t] = real ? *reinterpret_cast<const u32x4 *>(q + 32 * t) : (u32x4){};
            if (a.bf16) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[t][e] << 16)), fabsf(__uint_as_float(w[t][e] & 0xFFFF0000u))));
            }
        }
        scale = a.scale;
        if (a.bf16) {
            // times 2^(15 - e), top < 2^e: fp16's largest binade
            top = xor_max(xor_max(top, 16), 32);
            int e = 0;
            if (top > 0.0f && top < __builtin_inff()) frexpf(top, &e);
            const int up = 15 - e;
#pragma unroll
            for (int t = 0; t < KW; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x2 f = {ldexpf(__uint_as_float(w[t][j] << 16), up), ldexpf(__uint_as_float(w[t][j] & 0xFFFF0000u), up)};
                    w[t][j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, f16x2));
                }
            scale = ldexpf(scale, -up);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            float s = 0.0f;
#pragma unroll
            for (int t = g * KW / NG; t < (g + 1) * KW / NG; ++t) {
                x[t] = __builtin_bit_cast(f16x8, w[t]);
#pragma unroll
                for (int e = 0; e < 8; ++e) s += (float)x[t][e];
            }
            sum[g] = xor_add(xor_add(s, 16), 32);
        }
    }
};

__device__ __forceinline__ bool hidden(bool there, int slot, int sees) { return !there || slot >= sees; }

// Scores of the lane's eight tokens in its column, in log2; -inf where hidden.
template <int D64, int NG>
__device__ __forceinline__ void scores(float s[8], const Tile<D64, NG> &tile, const f16x8 kf[2][2 * D64], const Queries<D64, NG> &q,
                                       int slot, bool masked) {
    constexpr int KW = 2 * D64;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        float y[4] = {};
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            floatx4 acc = {};
#pragma unroll
            for (int w = g * KW / NG; w < (g + 1) * KW / NG; ++w) acc = mma(kf[t][w], q.x[w], acc);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t grid = tile.kg[g][t][i];
                const float v = fmaf(grid_zero_of(grid), q.sum[g], acc[i]), k = grid_scale_of(grid) * q.scale;
                y[i] = g == 0 ? k * v : fmaf(k, v, y[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[4 * t + i] = y[i];
    }
    if (masked) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (hidden(tile.there, slot + i, q.sees)) s[i] = kNegInf;
    }
}

template <int D64, int NG, int NT>
__global__ __launch_bounds__(kKvThreads) void attention_kernel(AttnArgs a) {
    constexpr int D = 64 * D64, KW = 2 * D64;
    extern __shared__ __attribute__((aligned(16))) float smem[];  // [wave][column][D] of one column tile, then (m, l)
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, kb = lane >> 4;
    const int h = blockIdx.y, col0 = blockIdx.z * (16 * NT);
    const Share sh = my_share(a);
    if (sh.b < 0) return;
    const int32_t *row = a.seqs.table + (int64_t)sh.b * a.seqs.width;
    const int last_block = (sh.len + 7) / 8 - 1;
    Queries<D64, NG> q[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) q[c].load(a, sh.b, h, sh.len, col0 + 16 * c + r);

    floatx4 acc[NT][D / 16] = {};
    float corr[NT][NG] = {}, sum[NT] = {}, top[NT];
    for (int c = 0; c < NT; ++c) top[c] = kNegInf;
    float vmax = 0.0f, vscale = 1.0f;  // a power of two above every s_v / 4, and 2^6 over it
    const Unpack un;
    const int clear = sh.len - a.n + 1;  // slots below this are visible to every column

    for (int tile = sh.first + wave; tile < sh.first + sh.tiles; tile += kKvWaves) {
        Tile<D64, NG> t;
        t.load(a.pool, a.seqs, row, tile, last_block, h);
        const int slot = tile * kKvTile + 8 * kb;
        const bool masked = (tile + 1) * kKvTile > clear || __any(!t.there);
        f16x8 kf[2][KW];
#pragma unroll
        for (int i = 0; i < KW; ++i) kf[0][i] = un.keys(t.k[0][i]), kf[1][i] = un.keys(t.k[1][i]);
        float p[NT][8];
        bool high = false;
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            scores<D64, NG>(p[c], t, kf, q[c], slot, masked);
            float m = p[c][0];
#pragma unroll
            for (int i = 1; i < 8; ++i) m = fmaxf(m, p[c][i]);
            high |= m > top[c] + kSlack;
        }
        float sv[NG][8], most = 0.0f;
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sv[g][i] = grid_scale_of(t.vg[g][i / 4][i % 4]);
                if (masked && hidden(t.there, slot + i, sh.len)) sv[g][i] = 0.0f;
                most = fmaxf(most, sv[g][i]);
            }
        if (__any(high || most > 4.0f * vmax)) {
            const float m4 = xor_max(xor_max(most, 16), 32);
            float down = 1.0f;
            if (m4 > vmax) {
                const float was = vscale;
                int e;
                frexpf(m4, &e);
                e = max(e, -118);  // 2^(6 - e) stays finite
                vmax = ldexpf(1.0f, e);
                vscale = ldexpf(1.0f, 6 - e);
                down = vscale / was;
            }
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                float m = p[c][0];
#pragma unroll
                for (int i = 1; i < 8; ++i) m = fmaxf(m, p[c][i]);
                m = fmaxf(top[c], xor_max(xor_max(m, 16), 32));
                const float f = top[c] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(top[c] - m);
                top[c] = m;
                sum[c] *= f;
#pragma unroll
                for (int g = 0; g < NG; ++g) corr[c][g] *= f * down;
#pragma unroll
                for (int d = 0; d < D / 16; ++d) acc[c][d] *= f * down;
            }
        }
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            const float base = top[c] == kNegInf ? 0.0f : top[c];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[c][i] = __builtin_amdgcn_exp2f(p[c][i] - base);
                sum[c] += p[c][i];
            }
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            f16x8 pf[NT];
#pragma unroll
            for (int i = 0; i < 8; ++i) sv[g][i] *= vscale;
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                float ps[8], z[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) ps[i] = p[c][i] * sv[g][i], z[i] = grid_zero_of(t.vg[g][i / 4][i % 4]);
                if (masked) {  // a hidden token's grid may hold anything
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (hidden(t.there, slot + i, q[c].sees)) ps[i] = z[i] = 0.0f;
                }
                u32x4 w;
#pragma unroll
                for (int i = 0; i < 8; i += 2)
                    w[i / 2] = __builtin_bit_cast(uint32_t, __builtin_convertvector(((f32x2){ps[i], ps[i + 1]}), f16x2));
                pf[c] = __builtin_bit_cast(f16x8, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) corr[c][g] = fmaf((float)pf[c][i], z[i], corr[c][g]);
            }
#pragma unroll
            for (int d = g * (D / 16) / NG; d < (g + 1) * (D / 16) / NG; ++d) {
                const f16x8 vf = un.values(t.v[d / 4], d % 4);
#pragma unroll
                for (int c = 0; c < NT; ++c) acc[c][d] = mma(vf, pf[c], acc[c][d]);
            }
        }
    }

    // The waves' sums, brought to the largest of their maxima and added in wave order.
    float2 *ml = reinterpret_cast<float2 *>(smem + kKvWaves * 16 * D);
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        const float l = xor_add(xor_add(sum[c], 16), 32);
        if (c) __syncthreads();
        if (kb == 0) ml[wave * 16 + r] = make_float2(top[c], l);
        __syncthreads();
        float m = kNegInf;
        for (int w = 0; w < kKvWaves; ++w) m = fmaxf(m, ml[w * 16 + r].x);
        const float f = (top[c] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(top[c] - m)) / vscale;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const float k = xor_add(xor_add(corr[c][g], 16), 32);
#pragma unroll
            for (int d = g * (D / 16) / NG; d < (g + 1) * (D / 16) / NG; ++d) {
                const floatx4 y = (acc[c][d] + k) * f;
                *reinterpret_cast<floatx4 *>(smem + (wave * 16 + r) * D + 16 * d + 4 * kb) = y;
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * D; i += kKvThreads) {
            const int cc = i / D, d = i % D, col = col0 + 16 * c + cc;
            if (col >= a.cols) break;
            float M = kNegInf, L = 0.0f, o = 0.0f;
            for (int w = 0; w < kKvWaves; ++w) M = fmaxf(M, ml[w * 16 + cc].x);
            for (int w = 0; w < kKvWaves; ++w) {
                const float2 v = ml[w * 16 + cc];
                L += v.x == kNegInf ? v.y : v.y * __builtin_amdgcn_exp2f(v.x - M);
                o += smem[(w * 16 + cc) * D + d];
            }
            const int64_t at = ((int64_t)blockIdx.x * gridDim.y + h) * a.cols + col;
            if (sh.splits == 1) {
                const float y = L == 0.0f ? 0.0f : o / L;
                const int tok = col / a.group;
                uint16_t *to = a.o + ((int64_t)sh.b * a.n + tok) * a.ldo + (int64_t)(h * a.group + col - tok * a.group) * D + d;
                *to = a.bf16 ? __builtin_bit_cast(uint16_t, (__bf16)y) : __builtin_bit_cast(uint16_t, (_Float16)y);
            } else {
                a.part[at * D + d] = o;
            }
            if (d == 0 && a.keep_stat) a.stat[at] = make_float2(M, L);
        }
    }
}

// The maximum and sum of a column over its sequence's items, by the 64 lanes of a wave.
__device__ __forceinline__ float2 joined_stat(const AttnArgs &a, const Share &sh, int h, int col) {
    const int lane = threadIdx.x & 63;
    float m = kNegInf, l = 0.0f;
    for (int x = lane; x < sh.splits; x += kWave) m = fmaxf(m, a.stat[((int64_t)(sh.base + x) * a.pool.heads + h) * a.cols + col].x);
    for (int o = 1; o < kWave; o *= 2) m = xor_max(m, o);
    for (int x = lane; x < sh.splits; x += kWave) {
        const float2 v = a.stat[((int64_t)(sh.base + x) * a.pool.heads + h) * a.cols + col];
        l += v.x == kNegInf ? v.y : v.y * __builtin_amdgcn_exp2f(v.x - m);
    }
    for (int o = 1; o < kWave; o *= 2) l = xor_add(l, o);
    return make_float2(m, l);
}

// Sequences of more than one item, or none: a wave per column.
template <int D64>
__global__ __launch_bounds__(kKvThreads) void combine_kernel(AttnArgs a) {
    constexpr int D = 64 * D64;
    const int lane = threadIdx.x & 63, h = blockIdx.y, b = blockIdx.x;
    const int col = blockIdx.z * kKvWaves + (threadIdx.x >> 6);
    const Share sh = share_of(a, b, true);
    if (sh.splits == 1 || col >= a.cols) return;
    const float2 ml = joined_stat(a, sh, h, col);
    float o[D64] = {};
    for (int x = 0; x < sh.splits; ++x) {
        const int64_t at = ((int64_t)(sh.base + x) * a.pool.heads + h) * a.cols + col;
        const float m = a.stat[at].x;
        const float f = m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m - ml.x);
#pragma unroll
        for (int u = 0; u < D64; ++u) o[u] += f * a.part[at * D + 64 * u + lane];
    }
    const int tok = col / a.group;
    uint16_t *to = a.o + ((int64_t)b * a.n + tok) * a.ldo + (int64_t)(h * a.group + col - tok * a.group) * D;
#pragma unroll
    for (int u = 0; u < D64; ++u) {
        const float y = ml.y == 0.0f ? 0.0f : o[u] / ml.y;
        to[64 * u + lane] = a.bf16 ? __builtin_bit_cast(uint16_t, (__bf16)y) : __builtin_bit_cast(uint16_t, (_Float16)y);
    }
}

// weight[token] = decay weight[token] + the sum of p over the columns, once maxima and sums are known.  Only the
// keys are read again; the same instructions give the same scores.
template <int D64, int NG>
__global__ __launch_bounds__(kKvThreads) void weights_kernel(AttnArgs a) {
    constexpr int KW = 2 * D64;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, kb = lane >> 4, h = blockIdx.y;
    const Share sh = my_share(a);
    if (sh.b < 0) return;
    const int32_t *row = a.seqs.table + (int64_t)sh.b * a.seqs.width;
    const int last_block = (sh.len + 7) / 8 - 1, clear = sh.len - a.n + 1;
    const Unpack un;
    for (int col0 = 0; col0 < a.cols; col0 += 16) {
        Queries<D64, NG> q;
        q.load(a, sh.b, h, sh.len, col0 + r);
        float2 ml = make_float2(0.0f, 0.0f);
        for (int c = 0; c < 16 && col0 + c < a.cols; ++c) {
            const float2 v = joined_stat(a, sh, h, col0 + c);
            if (c == r) ml = v;
        }
        const float inv = ml.y == 0.0f ? 0.0f : 1.0f / ml.y, base = ml.x == kNegInf ? 0.0f : ml.x;
        for (int tile = sh.first + wave; tile < sh.first + sh.tiles; tile += kKvWaves) {
            Tile<D64, NG> t;
            t.load(a.pool, a.seqs, row, tile, last_block, h);
            const int slot = tile * kKvTile + 8 * kb;
            f16x8 kf[2][KW];
#pragma unroll
            for (int i = 0; i < KW; ++i) kf[0][i] = un.keys(t.k[0][i]), kf[1][i] = un.keys(t.k[1][i]);
            float p[8];
            scores<D64, NG>(p, t, kf, q, slot, (tile + 1) * kKvTile > clear || __any(!t.there));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[i] = col0 + r < a.cols ? __builtin_amdgcn_exp2f(p[i] - base) * inv : 0.0f;
                for (int o = 1; o < 16; o *= 2) p[i] = xor_add(p[i], o);
            }
            const int page = slot < sh.len ? a.seqs.page_of(a.pool, row, slot) : -1;
            if (r == 0 && page >= 0) {
                float *w = a.pool.weight + a.pool.first(page, h) + (slot & (a.pool.page() - 1));
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (slot + i < sh.len) w[i] = col0 ? w[i] + p[i] : (a.decay == 0.0f ? p[i] : fmaf(a.decay, w[i], p[i]));
            }
        }
    }
}

struct Plan {
    int nt, items, target;
    bool direct;
    size_t part, stat;  // bytes
};
Plan plan_of(const gptq_kv_cache &c, int64_t n_seq, int64_t cols, int64_t max_len) {
    Plan p;
    p.nt = cols > 16 && c.head_dim <= 128 ? 2 : 1;  // two tiles of larger heads do not fit the registers
    const int64_t tiles = ceil_div(max_len, kKvTile), blocks = c.n_heads * ceil_div(cols, 16 * p.nt);
    p.target = (int)std::max<int64_t>(1, 1024 / blocks);
    const int64_t most = std::max<int64_t>(1, ceil_div(tiles, kKvLeast));
    p.items = (int)std::min<int64_t>(n_seq * most, p.target + n_seq);
    p.direct = most == 1;
    const size_t rows = (size_t)p.items * c.n_heads * cols;
    p.part = p.direct ? 0 : align_up(rows * c.head_dim * 4, 256);
    p.stat = align_up(rows * 8, 256);
    return p;
}

template <int D64, int NG>
hipError_t launch_attention(const AttnArgs &a, const Plan &p, int n_seq, bool weights, hipStream_t s) {
    const size_t lds = (size_t)kKvWaves * 16 * (64 * D64 * 4 + 8);
    const dim3 grid((unsigned)p.items, (unsigned)a.pool.heads, (unsigned)ceil_div(a.cols, 16 * p.nt));
    bool two = false;
    if constexpr (D64 <= 2) two = p.nt == 2;
    if constexpr (D64 <= 2) {
        if (two) attention_kernel<D64, NG, 2><<<grid, kKvThreads, lds, s>>>(a);
    }
    if (!two) attention_kernel<D64, NG, 1><<<grid, kKvThreads, lds, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (!p.direct) {
        combine_kernel<D64><<<dim3((unsigned)n_seq, (unsigned)a.pool.heads, (unsigned)ceil_div(a.cols, kKvWaves)), kKvThreads, 0, s>>>(a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (weights) {
        weights_kernel<D64, NG><<<dim3((unsigned)p.items, (unsigned)a.pool.heads), kKvThreads, 0, s>>>(a);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace

size_t kv_attention_ws_bytes(const gptq_kv_cache &c, int64_t n_seq, int64_t n, int64_t q_heads, int64_t max_len) {
    const Plan p = plan_of(c, n_seq, n * (q_heads / c.n_heads), max_len);
    return p.part + p.stat;
}

hipError_t run_kv_attention(const void *Q, gptq_dtype dt, int64_t n_seq, int64_t n, int64_t q_heads, int64_t ldq, const gptq_kv_cache &c,
                            const int32_t *table, int64_t width, const int32_t *lens, int64_t max_len, float scale, bool weights,
                            float decay, void *O, int64_t ldo, void *ws, hipStream_t s) {
    AttnArgs a;
    a.pool = kv_pool(c);
    a.seqs = {table, lens, (int32_t)n_seq, (int32_t)width, max_len};
    a.q = static_cast<const uint16_t *>(Q);
    a.ldq = ldq;
    a.o = static_cast<uint16_t *>(O);
    a.ldo = ldo;
    a.n = (int32_t)n;
    a.group = (int32_t)(q_heads / c.n_heads);
    a.cols = a.n * a.group;
    const Plan p = plan_of(c, n_seq, a.cols, max_len);
    a.part = static_cast<float *>(ws);
    a.stat = reinterpret_cast<float2 *>(static_cast<char *>(ws) + p.part);
    a.scale = scale * 1.44269504088896340736f;
    a.decay = decay;
    a.target = p.target;
    a.bf16 = dt == GPTQ_DT_BF16;
    a.direct = p.direct;
    a.keep_stat = weights || !p.direct;
    const int ng = a.pool.groups;
    switch (c.head_dim / 64) {
    case 1: return ng == 1 ? launch_attention<1, 1>(a, p, (int)n_seq, weights, s) : launch_attention<1, 2>(a, p, (int)n_seq, weights, s);
    case 2:
        return ng == 1 ? launch_attention<2, 1>(a, p, (int)n_seq, weights, s)
                       : (ng == 2 ? launch_attention<2, 2>(a, p, (int)n_seq, weights, s) : launch_attention<2, 4>(a, p, (int)n_seq, weights, s));
    case 3:
        return ng == 1 ? launch_attention<3, 1>(a, p, (int)n_seq, weights, s)
                       : (ng == 3 ? launch_attention<3, 3>(a, p, (int)n_seq, weights, s) : launch_attention<3, 6>(a, p, (int)n_seq, weights, s));
    default:
        return ng == 1 ? launch_attention<4, 1>(a, p, (int)n_seq, weights, s)
                       : (ng == 2 ? launch_attention<4, 2>(a, p, (int)n_seq, weights, s)
                                  : (ng == 4 ? launch_attention<4, 4>(a, p, (int)n_seq, weights, s) : launch_attention<4, 8>(a, p, (int)n_seq, weights, s)));
    }
}

}  // namespace gptq
