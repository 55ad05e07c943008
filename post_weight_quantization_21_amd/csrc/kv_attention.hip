// Attention of a few tokens over a 4-bit cache.
//
// The n G columns of a kv head (n tokens, G query heads each) are the B operand of
// v_mfma_f32_16x16x32_f16, sixteen at a time.  A wave takes tiles of 32 cached tokens:
//   S[token][column] = s_k (sum_d q_k x - z_k X),  X = sum_d x
// with the codes as fp16 numbers of one spacing (key_frag).  The A operand's row r of half
// t is token 8 (r / 4) + 4 t + r % 4, so a lane ends up with S of eight tokens next to each
// other in one column, which is what the second product
//   O[dim][column] = sum_token q_v (p s_v) - sum_token z_v (p s_v)
// wants of its B operand: p never leaves the lane.  It is held there as p s_v in fp16,
// scaled by a power of two that follows the largest s_v: for bf16 results one value, a
// rounding of 2^-11 of each term where theirs is 2^-8; for fp16 results two, the second
// what the first leaves (with one their error against 64 bits is 1.3 times a single
// rounding's; 16 x 4096 tokens of 32 heads take 53 us instead of 47, eight drafted tokens 45
// instead of 42).
// Values s_v more than 2^20 below the largest lose bits, those more than 2^31 below it vanish.
//
// What the sums lose: an instruction adds eight neighbouring products at a time to the fp32
// sum, each addition rounded to nearest, after it has cut off what lies 2^24 below the
// largest of the products' powers of two; there a subnormal operand counts as 2^-14
// (measured).  A code of one is therefore held as high as fp16's even spacing reaches, 2^-21
// and 2^-17: p s_v and queries lose what is below 2^-17 of the largest of their eight.  With
// codes in their lowest bits, which saves an instruction a word, that is 2^-14, always
// towards 0, and adds up over the tokens.  Errors against 64 bits (codes in the lowest bits;
// here; the result's own rounding): fp16, 16 x 4096 tokens 2.39e-4, 2.08e-4, 2.08e-4; bf16,
// 131072 tokens 1.86e-3, 1.66e-3, 1.65e-3; weights of a window of 16 tokens 1.7e-6, 7e-8.
// Times: 52.3, 53.4 us; 35.9, 36.1; 32 x 16384 tokens 83.5, 84.5.  The sums of q are 15 / 8
// as large as those of q - 8 would be, a bit of fp32; taking 8 p s_v off by more matrix
// instructions (tried with codes in the lowest bits) took 12 us more of 83 and left 2.29e-4.
//
// Queries of both types enter as fp16 times a power of two of their row, which takes no
// bit from a value above 2^-25 of the row's largest.
//
// One pass with a running maximum: the sums are rescaled only when a score passes the
// maximum they are held to by 2^6 (p may then be up to 64, which fp16 and fp32 hold).
//
// All tiles of all sequences are shared out evenly, 1024 workgroups of four waves on the
// chip at most; a sequence that several workgroups share is joined by a second launch.
// Bound by memory where the cache is long: one sequence of 131072 tokens, 64 heads on 8
// of 128 (143 MB), takes 36 us and 5.5 to join, 32 of up to 16384 (346 MB) 82-86; 16 of up
// to 4096, 32 heads on 32, fp16 (185 MB) 53, with 360 vector instructions a tile, units busy
// 0.42 of the time and waits 0.69 of the waves'.  With small groups by latency at two waves a
// SIMD: 8 drafted tokens of 8 x 8191 in groups of 32 issue 560 vector instructions a tile and
// sixteen columns, units busy 0.41, and take 41 us.  Short caches wait for loads (half and
// more of the waves' time, units busy 0.1 or less): 900 tokens 7 us, 5 x 6001 of one head of
// 256 11 us.
#include <algorithm>
#include <type_traits>

#include "kv_cache.h"

namespace gptq {
namespace {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

constexpr int kKvTile = 32;   // tokens of a tile
constexpr int kKvWaves = 4;   // waves of a workgroup, each with tiles of its own
constexpr int kKvThreads = kKvWaves * kWave;
constexpr int kMostSegments = 1024;  // of a sequence
constexpr float kSlack = 6.0f;
constexpr float kNegInf = -__builtin_inff();

struct AttnArgs {
    KvPool pool;
    KvSeqs seqs;
    const uint16_t *q;
    int64_t ldq;
    uint16_t *o;
    int64_t ldo;
    float *part;   // [segment][head][column][D]: the result over the segment alone
    float2 *stat;  // [segment][head][column]: maximum (of log2) and sum
    float2 *last;  // [sequence][head][column]: maximum and sum of a sequence of one segment, or NULL
    float scale;   // times log2 e
    float decay;
    int32_t n, group, cols, kept_cols;  // new tokens, query heads of a kv head, n * group; the columns of a tile in LDS
    int32_t target, least;  // workgroups that share the tiles; tiles of one at least
    int32_t weigh_target, weigh_tiles;  // those that weigh tokens; column tiles that they hold
    int32_t bf16, direct;
};

__device__ __forceinline__ float xor_max(float v, int o) { return fmaxf(v, __shfl_xor(v, o)); }
__device__ __forceinline__ float xor_add(float v, int o) { return v + __shfl_xor(v, o); }

// Nothing is computed or loaded on the other side of this.
__device__ __forceinline__ void keep_order() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// The thread's number as a value that nothing is computed from ahead of time: what a rare path derives from it would hold
// registers over the loops otherwise.
__device__ __forceinline__ int fresh_thread() {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
}

// How the cached tokens are shared out: the tiles of all sequences in a row, `chunk` to a workgroup, whose part of one
// sequence is a segment.  Workgroup x's segment of sequence b has the number x + b.
struct Share {
    int b, start, tiles, len;  // a sequence, its first tile in the row, its tiles and length
};
// 64 sequences at a time, a lane each; up to 64 are read once.
struct Row {
    const KvSeqs &seqs;
    int group = -1, len, tiles, upto;  // the lane's sequence; the tiles up to its end, from the group's first on
    int total = 0, chunk = 0;

    __device__ __forceinline__ void read(int g) {
        if (g == group) return;
        group = g;
        const int b = g * kWave + (threadIdx.x & 63);
        len = b < seqs.n ? seqs.len(b) : 0;
        tiles = (len + kKvTile - 1) / kKvTile;
        upto = wave_scan(tiles);
    }
    __device__ __forceinline__ Row(const KvSeqs &s) : seqs(s) {}
    __device__ __forceinline__ Row(const AttnArgs &a) : seqs(a.seqs) {
        for (int g = 0; g * kWave < seqs.n; ++g) {
            read(g);
            total += __builtin_amdgcn_readlane(upto, kWave - 1);
        }
        const int c = (total + a.target - 1) / a.target;
        chunk = max(a.least, (c + kKvWaves - 1) / kKvWaves * kKvWaves);
    }
    // The sequence that tile `at` of the row belongs to, or with `seq` sequence `at`.
    __device__ __forceinline__ Share find(int at, bool seq) {
        const int lane = threadIdx.x & 63;
        Share s = {};
        int base = 0;
        for (int g = 0; g * kWave < seqs.n; ++g) {
            read(g);
            const uint64_t hit = __ballot(seq ? g * kWave + lane == at : base + upto - tiles <= at && at < base + upto);
            if (hit) {
                const int l = __builtin_ctzll(hit);
                s.b = g * kWave + l;
                s.tiles = __builtin_amdgcn_readlane(tiles, l);
                s.start = base + __builtin_amdgcn_readlane(upto, l) - s.tiles;
                s.len = __builtin_amdgcn_readlane(len, l);
                break;
            }
            base += __builtin_amdgcn_readlane(upto, kWave - 1);
        }
        return s;
    }
};

__device__ __forceinline__ int tiles_of(const KvSeqs &s, int b) { return (s.len(b) + kKvTile - 1) / kKvTile; }

// The pages of a tile: one, or with pages of sixteen tokens one for each half.  -1: there is none.
struct TilePages {
    int lo, hi;
    __device__ __forceinline__ TilePages(const AttnArgs &a, const int32_t *row, int tile, int len) {
        const int slot = tile * kKvTile;
        lo = hi = a.seqs.page_of(a.pool, row, slot);
        if (a.pool.lg_page == 4) hi = slot + 16 < len ? a.seqs.page_of(a.pool, row, slot + 16) : lo;
    }
    __device__ __forceinline__ bool missing() const { return (lo | hi) < 0; }
};

// A wave's 32 cached tokens, as they come from memory.  Lane 16 kb + r holds key row r (token 8 (r / 4) + 4 t + r % 4 of
// half t), dims of lane row kb; of the values the eight tokens of block kb, dims 64 u + 16 j + r; and of the grids token
// lane % 32, keys in the lower lanes, values in the upper ones.
template <int D64, int NG>
struct Tile {
    static constexpr int D = 64 * D64, KW = D / 32;
    uint32_t k[2][KW];
    u32x4 v[D64];
    uint32_t grid[NG];

    template <typename T>
    __device__ __forceinline__ static const T *at(const char *base, uint32_t bytes) {
        return reinterpret_cast<const T *>(base + bytes);
    }
    __device__ __forceinline__ void key_words(const char *words, uint32_t off) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if constexpr (KW % 4 == 0) {
#pragma unroll
                for (int i = 0; i < KW; i += 4) {
                    const u32x4 w = *at<u32x4>(words, off + 2 * D * t + 4 * i);
                    k[t][i] = w[0], k[t][i + 1] = w[1], k[t][i + 2] = w[2], k[t][i + 3] = w[3];
                }
            } else {
#pragma unroll
                for (int i = 0; i < KW; i += 2) {
                    const u32x2 w = *at<u32x2>(words, off + 2 * D * t + 4 * i);
                    k[t][i] = w[0], k[t][i + 1] = w[1];
                }
            }
        }
    }
    // With the grids of the values, or those of the keys in all lanes.
    template <bool kBoth>
    __device__ __forceinline__ void load_keys(const AttnArgs &a, TilePages p, int tile, int h) {
        const char *k0 = reinterpret_cast<const char *>(a.pool.k);
        if (a.pool.lg_page > 4) {  // one page: its base is the same for all lanes
            const int lane = threadIdx.x & 63, r = lane & 15, kb = lane >> 4, row = 8 * (r >> 2) + (r & 3), tok = lane & 31;
            const char *g0 = reinterpret_cast<const char *>(!kBoth || lane < 32 ? a.pool.k_grid : a.pool.v_grid);
            const int64_t first = a.pool.first(max(p.lo, 0), h), in = tile * kKvTile & (a.pool.page() - 1);
            key_words(k0 + (first + in) * (D / 2), row * (D / 2) + kb * KW * 4);
#pragma unroll
            for (int g = 0; g < NG; ++g) grid[g] = *at<uint32_t>(g0 + (first * NG + in) * 4, 4 * tok + ((uint32_t)g << (a.pool.lg_page + 2)));
        } else {
            const int lane = fresh_thread() & 63, r = lane & 15, kb = lane >> 4, row = 8 * (r >> 2) + (r & 3), tok = lane & 31;
            const char *g0 = reinterpret_cast<const char *>(!kBoth || lane < 32 ? a.pool.k_grid : a.pool.v_grid);
            const int64_t lo = a.pool.first(max(p.lo, 0), h), hi = a.pool.first(max(p.hi, 0), h);
            const int64_t fk = r < 8 ? lo : hi, fg = tok < 16 ? lo : hi;
            key_words(k0 + fk * (D / 2), (row & 15) * (D / 2) + kb * KW * 4);
#pragma unroll
            for (int g = 0; g < NG; ++g) grid[g] = *at<uint32_t>(g0 + fg * (4 * NG), 4 * (tok & 15) + 64 * g);
        }
    }
    __device__ __forceinline__ void load_values(const AttnArgs &a, TilePages p, int tile, int h) {
        const char *v0 = reinterpret_cast<const char *>(a.pool.v);
        if (a.pool.lg_page > 4) {
            const int lane = threadIdx.x & 63, r = lane & 15, kb = lane >> 4;
            const int64_t first = a.pool.first(max(p.lo, 0), h), in = tile * kKvTile & (a.pool.page() - 1);
#pragma unroll
            for (int u = 0; u < D64; ++u) v[u] = *at<u32x4>(v0 + (first + in) * (D / 2), kb * 4 * D + r * 16 + 256 * u);
        } else {
            const int lane = fresh_thread() & 63, r = lane & 15, kb = lane >> 4;
            const int64_t lo = a.pool.first(max(p.lo, 0), h), hi = a.pool.first(max(p.hi, 0), h), fv = kb < 2 ? lo : hi;
#pragma unroll
            for (int u = 0; u < D64; ++u) v[u] = *at<u32x4>(v0 + fv * (D / 2), (kb & 1) * 4 * D + r * 16 + 256 * u);
        }
    }
};

// A code of 1 as the matrix cores see it.  Half of that exponent goes to the keys' scales and half to the queries', so that
// neither overflows before the scores do (keys up to 2^114, queries of any size).
constexpr float kCode = 1.0f / (1 << 21), kKeys = 1 << 9;

// The grids of a wave's tile in LDS, token by token: scales in fp32 (of keys times kKeys, of values times the wave's power
// of two) and -z in fp16.  Written by the lane that holds a token's word, read by the lanes that need eight.
template <int NG>
struct TileGrids {
    float scale[2][NG][kKvTile];
    uint16_t zero[2][NG][kKvTile];

    // `none`: of the upper lanes, those whose token has a value that is no number.  It makes the token's scores no numbers,
    // and so what sees them; to the others it is 0, since p = 0 does not make a product with it 0.
    __device__ __forceinline__ void put(const uint32_t grid[NG], float vscale, bool gone, uint64_t none) {
        const int lane = threadIdx.x & 63, side = lane >> 5, tok = lane & 31;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            float s = grid_scale_of(grid[g]);
            const bool odd = !(s == s);
            const _Float16 c = __builtin_bit_cast(f16x2, grid[g])[0];
            s = side ? (odd ? 0.0f : s * vscale) : s * kKeys;
            if (none && !side && (none >> (32 + tok) & 1)) s = __builtin_nanf("");
            scale[side][g][tok] = gone ? 0.0f : s;
            zero[side][g][tok] = __builtin_bit_cast(uint16_t, gone || odd ? (_Float16)0.0f : c - (_Float16)8.0f);
        }
    }
    // Eight tokens of block kb; t: four of them.
    __device__ __forceinline__ floatx4 scales(int side, int g, int kb, int t) const {
        return *reinterpret_cast<const floatx4 *>(&scale[side][g][8 * kb + 4 * t]);
    }
    __device__ __forceinline__ f16x8 zeros(int side, int g, int kb) const {
        return *reinterpret_cast<const f16x8 *>(&zero[side][g][8 * kb]);
    }
};
// What the wave has put into LDS is there for its other lanes.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Codes as fp16, masked in place: bits 3 to 6, q 2^-21, and 7 to 10, q 2^-17.  Bit 10 is the lowest of the exponent, and numbers
// below 2^-13 lie evenly, subnormal or not.
__device__ __forceinline__ uint32_t low(uint32_t w) { return w & 0x00780078u; }
__device__ __forceinline__ uint32_t high(uint32_t w) { return w & 0x07800780u; }
__device__ __forceinline__ f16x8 key_frag(uint32_t w) {  // pairs 0 and 2 are 2^4 smaller: the queries' are 2^4 larger there
    const uint32_t x = w << 3, y = w >> 5;
    const u32x4 f = {low(x), high(x), low(y), high(y)};
    return __builtin_bit_cast(f16x8, f);
}
// Dims j and j + 1 (j = 0, 2) of the four of each unit, eight tokens.
__device__ __forceinline__ void value_frags(f16x8 f[2], const u32x4 &w, int j) {
    u32x4 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = j ? w[i] >> 5 : w[i] << 3;
        a[i] = low(x);
        b[i] = high(x);
    }
    f[0] = __builtin_bit_cast(f16x8, a);
    f[1] = __builtin_bit_cast(f16x8, b);
}

__device__ __forceinline__ floatx4 mma(f16x8 a, f16x8 b, floatx4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }

// Sixteen columns of queries as B operands, times a power of two of their row, with their sums per group.
template <int D64, int NG>
struct Queries {
    static constexpr int KW = 2 * D64;
    f16x8 x[KW];
    float sum[NG];  // of the group's x, times kCode
    float scale;    // of scores, to log2
    int sees;       // slots below this are visible

    // The row's bits; prepare() turns them into x.
    __device__ __forceinline__ void load(const AttnArgs &a, int b, int h, int len, int col) {
        const int kb = (fresh_thread() & 63) >> 4;
        const bool real = col < a.cols;
        const int i = real ? col / a.group : 0, hq = h * a.group + (real ? col - i * a.group : 0);
        sees = real ? len - a.n + 1 + i : 0;
        const uint16_t *q = a.q + ((int64_t)b * a.n + i) * a.ldq + (int64_t)hq * (64 * D64) + 8 * kb;
#pragma unroll
        for (int t = 0; t < KW; ++t) x[t] = __builtin_bit_cast(f16x8, real ? *reinterpret_cast<const u32x4 *>(q + 32 * t) : (u32x4){});
    }
    __device__ __forceinline__ void prepare(const AttnArgs &a) {
        // the largest magnitude, whose bits order as the numbers do in both types; its binade becomes fp16's largest
        u16x2 most = {};
#pragma unroll
        for (int t = 0; t < KW; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, __builtin_bit_cast(u32x4, x[t])[j] & 0x7FFF7FFFu));
        const uint16_t m = most[0] > most[1] ? most[0] : most[1];
        float top = a.bf16 ? __uint_as_float((uint32_t)m << 16) : (float)__builtin_bit_cast(_Float16, m);
        top = xor_max(xor_max(top, 16), 32);
        int e = 0;
        if (top > 0.0f && top < __builtin_inff()) frexpf(top, &e);
        const int up = min(15 - e, 126);  // top < 2^e; (a power of two that fp32 holds)
        const float f0 = ldexpf(1.0f, up), f1 = ldexpf(1.0f, up - 4);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            float s = 0.0f;
#pragma unroll
            for (int t = g * KW / NG; t < (g + 1) * KW / NG; ++t) {
                const u32x4 w = __builtin_bit_cast(u32x4, x[t]);
                u32x4 y;
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // pair j of the fragment; the odd ones meet codes 2^4 larger
                    const uint32_t two = w[j];
                    f32x2 v = {__uint_as_float(two << 16), __uint_as_float(two & 0xFFFF0000u)};
                    if (!a.bf16) v = __builtin_convertvector(__builtin_bit_cast(f16x2, two), f32x2);
                    const float f = j & 1 ? f1 : f0;
                    const f16x2 hf = __builtin_convertvector(((f32x2){v[0] * f, v[1] * f}), f16x2);
                    const _Float16 one = j & 1 ? (_Float16)16.0f : (_Float16)1.0f;
                    s = __builtin_amdgcn_fdot2(hf, (f16x2){one, one}, s, false);
                    y[j] = __builtin_bit_cast(uint32_t, hf);
                }
                x[t] = __builtin_bit_cast(f16x8, y);
            }
            sum[g] = xor_add(xor_add(s, 16), 32) * kCode;
        }
        scale = ldexpf(a.scale, 12 - up);
    }
};

__device__ __forceinline__ bool hidden(bool there, int slot, int sees) { return !there || slot >= sees; }

// Scores of the lane's eight tokens in the columns, in log2 and less the columns' `base`, before any mask.  The queries are
// in registers, or `shared`: the lane's part of fragments in LDS.
template <int D64, int NG, int NT, bool kTight>
__device__ __forceinline__ void scores(float s[NT][8], const Tile<D64, NG> &tile, const TileGrids<NG> &grids, const Queries<D64, NG> q[NT],
                                       const f16x8 *shared, const float base[NT]) {
    constexpr int KW = 2 * D64, SG = KW / NG;  // matrix instructions of a group
    const int kb = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            floatx4 acc[NT] = {};
#pragma unroll
            for (int w = g * SG; w < (g + 1) * SG; ++w) {
                const f16x8 kf = key_frag(tile.k[t][w]);
#pragma unroll
                for (int c = 0; c < NT; ++c) acc[c] = mma(kf, shared ? shared[(c * KW + w) * kWave] : q[c].x[w], acc[c]);
            }
            const floatx4 scale = grids.scales(0, g, kb, t);
            const f16x8 zero = grids.zeros(0, g, kb);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < NT; ++c) {
                    const float v = fmaf((float)zero[4 * t + i], q[c].sum[g], acc[c][i]);
                    s[c][4 * t + i] = g == 0 ? scale[i] * v : fmaf(scale[i], v, s[c][4 * t + i]);
                }
            if (kTight) keep_order();  // fragments and grids of one group at a time: registers
        }
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[c][i] = fmaf(s[c][i], q[c].scale, -base[c]);
}

// A wave's sums over its tiles of a segment.
template <int D64, int NG, int NT>
struct Sums {
    static constexpr int D = 64 * D64;
    floatx4 acc[NT][D / 16];                  // of codes: kCode or, in odd dims of a unit, 16 kCode a step
    float corr[NT][NG], sum[NT], base[NT];    // base: what scores are taken less (0 as long as nothing is seen)
    float slack[NT];                          // a score above it raises base: kSlack, or anything as long as nothing is seen
    float vmax, vscale;                       // a power of two above every s_v / 4; 2^6 over it

    __device__ __forceinline__ Sums() {
#pragma unroll
        for (int c = 0; c < NT; ++c) {
#pragma unroll
            for (int d = 0; d < D / 16; ++d) acc[c][d] = (floatx4){};
#pragma unroll
            for (int g = 0; g < NG; ++g) corr[c][g] = 0.0f;
            sum[c] = base[c] = 0.0f;
            slack[c] = kNegInf;
        }
        vmax = 0.0f;
        vscale = 1.0f;
    }
    __device__ __forceinline__ void times(int c, float f) {
#pragma unroll
        for (int g = 0; g < NG; ++g) corr[c][g] *= f;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) acc[c][d] *= f;
    }
    // A new power of two for the values' scales, the largest of which is `most` (of the lane's).
    __device__ __forceinline__ void raise_values(float most) {
        for (int o = 1; o < kWave; o *= 2) most = xor_max(most, o);
        const float was = vscale;
        int e;
        frexpf(most, &e);
        e = max(e, -118);  // 2^(6 - e) stays finite
        vmax = ldexpf(1.0f, e);
        vscale = ldexpf(1.0f, 6 - e);
#pragma unroll
        for (int c = 0; c < NT; ++c) times(c, vscale / was);
    }
    // A new base from the lane's scores, of the columns that need one: what the others hold does not depend on who is beside them.
    __device__ __forceinline__ void raise(float s[NT][8]) {
#pragma unroll
        for (int c = 0; c < NT; ++c) {
            float m = s[c][0];
#pragma unroll
            for (int i = 1; i < 8; ++i) m = fmaxf(m, s[c][i]);
            m = xor_max(xor_max(m, 16), 32);
            const bool first = slack[c] == kNegInf;
            if (m > slack[c]) {
                times(c, first ? 1.0f : __builtin_amdgcn_exp2f(-m));  // (of nothing, the first time)
                sum[c] *= first ? 1.0f : __builtin_amdgcn_exp2f(-m);
                base[c] += m;
                slack[c] = kSlack;
#pragma unroll
                for (int i = 0; i < 8; ++i) s[c][i] -= m;
            }
        }
    }
    __device__ __forceinline__ float top(int c) const { return slack[c] == kNegInf ? kNegInf : base[c]; }
};

__device__ __forceinline__ int64_t result_at(const AttnArgs &a, int b, int h, int col, int D) {
    const int tok = col / a.group;
    return ((int64_t)b * a.n + tok) * a.ldo + (int64_t)(h * a.group + col - tok * a.group) * D;
}
__device__ __forceinline__ uint16_t result16(const AttnArgs &a, float y) {
    return a.bf16 ? __builtin_bit_cast(uint16_t, (__bf16)y) : __builtin_bit_cast(uint16_t, (_Float16)y);
}
// How much of a sum relative to `top` counts in one relative to `all`.
__device__ __forceinline__ float share_in(float top, float all) { return top == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(top - all); }

// The waves' sums, brought to the largest of their maxima and added in wave order: the result where the segment is all of
// its sequence, else its part.
template <int D64, int NG, int NT>
__device__ __forceinline__ void write_sums(const AttnArgs &a, const Sums<D64, NG, NT> &s, const Share &sh, bool whole, float *smem, int h, int col0) {
    constexpr int D = 64 * D64;
    const int thread = fresh_thread(), lane = thread & 63, wave = thread >> 6, r = lane & 15, kb = lane >> 4;
    const int kept = a.kept_cols;  // of a tile in LDS
    float2 *ml = reinterpret_cast<float2 *>(smem + kKvWaves * kept * D);
#pragma unroll
    for (int c = 0; c < NT; ++c) {
        const int left = a.cols - col0 - 16 * c;  // columns there are
        if (c && left <= 0) break;
        const float l = xor_add(xor_add(s.sum[c], 16), 32);
        __syncthreads();  // what the last round left in LDS has been read
        if (kb == 0) ml[wave * 16 + r] = make_float2(s.top(c), l);
        __syncthreads();
        float m = kNegInf, all = 0.0f;
#pragma unroll
        for (int w = 0; w < kKvWaves; ++w) m = fmaxf(m, ml[w * 16 + r].x);
#pragma unroll
        for (int w = 0; w < kKvWaves; ++w) {
            const float2 v = ml[w * 16 + r];
            all += v.x == kNegInf ? v.y : v.y * __builtin_amdgcn_exp2f(v.x - m);  // (a NaN stays)
        }
        const float inv = all == 0.0f ? 0.0f : 1.0f / all;
        // (in this order nothing overflows that the result does not)
        const float f = share_in(s.top(c), m) * inv * (1.0f / kCode), scale = 1.0f / s.vscale;
        const int64_t stat = ((int64_t)(blockIdx.x + sh.b) * a.pool.heads + h) * a.cols + col0 + 16 * c;
        if (r < left) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const float k = xor_add(xor_add(s.corr[c][g], 16), 32) * kCode;
#pragma unroll
                for (int d = g * (D / 16) / NG; d < (g + 1) * (D / 16) / NG; ++d)
                    *reinterpret_cast<floatx4 *>(smem + (wave * kept + r) * D + 16 * d + 4 * kb) = (s.acc[c][d] * (d & 1 ? 0.0625f : 1.0f) + k) * f * scale;
            }
            if (wave == 0 && kb == 0) {
                if (!whole)
                    a.stat[stat + r] = make_float2(m, all);
                else if (a.last)
                    a.last[((int64_t)sh.b * a.pool.heads + h) * a.cols + col0 + 16 * c + r] = make_float2(m, all);
            }
        }
        __syncthreads();
        for (int i = thread; i < min(left, 16) * (D / 4); i += kKvThreads) {
            const int cc = i / (D / 4), d = i % (D / 4) * 4;
            floatx4 o = *reinterpret_cast<const floatx4 *>(smem + cc * D + d);
#pragma unroll
            for (int w = 1; w < kKvWaves; ++w) o += *reinterpret_cast<const floatx4 *>(smem + (w * kept + cc) * D + d);
            if (whole) {
                uint16_t *to = a.o + result_at(a, sh.b, h, col0 + 16 * c + cc, D) + d;
#pragma unroll
                for (int e = 0; e < 4; ++e) to[e] = result16(a, o[e]);
            } else {
                *reinterpret_cast<floatx4 *>(a.part + (stat + cc) * D + d) = o;
            }
        }
    }
}

// Whether the queries stay in LDS, where registers are short.  (In LDS; in registers, us: heads of 128 in groups of 32 with two
// column tiles, 32 x 16384 tokens and 32 columns 186; 447, 256 in 64s and 192 in 32s, 8 x 8191 and 8 columns 24.6; 28 and 26;
// 30.  Below the border: 128 in 128s, 131072 tokens 38.8; 36.5, two column tiles 139; 125, 128 in 32s 34.6; 33.4, in 64s 25.5;
// 25.6.  256 in 32s, past it, would gain from registers: 34.0; 32.4.)
constexpr bool queries_in_lds(int D64, int NG, int NT) { return D64 * NG * NT >= 16; }
// Waves of a SIMD that the registers of a kernel allow (of 512, in steps of eight): its sums take 16 D64 NT, its queries
// 8 D64 NT, a tile 9 D64.  With a wave fewer; here; with one more, us, 16 x 8191 tokens and 4 columns where nothing else is said: 128
// in 128s 85; 83; - (32 x 16384, 8 columns) and 50; 53; 118 (fp16, 16 x 4096 of 32 heads), in 64s 28; 25; 49, in 32s 48; 34; 63; 64
// in 64s 20; 22; 21 and 107; 92; - (32 x 16384, 32 columns one tile at a time), in 32s 20; 22; 38; 8 x 8191 and 8 columns: 192 in
// 192s 20; 19; 17, in 64s 22; 20; 28, in 32s 26; 26; 67; 256 in 256s 24; 23; 26, in 64s 27; 25; 56, in 32s -; 34; 93.  128 in 128s
// spills three registers, or five, at four waves; at three it spills none.
constexpr int occupancy(int D64, int NG, int NT) {
    if (D64 * NT == 1 || (D64 == 2 && NT == 1 && NG == 1)) return 4;
    if ((D64 == 2 && NT == 1 && NG == 2) || (D64 == 1 && NG == 1)) return 3;
    return D64 * NG * NT < 32 ? 2 : 1;
}

template <int D64, int NG, int NT, bool kBf16>
__global__ __launch_bounds__(kKvThreads, occupancy(D64, NG, NT)) void attention_kernel(AttnArgs a) {
    constexpr int D = 64 * D64;
    constexpr bool kShared = queries_in_lds(D64, NG, NT);
    extern __shared__ __attribute__((aligned(16))) float smem[];  // [wave][column][D] of one column tile, then (m, l), then grids
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, kb = lane >> 4;
    const int h = blockIdx.y, col0 = blockIdx.z * (16 * NT);
    TileGrids<NG> &grids = reinterpret_cast<TileGrids<NG> *>(smem + kKvWaves * (a.kept_cols * D + 32))[wave];
    int from = 0, to;  // of the row of tiles
    Share sh;
    if (a.direct) {  // a sequence to a workgroup
        sh = {(int)blockIdx.x, 0, tiles_of(a.seqs, blockIdx.x), a.seqs.len(blockIdx.x)};
        to = sh.tiles;
    } else {
        Row rows(a);
        from = blockIdx.x * rows.chunk;
        to = min(from + rows.chunk, rows.total);
        if (from >= to) return;
        sh = rows.find(from, false);
    }
    for (;;) {
        const int32_t *row = a.seqs.table + (int64_t)sh.b * a.seqs.width;
        const int t0 = from - sh.start, t1 = min(to - sh.start, sh.tiles);  // of the sequence
        Queries<D64, NG> q[NT];
#pragma unroll
        for (int c = 0; c < NT; ++c) q[c].load(a, sh.b, h, sh.len, col0 + 16 * c + r);
        Sums<D64, NG, NT> sums;
        const int clear = sh.len - a.n + 1;  // slots below this are visible to every column
        int tile = t0 + wave;
        Tile<D64, NG> t;
        TilePages pages = {a, row, max(min(tile, t1 - 1), 0), sh.len};
        if (tile < t1) {
            t.template load_keys<true>(a, pages, tile, h);
            t.load_values(a, pages, tile, h);
        }
#pragma unroll
        for (int c = 0; c < NT; ++c) q[c].prepare(a);
        const f16x8 *shared = nullptr;
        if constexpr (kShared) {  // all waves have the same ones
            f16x8 *to = reinterpret_cast<f16x8 *>(smem + kKvWaves * (a.kept_cols * D + 32 + (int)(sizeof(TileGrids<NG>) / 4))) + lane;
            if (wave == 0) {
#pragma unroll
                for (int c = 0; c < NT; ++c)
#pragma unroll
                    for (int w = 0; w < 2 * D64; ++w) to[(c * 2 * D64 + w) * kWave] = q[c].x[w];
            }
            __syncthreads();
            shared = to;
        }
        // The keys of the next tile are on their way during the second product, its values during the first of the next.
        while (tile < t1) {
            const int next = tile + kKvWaves;
            const TilePages coming = {a, row, min(next, t1 - 1), sh.len};
            const bool masked = (tile + 1) * kKvTile > clear || pages.missing();
            const bool gone = masked && hidden(((lane & 16) ? pages.hi : pages.lo) >= 0, tile * kKvTile + (lane & 31), sh.len);
            float most = 0.0f;
            bool odd = false;
            if (lane >= 32 && !gone) {
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float s = grid_scale_of(t.grid[g]);
                    most = fmaxf(most, s);
                    odd |= !(s == s);
                }
            }
            if (__any(most > 4.0f * sums.vmax)) sums.raise_values(most);
            grids.put(t.grid, sums.vscale, gone, __ballot(odd));
            wave_fence();
            float p[NT][8];
            scores<D64, NG, NT, NG == 1>(p, t, grids, q, shared, sums.base);
            if (next < t1) t.template load_keys<true>(a, coming, next, h);
            const int slot = tile * kKvTile + 8 * kb;
            const bool there = (kb < 2 ? pages.lo : pages.hi) >= 0;
            if (masked) {
#pragma unroll
                for (int c = 0; c < NT; ++c)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (hidden(there, slot + i, q[c].sees)) p[c][i] = kNegInf;
            }
            bool high = false;
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                float m = p[c][0];
#pragma unroll
                for (int i = 1; i < 8; ++i) m = fmaxf(m, p[c][i]);
                high |= m > sums.slack[c];
            }
            if (__any(high)) sums.raise(p);
#pragma unroll
            for (int c = 0; c < NT; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    p[c][i] = __builtin_amdgcn_exp2f(p[c][i]);
                    sums.sum[c] += p[c][i];
                }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const floatx4 s0 = grids.scales(1, g, kb, 0), s1 = grids.scales(1, g, kb, 1);
                const f16x8 zero = grids.zeros(1, g, kb);
                f16x8 pf[NT], rest[NT];  // p s_v, and what fp16 leaves of it
#pragma unroll
                for (int c = 0; c < NT; ++c) {
                    float ps[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) ps[i] = p[c][i] * (i < 4 ? s0[i] : s1[i - 4]);
                    u32x4 w, v;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f16x2 z = {zero[2 * i], zero[2 * i + 1]};
                        const f16x2 f = __builtin_convertvector(((f32x2){ps[2 * i], ps[2 * i + 1]}), f16x2);
                        sums.corr[c][g] = __builtin_amdgcn_fdot2(f, z, sums.corr[c][g], false);
                        w[i] = __builtin_bit_cast(uint32_t, f);
                        if constexpr (!kBf16) {
                            const f16x2 y = __builtin_convertvector(((f32x2){ps[2 * i] - (float)f[0], ps[2 * i + 1] - (float)f[1]}), f16x2);
                            sums.corr[c][g] = __builtin_amdgcn_fdot2(y, z, sums.corr[c][g], false);
                            v[i] = __builtin_bit_cast(uint32_t, y);
                        }
                    }
                    pf[c] = __builtin_bit_cast(f16x8, w);
                    if constexpr (!kBf16) rest[c] = __builtin_bit_cast(f16x8, v);
                }
#pragma unroll
                for (int d = g * (D / 16) / NG; d < (g + 1) * (D / 16) / NG; d += 2) {
                    f16x8 vf[2];
                    value_frags(vf, t.v[d / 4], d % 4);
#pragma unroll
                    for (int c = 0; c < NT; ++c) {
                        sums.acc[c][d] = mma(vf[0], pf[c], sums.acc[c][d]);
                        sums.acc[c][d + 1] = mma(vf[1], pf[c], sums.acc[c][d + 1]);
                        if constexpr (!kBf16) {
                            sums.acc[c][d] = mma(vf[0], rest[c], sums.acc[c][d]);
                            sums.acc[c][d + 1] = mma(vf[1], rest[c], sums.acc[c][d + 1]);
                        }
                    }
                    keep_order();
                }
            }
            if (next < t1) t.load_values(a, coming, next, h);
            tile = next;
            pages = coming;
        }
        write_sums<D64, NG, NT>(a, sums, sh, t0 == 0 && t1 == sh.tiles, smem, h, col0);
        if (from + (t1 - t0) >= to) break;
        from += t1 - t0;
        sh = Row(a.seqs).find(from, false);
    }
}

// The segments of a sequence: the first, and how many.
struct Segments {
    int first, n;
    __device__ __forceinline__ Segments(const Share &sh, int chunk)
        : first(sh.start / chunk + sh.b), n(sh.tiles ? (sh.start + sh.tiles - 1) / chunk - sh.start / chunk + 1 : 0) {}
};

// The result of a column of a sequence with several segments, or none, by a workgroup: a thread takes four dims of every
// kLanes-th segment (five rows of 48 threads for heads of 192).
template <int D64>
__device__ __forceinline__ void combine(const AttnArgs &a, int col, int h, int b) {
    constexpr int D = 64 * D64, kRow = D / 4, kLanes = kKvThreads / kRow;
    __shared__ float share[kMostSegments];
    __shared__ float red[2][kKvWaves];
    __shared__ floatx4 sums[kKvThreads];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    Row rows(a);
    const Segments seg(rows.find(b, true), rows.chunk);
    if (seg.n == 1) return;
    const int64_t at0 = ((int64_t)seg.first * a.pool.heads + h) * a.cols + col, step = (int64_t)a.pool.heads * a.cols;
    float m = kNegInf, l = 0.0f;
    for (int x = threadIdx.x; x < seg.n; x += kKvThreads) m = fmaxf(m, a.stat[at0 + x * step].x);
    for (int o = 1; o < kWave; o *= 2) m = xor_max(m, o);
    if (lane == 0) red[0][wave] = m;
    __syncthreads();
    for (int w = 0; w < kKvWaves; ++w) m = fmaxf(m, red[0][w]);
    for (int x = threadIdx.x; x < seg.n; x += kKvThreads) {
        const float2 v = a.stat[at0 + x * step];
        share[x] = v.x == kNegInf ? v.y : v.y * share_in(v.x, m);  // (a NaN stays)
        l += share[x];
    }
    for (int o = 1; o < kWave; o *= 2) l = xor_add(l, o);
    if (lane == 0) red[1][wave] = l;
    __syncthreads();
    l = 0.0f;
    for (int w = 0; w < kKvWaves; ++w) l += red[1][w];
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int mine = threadIdx.x / kRow, d4 = threadIdx.x % kRow;
    floatx4 o = {};
    if (mine < kLanes) {
#pragma unroll 4
        for (int x = mine; x < seg.n; x += kLanes) o += share[x] * inv * *reinterpret_cast<const floatx4 *>(a.part + (at0 + x * step) * D + 4 * d4);
    }
    sums[threadIdx.x] = o;
    __syncthreads();
    if (threadIdx.x < kRow) {
        for (int y = 1; y < kLanes; ++y) o += sums[y * kRow + threadIdx.x];
        uint16_t *to = a.o + result_at(a, b, h, col, D) + 4 * threadIdx.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i] = result16(a, o[i]);
    }
}
template <int D64>
__global__ __launch_bounds__(kKvThreads) void combine_kernel(AttnArgs a) {
    combine<D64>(a, blockIdx.x, blockIdx.y, blockIdx.z);
}

template <int kCtrl>
__device__ __forceinline__ float lane_of(float v) {  // of the lane that a DPP control names
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, 0xF, 0xF, true));
}
// Eight sums over a row of sixteen lanes, of which lane r has number r / 2: at each step a lane keeps half of the numbers
// and hands the others to a lane that keeps those.
__device__ __forceinline__ float row_sums(const float w[8], int r) {
    float u[4], v[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = (r & 8 ? w[i + 4] : w[i]) + lane_of<0x128>(r & 8 ? w[i] : w[i + 4]);  // row_ror:8
#pragma unroll
    for (int i = 0; i < 2; ++i) v[i] = (r & 4 ? u[i + 2] : u[i]) + lane_of<0x141>(r & 4 ? u[i] : u[i + 2]);  // row_half_mirror
    const float z = (r & 2 ? v[1] : v[0]) + lane_of<0x4E>(r & 2 ? v[0] : v[1]);  // quad_perm 2 3 0 1
    return z + lane_of<0xB1>(z);  // quad_perm 1 0 3 2
}

// What a column needs beside its queries.
template <int NG>
struct Column {
    float sum[NG], scale, base, inv;  // inv: 1 / the sum of exp; 0 where nothing is seen, or there is no column
    int sees;
};
constexpr int kWeighTiles = 8;  // column tiles of a pass over the tokens
template <int D64, int NG>
constexpr int weigh_bytes(int tiles) {
    return kKvWaves * (int)sizeof(TileGrids<NG>) + tiles * (2 * D64 * 1024 + 16 * (int)sizeof(Column<NG>));
}

// weight[token] = decay weight[token] + the sum of p over the columns, once the columns' maxima and sums are known.  Only
// the keys are read again; the same instructions give the same scores.  The queries are in LDS, up to kWeighTiles tiles of
// them, and each of the wave's tiles of tokens goes through all; more columns take further passes.  Vector
// instructions (260 a tile) are busy half of the time: 32 sequences of up to 16384 tokens, 64 heads on 8, take 64-67 us with
// the joins of their segments, 3 TB/s; loading the next tile ahead changed nothing.  A window of 16 tokens with 128 columns (2 x
// 5003) takes 19 us, 0.63 of its waves' time waits and units busy 0.08.  (Not built: the first pass could write its scores, 4
// bytes a token and column to write and to read; up to 8 columns that is 64 bytes against the keys' 68, and no second product.)
template <int D64, int NG>
__device__ __forceinline__ void weigh(const AttnArgs &a, int item, int h, unsigned char *smem) {
    constexpr int KW = 2 * D64;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, kb = lane >> 4;
    TileGrids<NG> &grids = reinterpret_cast<TileGrids<NG> *>(smem)[wave];
    f16x8 *frags = reinterpret_cast<f16x8 *>(smem + kKvWaves * sizeof(TileGrids<NG>));
    Column<NG> *columns = reinterpret_cast<Column<NG> *>(frags + a.weigh_tiles * KW * kWave);
    int from, to, chunk;
    {
        const Row rows(a);
        chunk = rows.chunk;
        const int c = (rows.total + a.weigh_target - 1) / a.weigh_target, mine = (c + kKvWaves - 1) / kKvWaves * kKvWaves;
        from = item * mine;
        to = min(from + mine, rows.total);
    }
    while (from < to) {
        const Share sh = Row(a.seqs).find(from, false);
        const Segments seg(sh, chunk);
        const int32_t *row = a.seqs.table + (int64_t)sh.b * a.seqs.width;
        const int t0 = from - sh.start, t1 = min(to - sh.start, sh.tiles), clear = sh.len - a.n + 1;
        for (int col0 = 0; col0 < a.cols; col0 += 16 * kWeighTiles) {
            const int tiles = min((a.cols - col0 + 15) / 16, kWeighTiles);
            __syncthreads();  // the last pass has read its columns
            for (int c = wave; c < tiles; c += kKvWaves) {
                const int col = col0 + 16 * c + r;
                Queries<D64, NG> q;
                q.load(a, sh.b, h, sh.len, col);
                float m = kNegInf, l = 0.0f;
                if (a.direct || seg.n == 1) {
                    if (col < a.cols) {
                        const float2 v = a.last[((int64_t)sh.b * a.pool.heads + h) * a.cols + col];
                        m = v.x, l = v.y;
                    }
                } else {
                    const int64_t at0 = ((int64_t)seg.first * a.pool.heads + h) * a.cols + min(col, a.cols - 1), step = (int64_t)a.pool.heads * a.cols;
                    for (int x = kb; x < seg.n; x += 4) m = fmaxf(m, a.stat[at0 + x * step].x);
                    m = xor_max(xor_max(m, 16), 32);
                    for (int x = kb; x < seg.n; x += 4) {
                        const float2 v = a.stat[at0 + x * step];
                        l += v.x == kNegInf ? v.y : v.y * __builtin_amdgcn_exp2f(v.x - m);
                    }
                    l = xor_add(xor_add(l, 16), 32);
                }
                q.prepare(a);
#pragma unroll
                for (int w = 0; w < KW; ++w) frags[(c * KW + w) * kWave + lane] = q.x[w];
                if (kb == 0) {
                    Column<NG> &k = columns[16 * c + r];
#pragma unroll
                    for (int g = 0; g < NG; ++g) k.sum[g] = q.sum[g];
                    k.scale = q.scale;
                    // Where the sum is no number, so is base, and inv is 1: what the column sees gets no number, what is hidden from it 0.
                    const bool none = !(l == l);
                    k.base = none ? l : m == kNegInf ? 0.0f : m;
                    k.inv = l == 0.0f || col >= a.cols ? 0.0f : none ? 1.0f : 1.0f / l;
                    k.sees = q.sees;
                }
            }
            __syncthreads();
            const float decay = col0 ? 1.0f : a.decay;
            // the token whose weight this lane has in the end, of the tile's page
            const int mine = 8 * kb + (r >> 1);
            auto weight_of = [&](TilePages p, int tile) {
                const int page = kb < 2 ? p.lo : p.hi, slot = tile * kKvTile + mine;
                return page < 0 || slot >= sh.len || (r & 1) ? nullptr : a.pool.weight + a.pool.first(page, h) + (slot & (a.pool.page() - 1));
            };
            int tile = t0 + wave;
            Tile<D64, NG> t;
            TilePages pages = {a, row, min(tile, t1 - 1), sh.len};
            float *at = nullptr, old = 0.0f;
            if (tile < t1) {
                t.template load_keys<false>(a, pages, tile, h);
                at = weight_of(pages, tile);
                if (at && decay != 0.0f) old = *at;
            }
            while (tile < t1) {
                const int next = tile + kKvWaves;
                const TilePages coming = {a, row, min(next, t1 - 1), sh.len};
                const int slot = tile * kKvTile + 8 * kb;
                const bool masked = (tile + 1) * kKvTile > clear || pages.missing(), there = (kb < 2 ? pages.lo : pages.hi) >= 0;
                float w[8] = {};
                grids.put(t.grid, 1.0f, false, 0);
                wave_fence();
                for (int c = 0; c < tiles; ++c) {
                    const Column<NG> &k = columns[16 * c + r];
                    Queries<D64, NG> q;
#pragma unroll
                    for (int g = 0; g < NG; ++g) q.sum[g] = k.sum[g];
                    q.scale = k.scale;
                    const float base = k.base, inv = k.inv;
                    float p[1][8];
                    scores<D64, NG, 1, true>(p, t, grids, &q, frags + c * KW * kWave + lane, &base);
                    if (masked) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (hidden(there, slot + i, k.sees)) p[0][i] = kNegInf;
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] += inv != 0.0f ? __builtin_amdgcn_exp2f(p[0][i]) * inv : 0.0f;
                }
                float *const here = at;
                const float before = old;
                at = nullptr;
                if (next < t1) {
                    t.template load_keys<false>(a, coming, next, h);
                    at = weight_of(coming, next);
                    if (at && decay != 0.0f) old = *at;
                }
                const float sum = row_sums(w, r);
                if (here) *here = decay == 0.0f ? sum : fmaf(decay, before, sum);
                tile = next;
                pages = coming;
            }
        }
        from += t1 - t0;
    }
}
// The two together: the first `combining` workgroups join the segments' results, the others weigh tokens.
template <int D64, int NG>
__global__ __launch_bounds__(kKvThreads, D64 == 4 ? (NG < 4 ? 3 : 2) : (D64 * NG <= 4 ? 4 : 3)) void finish_kernel(AttnArgs a, int combining) {
    extern __shared__ __attribute__((aligned(16))) unsigned char finish_smem[];
    int x = blockIdx.x;
    if (x < combining) {
        const int col = x % a.cols, y = x / a.cols;
        combine<D64>(a, col, y % a.pool.heads, y / a.pool.heads);
    } else {
        x -= combining;
        weigh<D64, NG>(a, x / a.pool.heads, x % a.pool.heads, finish_smem);
    }
}

struct Plan {
    int nt, items, target, least, weigh_items, weigh_target;
    bool direct;
    size_t part, stat, last;  // bytes
};
Plan plan_with(int nt, const gptq_kv_cache &c, int64_t n_seq, int64_t cols, int64_t max_len) {
    Plan p;
    p.nt = nt;
    const int64_t tiles = ceil_div(max_len, kKvTile), blocks = c.n_heads * ceil_div(cols, 16 * p.nt);
    // as many workgroups as the chip holds at once, but no more than combine() takes of one sequence
    p.target = (int)std::min<int64_t>(kMostSegments, std::max<int64_t>(1, 256 * occupancy(c.head_dim / 64, kv_pool(c).groups, p.nt) / blocks));
    // A tile for each wave, or two where the columns take several workgroups, each with parts to join (the last 16 tokens of
    // two prompts of up to 5003, 128 columns: 34 us instead of 39; 900 tokens, 4 columns: 12.2 instead of 11.5).
    p.least = kKvWaves * (cols > 16 * p.nt ? 2 : 1);
    p.direct = tiles <= p.least;
    const int64_t all = std::max<int64_t>(1, n_seq * tiles);
    p.items = (int)(p.direct ? n_seq : std::min<int64_t>(p.target, ceil_div(all, p.least)));
    p.weigh_target = (int)std::max<int64_t>(1, 256 * 4 / c.n_heads);
    p.weigh_items = (int)std::min<int64_t>(p.weigh_target, ceil_div(all, kKvWaves));
    const size_t rows = (size_t)c.n_heads * cols, segments = p.direct ? 0 : rows * (p.items + n_seq);
    p.part = align_up(segments * c.head_dim * 4, 256);
    p.stat = align_up(segments * 8, 256);
    p.last = align_up(rows * n_seq * 8, 256);
    return p;
}
// Two column tiles a wave share the tokens' loads and unpacking, and halve the waves that can be at work.  They take over where
// 2048 waves would have sixteen tiles of tokens each.  One column tile a wave; two, us, by the tiles that each would have, 17 to
// 64 columns of heads of 128 in 128s where nothing else is said: 1: 12.3; 15.7 (a window's 128 columns of heads of 64), 4: 27; 29
// and 22; 29 (in 64s), 8: 31; 31 and 37; 42 (in 32s), 16: 53; 52, 55; 53 and 33; 32 (heads of 64), 32: 96; 90 (fp16),
// 64: 132; 124 and 189; 186 (in 32s), 128: 245; 211.  Two tiles of larger heads do not fit the registers.
bool pairs(const gptq_kv_cache &c, int64_t cols) { return cols > 16 && c.head_dim <= 128; }
Plan plan_of(const gptq_kv_cache &c, int64_t n_seq, int64_t cols, int64_t max_len) {
    const bool long_waves = n_seq * ceil_div(max_len, kKvTile) * c.n_heads * ceil_div(cols, 32) >= 16 * 2048;
    return plan_with(pairs(c, cols) && long_waves ? 2 : 1, c, n_seq, cols, max_len);
}

template <int D64, int NG, int NT>
hipError_t launch_tiles(AttnArgs a, const Plan &p, int n_seq, bool weights, hipStream_t s) {
    const size_t lds = (size_t)kKvWaves * (a.kept_cols * 64 * D64 * 4 + 16 * 8 + sizeof(TileGrids<NG>)) + (queries_in_lds(D64, NG, NT) ? (size_t)NT * 2 * D64 * 1024 : 0);
    (a.bf16 ? attention_kernel<D64, NG, NT, true> : attention_kernel<D64, NG, NT, false>)<<<
        dim3((unsigned)p.items, (unsigned)a.pool.heads, (unsigned)ceil_div(a.cols, 16 * NT)), kKvThreads, lds, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (weights) {
        const int combining = p.direct ? 0 : a.cols * a.pool.heads * n_seq;
        finish_kernel<D64, NG><<<dim3((unsigned)(combining + p.weigh_items * a.pool.heads)), kKvThreads, (size_t)weigh_bytes<D64, NG>(a.weigh_tiles), s>>>(a, combining);
    } else if (!p.direct) {
        combine_kernel<D64><<<dim3((unsigned)a.cols, (unsigned)a.pool.heads, (unsigned)n_seq), kKvThreads, 0, s>>>(a);
    }
    return hipGetLastError();
}
template <int D64, int NG>
hipError_t launch_attention(const AttnArgs &a, const Plan &p, int n_seq, bool weights, hipStream_t s) {
    if constexpr (D64 <= 2) {
        if (p.nt == 2) return launch_tiles<D64, NG, 2>(a, p, n_seq, weights, s);
    }
    return launch_tiles<D64, NG, 1>(a, p, n_seq, weights, s);
}

}  // namespace

size_t kv_attention_ws_bytes(const gptq_kv_cache &c, int64_t n_seq, int64_t n, int64_t q_heads, int64_t max_len) {
    // (either column tiling's, so that fewer sequences or tokens never need more)
    const int64_t cols = n * (q_heads / c.n_heads);
    size_t most = 0;
    for (int nt = 1; nt <= (pairs(c, cols) ? 2 : 1); ++nt) {
        const Plan p = plan_with(nt, c, n_seq, cols, max_len);
        most = std::max(most, p.part + p.stat + p.last);
    }
    return most;
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
    a.last = weights ? reinterpret_cast<float2 *>(static_cast<char *>(ws) + p.part + p.stat) : nullptr;
    a.scale = scale * 1.44269504088896340736f;
    a.decay = decay;
    a.target = p.target;
    a.least = p.least;
    a.kept_cols = std::min(a.cols, 16);
    a.weigh_target = p.weigh_target;
    a.weigh_tiles = (int)std::min<int64_t>(ceil_div(a.cols, 16), kWeighTiles);
    a.bf16 = dt == GPTQ_DT_BF16;
    a.direct = p.direct;
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
