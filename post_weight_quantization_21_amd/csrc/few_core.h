// Products of at most sixteen rows of activations with packed b-bit weights
// (b = 2, 3, 4, 8): the part one wave computes, shared by the matrix-vector
// products (gemv.hip) and the experts' products (moe.hip).
//
//   acc[m][o] = sum_k x[m][k] (q[o][k] - z[o][k/g]) s[o][k/g]
//
// A row's codes are a little-endian bit stream; 32 codes (a "unit") are b whole
// words.  A wave owns 16 weight rows per tile and walks K in steps of 128
// columns: lane l = 16 kb + r reads unit 4 step + kb of row r and turns it into
// four fragments of eight 16-bit floats; v_mfma_f32_16x16x32 multiplies a
// fragment (lane: column r of B, eight K values) with the same columns of x
// (lane: row m = l % 16 of A).  Which K a slot holds does not matter as long as
// x and the weights agree, so a fragment takes the codes in whatever order they
// unpack cheapest, and x follows.
//
// The result has its weight row in the lane's column (D[4 kb + i][r], i = 0..3,
// m = 4 kb + i), so scale and zero are one value per lane.  The matrix cores
// are not what bounds these products: at full HBM rate they are busy a quarter
// of the time for one token as for sixteen, so M <= 16 runs on them throughout.
#pragma once

#include <algorithm>

#include "common.h"

namespace gptq {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kFewRows = 16;    // rows of activations
constexpr int kTileRows = 16;   // weight rows of a tile
constexpr int kUnit = 32;       // codes of a unit: b words
constexpr int kStep = 128;      // columns of a step: one unit per lane row
constexpr int64_t kFewMaxIn = (int64_t)1 << 20;  // columns a packed matrix may have (32-bit offsets within a row)

// Exact quotients n / d of small numbers: n, d < 2^15 (units and steps of a row).
struct SmallDiv {
    uint32_t magic;  // floor(2^32 / d) + 1, or 0 for d = 1
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return magic ? __umulhi(n, magic) : n; }
};
inline SmallDiv small_div(uint32_t d) { return {d <= 1 ? 0u : (uint32_t)((uint64_t(1) << 32) / d + 1)}; }

// One stack of packed matrices as the kernels see it.
struct PackedDev {
    const uint32_t *packed;
    const float *scales, *zeros;
    int32_t d_out, words, groups;  // rows, words per row, groups per row
    int32_t units;                 // units per row (d_in / 32)
    int32_t split;                 // a group ends inside a step: fold per unit
    SmallDiv by;                   // steps (split: units) per group
};

PackedDev packed_dev(const gptq_packed &w);  // gemv.hip

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void swap32(uint32_t &a, uint32_t &b) {  // a's upper half with b's lower half
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t &a, uint32_t &b) {  // a's odd rows of 16 lanes with b's even rows
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
// Registers i x lane rows kb transposed: out[i] in lane row kb = in[kb] of lane row i.
__device__ __forceinline__ void transpose4(uint32_t &a, uint32_t &b, uint32_t &c, uint32_t &d) {
    swap32(a, c);
    swap32(b, d);
    swap16(a, b);
    swap16(c, d);
}
// out[j] = v of lane row j, in every lane row.
__device__ __forceinline__ void spread4(float v, float out[4]) {
    uint32_t a = __float_as_uint(v), b = a;
    swap32(a, b);
    uint32_t c = a, d = b;
    swap16(a, c);
    swap16(b, d);
    out[0] = __uint_as_float(a);
    out[1] = __uint_as_float(c);
    out[2] = __uint_as_float(b);
    out[3] = __uint_as_float(d);
}

template <typename T>
struct Vec8;
template <>
struct Vec8<_Float16> {
    typedef f16x8 V;
    __device__ static floatx4 mma(V a, V b, floatx4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
};
template <>
struct Vec8<__bf16> {
    typedef bf16x8 V;
    __device__ static floatx4 mma(V a, V b, floatx4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
};

// Bits [at, at + b) of a unit, at a compile-time position.
template <int b>
__device__ __forceinline__ uint32_t code_at(const uint32_t *w, int c) {
    const int at = b * c, i = at >> 5, sh = at & 31;
    uint32_t v = sh + b > 32 ? __builtin_amdgcn_alignbit(w[i + 1], w[i], sh) : w[i] >> sh;
    return sh + b == 32 ? v : v & ((1u << b) - 1u);
}

// Fragment i of a unit (eight codes) as 16-bit floats of which column j comes
// from code col(i, j).  fp16 gives q - z, exactly: masking a code into mantissa
// bits [s, s + b) of an fp16 with exponent 10 makes 1024 + q 2^s, and a packed
// multiply-add with 2^-s takes the rest away without rounding.  bf16 has no
// packed arithmetic, so it gives 2^b + q (the code shifted to the top of the
// mantissa) and the caller takes (2^b + z) sum x away with one more matrix
// instruction per fragment, whose B operand is the constant -(2^b + z); only
// the fp32 sums round.  Eight-bit codes fill bf16's significand, so they go
// through fp32: q - z is an integer of at most 255 and exact in bf16.
template <int b, typename T>
struct Codes {
    typedef typename Vec8<T>::V V;
    static constexpr bool kHalf = sizeof(T) == 2 && !__is_same(T, __bf16);
    static constexpr bool kOffset = !kHalf && b < 8;  // fragments hold 2^b + q
    uint32_t magic;
    uint32_t zb;       // offset form: the pair -(2^b + z) in bf16
    f16x2 z16[5];      // fp16: the pair 2^(10 - s) + z for s = 0, 2, 4, 6, 8
    float z;

    __device__ __forceinline__ Codes() {
        magic = kHalf ? 0x64006400u : (uint32_t)(0x3F80 + 128 * b) * 0x10001u;  // fp16 1024, bf16 2^b
        asm volatile("" : "+v"(magic));  // a register operand: VOP3 takes no literal
    }
    __device__ __forceinline__ void set_zero(float zero) {
        z = zero;
        if constexpr (kOffset) {
            zb = __builtin_bit_cast(uint32_t, (bf16x2){(__bf16)(-((float)(1 << b) + zero)), (__bf16)(-((float)(1 << b) + zero))});
        }
        if constexpr (kHalf) {
#pragma unroll
            for (int i = 0; i < 5; ++i) {
                const _Float16 v = (_Float16)((float)(1024 >> (2 * i)) + zero);
                z16[i] = (f16x2){v, v};
            }
        }
    }
    __device__ __forceinline__ V zero_frag() const {
        u32x4 v = {zb, zb, zb, zb};
        return __builtin_bit_cast(V, v);
    }
    // Column of the unit that slot j of fragment i holds.
    __host__ __device__ static constexpr int col(int i, int j) {
        if (b == 4) return 8 * i + (j >> 1) + 4 * (j & 1);
        if (b == 2) return 16 * (i >> 1) + 4 * (i & 1) + (j >> 1) + 8 * (j & 1);
        return 8 * i + j;
    }
    // Pair p (slots 2p and 2p + 1) of fragment i.
    __device__ __forceinline__ uint32_t pair(const uint32_t *w, int i, int p) const {
        constexpr uint32_t m = ((1u << b) - 1u) * 0x10001u;
        if constexpr (b == 8) {
            const uint32_t v = w[2 * i + (p >> 1)];
            if constexpr (kHalf) {
                const uint32_t h = __builtin_amdgcn_perm(magic, v, p & 1 ? 0x07030702u : 0x07010700u);
                return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, h) - z16[0]);
            } else {
                const float lo = (float)((v >> (16 * (p & 1))) & 255u) - z, hi = (float)((v >> (16 * (p & 1) + 8)) & 255u) - z;
                return __builtin_bit_cast(uint32_t, (bf16x2){(__bf16)lo, (__bf16)hi});
            }
        } else if constexpr (b == 3) {
            const uint32_t v = code_at<3>(w, 8 * i + 2 * p) | (code_at<3>(w, 8 * i + 2 * p + 1) << 16);
            if constexpr (kHalf) return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, v | magic) - z16[0]);
            return (v << 4) | magic;
        } else {  // codes b c and b c + 16 of a word
            const uint32_t v = b == 4 ? w[i] : w[i >> 1];
            const int at = b == 4 ? 4 * p : 2 * (4 * (i & 1) + p);
            if constexpr (kHalf) {
                const int base = at >= 8 ? 8 : 0, s = at - base;  // masked in place at shifts of 0 .. 6
                const f16x2 h = __builtin_bit_cast(f16x2, ((base ? v >> base : v) & (m << s)) | magic);
                if (s == 0) return __builtin_bit_cast(uint32_t, h - z16[0]);
                const _Float16 f = (_Float16)(1.0f / (float)(1 << s));
                return __builtin_bit_cast(uint32_t, h * (f16x2){f, f} - z16[s / 2]);
            }
            constexpr int top = 7 - b;  // the code's place in the mantissa
            return ((at > top ? v >> (at - top) : v << (top - at)) & (m << top)) | magic;
        }
    }
    __device__ __forceinline__ V frag(const uint32_t *w, int i) const {
        u32x4 v = {pair(w, i, 0), pair(w, i, 1), pair(w, i, 2), pair(w, i, 3)};
        return __builtin_bit_cast(V, v);
    }
    // Fragment i of x from the unit's 32 columns in their own order (16 words).
    __device__ __forceinline__ static V xfrag(const uint32_t *x, int i) {
        u32x4 v;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int c0 = col(i, 2 * p), c1 = col(i, 2 * p + 1);
            if (c1 == c0 + 1)
                v[p] = x[c0 / 2];
            else
                v[p] = __builtin_amdgcn_perm(x[c1 / 2], x[c0 / 2], c0 & 1 ? 0x07060302u : 0x05040100u);
        }
        return __builtin_bit_cast(V, v);
    }
};

template <typename V>
__device__ __forceinline__ void transpose_frags(V f[4]) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        u32x4 a = __builtin_bit_cast(u32x4, f[0]), c = __builtin_bit_cast(u32x4, f[1]);
        u32x4 d = __builtin_bit_cast(u32x4, f[2]), e = __builtin_bit_cast(u32x4, f[3]);
        uint32_t q0 = a[p], q1 = c[p], q2 = d[p], q3 = e[p];
        transpose4(q0, q1, q2, q3);
        a[p] = q0;
        c[p] = q1;
        d[p] = q2;
        e[p] = q3;
        f[0] = __builtin_bit_cast(V, a);
        f[1] = __builtin_bit_cast(V, c);
        f[2] = __builtin_bit_cast(V, d);
        f[3] = __builtin_bit_cast(V, e);
    }
}

template <int b>
__device__ __forceinline__ void load_unit(const uint32_t *p, uint32_t *w) {
    if constexpr (b == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x, w[1] = v.y;
    } else if constexpr (b == 3) {
        const uint3 v = *reinterpret_cast<const uint3 *>(p);  // 4-byte aligned: a row of 32 n codes is 12 n bytes
        w[0] = v.x, w[1] = v.y, w[2] = v.z;
    } else {
#pragma unroll
        for (int i = 0; i < b / 4; ++i) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p + 4 * i);
            w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
    }
}

// How a workgroup of kFewWaves waves shares a product: 2^lg waves (slices) split
// K between them on each of kFewWaves >> lg row tiles.
constexpr int kFewWaves = 8;
constexpr int kFewThreads = kFewWaves * kWave;
constexpr int kFewOccupancy = 4;             // waves per SIMD, which the kernels' registers allow
constexpr int kFewResident = 256 * 4 * kFewOccupancy;  // waves of the chip at once
// x is staged in LDS in chunks, a unit of a row per thread, two buffers.
constexpr int kXPad = 8;  // values after each staged row: sixteen rows start in different banks

// Rows of activations: row m of plane p is base + p * plane + row(m) * ld.
struct XRows {
    const uint16_t *base;
    int64_t ld, plane;
    bool gathered;  // rows are numbered by `row` of lane m, else m itself
    int32_t row;
};

__host__ __device__ inline int ceil_log2(int n) { return n <= 1 ? 0 : 32 - __builtin_clz((unsigned)(n - 1)); }
// Steps of K that a chunk of `rows` staged rows (P M) holds, at most all of them.
__host__ __device__ inline int chunk_steps(int rows, int steps) {
    const int c = (kFewThreads / 4) >> ceil_log2(rows);
    return c < steps ? c : steps;
}
__host__ __device__ inline int staged_ld(int chunk) { return chunk * kStep + kXPad; }
// LDS bytes of a product of 1 .. max_rows rows of `planes` planes: the staged
// activations, or the waves' sums after it.
inline size_t few_lds_bytes(int max_rows, int planes, int units) {
    const int steps = (units + 3) / 4;
    size_t bytes = (size_t)kFewWaves * max_rows * kTileRows * 4;
    for (int m = 1; m <= max_rows; ++m) {
        const int chunk = chunk_steps(planes * m, steps);
        const size_t one = (size_t)planes * m * staged_ld(chunk) * 2;
        bytes = std::max(bytes, chunk < steps ? 2 * one : one);
    }
    return bytes;
}

// Columns [128 c0, 128 (c0 + n)) of the M rows (P planes of them) staged for the
// matrix cores: row-major, each unit's four fragments in slot order, zeros past
// the last unit (a step may hold fewer than four).
template <int b, typename T, int P>
struct StageX {
    typedef typename Vec8<T>::V V;
    int r, u;             // the thread's staged row (r >= P M: none) and its unit in the chunk
    const uint16_t *src;  // the row's columns
    uint4 v[4];
    __device__ __forceinline__ void init(const XRows &x, int M) {
        const int lg = 9 - ceil_log2(P * M);  // log2 of the threads per row
        static_assert(kFewThreads == 512, "threads per row");
        r = threadIdx.x >> lg;
        u = threadIdx.x & ((1 << lg) - 1);
        const int p = P == 1 ? 0 : (r >= M) + (P > 2 && r >= 2 * M), m = r - p * M;
        const int row = x.gathered ? __shfl(x.row, m) : m;
        src = x.base + (r < P * M ? p * x.plane + row * x.ld : 0);
    }
    __device__ __forceinline__ void load(int M, int c0, int n, int units) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = make_uint4(0, 0, 0, 0);
        if (r < P * M && u < 4 * n && 4 * c0 + u < units) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = reinterpret_cast<const uint4 *>(src + (4 * c0 + u) * kUnit)[i];
        }
    }
    __device__ __forceinline__ void store(uint16_t *xs, int M, int n, int ld) const {
        if (r >= P * M || u >= 4 * n) return;
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[4 * i] = v[i].x, w[4 * i + 1] = v[i].y, w[4 * i + 2] = v[i].z, w[4 * i + 3] = v[i].w;
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<V *>(xs + r * ld + u * kUnit + 8 * i) = Codes<b, T>::xfrag(w, i);
    }
};

// The wave's sums for a tile of 16 weight rows over its slice of K, from x
// staged chunk by chunk; every wave of the workgroup calls it, with the same x.
// row0: the tile's first row in the stack w, rows: its rows there.  kSplit:
// groups end inside a step, so the fragments of the four lane rows are
// transposed to make each matrix instruction cover one unit, and the fold with
// the scale runs per unit; otherwise it runs per step.
//
// The weights stream through registers: a body of S steps is loaded while the
// one before it is computed, so a wave keeps S to 2S KB (4 bits) in flight.
// Scales and zeros come with it: without kSplit lane row kb reads those of step
// kb of the body and the rows trade them (spread4), one load for four steps.
template <int b, typename T, int P, bool kSplit>
__device__ __forceinline__ floatx4 few_product(const PackedDev &w, int64_t row0, int rows, const XRows &x, int M,
                                               int slice, int lg, uint16_t *lds) {
    typedef typename Vec8<T>::V V;
    typedef Codes<b, T> C;
    constexpr int S = b == 8 || (kSplit && P > 1) ? 2 : 4;
    constexpr int NS = kSplit ? S : 1;
    const int lane = threadIdx.x % kWave, kb = lane >> 4;
    const int units = w.units, steps = (units + 3) / 4;
    const int chunk = chunk_steps(P * M, steps), ld = staged_ld(chunk);
    const int rl = std::min(lane & 15, rows - 1);
    const uint32_t *wp = w.packed + row0 * w.words + (int64_t)rl * w.words;
    const float *sp = w.scales + row0 * w.groups + rl * w.groups, *zp = w.zeros + row0 * w.groups + rl * w.groups;
    const SmallDiv by = w.by;
    struct Body {
        uint32_t w[S][b];
        float s[NS], z[NS];
    } nxt, cur;
    auto load = [&](Body &d, int step) {
#pragma unroll
        for (int j = 0; j < S; ++j) {
            const int u = std::min(4 * (step + j) + kb, units - 1);  // past the end: loaded again, not used
            load_unit<b>(wp + u * b, d.w[j]);
            if constexpr (kSplit) {
                const uint32_t gi = by.div(u);
                d.s[j] = sp[gi], d.z[j] = zp[gi];
            }
        }
        if constexpr (!kSplit) {
            const uint32_t gi = by.div(std::min(step + (kb & (S - 1)), steps - 1));
            d.s[0] = sp[gi], d.z[0] = zp[gi];
        }
    };
    floatx4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    StageX<b, T, P> stage;
    stage.init(x, M);
    stage.load(M, 0, chunk, units);
    int s = slice * chunk >> lg, end = (slice + 1) * chunk >> lg;  // of the first chunk
    load(nxt, s);
    stage.store(lds, M, chunk, ld);
    __syncthreads();
    uint16_t *buf = lds, *other = lds + P * M * ld;
    C codes;
    const int m = std::min(lane & 15, M - 1);
    for (int c0 = 0; c0 < steps; c0 += chunk) {
        const int c1 = c0 + chunk, n1 = std::min(chunk, steps - c1);  // the next chunk, if n1 > 0
        if (n1 > 0) stage.load(M, c1, n1, units);
        const int next = c1 + (slice * n1 >> lg);
        const uint16_t *xl = buf + m * ld + kb * (kSplit ? 8 : kUnit);
        if (s >= end) load(nxt, next);  // fewer steps than slices: nothing here for this wave
        for (; s < end; s += S) {
            cur = nxt;
            load(nxt, s + S < end ? s + S : next);
            float sc[4], zc[4];
            if constexpr (!kSplit) {
                spread4(cur.s[0], sc);
                spread4(cur.z[0], zc);
            }
#pragma unroll
            for (int j = 0; j < S; ++j) {
                if (s + j >= end) break;
                V xf[P][4];
#pragma unroll
                for (int p = 0; p < P; ++p)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        xf[p][i] = *reinterpret_cast<const V *>(xl + p * M * ld + (s + j - c0) * kStep + i * (kSplit ? kUnit : 8));
                V wf[4];
                if constexpr (kSplit) {
                    if constexpr (!C::kOffset) codes.set_zero(cur.z[j]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) wf[i] = codes.frag(cur.w[j], i);
                    spread4(cur.s[j], sc);
                    if constexpr (C::kOffset) spread4(cur.z[j], zc);
                    transpose_frags(wf);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        floatx4 g = {0.0f, 0.0f, 0.0f, 0.0f};
                        if constexpr (C::kOffset) codes.set_zero(zc[i]);
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            if constexpr (C::kOffset) g = Vec8<T>::mma(xf[p][i], codes.zero_frag(), g);
                            g = Vec8<T>::mma(xf[p][i], wf[i], g);
                        }
#pragma unroll
                        for (int t = 0; t < 4; ++t) acc[t] = fmaf(sc[i], g[t], acc[t]);
                    }
                } else {
                    codes.set_zero(zc[j]);
                    floatx4 g = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        wf[i] = codes.frag(cur.w[j], i);
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            if constexpr (C::kOffset) g = Vec8<T>::mma(xf[p][i], codes.zero_frag(), g);
                            g = Vec8<T>::mma(xf[p][i], wf[i], g);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < 4; ++t) acc[t] = fmaf(sc[j], g[t], acc[t]);
                }
            }
        }
        if (n1 > 0) {
            stage.store(other, M, n1, ld);
            __syncthreads();  // the next chunk is staged; this one's buffer is written again a barrier later
            uint16_t *t = buf;
            buf = other;
            other = t;
            s = next;
            end = c1 + ((slice + 1) * n1 >> lg);
        }
    }
    return acc;
}

// The waves' sums through LDS: after it, sums[(wave * M + m) * 16 + row] of the workgroup.
__device__ __forceinline__ void few_share(float *sums, int wave, const floatx4 &acc, int M) {
    const int lane = threadIdx.x % kWave;
    __syncthreads();  // the staged activations are no longer read
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int m = 4 * (lane >> 4) + t;
        if (m < M) sums[(wave * M + m) * kTileRows + (lane & 15)] = acc[t];
    }
    __syncthreads();
}
// Sum over the 2^lg waves from `wave` on of row c of their tile and token m.
__device__ __forceinline__ float few_sum(const float *sums, int wave, int lg, int M, int m, int c) {
    float v = 0.0f;
    for (int k = 0; k < 1 << lg; ++k) v += sums[((wave + k) * M + m) * kTileRows + c];
    return v;
}
// The wave's number in the workgroup, known to be the same in all its lanes.
__device__ __forceinline__ int few_wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x / kWave); }

// log2 of the waves that split K for one row tile, at most `most`: as many as
// `tiles` tiles leave room for on the chip at once while a wave keeps a body of steps.
int few_slices(int64_t tiles, int units, int most);

// Rounding of a result to the output's type, to nearest even.
__device__ __forceinline__ void store_as(void *y, int64_t i, gptq_dtype dt, float v) {
    if (dt == GPTQ_DT_F32)
        static_cast<float *>(y)[i] = v;
    else if (dt == GPTQ_DT_BF16)
        static_cast<__bf16 *>(y)[i] = (__bf16)v;
    else
        static_cast<_Float16 *>(y)[i] = (_Float16)v;
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + expf(-g)) * u; }

}  // namespace gptq
