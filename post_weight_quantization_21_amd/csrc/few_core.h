// Products of at most sixteen rows of activations with packed b-bit weights
// (b = 2, 3, 4, 8), shared by the matrix-vector products (gemv.hip) and the
// experts' products (moe.hip).
//
//   acc[m][o] = sum_k x[m][k] (q[o][k] - z[o][k/g]) s[o][k/g]
//
// A row's codes are a little-endian bit stream; 32 codes (a "unit") are b whole
// words.  A wave owns a tile of 16 weight rows and walks K in steps of 128
// columns, four steps a quad: lane l = 16 kb + r reads unit 4 step + kb of row r
// and turns it into four fragments of eight 16-bit floats; v_mfma_f32_16x16x32
// multiplies a fragment (lane: column r of B, eight K values) with the same
// columns of x (lane: row m = l % 16 of A).  Which K a slot holds does not
// matter as long as x and the weights agree, so a fragment takes the codes in
// whatever order they unpack cheapest, and x follows ("prepared" x, below).
//
// The result has its weight row in the lane's column (D[4 kb + i][r], i = 0..3,
// m = 4 kb + i), so scale and zero are one value per lane.
//
// What bounds it: start and staging where the layer is small, its bytes where it is
// large, and beside them the instructions that unpack: one token of 28672 x 8192
// issues 75 vector instructions per step of 16 x 128 codes (36-40 unpack), which
// keep the vector units busy for 0.38 of the time, and eight gated tokens in groups
// of 64 issue 115 for 0.55 of it (counters).  Hence scales and zero constants come
// ready from LDS, weights through buffer loads with scalar offsets, and two quads of
// registers take turns without copies.  The matrix cores are busy for 0.03 to 0.16
// of the time, so all M run on them.
#pragma once

#include <algorithm>

#include "common.h"

namespace gptq {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x3 __attribute__((ext_vector_type(3)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kFewRows = 16;   // rows of activations
constexpr int kTileRows = 16;  // weight rows of a tile
constexpr int kUnit = 32;      // codes of a unit: b words
constexpr int kStep = 128;     // columns of a step: one unit per lane row
constexpr int kQuad = 512;     // columns of a quad of steps: what a wave takes at least

// How a workgroup of kFewWaves waves shares a product: 2^lg waves (slices) split
// K between them on each of kFewWaves >> lg row tiles.
constexpr int kFewWaves = 8;
constexpr int kFewThreads = kFewWaves * kWave;
constexpr int kFewOccupancy = 4;                       // waves per SIMD, which the kernels' registers allow
constexpr int kFewResident = 256 * 4 * kFewOccupancy;  // waves of the chip at once

// LDS of a workgroup: the waves' sums, then, for a phase of quads, the scales and
// zero constants of its rows and x.  Two workgroups share a compute unit's 160
// KB; one takes most of it where there are no more workgroups than compute units.
constexpr int kSumsBytes = kFewWaves * kFewRows * kTileRows * 4;
constexpr int kLdsShared = 80 * 1024, kLdsAlone = 156 * 1024;

__host__ __device__ inline int few_steps(int units) { return (units + 3) / 4; }
__host__ __device__ inline int few_quads(int units) { return (units + 15) / 16; }
__host__ __device__ inline int ceil_log2(int n) { return n <= 1 ? 0 : 32 - __builtin_clz((unsigned)(n - 1)); }

// Exact quotients n / d of small numbers: n, d < 2^15 (units and steps of a row).
struct SmallDiv {
    uint32_t magic;  // floor(2^32 / d) + 1, or 0 for d = 1
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return magic ? __umulhi(n, magic) : n; }
};
inline SmallDiv small_div(uint32_t d) { return {d <= 1 ? 0u : (uint32_t)((uint64_t(1) << 32) / d + 1)}; }

// Stacks of packed matrices as the kernels see them: the pointers, and the shape
// that gate and up share.
struct FewMat {
    const uint32_t *packed;
    const float *scales, *zeros;
};
struct FewShape {
    int32_t d_out, words, groups;  // rows, words per row, groups per row
    int32_t units;                 // units per row (d_in / 32)
    int32_t lg;                    // log2 of the slices
    int32_t lds, quad_entries;     // LDS bytes; bytes of a quad's entries
    SmallDiv by;                   // steps per group, or units per group where groups end inside a step
};
FewMat few_mat(const gptq_packed &w);  // gemv.hip
// tiles: row tiles that share the chip; most: slices at most; rows: of x (all
// its planes) as expected, and at most.
FewShape few_shape(const gptq_packed &w, double tiles, int most, int rows, int max_rows);
// Groups end inside a step: the fragments are transposed so that a matrix
// instruction covers one unit, and the fold with the scale runs per unit.
bool few_split(const gptq_packed &w);

// LDS bytes that a phase does not grow: the sums and the entries' odd row ends.
__host__ __device__ inline int few_fixed(int lg) { return kSumsBytes + (kFewWaves >> lg) * kTileRows * 3 * 8; }
// Quads of a phase: as many as fit.
__host__ __device__ inline int few_phase(const FewShape &w, int rows) {
    const int q = (w.lds - few_fixed(w.lg)) / (rows * kQuad * 2 + w.quad_entries), quads = few_quads(w.units);
    return q < quads ? q : quads;
}

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

// Column of its unit that slot j of fragment f holds, and the way back.
template <int b>
__host__ __device__ constexpr int slot_col(int f, int j) {
    if (b == 4) return 8 * f + (j >> 1) + 4 * (j & 1);
    if (b == 2) return 16 * (f >> 1) + 4 * (f & 1) + (j >> 1) + 8 * (j & 1);
    return 8 * f + j;
}
template <int b>
__host__ __device__ constexpr int col_slot(int c) {  // 8 f + j
    if (b == 4) return (c & ~7) + 2 * (c & 3) + (c >> 2 & 1);
    if (b == 2) return (c & 16) + 8 * (c >> 2 & 1) + 2 * (c & 3) + (c >> 3 & 1);
    return c;
}

// Bits [b c, b c + b) of a unit, at a compile-time position.
template <int b>
__device__ __forceinline__ uint32_t code_at(const uint32_t *w, int c) {
    const int at = b * c, i = at >> 5, sh = at & 31;
    uint32_t v = sh + b > 32 ? __builtin_amdgcn_alignbit(w[i + 1], w[i], sh) : w[i] >> sh;
    return sh + b == 32 ? v : v & ((1u << b) - 1u);
}

// Fragment f of a unit (eight codes) as 16-bit floats.  fp16 gives q - z,
// exactly: masking a code into mantissa bits [s, s + b) of an fp16 with exponent
// 10 makes 1024 + q 2^s, and a packed multiply-add with 2^-s takes the rest away
// without rounding.  bf16 has no packed arithmetic, so it gives 2^b + q (the code
// shifted to the top of the mantissa) and the caller takes (2^b + z) sum x away
// with one more matrix instruction per fragment, whose B operand is the constant
// -(2^b + z); only the fp32 sums round.  Eight-bit codes fill bf16's significand,
// so they go through fp32: q - z is an integer of at most 255 and exact in bf16.
// bf16's 2^b + q and 2^b + z are held less an exponent, below 1, and the sums are
// multiplied by kScaled at the end: x may be as large as fp32 itself holds, and
// products with 2^b + q would leave fp32 where the result does not.  (Of eight bits, whose x may
// be 2^8 times smaller, that multiply-add with a literal instead of a subtraction
// takes 13.2 us instead of 11.4 for seven tokens of 5003 x 2720.)
template <int b, typename T>
struct Codes {
    typedef typename Vec8<T>::V V;
    static constexpr bool kF16 = __is_same(T, _Float16);
    static constexpr bool kOffset = !kF16 && b < 8;  // fragments hold 2^b + q
    static constexpr float kScaled = 2 << b;  // a power of two: nothing rounds
    uint32_t magic;
    uint32_t zc;  // constant(z)
    f16x2 z2;     // fp16, two bits: 256 + z, 16 + z

    __device__ __forceinline__ Codes() {
        magic = kF16 ? 0x64006400u : 0x3F003F00u;  // fp16 1024, bf16 2^b / kScaled
        asm volatile("" : "+v"(magic));  // a register operand: VOP3 takes no literal
    }
    // What the unpacking needs of a zero point: fp16 the pair 1024 + z, 64 + z;
    // bf16 twice -(2^b + z) / kScaled; bf16 of eight bits z in fp32.
    __device__ __forceinline__ static uint32_t constant(float z) {
        if constexpr (kF16) return __builtin_bit_cast(uint32_t, (f16x2){(_Float16)(1024.0f + z), (_Float16)(64.0f + z)});
        if constexpr (!kOffset) return __float_as_uint(z);
        const __bf16 v = (__bf16)fmaf(z, -1.0f / kScaled, -0.5f);
        return __builtin_bit_cast(uint32_t, (bf16x2){v, v});
    }
    __device__ __forceinline__ void set(uint32_t c) {
        zc = c;
        if constexpr (kF16 && b == 2) z2 = __builtin_bit_cast(f16x2, c) - (f16x2){(_Float16)768.0f, (_Float16)48.0f};
    }
    __device__ __forceinline__ V zero_frag() const {
        const u32x4 v = {zc, zc, zc, zc};
        return __builtin_bit_cast(V, v);
    }
    // 2^(10 - s) + z, twice
    __device__ __forceinline__ f16x2 bias(int s) const {
        const f16x2 z = __builtin_bit_cast(f16x2, zc);
        const _Float16 v = s == 0 ? z[0] : (s == 4 ? z[1] : (s == 2 ? z2[0] : z2[1]));
        return (f16x2){v, v};
    }
    // Pair p (slots 2p and 2p + 1) of fragment f.
    __device__ __forceinline__ uint32_t pair(const uint32_t *w, int f, int p) const {
        constexpr uint32_t m = ((1u << b) - 1u) * 0x10001u;
        if constexpr (b == 8) {
            const uint32_t v = w[2 * f + (p >> 1)];
            if constexpr (kF16) {
                const uint32_t h = __builtin_amdgcn_perm(magic, v, p & 1 ? 0x07030702u : 0x07010700u);
                return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, h) - bias(0));
            } else {
                const float z = __uint_as_float(zc);
                const float lo = (float)((v >> (16 * (p & 1))) & 255u) - z, hi = (float)((v >> (16 * (p & 1) + 8)) & 255u) - z;
                return __builtin_bit_cast(uint32_t, (bf16x2){(__bf16)lo, (__bf16)hi});
            }
        } else if constexpr (b == 3) {
            const uint32_t v = code_at<3>(w, 8 * f + 2 * p) | (code_at<3>(w, 8 * f + 2 * p + 1) << 16);
            if constexpr (kF16) return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, v | magic) - bias(0));
            return (v << 4) | magic;
        } else {  // codes b c and b c + 16 of a word
            const uint32_t v = b == 4 ? w[f] : w[f >> 1];
            const int at = b == 4 ? 4 * p : 2 * (4 * (f & 1) + p);
            if constexpr (kF16) {
                const int base = at >= 8 ? 8 : 0, s = at - base;  // masked in place at shifts of 0 .. 6
                const f16x2 h = __builtin_bit_cast(f16x2, ((base ? v >> base : v) & (m << s)) | magic);
                if (s == 0) return __builtin_bit_cast(uint32_t, h - bias(0));
                const _Float16 r = (_Float16)(1.0f / (float)(1 << s));
                return __builtin_bit_cast(uint32_t, h * (f16x2){r, r} - bias(s));
            }
            constexpr int top = 7 - b;  // the code's place in the mantissa
            return ((at > top ? v >> (at - top) : v << (top - at)) & (m << top)) | magic;
        }
    }
    __device__ __forceinline__ V frag(const uint32_t *w, int f) const {
        const u32x4 v = {pair(w, f, 0), pair(w, f, 1), pair(w, f, 2), pair(w, f, 3)};
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

// A unit's words through a buffer descriptor: `at` not below the descriptor's
// size reads nothing and gives zeros, whether or not the hardware counts the
// scalar offset `base` in, as long as base alone is no more than that size.
template <int b>
__device__ __forceinline__ void load_unit(__amdgpu_buffer_rsrc_t p, uint32_t at, uint32_t base, uint32_t *w) {
    if constexpr (b == 2) {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(p, at, base, 0);
        w[0] = v[0], w[1] = v[1];
    } else if constexpr (b == 3) {
        const u32x3 v = __builtin_amdgcn_raw_buffer_load_b96(p, at, base, 0);
        w[0] = v[0], w[1] = v[1], w[2] = v[2];
    } else {
#pragma unroll
        for (int i = 0; i < b / 4; ++i) {
            const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(p, at + 16 * i, base, 0);
            w[4 * i] = v[0], w[4 * i + 1] = v[1], w[4 * i + 2] = v[2], w[4 * i + 3] = v[3];
        }
    }
}

// Prepared x: M rows of whole quads as pieces of eight 16-bit values in slot
// order, piece (4 (4 step + u) + f) M + m holding fragment f of unit u of row m;
// columns past the last unit are zero.  A lane's operand of a matrix instruction
// is one piece, the rows of a lane row next to each other.
__host__ __device__ inline int64_t prepared_values(int64_t rows, int units) { return rows * few_quads(units) * kQuad; }
template <int b>
__device__ __forceinline__ int64_t prepared_at(int col, int M, int m) {
    const int s = col_slot<b>(col % kUnit);
    return ((int64_t)(col / kUnit * 4 + (s >> 3)) * M + m) * 8 + (s & 7);
}

// Activations of a product: rows as they are, rows whose columns are read in
// packed order, prepared in memory, or fp32 rows, which become two planes of fp16
// that follow each other in LDS: each value times its row's power of two rounded
// to fp16, and the rest rounded to fp16.
enum FewX { kRawX, kOrderedX, kPreparedX, kFloatX };
struct XRows {
    const void *base;
    int64_t ld;            // between rows (not prepared)
    bool gathered;         // raw and ordered: rows are numbered by `row` of lane m, else m itself
    int32_t row;
    const int32_t *order;  // ordered: x's column of each packed one
    float scale;           // fp32: the power of two of row m in lane m
};

// A phase's x on its way into LDS, in batches of a unit a thread (fp32: half of one).
template <int b, FewX kX>
struct StageX {
    u32x4 v[4];
    uint32_t magic;                    // raw: of the division by the units of a row; fp32: by its pieces
    int per_row, items, first, total;  // units of a row and of all in the phase, its first unit, batches
    __device__ __forceinline__ void init(int M, int units, int q0, int nq) {
        per_row = 16 * nq;
        magic = 0xFFFFFFFFu / (uint32_t)(kX == kFloatX ? 4 * per_row : per_row) + 1;
        items = M * per_row;  // units
        first = 16 * q0;
        total = ((kX == kFloatX ? 2 * items : items) + kFewThreads - 1) / kFewThreads;
    }
    // Raw: unit i of the phase is unit u of row r.  Prepared: piece i of the phase, four a thread.  Ordered: pieces as
    // prepared, each gathered value by value.  fp32: piece i, two a thread, is piece p of row r.
    __device__ __forceinline__ void load(const XRows &x, int M, int units, int batch) {
        const uint16_t *base = static_cast<const uint16_t *>(x.base);
        if constexpr (kX == kRawX) {
            const int i = threadIdx.x + batch * kFewThreads;
            const int r = __umulhi(i, magic), u = first + i - r * per_row;
            const int row = x.gathered ? __shfl(x.row, r & (kWave - 1)) : r;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = (u32x4){0, 0, 0, 0};
            if (i < items && u < units) {
                const u32x4 *src = reinterpret_cast<const u32x4 *>(base + row * x.ld + u * kUnit);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = src[j];
            }
        } else if constexpr (kX == kOrderedX) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = threadIdx.x + (4 * batch + j) * kFewThreads, piece = (int)((uint32_t)i / (uint32_t)M);
                const int u = first + (piece >> 2), f = piece & 3, f0 = b == 2 ? 16 * (f >> 1) + 4 * (f & 1) : 8 * f;
                const int r = i - piece * M, m = x.gathered ? __shfl(x.row, r & (kWave - 1)) : r;
                v[j] = (u32x4){0, 0, 0, 0};
                if (i < 4 * items && u < units) {
                    const uint16_t *row = base + m * x.ld;
                    const int32_t *at = x.order + u * kUnit + f0;
                    uint32_t h[8];
#pragma unroll
                    for (int n = 0; n < 8; ++n) h[n] = row[std::min(std::max(at[slot_col<b>(0, n)], 0), units * kUnit - 1)];
                    v[j] = (u32x4){h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16};
                }
            }
        } else if constexpr (kX == kFloatX) {
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                const int i = threadIdx.x + (2 * batch + j / 2) * kFewThreads, r = __umulhi(i, magic), p = i - r * 4 * per_row;
                const int u = first + (p >> 2), f = p & 3, f0 = b == 2 ? 16 * (f >> 1) + 4 * (f & 1) : 8 * f;
                v[j] = v[j + 1] = (u32x4){0, 0, 0, 0};
                if (i < 4 * items && u < units) {
                    const float *src = static_cast<const float *>(x.base) + r * x.ld + u * kUnit + f0;
                    v[j] = *reinterpret_cast<const u32x4 *>(src);  // the piece's two runs of four columns
                    v[j + 1] = *reinterpret_cast<const u32x4 *>(src + (b == 2 ? 8 : 4));
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = threadIdx.x + (4 * batch + j) * kFewThreads;
                v[j] = (u32x4){0, 0, 0, 0};  // (left alone, it would be kept through the phase before)
                if (i < 4 * items) v[j] = *reinterpret_cast<const u32x4 *>(base + ((int64_t)4 * first * M + i) * 8);
            }
        }
    }
    __device__ __forceinline__ void store(uint16_t *xs, const XRows &x, int M, int batch) const {
        u32x4 *dst = reinterpret_cast<u32x4 *>(xs);
        if constexpr (kX == kRawX) {
            const int i = threadIdx.x + batch * kFewThreads;
            const int r = __umulhi(i, magic), u = i - r * per_row;
            if (i >= items) return;
            uint32_t t[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) t[j] = v[j / 4][j % 4];
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                u32x4 o;
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    constexpr int apart = b == 4 ? 4 : 8;
                    const int c0 = slot_col<b>(f, 2 * p), c1 = slot_col<b>(f, 2 * p + 1);
                    o[p] = c1 == c0 + 1 ? t[c0 / 2]
                                        : __builtin_amdgcn_perm(t[(c0 + apart) / 2], t[c0 / 2], c0 & 1 ? 0x07060302u : 0x05040100u);
                }
                dst[(4 * u + f) * M + r] = o;
            }
        } else if constexpr (kX == kFloatX) {
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                const int i = threadIdx.x + (2 * batch + j / 2) * kFewThreads, r = __umulhi(i, magic), p = i - r * 4 * per_row;
                const float scale = __shfl(x.scale, r & (kWave - 1));
                if (i >= 4 * items) continue;
                _Float16 hi[8], lo[8];
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    const int c = slot_col<b>(0, n), run = c >= (b == 2 ? 8 : 4);
                    const float a = __uint_as_float(v[j + run][c & 3]) * scale;
                    hi[n] = (_Float16)a;
                    lo[n] = (_Float16)(a - (float)hi[n]);
                }
                dst[p * M + r] = __builtin_bit_cast(u32x4, (f16x8){hi[0], hi[1], hi[2], hi[3], hi[4], hi[5], hi[6], hi[7]});
                dst[4 * items + p * M + r] = __builtin_bit_cast(u32x4, (f16x8){lo[0], lo[1], lo[2], lo[3], lo[4], lo[5], lo[6], lo[7]});
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = threadIdx.x + (4 * batch + j) * kFewThreads;
                if (i < 4 * items) dst[i] = v[j];
            }
        }
    }
};

// Scales and zero constants of groups [ga, ga + n) of the workgroup's rows into
// LDS, entry row * ld + group, ld odd so that sixteen rows lie in different
// banks.  Row i of the workgroup: row i % 16 of tile i / 16; tile t is that of
// wave t << lg.  (Read where they are used, a few bytes a row at a time, the
// requests at L2 cost 7 of 33 us at 28672 x 8192 with groups of 128, and half
// the time with groups of 64.)
template <int b, typename T, int kMats>
struct StageGroups {
    static constexpr int kBatch = 8;  // loads of a thread before its first store
    const char *sb[kMats], *zb[kMats];  // of row tile 0
    int rows, groups;                   // from row tile 0 to the matrix's end; groups per row
    int ga, n, ld, items, total;        // the phase's groups; entries of a matrix, loads of a thread
    uint32_t magic;                     // of the division by n
    float s[kBatch], z[kBatch];

    __device__ __forceinline__ void init(int first, int last, int count) {
        ga = first;
        n = last - first + 1;
        ld = n | 1;
        magic = n > 1 ? 0xFFFFFFFFu / (uint32_t)n + 1 : 0;
        items = count / kMats * n;
        total = (items + kFewThreads - 1) / kFewThreads * kMats;
    }
    __device__ __forceinline__ int row_of(int i) const { return magic ? __umulhi(i, magic) : i; }
    __device__ __forceinline__ void load(int t0) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            s[k] = z[k] = 0.0f;
            if (t0 + k >= total) continue;
            const int i = threadIdx.x + (t0 + k) / kMats * kFewThreads, r = row_of(i);
            if (i >= items) continue;
            const uint32_t at = 4u * (std::min(r, rows - 1) * groups + ga + i - r * n);
            s[k] = *reinterpret_cast<const float *>(sb[k % kMats] + at);
            z[k] = *reinterpret_cast<const float *>(zb[k % kMats] + at);
        }
    }
    __device__ __forceinline__ void store(uint2 *entries, int t0) const {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (t0 + k >= total) continue;
            const int i = threadIdx.x + (t0 + k) / kMats * kFewThreads, r = row_of(i);
            const int row = kMats > 1 ? (r >> 4) * 32 + k % kMats * 16 + (r & 15) : r;  // of the workgroup
            if (i < items) entries[row * ld + i - r * n] = make_uint2(__float_as_uint(s[k]), Codes<b, T>::constant(z[k]));
        }
    }
};

// The workgroup's product: the calling wave's sums for its tile and slice.
// mats[t % kMats]: the matrix of the workgroup's tile t, whose rows are those of
// row tile t / kMats; row0: the first row of row tile 0 in the stack, rows: from
// there to the matrix's end (at least 1).  Every wave of the workgroup calls it.
//
// K runs in phases whose x and entries fit in LDS (mostly one); in a phase the
// waves of a tile take equal runs of quads.  Weights stream through two sets of
// registers, one computed while the other is loaded (4 to 8 KB of a wave in
// flight at 4 bits); past the wave's run nothing is read.  x is zero past the
// last unit.
template <int b, typename T, int kMats, bool kSplit, FewX kX>
__device__ __forceinline__ floatx4 few_product(const FewMat *mats, const FewShape &w, int64_t row0, int rows, const XRows &x,
                                               int M, int wave, unsigned char *smem) {
    typedef typename Vec8<T>::V V;
    typedef Codes<b, T> C;
    constexpr int P = kX == kFloatX ? 2 : 1;  // planes of x
    const int lane = threadIdx.x % kWave, kb = lane >> 4, lg = w.lg;
    const int units = w.units, quads = few_quads(units), phase_quads = few_phase(w, P * M);
    const int tile = wave >> lg, slice = wave & ((1 << lg) - 1), tiles = kFewWaves >> lg;
    const int m = std::min(lane & 15, M - 1);
    uint16_t *xs = reinterpret_cast<uint16_t *>(smem + kSumsBytes);
    uint2 *entries = reinterpret_cast<uint2 *>(smem + kSumsBytes + phase_quads * P * M * kQuad * 2);
    const FewMat &mat = mats[kMats > 1 ? tile % kMats : 0];
    const int t0 = std::min(tile / kMats * kTileRows, rows - 1), tr = std::min(kTileRows, rows - t0), rl = std::min(lane & 15, tr - 1);
    const uint32_t bytes = 4u * tr * w.words, wo = 4u * (rl * w.words + kb * b);
    const auto wr = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint32_t *>(mat.packed + (row0 + t0) * w.words), 0, bytes, 0x00020000);
    // bytes of prepared x in LDS: the lane's first piece, between its pieces of a step
    const uint32_t xlane = 16u * ((kSplit ? kb : 4 * kb) * M + m), xnext = (kSplit ? 64u : 16u) * M;

    constexpr int kS = b == 8 ? 2 : 4;  // steps of a set of registers
    uint32_t wa[kS][b], wb[kS][b];
    auto load = [&](uint32_t (*dst)[b], int set, int end) {
#pragma unroll
        for (int j = 0; j < kS; ++j) {
            const int u = 4 * (kS * set + j) + kb;
            load_unit<b>(wr, set < end && u < units ? wo : bytes, std::min(16u * b * (kS * set + j), bytes), dst[j]);
        }
    };
    floatx4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    C codes;
    StageX<b, kX> stage;
    StageGroups<b, T, kMats> groups;
#pragma unroll
    for (int k = 0; k < kMats; ++k) {
        groups.sb[k] = reinterpret_cast<const char *>(mats[k].scales + row0 * w.groups);
        groups.zb[k] = reinterpret_cast<const char *>(mats[k].zeros + row0 * w.groups);
    }
    groups.rows = rows;
    groups.groups = w.groups;
    for (int q0 = 0; q0 < quads; q0 += phase_quads) {
        const int nq = std::min(phase_quads, quads - q0);
        const int qs = q0 + (slice * nq >> lg), qe = q0 + ((slice + 1) * nq >> lg);
        const int hs = qs * 4 / kS, he = qe * 4 / kS;
        // the phase's groups: of its first and last column
        const int ga = w.by.div(kSplit ? 16 * q0 : 4 * q0);
        const int gb = w.by.div(kSplit ? std::min(16 * (q0 + nq), units) - 1 : std::min(4 * (q0 + nq), few_steps(units)) - 1);
        if (q0 > 0) __syncthreads();  // the phase before is done with LDS
        // loads return in order: what the barrier waits for goes before the weights
        stage.init(M, units, q0, nq);
        stage.load(x, M, units, 0);
        groups.init(ga, gb, tiles * kTileRows);
        groups.load(0);
        load(wa, hs, he);
        stage.store(xs, x, M, 0);
        groups.store(entries, 0);
        for (int t = 1; t < stage.total; ++t) {
            stage.load(x, M, units, t);
            stage.store(xs, x, M, t);
        }
        for (int t = groups.kBatch; t < groups.total; t += groups.kBatch) {
            groups.load(t);
            groups.store(entries, t);
        }
        load(wb, hs + 1, he);
        __syncthreads();
        const uint2 *el = entries + (tile * kTileRows + (lane & 15)) * groups.ld - ga;
        const char *xb = reinterpret_cast<const char *>(xs);
        const uint32_t xplane = 1024u * nq * M;
        auto set = [&](uint32_t (*wq)[b], int h) {
#pragma unroll
            for (int j = 0; j < kS; ++j) {
                const int step = kS * h + j;
                if (4 * step >= units) break;  // the last quad's steps past the end
                V xf[P][4], wf[4];
                uint32_t at = xlane + 256u * M * (step - 4 * q0);
                asm volatile("" : "+v"(at));  // one address a step: an induction variable each would fill the registers
#pragma unroll
                for (int p = 0; p < P; ++p)
#pragma unroll
                    for (int i = 0; i < 4; ++i) xf[p][i] = *reinterpret_cast<const V *>(xb + (at + p * xplane + i * xnext));
                if constexpr (kSplit) {
                    if constexpr (!C::kOffset) codes.set(el[w.by.div(std::min(4 * step + kb, units - 1))].y);
#pragma unroll
                    for (int i = 0; i < 4; ++i) wf[i] = codes.frag(wq[j], i);
                    transpose_frags(wf);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint2 e = el[w.by.div(std::min(4 * step + i, units - 1))];
                        floatx4 g = {0.0f, 0.0f, 0.0f, 0.0f};
                        if constexpr (C::kOffset) codes.set(e.y);
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            if constexpr (C::kOffset) g = Vec8<T>::mma(xf[p][i], codes.zero_frag(), g);
                            g = Vec8<T>::mma(xf[p][i], wf[i], g);
                        }
#pragma unroll
                        for (int t = 0; t < 4; ++t) acc[t] = fmaf(__uint_as_float(e.x), g[t], acc[t]);
                    }
                } else {
                    const uint2 e = el[w.by.div(step)];
                    codes.set(e.y);
                    floatx4 g[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};  // two chains: half the latency
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        wf[i] = codes.frag(wq[j], i);
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            if constexpr (C::kOffset) g[i & 1] = Vec8<T>::mma(xf[p][i], codes.zero_frag(), g[i & 1]);
                            g[i & 1] = Vec8<T>::mma(xf[p][i], wf[i], g[i & 1]);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < 4; ++t) acc[t] = fmaf(__uint_as_float(e.x), g[0][t] + g[1][t], acc[t]);
                }
            }
        };
        for (int h = hs; h < he; h += 2) {
            set(wa, h);
            load(wa, h + 2, he);
            if (h + 1 >= he) break;
            set(wb, h + 1);
            load(wb, h + 3, he);
        }
    }
    if constexpr (C::kOffset) {
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[t] *= C::kScaled;
    }
    return acc;
}

// The waves' sums through LDS: after it, sums[(wave * M + m) * 16 + row] of the workgroup.
__device__ __forceinline__ void few_share(float *sums, int wave, const floatx4 &acc, int M) {
    const int lane = threadIdx.x % kWave;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int m = 4 * (lane >> 4) + t;
        if (m < M) sums[(wave * M + m) * kTileRows + (lane & 15)] = acc[t];
    }
    __syncthreads();
}
// Sum over the 2^lg waves from `wave` on of row c of their tile and token m.
__device__ __forceinline__ float few_sum(const float *sums, int wave, int lg, int M, int m, int c) {
    float t[kFewWaves];
#pragma unroll
    for (int k = 0; k < kFewWaves; ++k) t[k] = sums[((wave + (k & ((1 << lg) - 1))) * M + m) * kTileRows + c];
    float v = t[0];
#pragma unroll
    for (int k = 1; k < kFewWaves; ++k) v += k >> lg ? 0.0f : t[k];
    return v;
}
// The wave's number in the workgroup, known to be the same in all its lanes.
__device__ __forceinline__ int few_wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x / kWave); }

// Rounding of a result to the output's type, to nearest even.
__device__ __forceinline__ void store_as(void *y, int64_t i, gptq_dtype dt, float v) {
    if (dt == GPTQ_DT_F32)
        static_cast<float *>(y)[i] = v;
    else if (dt == GPTQ_DT_BF16)
        static_cast<__bf16 *>(y)[i] = (__bf16)v;
    else
        static_cast<_Float16 *>(y)[i] = (_Float16)v;
}

// silu(g) u.  Below -80 exp(-g) nears fp32's end (and passes it at -88.7) while u
// may bring the result back: exp(g) in two halves, and 1 + exp(g) is 1.
__device__ __forceinline__ float silu_mul(float g, float u) {
    if (g < -80.0f) {
        const float e = expf(0.5f * g);
        return g * e * (e * u);
    }
    return g / (1.0f + expf(-g)) * u;
}

}  // namespace gptq
