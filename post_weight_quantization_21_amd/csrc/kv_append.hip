// New keys and values into the pages of a 4-bit cache.
//
// A group's grid (all decisions binary32, round half to even):
//   asymmetric  lo = min(min x, 0), hi = max(max x, 0), s = bf16((hi - lo) (1/15)),
//               z = clamp(rint(-lo / s), 0, 15), q = clamp(rint(x / s + z), 0, 15)
//   symmetric   s = bf16(max|x| (1/7)), z = 8, q = clamp(rint(x / s), -7, 7) + 8
// with s = 1 where it would be 0 (1/15 and 1/7: the nearest binary32; a quotient, as the
// layers' grids have it, gives another bf16 number only where it lies halfway between two:
// 0.1 to 0.3 % of asymmetric groups of normally distributed fp16 values, none of bf16 ones
// and no symmetric one).  The scale is rounded before the codes are chosen, so its sixteen
// bits cost no accuracy beyond the last code's (a range may end 0.06 of a step past code
// 15).  A group with a value that is not finite, or whose scale
// is not, is stored with a scale that is no number.
#include "kv_cache.h"

namespace gptq {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

struct AppendArgs {
    KvPool pool;
    KvSeqs seqs;
    const uint16_t *x[2];  // keys, values: [T][ld]
    int64_t ld[2];
    uint16_t *out[2];  // the values as stored, or NULL
    int64_t ld_out[2];
    const int32_t *offs;
    int64_t T, per;  // tokens; tokens of a sequence where there are no offsets
    int32_t bf16, symmetric;
};

// Two values of a word in fp32, and back.
template <bool kBf16>
__device__ __forceinline__ f32x2 unpack2(uint32_t w) {
    if constexpr (kBf16) return (f32x2){__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)};
    return __builtin_convertvector(__builtin_bit_cast(f16x2, w), f32x2);
}
template <bool kBf16>
__device__ __forceinline__ uint32_t pack2(f32x2 v) {
    if constexpr (kBf16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}

// A step of a reduction over neighbouring lanes: the value of the lane's partner.
template <int kStep>
__device__ __forceinline__ float partner(float v) {
    const int x = __float_as_int(v);
    if constexpr (kStep == 16) {
        return __shfl_xor(v, 16);
    } else {  // pairs, quads, halves of eight, halves of a row
        constexpr int ctrl = kStep == 1 ? 0xB1 : kStep == 2 ? 0x4E : kStep == 4 ? 0x141 : 0x140;
        return __int_as_float(__builtin_amdgcn_update_dpp(0, x, ctrl, 0xF, 0xF, true));
    }
}

// The range of a group, which always holds 0, and the sum of its values times 0: no number if one of them is not finite.  (The
// values' own sum reaches both infinities over lanes whose values are finite.)
struct Range {
    float lo, hi, none;
    template <int kStep, int W>  // over W neighbouring lanes
    __device__ __forceinline__ void reduce() {
        if constexpr (kStep < W) {
            lo = fminf(lo, partner<kStep>(lo));
            hi = fmaxf(hi, partner<kStep>(hi));
            none += partner<kStep>(none);
            reduce<2 * kStep, W>();
        }
    }
};

// x / s is the correctly rounded quotient by Markstein's correction, as in quant_grid.h: with r = RN(1 / s) and q = RN(x r),
// RN(q + (x - q s) r).  |x / s| stays below 16, since s comes from the group's own range; scales outside 2^-100 .. 2^100
// are brought back by a power of two m, so that no step over- or underflows (where x / s is tiny, it rounds away anyway).
struct Grid4 {
    float s, m, ss, r, z, lo, hi, zadd;
    bool bad;

    __device__ __forceinline__ Grid4(const Range &g, bool symmetric) {
#pragma clang fp contract(off)
        s = symmetric ? fmaxf(-g.lo, g.hi) * (1.0f / 7.0f) : (g.hi - g.lo) * (1.0f / 15.0f);
        s = (float)(__bf16)s;
        if (s == 0.0f) s = 1.0f;
        bad = !(s < __builtin_inff()) || !(g.none == g.none);
        m = s < 0x1p-100f ? 0x1p100f : s > 0x1p100f ? 0x1p-100f : 1.0f;
        ss = s * m;
        r = 1.0f / ss;
        z = symmetric ? 0.0f : __builtin_amdgcn_fmed3f(rintf(quotient(-g.lo * m)), 0.0f, 15.0f);
        lo = symmetric ? -7.0f : 0.0f;
        hi = symmetric ? 7.0f : 15.0f;
        zadd = symmetric ? 8.0f : 0.0f;
        if (bad) s = __builtin_nanf("");
    }
    __device__ __forceinline__ float quotient(float x) const {
        const float q = x * r;
        return fmaf(fmaf(-q, ss, x), r, q);
    }
    // The code less zadd of x m, and the value that one stands for.
    __device__ __forceinline__ float level(float x) const {
#pragma clang fp contract(off)
        return __builtin_amdgcn_fmed3f(rintf(quotient(x) + z), lo, hi);
    }
    __device__ __forceinline__ float value(float level) const { return s * (level - z); }
    __device__ __forceinline__ uint32_t word() const {
        const uint32_t top = bad ? 0x7FC0u : __float_as_uint(s) >> 16;
        return top << 16 | __builtin_bit_cast(uint16_t, (_Float16)(bad ? 0.0f : 8.0f - (zadd + z)));
    }
};

// Four levels as the codes' sixteen bits, the first lowest (sums below 2^16 are exact).
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float zadd) {
    return (uint32_t)fmaf(fmaf(fmaf(d, 16.0f, c), 16.0f, b), 16.0f, fmaf(zadd, 4369.0f, a));
}

constexpr int kBlockTokens = 32;  // tokens of a workgroup that stages values

// A workgroup takes tokens of one head and side, a thread eight neighbouring dims of one: a word of keys.  Values: eight
// lanes hold a set of 64 dims, lane i dims 16 j + 8 (i % 2) .. + 7 with j = i / 2; they trade words so that each has two
// units of all four j.  Units of neighbouring tokens share sixteen bytes: staged, whole blocks of eight tokens are put
// together in LDS and stored at once, else each token's two bytes are.
//
// Bound by vector instructions and memory alike where tokens are many (270 a thread, two thirds of them choose eight codes
// and their values): 32768 tokens of 8 heads of 128 values with the values returned (305 MB) take 69 us, 4.4 TB/s, and 85
// without staging; by the launch where they are few: 32 tokens of 32 sequences 3.7 us, 4.9 staged.
template <int D64, int GROUP, bool kStaged, bool kBf16>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a) {
    constexpr int D = 64 * D64, NG = D / GROUP, kLanes = D64 == 1 ? 8 : (D64 == 2 ? 16 : 32), kPass = 256 / kLanes;
    constexpr int kPasses = kStaged ? kBlockTokens / kPass : 1, kTokens = kPass * kPasses, kCols = kTokens + 8;
    __shared__ int64_t place[kTokens];  // tokens counted over the pool, of the head; -1: stored nowhere, -2: in no sequence
    __shared__ int whole;               // the slot of the first token where all of them follow it on pages that exist, else -1
    __shared__ __attribute__((aligned(16))) uint16_t units[kStaged ? D / 4 : 1][kCols];
    const bool values = blockIdx.z != 0;
    const int h = blockIdx.y, i = threadIdx.x % kLanes, mask = a.pool.page() - 1;
    const int64_t t0 = (int64_t)blockIdx.x * kTokens;
    u32x4 x[kPasses];
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const int64_t t = t0 + p * kPass + threadIdx.x / kLanes;
        x[p] = (u32x4){};
        if (t < a.T && i < D / 8) x[p] = *reinterpret_cast<const u32x4 *>(a.x[values] + t * a.ld[values] + h * D + 8 * i);
    }
    if (threadIdx.x < 64) {  // the first wave finds the tokens' places
        const int64_t t = t0 + threadIdx.x;
        int b = a.seqs.n, slot = -1;
        if (threadIdx.x < kTokens && t < a.T) {
            if (!a.offs) {
                b = (int)(t / a.per);
                slot = a.seqs.len(b) - (int)((int64_t)(b + 1) * a.per - t);
            } else {
                int lo = 0, hi = a.seqs.n;  // the first sequence that ends behind t
                while (lo < hi) {
                    const int mid = (lo + hi) / 2;
                    if (a.offs[mid + 1] > t)
                        hi = mid;
                    else
                        lo = mid + 1;
                }
                b = lo;
                if (b < a.seqs.n) slot = a.seqs.len(b) - (int)(a.offs[b + 1] - t);
            }
        }
        int page = -1;
        if (b < a.seqs.n && slot >= 0 && slot < a.seqs.capacity) page = a.seqs.page_of(a.pool, a.seqs.table + (int64_t)b * a.seqs.width, slot);
        if (threadIdx.x < kTokens) place[threadIdx.x] = page >= 0 ? a.pool.first(page, h) + (slot & mask) : (b < a.seqs.n ? -1 : -2);
        if constexpr (kStaged) {
            const bool same = b == __shfl(b, 0) && page >= 0;
            const uint64_t all = __ballot(same || threadIdx.x >= kTokens);
            if (threadIdx.x == 0) whole = ~all ? -1 : slot;
        }
    }
    __syncthreads();
    const bool wide = kStaged && values && whole >= 0;
    const int shift = kStaged ? whole & 7 : 0;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const int n = p * kPass + threadIdx.x / kLanes;  // of the workgroup's tokens
        const int64_t t = t0 + n, at = place[n];
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const uint32_t two = x[p][e / 2];
            const f32x2 v = unpack2<kBf16>(two);
            f[e] = v[0], f[e + 1] = v[1];
        }
        Range range = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            range.lo = fminf(range.lo, fminf(f[e], f[e + 1]));
            range.hi = fmaxf(range.hi, fmaxf(f[e], f[e + 1]));
            range.none = fmaf(f[e], 0.0f, fmaf(f[e + 1], 0.0f, range.none));
        }
        range.template reduce<1, (GROUP == 192 ? 32 : GROUP / 8)>();
        const Grid4 g(range, a.symmetric);
        if (__any(g.m != 1.0f)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= g.m;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = g.level(f[e]);
        if (a.out[values] && at > -2 && t < a.T && i < D / 8) {
            u32x4 y;
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = pack2<kBf16>((f32x2){g.value(f[2 * e]), g.value(f[2 * e + 1])});
            *reinterpret_cast<u32x4 *>(a.out[values] + t * a.ld_out[values] + h * D + 8 * i) = y;
        }
        uint32_t w;
        if (!values) {  // dim e at bits 4 (e / 2 + 4 (e % 2))
            w = codes4(f[0], f[2], f[4], f[6], g.zadd) | codes4(f[1], f[3], f[5], f[7], g.zadd) << 16;
            if (g.bad) w = 0x88888888u;
        } else {
            uint32_t nib = codes4(f[0], f[1], f[2], f[3], g.zadd) | codes4(f[4], f[5], f[6], f[7], g.zadd) << 16;
            if (g.bad) nib = 0x88888888u;
            // this lane's units m = 2 (i % 8), + 1: nibbles 2 (i % 4), + 1 of the lanes with their half of the dims
            const int lane = threadIdx.x & 63, from = (lane & ~7) + (i % 8) / 4, down = 8 * (i % 4);
            w = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t two = (uint32_t)__shfl((int)nib, from + 2 * j) >> down;
                w |= (two & 15u) << (4 * j) | (two & 0xF0u) << (12 + 4 * j);
            }
        }
        if (at < 0 || i >= D / 8) continue;
        const int64_t first = at & ~(int64_t)mask;
        const int in = (int)(at & mask), unit = 2 * i;  // 16 u + m of the first of the two units
        if (8 * i % GROUP == 0) {
            uint32_t *grid = (values ? a.pool.v_grid : a.pool.k_grid) + first * NG + ((int64_t)(8 * i / GROUP) << a.pool.lg_page);
            grid[in] = g.word();
        }
        if (!values) {
            a.pool.k[at * (D / 8) + (i & 3) * (D / 32) + (i >> 2)] = w;
            if (i == 0 && a.pool.weight) a.pool.weight[at] = 0.0f;
        } else if (wide) {
            if constexpr (kStaged) {
                units[unit][n + shift] = (uint16_t)w;
                units[unit + 1][n + shift] = (uint16_t)(w >> 16);
            }
        } else {
            uint16_t *v = a.pool.v + (at & ~(int64_t)7) * (D / 4) + unit * 8 + (at & 7);
            v[0] = (uint16_t)w;
            v[8] = (uint16_t)(w >> 16);
        }
    }
    if constexpr (kStaged) {
        if (!wide) return;
        __syncthreads();
        for (int j = threadIdx.x; j < kCols / 8 * (D / 4); j += 256) {
            const int c = j / (D / 4) * 8, unit = j % (D / 4);  // columns c .. c + 7 are tokens c - shift ..
            const int lo = max(c - shift, 0), hi = min(c - shift + 8, kTokens);
            if (lo >= hi) continue;
            uint16_t *v = a.pool.v + (place[lo] & ~(int64_t)7) * (D / 4) + unit * 8;
            if (hi - lo == 8) {
                *reinterpret_cast<u32x4 *>(v) = *reinterpret_cast<const u32x4 *>(&units[unit][c]);
            } else {
                for (int n = lo; n < hi; ++n) v[(n + shift) & 7] = units[unit][n + shift];
            }
        }
    }
}

template <int D64, int GROUP>
void launch_append(const AppendArgs &a, hipStream_t s) {
    constexpr int kPass = 256 / (D64 == 1 ? 8 : (D64 == 2 ? 16 : 32));
    // Staged where there are workgroups of 32 tokens for every compute unit (both sides: above).
    if (ceil_div(a.T, kBlockTokens) * a.pool.heads * 2 >= 512)
        (a.bf16 ? append_kernel<D64, GROUP, true, true> : append_kernel<D64, GROUP, true, false>)<<<dim3((unsigned)ceil_div(a.T, kBlockTokens), (unsigned)a.pool.heads, 2), 256, 0, s>>>(a);
    else
        (a.bf16 ? append_kernel<D64, GROUP, false, true> : append_kernel<D64, GROUP, false, false>)<<<dim3((unsigned)ceil_div(a.T, kPass), (unsigned)a.pool.heads, 2), 256, 0, s>>>(a);
}
template <int D64>
hipError_t launch_append(const AppendArgs &a, int group, hipStream_t s) {
    if (group == 64 * D64)
        launch_append<D64, 64 * D64>(a, s);
    else if (group == 32)
        launch_append<D64, 32>(a, s);
    else if (group == 64)
        launch_append<D64, 64>(a, s);
    else if constexpr (D64 == 4)
        launch_append<D64, 128>(a, s);
    return hipGetLastError();
}

}  // namespace

KvPool kv_pool(const gptq_kv_cache &c) {
    const int group = c.group_size ? c.group_size : c.head_dim;
    return {c.k, c.v, c.k_grid, c.v_grid, c.weight, (int32_t)c.n_pages, c.n_heads, __builtin_ctz(c.page), c.head_dim / group};
}

hipError_t run_kv_append(const void *K, int64_t ldk, const void *V, int64_t ldv, gptq_dtype dt, int64_t T, const int32_t *offs,
                         const gptq_kv_cache &c, const int32_t *table, int64_t width, const int32_t *lens, int64_t n_seq, void *K_out,
                         int64_t ldko, void *V_out, int64_t ldvo, hipStream_t s) {
    AppendArgs a;
    a.pool = kv_pool(c);
    a.seqs = {table, lens, (int32_t)n_seq, (int32_t)width, width * c.page};
    a.x[0] = static_cast<const uint16_t *>(K);
    a.x[1] = static_cast<const uint16_t *>(V);
    a.ld[0] = ldk;
    a.ld[1] = ldv;
    a.out[0] = static_cast<uint16_t *>(K_out);
    a.out[1] = static_cast<uint16_t *>(V_out);
    a.ld_out[0] = ldko;
    a.ld_out[1] = ldvo;
    a.offs = offs;
    a.T = T;
    a.per = T / n_seq;
    a.bf16 = dt == GPTQ_DT_BF16;
    a.symmetric = c.symmetric;
    const int group = c.group_size ? c.group_size : c.head_dim;
    switch (c.head_dim) {
    case 64: return launch_append<1>(a, group, s);
    case 128: return launch_append<2>(a, group, s);
    case 192: return launch_append<3>(a, group, s);
    default: return launch_append<4>(a, group, s);
    }
}

}  // namespace gptq
