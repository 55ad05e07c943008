// New keys and values into the pages of a 4-bit cache.
//
// A group's grid (all decisions binary32, round half to even):
//   asymmetric  lo = min(min x, 0), hi = max(max x, 0), s = bf16((hi - lo) (1/15)),
//               z = clamp(rint(-lo / s), 0, 15), q = clamp(rint(x / s + z), 0, 15)
//   symmetric   s = bf16(max|x| (1/7)), z = 8, q = clamp(rint(x / s), -7, 7) + 8
// with s = 1 where it would be 0 (1/15 and 1/7: the nearest binary32).  The scale is
// rounded before the codes are chosen, so its sixteen bits cost no accuracy beyond the
// last code's (a range may end 0.06 of a step past code 15).  A group with a value that is not finite, or whose scale
// is not, is stored with a scale that is no number.
#include "kv_cache.h"

namespace gptq {
namespace {

struct AppendArgs {
    KvPool pool;
    KvSeqs seqs;
    const uint16_t *x[2];  // keys, values: [T][ld]
    int64_t ld[2];
    uint16_t *out[2];  // the values as stored, or NULL
    int64_t ld_out[2];
    const int32_t *offs;
    int64_t T;
    int32_t bf16, symmetric;
};

__device__ __forceinline__ float load16(uint16_t h, bool bf16) {
    return bf16 ? __uint_as_float((uint32_t)h << 16) : (float)__builtin_bit_cast(_Float16, h);
}
__device__ __forceinline__ uint16_t store16(float f, bool bf16) {
    return bf16 ? __builtin_bit_cast(uint16_t, (__bf16)f) : __builtin_bit_cast(uint16_t, (_Float16)f);
}

struct Range {
    float lo, hi;
    bool bad;
    __device__ __forceinline__ void add(float x) {
        lo = fminf(lo, x);
        hi = fmaxf(hi, x);
        bad |= !(fabsf(x) < __builtin_inff());
    }
    __device__ __forceinline__ void add(const Range &r) {
        lo = fminf(lo, r.lo);
        hi = fmaxf(hi, r.hi);
        bad |= r.bad;
    }
    template <int W>  // over W neighbouring lanes
    __device__ __forceinline__ void reduce() {
#pragma unroll
        for (int o = 1; o < W; o *= 2) {
            const Range r = {__shfl_xor(lo, o), __shfl_xor(hi, o), (bool)__shfl_xor((int)bad, o)};
            add(r);
        }
    }
};

struct Grid4 {
    float s, z, qlo, qhi, zadd;
    bool bad;
};
__device__ __forceinline__ Grid4 fit4(const Range &r, bool symmetric) {
#pragma clang fp contract(off)
    Grid4 g;
    const float s = symmetric ? fmaxf(-r.lo, r.hi) * (1.0f / 7.0f) : (r.hi - r.lo) * (1.0f / 15.0f);
    g.s = (float)(__bf16)s;
    if (g.s == 0.0f) g.s = 1.0f;
    g.bad = r.bad || !(g.s < __builtin_inff());
    g.z = symmetric ? 0.0f : fminf(fmaxf(rintf(-r.lo / g.s), 0.0f), 15.0f);
    g.qlo = symmetric ? -7.0f : 0.0f;
    g.qhi = symmetric ? 7.0f : 15.0f;
    g.zadd = symmetric ? 8.0f : 0.0f;
    return g;
}
__device__ __forceinline__ uint32_t code4(const Grid4 &g, float x) {
#pragma clang fp contract(off)
    const float q = fminf(fmaxf(rintf(x / g.s + g.z), g.qlo), g.qhi) + g.zadd;
    return g.bad ? 8u : (uint32_t)q;
}
__device__ __forceinline__ uint32_t word4(const Grid4 &g) {
    const uint32_t s = g.bad ? 0x7FC0u : __float_as_uint(g.s) >> 16;
    const float c = g.bad ? 0.0f : 8.0f - (g.zadd + g.z);
    return (s << 16) | __builtin_bit_cast(uint16_t, (_Float16)c);
}
__device__ __forceinline__ float value4(const Grid4 &g, uint32_t q) {
    return g.bad ? __builtin_nanf("") : g.s * ((float)q - (g.zadd + g.z));
}

// A thread takes eight values of one token, head and side: of keys a word, eight dims
// next to each other; of values two units, dims 64 u + 16 j + m, + 1 for j = 0 .. 3.
template <int D64, int GROUP>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a) {
    constexpr int D = 64 * D64, NG = D / GROUP, kLanes = D64 == 1 ? 8 : (D64 == 2 ? 16 : 32);
    const bool values = blockIdx.y != 0;
    const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) / kLanes;  // (token, head)
    const int i = threadIdx.x % kLanes, heads = a.pool.heads;
    const int64_t t = row / heads;
    const int h = (int)(row - t * heads);
    // the token's sequence and slot
    int b, slot = -1;
    if (!a.offs) {
        const int64_t per = a.T / a.seqs.n;
        b = (int)(t / per);
        if (t < a.T) slot = a.seqs.len(b) - (int)((b + 1) * per - t);
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
        if (t < a.T && b < a.seqs.n) slot = a.seqs.len(b) - (int)(a.offs[b + 1] - t);
    }
    const bool in = t < a.T && b < a.seqs.n, mine = i < D / 8;
    int page = -1;
    if (in && slot >= 0 && slot < a.seqs.capacity) page = a.seqs.page_of(a.pool, a.seqs.table + (int64_t)b * a.seqs.width, slot);
    uint16_t x16[8];
    Range r[2] = {};
    const int u = i / 8, m = 2 * (i % 8);
    if (in && mine) {
        const uint16_t *x = a.x[values] + t * a.ld[values] + h * D;
        if (!values) {
            const u32x4 w = *reinterpret_cast<const u32x4 *>(x + 8 * i);
#pragma unroll
            for (int e = 0; e < 8; ++e) x16[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t w = *reinterpret_cast<const uint32_t *>(x + 64 * u + 16 * j + m);
                x16[2 * j] = (uint16_t)w;
                x16[2 * j + 1] = (uint16_t)(w >> 16);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) r[values ? e / 4 : 0].add(load16(x16[e], a.bf16));
    }
    // The group's range: of keys over the lanes that hold it; of values a group of 32
    // is half of every lane's share of a set of 64.
    Grid4 g[2];
    if (!values) {
        r[0].template reduce<(GROUP == 32 ? 4 : GROUP == 64 ? 8 : GROUP == 128 ? 16 : 32)>();
        g[0] = g[1] = fit4(r[0], a.symmetric);
    } else if constexpr (GROUP == 32) {
        r[0].template reduce<8>();
        r[1].template reduce<8>();
        g[0] = fit4(r[0], a.symmetric);
        g[1] = fit4(r[1], a.symmetric);
    } else {
        r[0].add(r[1]);
        r[0].template reduce<(GROUP == 64 ? 8 : GROUP == 128 ? 16 : 32)>();
        g[0] = g[1] = fit4(r[0], a.symmetric);
    }
    if (!in || !mine) return;
    uint32_t q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = code4(g[values ? e / 4 : 0], load16(x16[e], a.bf16));
    if (a.out[values]) {
        uint16_t *o = a.out[values] + t * a.ld_out[values] + h * D, y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = store16(value4(g[values ? e / 4 : 0], q[e]), a.bf16);
        if (!values) {
            u32x4 w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = y[2 * e] | (uint32_t)y[2 * e + 1] << 16;
            *reinterpret_cast<u32x4 *>(o + 8 * i) = w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint32_t *>(o + 64 * u + 16 * j + m) = y[2 * j] | (uint32_t)y[2 * j + 1] << 16;
        }
    }
    if (page < 0) return;
    const int at = slot & (a.pool.page() - 1);
    const int64_t first = a.pool.first(page, h);
    if (!values) {
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) w |= q[e] << (4 * (e / 2 + 4 * (e & 1)));
        a.pool.k[(first + at) * (D / 8) + (i & 3) * (D / 32) + (i >> 2)] = w;
        if (8 * i % GROUP == 0) a.pool.k_grid[first * NG + (int64_t)(8 * i / GROUP) * a.pool.page() + at] = word4(g[0]);
        if (i == 0 && a.pool.weight) a.pool.weight[first + at] = 0.0f;
    } else {
        uint16_t *v = a.pool.v + ((first + (at & ~7)) * (D / 4) + (16 * u + m) * 8 + (at & 7));
#pragma unroll
        for (int k = 0; k < 2; ++k)
            v[8 * k] = (uint16_t)(q[k] | q[2 + k] << 4 | q[4 + k] << 8 | q[6 + k] << 12);
        uint32_t *grid = a.pool.v_grid + first * NG + at;
        if constexpr (GROUP == 32) {
            if (i % 8 < 2) grid[(int64_t)(2 * u + i % 8) * a.pool.page()] = word4(i % 8 ? g[1] : g[0]);
        } else {
            if (8 * i % GROUP == 0) grid[(int64_t)(8 * i / GROUP) * a.pool.page()] = word4(g[0]);
        }
    }
}

template <int D64>
hipError_t launch_append(const AppendArgs &a, int group, hipStream_t s) {
    constexpr int kLanes = D64 == 1 ? 8 : (D64 == 2 ? 16 : 32);
    const dim3 grid((unsigned)ceil_div(a.T * a.pool.heads, 256 / kLanes), 2);
    void (*kernel)(AppendArgs) = nullptr;
    if (group == 64 * D64)
        kernel = append_kernel<D64, 64 * D64>;
    else if (group == 32)
        kernel = append_kernel<D64, 32>;
    else if (group == 64)
        kernel = append_kernel<D64, 64>;
    else if constexpr (D64 == 4)
        kernel = append_kernel<D64, 128>;
    kernel<<<grid, 256, 0, s>>>(a);
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
