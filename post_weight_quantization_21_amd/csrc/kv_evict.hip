// Thinning out a 4-bit cache: of every sequence and kv head, the last `recent`
// tokens and the heaviest others by accumulated weight, `budget` in all, are copied to
// other pages in slot order.
#include "kv_cache.h"

namespace gptq {
namespace {

constexpr int kSelectThreads = 1024, kSelectWaves = kSelectThreads / kWave;

struct EvictArgs {
    KvPool pool;
    KvSeqs seqs;
    const int32_t *to;  // [n][to_width] pages
    int32_t to_width, budget, recent;
    int32_t *kept;      // [n][heads][budget] slots, -1 behind the last
    int32_t *new_lens;  // or NULL
};

// Weights in ascending order of an unsigned integer: NaN, negative numbers, zeros of either sign, positive ones.
__device__ __forceinline__ uint32_t rank_of(float w) {
    if (!(w == w)) return 0;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint32_t rank_at(const EvictArgs &a, const int32_t *row, int h, int slot) {
    const int page = a.seqs.page_of(a.pool, row, slot);
    return page < 0 ? 0u : rank_of(a.pool.weight[a.pool.first(page, h) + (slot & (a.pool.page() - 1))]);
}

// The `heavy`-th largest rank of slots below `safe`, digit by digit from the highest (a histogram of 256 each), then
// the kept slots in order: all above that rank, and of those at it the first ones.
__global__ __launch_bounds__(kSelectThreads) void select_kernel(EvictArgs a) {
    __shared__ uint32_t hist[256], found[2];
    __shared__ int counts[2][kSelectWaves];
    const int h = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int32_t *row = a.seqs.table + (int64_t)b * a.seqs.width;
    const int len = a.seqs.len(b), keep = min(len, a.budget), recent = min(a.recent, keep);
    const int safe = len - recent, heavy = keep - recent;  // heavy of the first `safe` slots stay
    int32_t *kept = a.kept + ((int64_t)b * a.pool.heads + h) * a.budget;
    for (int i = keep + threadIdx.x; i < a.budget; i += kSelectThreads) kept[i] = -1;
    if (a.new_lens && h == 0 && threadIdx.x == 0) a.new_lens[b] = keep;
    uint32_t edge = 0;  // the rank of the last that stays; `ties` of those that have it stay
    int ties = heavy;
    if (heavy > 0 && heavy < safe) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (threadIdx.x < 256) hist[threadIdx.x] = 0;
            __syncthreads();
            for (int i = threadIdx.x; i < safe; i += kSelectThreads) {
                const uint32_t k = rank_at(a, row, h, i);
                if (shift == 24 || k >> (shift + 8) == edge >> (shift + 8)) atomicAdd(&hist[k >> shift & 255], 1u);
            }
            __syncthreads();
            if (threadIdx.x == 0) {
                uint32_t left = ties;
                int d = 255;
                while (d > 0 && hist[d] < left) left -= hist[d--];
                found[0] = d;
                found[1] = left;
            }
            __syncthreads();
            edge |= found[0] << shift;
            ties = found[1];
        }
    }
    // heavy == safe: every rank is at or above 0, and ties is enough for all of them
    int above0 = 0, ties0 = 0;  // kept above the edge, and seen at it, before this round
    for (int i0 = 0; i0 < len; i0 += kSelectThreads) {
        const int i = i0 + threadIdx.x;
        bool above = false, at = false;
        if (i < safe && heavy > 0) {
            const uint32_t k = rank_at(a, row, h, i);
            above = k > edge;
            at = k == edge;
        } else if (i >= safe && i < len) {
            above = true;
        }
        const uint64_t va = __ballot(above), vt = __ballot(at), below = (1ull << lane) - 1;
        if (lane == 0) counts[0][wave] = __popcll(va), counts[1][wave] = __popcll(vt);
        __syncthreads();
        int na = above0 + __popcll(va & below), nt = ties0 + __popcll(vt & below);
        for (int w = 0; w < kSelectWaves; ++w) {
            if (w < wave) na += counts[0][w], nt += counts[1][w];
            above0 += counts[0][w];
            ties0 += counts[1][w];
        }
        if (above || (at && nt < ties)) kept[na + min(nt, ties)] = i;
        __syncthreads();
    }
}

// The kept tokens to their new pages: 32 of one head a workgroup.
template <int D64>
__global__ __launch_bounds__(256) void move_kernel(EvictArgs a) {
    constexpr int D = 64 * D64;
    __shared__ int64_t from[32], to[32];  // tokens counted over the pool, from -1: none
    const int h = blockIdx.y, b = blockIdx.z, j0 = blockIdx.x * 32;
    const int32_t *kept = a.kept + ((int64_t)b * a.pool.heads + h) * a.budget;
    const int mask = a.pool.page() - 1;
    if (threadIdx.x < 32) {
        const int j = j0 + threadIdx.x, slot = j < a.budget ? kept[j] : -1;
        from[threadIdx.x] = -1;
        if (slot >= 0) {
            const int src = a.seqs.page_of(a.pool, a.seqs.table + (int64_t)b * a.seqs.width, slot);
            const int dst = a.seqs.page_of(a.pool, a.to + (int64_t)b * a.to_width, j);
            if (src >= 0 && dst >= 0) {
                from[threadIdx.x] = a.pool.first(src, h) + (slot & mask);
                to[threadIdx.x] = a.pool.first(dst, h) + (j & mask);
            }
        }
    }
    __syncthreads();
    if (from[0] < 0 && kept[j0] < 0) return;
    for (int i = threadIdx.x; i < 32 * (D / 32); i += 256) {  // keys, sixteen bytes each
        const int j = i / (D / 32), w = i % (D / 32);
        if (from[j] >= 0)
            *reinterpret_cast<u32x4 *>(a.pool.k + to[j] * (D / 8) + 4 * w) = *reinterpret_cast<const u32x4 *>(a.pool.k + from[j] * (D / 8) + 4 * w);
    }
    for (int i = threadIdx.x; i < 4 * (D / 4); i += 256) {  // values: a unit's eight tokens
        const int j = 8 * (i / (D / 4)), unit = i % (D / 4);
        uint16_t x[8];
        bool all = true;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t f = from[j + e];
            all &= f >= 0;
            x[e] = f < 0 ? 0 : a.pool.v[(f & ~(int64_t)7) * (D / 4) + unit * 8 + (f & 7)];
        }
        if (all) {
            uint16_t *v = a.pool.v + to[j] * (D / 4) + unit * 8;  // to[j] starts a block of eight
            u32x4 w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = x[2 * e] | (uint32_t)x[2 * e + 1] << 16;
            *reinterpret_cast<u32x4 *>(v) = w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (from[j + e] >= 0) a.pool.v[(to[j + e] & ~(int64_t)7) * (D / 4) + unit * 8 + (to[j + e] & 7)] = x[e];
        }
    }
    for (int i = threadIdx.x; i < 32 * (2 * a.pool.groups + 1); i += 256) {  // grids and weights
        const int j = i % 32, which = i / 32;
        if (from[j] < 0) continue;
        if (which == 2 * a.pool.groups) {
            a.pool.weight[to[j]] = a.pool.weight[from[j]];
        } else {
            uint32_t *grid = which & 1 ? a.pool.v_grid : a.pool.k_grid;
            const int g = which / 2;
            const int64_t f = from[j] & ~(int64_t)mask, t = to[j] & ~(int64_t)mask;
            grid[t * a.pool.groups + ((int64_t)g << a.pool.lg_page) + (to[j] & mask)] =
                grid[f * a.pool.groups + ((int64_t)g << a.pool.lg_page) + (from[j] & mask)];
        }
    }
}

}  // namespace

size_t kv_evict_ws_bytes(const gptq_kv_cache &, int64_t, int64_t, int64_t) { return 0; }

hipError_t run_kv_evict(const gptq_kv_cache &c, const int32_t *table, int64_t width, const int32_t *lens, int64_t n_seq, int64_t max_len,
                        const int32_t *to, int64_t to_width, int64_t budget, int64_t recent, int32_t *kept, int32_t *new_lens, void *,
                        hipStream_t s) {
    EvictArgs a;
    a.pool = kv_pool(c);
    a.seqs = {table, lens, (int32_t)n_seq, (int32_t)width, max_len};
    a.to = to;
    a.to_width = (int32_t)to_width;
    a.budget = (int32_t)budget;
    a.recent = (int32_t)recent;
    a.kept = kept;
    a.new_lens = new_lens;
    select_kernel<<<dim3((unsigned)c.n_heads, (unsigned)n_seq), kSelectThreads, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)ceil_div(budget, 32), (unsigned)c.n_heads, (unsigned)n_seq);
    switch (c.head_dim) {
    case 64: move_kernel<1><<<grid, 256, 0, s>>>(a); break;
    case 128: move_kernel<2><<<grid, 256, 0, s>>>(a); break;
    case 192: move_kernel<3><<<grid, 256, 0, s>>>(a); break;
    default: move_kernel<4><<<grid, 256, 0, s>>>(a); break;
    }
    return hipGetLastError();
}

}  // namespace gptq
