// Thinning out a 4-bit cache: of every sequence and kv head, the last `recent`
// tokens and the heaviest others by accumulated weight, `budget` in all, are copied to
// other pages in slot order.  What a missing page would hold are no tokens and are left
// out, so that every place below the new length is written; which pages are missing is the
// same for all heads of a sequence, and so is the new length.
#include <algorithm>

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

// Weights in ascending order of an unsigned integer, above 0 (no token) and below kLate (a token that stays whatever its
// weight): NaN, negative numbers, zeros of either sign, positive ones.
constexpr uint32_t kLate = 0xFFFFFFFF;
__device__ __forceinline__ uint32_t rank_of(float w) {
    if (!(w == w)) return 1;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
// Of four neighbouring slots from a multiple of four on, which share a page; those from `late` on stay.
__device__ __forceinline__ u32x4 ranks_at(const EvictArgs &a, const int32_t *row, int h, int slot, int late) {
    const int page = a.seqs.page_of(a.pool, row, slot);
    if (page < 0) return (u32x4){};
    const floatx4 w = *reinterpret_cast<const floatx4 *>(a.pool.weight + a.pool.first(page, h) + (slot & (a.pool.page() - 1)));
    u32x4 k = {rank_of(w[0]), rank_of(w[1]), rank_of(w[2]), rank_of(w[3])};
    if (slot + 3 >= late) {
#pragma unroll
        for (int e = 0; e < 4; ++e) k[e] = slot + e >= late ? kLate : k[e];
    }
    return k;
}

// The rank of the `heavy`-th largest of the slots below `safe`, digit by digit from the highest (11, 11 and 10 bits, a
// histogram of each), then the kept slots in order: all above that rank, and of those at it the first ones.  Ranks stay in
// LDS where they fit, `in_lds` of them (a multiple of four); a wave walks slots next to each other, so that order is a matter
// of sums over its lanes.
//
// A workgroup for a sequence and head, bound by its own steps: 10 us for 16 sequences of 2112 tokens (1.3 for the weights,
// 1.3 a digit, 1 for the order, the launch), 34.3 for four of up to 32768, on 32 compute units (of 19968 ranks 6 to load, 4-5
// a digit, 4.5 for the order; LDS conflicts are 3 % of it).  To know that no page is missing costs 0.3 and 0.7 of these.
// Not built: more workgroups for a head (one launch more, with the ranks that share the edge's first digit brought together), and
// the second and third digit over those ranks alone.
constexpr int kBins = 2048, kRanksInLds = 36 * 1024;  // 144 KB
__global__ __launch_bounds__(kSelectThreads) void select_kernel(EvictArgs a, int in_lds) {
    extern __shared__ uint32_t ranks[];
    __shared__ uint32_t hist[kBins + kWave], found[2], sums[kSelectWaves];
    __shared__ int counts[2][kSelectWaves];
    const int h = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int32_t *row = a.seqs.table + (int64_t)b * a.seqs.width;
    const int len = a.seqs.len(b), lg = a.pool.lg_page, pages = (len + a.pool.page() - 1) >> lg;
    auto tokens_of = [&](int p) { return p >= 0 && a.seqs.page_of(a.pool, row, p << lg) >= 0 ? min(a.pool.page(), len - (p << lg)) : 0; };
    int here = 0;
    bool gone = false;  // a page of the thread's
    for (int p = threadIdx.x; p < pages; p += kSelectThreads) {
        const int n = tokens_of(p);
        here += n;
        gone |= n == 0;
    }
    int keep = min(len, a.budget), recent = min(a.recent, keep);
    int safe = len - recent, heavy = keep - recent, late = 0x7FFFFFFF;  // heavy of the first `safe` slots stay
    int32_t *kept = a.kept + ((int64_t)b * a.pool.heads + h) * a.budget;
    if (!__syncthreads_or(gone)) {
        for (int i = threadIdx.x; i < recent; i += kSelectThreads) kept[heavy + i] = safe + i;
    } else {  // of all slots, the last `recent` tokens and the heaviest others
        here = wave_scan(here);
        if (lane == 63) sums[wave] = here;
        __syncthreads();
        keep = 0;
        for (int w = 0; w < kSelectWaves; ++w) keep += sums[w];
        keep = min(keep, a.budget);
        recent = min(a.recent, keep);
        safe = late = len;
        heavy = keep;
        if (recent > 0) {  // `late` has `recent` tokens from it on: 1024 pages at a time from the last
            int before = 0;
            for (int top = pages - 1; top >= 0 && before < recent; top -= kSelectThreads) {
                const int p = top - (int)threadIdx.x, n = tokens_of(p), upto = wave_scan(n);
                __syncthreads();  // sums have been read
                if (lane == 63) sums[wave] = upto;
                __syncthreads();
                int mine = before + upto - n;  // on the pages behind this one
                for (int w = 0; w < kSelectWaves; ++w) {
                    mine += w < wave ? sums[w] : 0;
                    before += sums[w];
                }
                if (mine < recent && recent <= mine + n) found[0] = (p << lg) + n - (recent - mine);
            }
            __syncthreads();
            late = found[0];
        }
    }
    for (int i = keep + threadIdx.x; i < a.budget; i += kSelectThreads) kept[i] = -1;
    if (a.new_lens && h == 0 && threadIdx.x == 0) a.new_lens[b] = keep;
    if (heavy == 0) return;
    if (heavy == safe) {
        for (int i = threadIdx.x; i < safe; i += kSelectThreads) kept[i] = i;
        return;
    }
    u32x4 *four = reinterpret_cast<u32x4 *>(ranks);
    auto rank4 = [&](int i) { return i < in_lds ? four[i / 4] : ranks_at(a, row, h, i, late); };
    uint32_t edge = 0, ties = heavy;  // the rank of the last that stays; `ties` of those that have it stay
    for (int shift = 21, bits = 11; shift >= 0;) {
        for (int i = threadIdx.x; i < kBins; i += kSelectThreads) hist[i] = 0;
        __syncthreads();
        const uint32_t digits = (1u << bits) - 1;
        const int above = shift + bits;
        // A rank that differs from the edge above these bits counts in a bin of its lane's, past the others (a branch costs more).
        auto count = [&](const u32x4 &k, int i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool in = i + e < safe && (above == 32 || (k[e] ^ edge) >> above == 0);
                atomicAdd(&hist[in ? k[e] >> shift & digits : kBins + lane], 1u);
            }
        };
        if (shift == 21) {
#pragma unroll 8
            for (int i = 4 * threadIdx.x; i < safe; i += 4 * kSelectThreads) {
                const u32x4 k = ranks_at(a, row, h, i, late);
                if (i < in_lds) four[i / 4] = k;
                count(k, i);
            }
        } else {
#pragma unroll 4
            for (int i = 4 * threadIdx.x; i < safe; i += 4 * kSelectThreads) count(rank4(i), i);
        }
        __syncthreads();
        // thread i holds bins kBins - 2 i - 1 and - 2: sums from the highest bin down
        const uint32_t h0 = hist[kBins - 1 - 2 * threadIdx.x], h1 = hist[kBins - 2 - 2 * threadIdx.x];
        const uint32_t upto = (uint32_t)wave_scan((int)(h0 + h1));
        if (lane == 63) sums[wave] = upto;
        __syncthreads();
        uint32_t before = upto - h0 - h1;
        for (int w = 0; w < wave; ++w) before += sums[w];
        if (before < ties && ties <= before + h0)
            found[0] = kBins - 1 - 2 * threadIdx.x, found[1] = ties - before;
        else if (before + h0 < ties && ties <= before + h0 + h1)
            found[0] = kBins - 2 - 2 * threadIdx.x, found[1] = ties - before - h0;
        __syncthreads();
        edge |= found[0] << shift;
        ties = found[1];
        bits = shift < 11 ? 10 : 11;
        shift = shift == 21 ? 10 : shift == 10 ? 0 : -1;
    }
    // A wave's share of the slots in rounds of 256, four neighbouring ones a lane.
    const int share = (safe + 4 * kSelectThreads - 1) / (4 * kSelectThreads) * (4 * kWave), i0 = wave * share, i1 = min(i0 + share, safe);
    int na = 0, nt = 0;
    for (int i = i0 + 4 * lane; i < i1; i += 4 * kWave) {
        const u32x4 k = rank4(i);
#pragma unroll
        for (int e = 0; e < 4; ++e) na += i + e < i1 && k[e] > edge, nt += i + e < i1 && k[e] == edge;
    }
    na = wave_scan(na);
    nt = wave_scan(nt);
    if (lane == 63) counts[0][wave] = na, counts[1][wave] = nt;
    __syncthreads();
    na = nt = 0;
    for (int w = 0; w < wave; ++w) na += counts[0][w], nt += counts[1][w];
    for (int j = i0; j < i1; j += 4 * kWave) {
        const int i = j + 4 * lane;
        const u32x4 k = i < i1 ? rank4(i) : (u32x4){};
        bool above[4], at[4];
        int ma = 0, mt = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            above[e] = i + e < i1 && k[e] > edge;
            at[e] = i + e < i1 && k[e] == edge;
            ma += above[e];
            mt += at[e];
        }
        const int sa = wave_scan(ma), st = wave_scan(mt);
        int pa = na + sa - ma, pt = nt + st - mt;  // before this lane's
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (above[e] || (at[e] && pt < (int)ties)) kept[pa + min(pt, (int)ties)] = i + e;
            pa += above[e];
            pt += at[e];
        }
        na += __builtin_amdgcn_readlane(sa, 63);
        nt += __builtin_amdgcn_readlane(st, 63);
    }
}

// The kept tokens to their new pages: 32 of one head a workgroup.  Keys, grids and weights move by the token; values by the
// unit of eight tokens that it writes, gathered two bytes each.  Bound by memory: 16 x 2048 tokens of 8 heads of 128 (74 MB)
// take 17.2 us, 4.3 TB/s.
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
    const int in_lds = (int)std::min<int64_t>(align_up(max_len, 4), kRanksInLds);
    select_kernel<<<dim3((unsigned)c.n_heads, (unsigned)n_seq), kSelectThreads, (size_t)in_lds * 4, s>>>(a, in_lds);
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
