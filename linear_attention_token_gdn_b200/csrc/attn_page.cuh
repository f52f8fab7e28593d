// attn_page.cuh -- the choice of cache pages that a new token attends to: the mean key of each page, kept up
// as pages fill, and for each (row, key head) the pages whose mean key scores highest.
//
//   mean_p = sum of the page's keys inside the row's length / their count            (fp32)
//   score_p = max over the query heads h of the key head's group of q_h . mean_p      (fp64)
// The first n_first and the last n_last pages are always chosen, the rest by score, ties to the lower page;
// the list is ascending, -1 behind its end.
//
// Scores are summed in fp64: which page is the last to be chosen can hang on the last bits of two scores,
// and with 2^-53 the order of the sum (so the tile, or another build) no longer decides it in practice.
#pragma once
#include "attn_decode.cuh"

namespace gdn {

// ---------------------------------------------------------------- mean keys

constexpr int kMeanThreads = 128;

struct AttnMeanArgs {
    const void* k_cache;
    const int32_t *table, *lens, *starts;       // starts: first new position of each row (NULL: 0)
    int B, Hkv, num_pages, page_size, max_pages;
    float* mean;                                // [num_pages, Hkv, D]
};

// Pages of row b that hold a position in [starts[b], lens[b]): first page, and their number.
__device__ __forceinline__ int attn_touched(const AttnMeanArgs& a, int b, int& first) {
    const int len = attn_len(a.lens, b, (long long)a.max_pages * a.page_size);
    const int start = a.starts == nullptr ? 0 : max(a.starts[b], 0);
    first = 0;
    if (start >= len) return 0;
    first = start / a.page_size;
    return (len + a.page_size - 1) / a.page_size - first;
}

// HBM-bound: a CTA reads a page of one key head (page_size x D, contiguous) with 16-byte loads, all of them
// in flight at once for pages of 64 keys of 128 channels, and adds in fp32 in a fixed order.
template <bool BF, int D>
__global__ void __launch_bounds__(kMeanThreads) attn_page_mean_kernel(const AttnMeanArgs a) {
    constexpr int LPR = D / 8, RPP = kMeanThreads / LPR, U = 8;  // lanes of a key, keys of a pass, passes in flight
    __shared__ __align__(16) float s_sum[RPP][D];  // written 16 bytes at a time
    const int tid = threadIdx.x, l = tid % LPR, sub = tid / LPR;
    long long share = 0;
    const AttnPlace place = attn_locate<kMeanThreads>(
        a.B,
        [&](int b) {
            int first;
            return (long long)attn_touched(a, b, first) * a.Hkv;
        },
        [&](long long total) {
            share = (total + gridDim.x - 1) / gridDim.x;
            return share * blockIdx.x;
        });
    long long at = share * blockIdx.x;
    const long long end = min(at + share, place.total);
    int b = place.b, first = 0, n = 0;
    long long row_base = place.before;
    if (at < end) n = attn_touched(a, b, first);
    for (; at < end; ++at) {
        while (at >= row_base + (long long)n * a.Hkv) {
            row_base += (long long)n * a.Hkv;
            n = attn_touched(a, ++b, first);
        }
        const int i = (int)((at - row_base) / a.Hkv), hk = (int)(at - row_base - (long long)i * a.Hkv);
        const int page = first + i;
        const int count = min(a.page_size, a.lens[b] - page * a.page_size);
        const int phys = a.table[(size_t)b * a.max_pages + page];
        if (phys < 0 || phys >= a.num_pages || count <= 0) {  // uniform
            if (tid == 0) raise_error(kErrPage);
            continue;
        }
        const size_t slot = (size_t)phys * a.Hkv + hk;
        if (!in_bounds((long long)slot, (long long)a.num_pages * a.Hkv)) continue;
        const uint16_t* keys = reinterpret_cast<const uint16_t*>(a.k_cache) + slot * a.page_size * D + 8 * l;
        float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int r0 = sub; r0 < count; r0 += U * RPP) {
            uint4 x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                x[u] = make_uint4(0, 0, 0, 0);
                if (r0 + u * RPP < count) x[u] = *reinterpret_cast<const uint4*>(keys + (size_t)(r0 + u * RPP) * D);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = unpack2<BF>(w[e]);
                    sum[2 * e] += f.x;
                    sum[2 * e + 1] += f.y;
                }
            }
        }
        __syncthreads();  // the previous page's sums have been read
        stv<kF32, 8>(s_sum[sub], 8 * l, sum);
        __syncthreads();
        for (int c = tid; c < D; c += kMeanThreads) {
            float total = 0.0f;
#pragma unroll
            for (int r = 0; r < RPP; ++r) total += s_sum[r][c];
            a.mean[slot * D + c] = total / (float)count;
        }
    }
}

// ---------------------------------------------------------------- scores

struct AttnSelectArgs {
    const void* q;
    const float* mean;
    const int32_t *table, *lens;
    int B, Hq, Hkv, group, num_pages, page_size, max_pages, n_sel, n_first, n_last;
    unsigned long long* keys;                   // [B, Hkv, max_pages]
    int32_t* pages;                             // [B, Hkv, n_sel]
};

constexpr int kScoreThreads = 128, kScorePages = kScoreThreads, kScoreHeads = 8, kScoreSlab = 32;

// A double as an unsigned number of the same order; NaN is the lowest.
__device__ __forceinline__ unsigned long long sort_key(double x) {
    if (x != x) return 0ull;
    const long long bits = __double_as_longlong(x + 0.0);  // -0 as 0
    return bits < 0 ? ~(unsigned long long)bits : (unsigned long long)bits | 0x8000000000000000ull;
}

// One thread per page: 128 pages of a (row, key head) at a time, their means brought into shared memory 32
// channels at a time (rows padded by 16 bytes: a quarter warp's 16-byte reads then cover all banks), 8 heads'
// sums per thread.  Bound by the fp64 units: 8 fused multiply-adds per 4 bytes of mean key at a group of 8.
template <bool BF, int D>
__global__ void __launch_bounds__(kScoreThreads) attn_score_kernel(const AttnSelectArgs a) {
    constexpr int ROW = kScoreSlab + 4;
    __shared__ __align__(16) float s_mean[kScorePages][ROW];
    __shared__ __align__(16) double s_q[D][kScoreHeads];
    __shared__ int s_phys[kScorePages];
    const int tid = threadIdx.x;
    const long long capacity = (long long)a.max_pages * a.page_size;
    auto pages_of = [&](int b) { return (attn_len(a.lens, b, capacity) + a.page_size - 1) / a.page_size; };
    auto blocks_of = [&](int pages) { return pages > a.n_sel ? (pages + kScorePages - 1) / kScorePages : 0; };
    long long share = 0;
    const AttnPlace place = attn_locate<kScoreThreads>(
        a.B, [&](int b) { return (long long)blocks_of(pages_of(b)) * a.Hkv; },
        [&](long long total) {
            share = (total + gridDim.x - 1) / gridDim.x;
            return share * blockIdx.x;
        });
    long long at = share * blockIdx.x;
    const long long end = min(at + share, place.total);
    int b = place.b, n = 0;
    long long row_base = place.before;
    if (at < end) n = blocks_of(pages_of(b));
    for (; at < end; ++at) {
        while (at >= row_base + (long long)n * a.Hkv) {
            row_base += (long long)n * a.Hkv;
            n = blocks_of(pages_of(++b));
        }
        const int hk = (int)((at - row_base) / n);
        const int page = (int)(at - row_base - (long long)hk * n) * kScorePages + tid;
        const int pages = pages_of(b);
        int phys = -1;
        if (page < pages) phys = attn_page(a.table, a.max_pages, a.num_pages, b, page);
        __syncthreads();  // the previous block's shared values have been read
        s_phys[tid] = phys;
        double best = -INFINITY;
        bool any = false;
        for (int h0 = 0; h0 < a.group; h0 += kScoreHeads) {
            const int heads = min(kScoreHeads, a.group - h0);
            if (h0 > 0) __syncthreads();
            for (int i = tid; i < D * kScoreHeads; i += kScoreThreads) {
                const int h = i / D, c = i - h * D;
                s_q[c][h] = h < heads ? (double)ld1(a.q, BF ? kBF16 : kF16,
                                                    ((size_t)b * a.Hq + hk * a.group + h0 + h) * D + c)
                                      : 0.0;
            }
            double sum[kScoreHeads];
#pragma unroll
            for (int h = 0; h < kScoreHeads; ++h) sum[h] = 0.0;
            for (int c0 = 0; c0 < D; c0 += kScoreSlab) {
                __syncthreads();
#pragma unroll
                for (int i = tid; i < kScorePages * kScoreSlab / 4; i += kScoreThreads) {
                    const int r = i / (kScoreSlab / 4), c = 4 * (i - r * (kScoreSlab / 4));
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (s_phys[r] >= 0)
                        x = *reinterpret_cast<const float4*>(a.mean + ((size_t)s_phys[r] * a.Hkv + hk) * D + c0 + c);
                    *reinterpret_cast<float4*>(&s_mean[r][c]) = x;
                }
                __syncthreads();
#pragma unroll 2
                for (int c = 0; c < kScoreSlab; c += 4) {
                    const float4 x4 = *reinterpret_cast<const float4*>(&s_mean[tid][c]);
                    const float x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const double xd = (double)x[e];
#pragma unroll
                        for (int h = 0; h < kScoreHeads; h += 2) {
                            const double2 qd = *reinterpret_cast<const double2*>(&s_q[c0 + c + e][h]);
                            sum[h] = fma(qd.x, xd, sum[h]);
                            sum[h + 1] = fma(qd.y, xd, sum[h + 1]);
                        }
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < kScoreHeads; ++h) {
                if (h < heads && sum[h] == sum[h]) {
                    best = fmax(best, sum[h]);
                    any = true;
                }
            }
        }
        if (page < pages) {
            const bool kept = page < a.n_first || page >= pages - a.n_last;
            a.keys[((size_t)b * a.Hkv + hk) * a.max_pages + page] =
                kept ? ~0ull : phys < 0 || !any ? 0ull : sort_key(best);
        }
    }
}

// ---------------------------------------------------------------- choice

constexpr int kSelectThreads = 512;

// Per (row, key head): the n_sel-th largest key by 8-bit digits from the top, each digit's counts in shared
// memory (lanes with the same digit add once: the top digits of scores are nearly all alike), then the pages
// above it, and the first ones equal to it, in page order.
__global__ void __launch_bounds__(kSelectThreads) attn_select_kernel(const AttnSelectArgs a) {
    constexpr int WARPS = kSelectThreads / 32;
    __shared__ int s_count[256], s_warp[WARPS], s_digit, s_need;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / a.Hkv;
    const unsigned long long* keys = a.keys + (size_t)blockIdx.x * a.max_pages;
    int32_t* out = a.pages + (size_t)blockIdx.x * a.n_sel;
    const int len = attn_len(a.lens, b, (long long)a.max_pages * a.page_size);
    const int n = (len + a.page_size - 1) / a.page_size;
    if (n <= a.n_sel) {  // all of them
        for (int i = tid; i < a.n_sel; i += kSelectThreads) out[i] = i < n ? i : -1;
        return;
    }
    unsigned long long prefix = 0, mask = 0;
    int need = a.n_sel;  // of the keys that match the prefix
    for (int shift = 56; shift >= 0; shift -= 8) {
        if (tid < 256) s_count[tid] = 0;
        __syncthreads();
        for (int i0 = 0; i0 < n; i0 += kSelectThreads) {
            const int i = i0 + tid;
            const unsigned long long key = i < n ? keys[i] : 0;
            const int digit = i < n && (key & mask) == prefix ? (int)(key >> shift & 255) : -1;
            const unsigned same = __match_any_sync(0xffffffffu, digit);
            if (digit >= 0 && lane == __ffs(same) - 1) atomicAdd(&s_count[digit], __popc(same));
        }
        __syncthreads();
        if (warp == 0) {  // lane l: digits 255 - 8 l down to 248 - 8 l
            int sum = 0;
#pragma unroll
            for (int u = 0; u < 8; ++u) sum += s_count[255 - 8 * lane - u];
            int above = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, above, o);
                if (lane >= o) above += y;
            }
            above -= sum;  // keys with a digit above this lane's
            if (above < need && need <= above + sum) {
                int d = 255 - 8 * lane;
                while (above + s_count[d] < need) above += s_count[d--];
                s_digit = d;
                s_need = need - above;
            }
        }
        __syncthreads();
        need = s_need;
        prefix |= (unsigned long long)s_digit << shift;
        mask |= 255ull << shift;
        const bool all = s_count[s_digit] == need;
        __syncthreads();
        if (all) break;
    }
    int written = 0, ties = 0;
    for (int i0 = 0; i0 < n; i0 += kSelectThreads) {
        const int i = i0 + tid;
        const unsigned long long key = i < n ? keys[i] & mask : 0;
        const bool tie = i < n && key == prefix;
        const unsigned tied = __ballot_sync(0xffffffffu, tie);
        if (lane == 0) s_warp[warp] = __popc(tied);
        __syncthreads();
        int rank = ties + __popc(tied & ((1u << lane) - 1u));
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            if (w < warp) rank += s_warp[w];
            ties += s_warp[w];
        }
        __syncthreads();
        const bool take = i < n && (key > prefix || (tie && rank < need));
        const unsigned taken = __ballot_sync(0xffffffffu, take);
        if (lane == 0) s_warp[warp] = __popc(taken);
        __syncthreads();
        int to = written + __popc(taken & ((1u << lane) - 1u));
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            if (w < warp) to += s_warp[w];
            written += s_warp[w];
        }
        if (take && in_bounds(to, a.n_sel)) out[to] = i;
        __syncthreads();
    }
}

}  // namespace gdn
