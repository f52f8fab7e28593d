// attn_page.cuh -- the choice of cache pages that a new token attends to: the mean key of each page, kept up
// as pages fill, and for each (row, key head) the pages whose mean key scores highest.
//
//   mean_p = sum of the page's keys inside the row's length / their count            (fp32)
//   score_p = max over the query heads h of the key head's group of q_h . mean_p      (fp64)
// The first n_first and the last n_last pages are always chosen, the rest by score, ties to the lower page;
// the list is ascending, -1 behind its end.  The score is this library's own; the architecture's sparse attention has an indexer
// of its own, which this is not.
//
// Scores are summed in fp64: which page is the last to be chosen can hang on the last bits of two scores,
// and with 2^-53 the order of the sum (so the tile, or another build) no longer decides it in practice.
#pragma once
#include "attn_decode.cuh"

namespace gdn {

// ---------------------------------------------------------------- mean keys

constexpr int kMeanThreads = 128, kMeanPerSm = 7;  // CTAs an SM: the grid is one resident wave

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

// HBM-bound: a CTA takes one page of one key head (page_size x D, contiguous) after another with 16-byte loads, U of
// them in flight per thread, which is all of a page of 64 keys of 128 channels.  The next page's loads are issued before
// this one's sums are joined over the CTA, and its place in the cache is looked up one page earlier still, so memory
// never waits for the join.  Sums are fp32, in a fixed order.  Measured: 133 MB of keys on 64-key pages of 8 heads of 128,
// 26 us, 5.1 TB/s with a prologue of 5 us; looking a page up when it is its turn, 40 us.
template <bool BF, int D>
__global__ void __launch_bounds__(kMeanThreads, kMeanPerSm) attn_page_mean_kernel(const AttnMeanArgs a) {
    constexpr int LPR = D / 8, RPP = kMeanThreads / LPR, U = 8;  // lanes of a key, keys of a pass, passes in flight
    __shared__ __align__(16) float s_sum[2][RPP][D];  // written 16 bytes at a time
    const int tid = threadIdx.x, l = tid % LPR, sub = tid / LPR;
    tc::wait_prerequisites();
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
    // the walk along the line: row b, its page `first + i`, key head hk; a row's pages outside, its key heads inside
    int b = place.b, first = 0, n = 0, i = 0, hk = 0, len = 0;
    if (at < end) {
        n = attn_touched(a, b, first);
        len = a.lens[b];
        i = (int)((at - place.before) / a.Hkv);
        hk = (int)(at - place.before - (long long)i * a.Hkv);
    }
    // Next item of the line: its (page, key head) in the cache, or -1, and its keys inside the row.
    struct Item {
        long long slot;
        int count;
    };
    auto find = [&](bool more) -> Item {
        Item it{-1, 0};
        if (!more) return it;
        while (i == n) {
            n = attn_touched(a, ++b, first);
            len = a.lens[b];
            i = 0;
        }
        const int page = first + i;
        it.count = min(a.page_size, len - page * a.page_size);
        const int phys = a.table[(size_t)b * a.max_pages + page];
        if (phys < 0 || phys >= a.num_pages || it.count <= 0) {  // uniform
            if (tid == 0) raise_error(kErrPage);
        } else {
            it.slot = (long long)phys * a.Hkv + hk;
            if (!in_bounds(it.slot, (long long)a.num_pages * a.Hkv)) it.slot = -1;
        }
        if (++hk == a.Hkv) {
            hk = 0;
            ++i;
        }
        return it;
    };
    uint4 x[U];
    const uint16_t* cache = reinterpret_cast<const uint16_t*>(a.k_cache) + 8 * l;
    auto load = [&](const Item& it, int r0) {
        const uint16_t* keys = cache + it.slot * a.page_size * D;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u] = make_uint4(0, 0, 0, 0);
            if (it.slot >= 0 && r0 + u * RPP < it.count) x[u] = *reinterpret_cast<const uint4*>(keys + (size_t)(r0 + u * RPP) * D);
        }
    };

    Item now = find(at < end), next = find(at + 1 < end);
    load(now, sub);
    int parity = 0;
    for (; at < end; ++at) {
        float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int r0 = sub;;) {
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
            r0 += U * RPP;
            if (r0 >= now.count) break;
            load(now, r0);
        }
        const Item done = now;
        now = next;
        load(now, sub);
        next = find(at + 2 < end);
        if (done.slot < 0) continue;  // uniform
        stv<kF32, 8>(s_sum[parity][sub], 8 * l, sum);
        __syncthreads();  // the other buffer's readers have passed the sync before
        for (int c = tid; c < D; c += kMeanThreads) {
            float total = 0.0f;
#pragma unroll
            for (int r = 0; r < RPP; ++r) total += s_sum[parity][r][c];
            a.mean[done.slot * D + c] = total / (float)done.count;
        }
        parity ^= 1;
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

constexpr int kScoreThreads = 128, kScorePages = 8 * kScoreThreads / 32;  // 8 pages a warp

// CTAs an SM, by the registers that two pages' loads take: the grid is one resident wave.
__host__ __device__ constexpr int attn_score_per_sm(int d) { return d == 256 ? 2 : d == 128 ? 4 : 5; }

// A double as an unsigned number of the same order; NaN is the lowest.
__device__ __forceinline__ unsigned long long sort_key(double x) {
    if (x != x) return 0ull;
    const long long bits = __double_as_longlong(x + 0.0);  // -0 as 0
    return bits < 0 ? ~(unsigned long long)bits : (unsigned long long)bits | 0x8000000000000000ull;
}

__device__ __forceinline__ void dmma(double (&c)[2], double a, double b) {
    asm volatile("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0,%1}, {%2}, {%3}, {%0,%1};"
                 : "+d"(c[0]), "+d"(c[1])
                 : "d"(a), "d"(b));
}

// Scores of 32 pages of a (row, key head) at a time, 8 per warp in 8 x 8 x 4 fp64 products, whose 8 columns are
// query heads.  The contraction runs over channels in any order, so a lane's 4 channels of a page are one 16-byte load,
// all of a page's loads (8 at d = 128) are in flight together, and nothing of the means goes through shared memory;
// only the queries do, as doubles in fragment order, once per (row, key head).  The next pages' means load under this
// one's products, their places in the cache having been looked up one step earlier; four independent sums keep a step's
// products from waiting for one another.  What bounds it: HBM (the means), the products
// (8.5 us below) and the conversions to fp64, 16 a clock and SM.  12 bytes a thread spill at d = 64 and 128.  Measured: 16,800 pages of 64 rows, 8 key heads of 128,
// groups of 4: 22 us (means through shared memory and fused multiply-adds: 95); 7900 pages of 4 rows, 4 key heads: 11 us.
template <bool BF, int D>
__global__ void __launch_bounds__(kScoreThreads, attn_score_per_sm(D)) attn_score_kernel(const AttnSelectArgs a) {
    constexpr int KB = D / 16;  // 16-byte loads of a page
    __shared__ double s_q[D / 4][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    tc::wait_prerequisites();
    tc::launch_dependents();
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
    // the walk along the line: row b, key head hk, block blk of its pages; key heads outside, blocks inside
    int b = place.b, pages = 0, n = 0, hk = 0, blk = 0;
    if (at < end) {
        n = blocks_of(pages = pages_of(b));
        hk = (int)((at - place.before) / n);
        blk = (int)(at - place.before - (long long)hk * n);
    }
    struct Item {
        int b, hk, page, phys;  // this lane's page (-1: behind the row's last) and its place in the cache (-1: none)
    };
    auto find = [&](bool more) -> Item {
        Item it{0, 0, -1, -1};
        if (!more) return it;
        while (hk == a.Hkv || n == 0) {
            n = blocks_of(pages = pages_of(++b));
            hk = 0;
        }
        it.b = b;
        it.hk = hk;
        const int page = blk * kScorePages + warp * 8 + g;
        if (page < pages) {
            it.page = page;
            it.phys = attn_page(a.table, a.max_pages, a.num_pages, b, page);
            if (it.phys >= 0 && !in_bounds(it.phys, a.num_pages)) it.phys = -1;
        }
        if (++blk == n) {
            blk = 0;
            ++hk;
        }
        return it;
    };
    float4 x[KB];
    auto load = [&](const Item& it) {
        const float* mean = a.mean + ((size_t)it.phys * a.Hkv + it.hk) * D + 4 * t;
#pragma unroll
        for (int c = 0; c < KB; ++c) {
            x[c] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (it.phys >= 0) x[c] = *reinterpret_cast<const float4*>(mean + 16 * c);
        }
    };

    // The first 8 heads' queries of an item, 16 bytes at a time; heads that the group does not have are zeros.
    constexpr int QN = (D + kScoreThreads - 1) / kScoreThreads;
    uint4 raw[QN];
    auto load_q = [&](const Item& it, int h0) {
        const int heads = min(8, a.group - h0);
#pragma unroll
        for (int u = 0; u < QN; ++u) {
            const int i = tid + u * kScoreThreads, h = i / (D / 8), c = 8 * (i - h * (D / 8));
            raw[u] = make_uint4(0, 0, 0, 0);
            if (h < heads)
                raw[u] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.q) +
                                                         ((size_t)it.b * a.Hq + it.hk * a.group + h0 + h) * D + c);
        }
    };

    // channel 16 m + 4 t + j of head h stands at step 4 m + j, lane 4 h + t
    auto store_q = [&]() {
#pragma unroll
        for (int u = 0; u < QN; ++u) {
            const int i = tid + u * kScoreThreads, h = i / (D / 8), c0 = 8 * (i - h * (D / 8));
            const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
            if (h < 8) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int c = c0 + e;
                    const float2 f = unpack2<BF>(w[e >> 1]);
                    s_q[c / 16 * 4 + (c & 3)][4 * h + (c >> 2 & 3)] = (double)(e & 1 ? f.y : f.x);
                }
            }
        }
    };

    Item now = find(at < end);
    load(now);
    if (at < end) load_q(now, 0);
    Item next = find(at + 1 < end);
    int held = -1;  // the (row, key head) whose queries are in s_q
    for (; at < end; ++at) {
        float4 m[KB];
#pragma unroll
        for (int c = 0; c < KB; ++c) m[c] = x[c];
        const Item item = now;
        if (held != item.b * a.Hkv + item.hk || a.group > 8) {
            if (held >= 0 && a.group > 8) load_q(item, 0);  // the last ones loaded were another part of the group
            __syncthreads();                                // the queries before them have been read
            held = item.b * a.Hkv + item.hk;
            store_q();
            __syncthreads();
        }
        now = next;
        load(now);
        if (at + 1 < end && a.group <= 8 && (now.b != item.b || now.hk != item.hk)) load_q(now, 0);
        next = find(at + 2 < end);
        unsigned long long best = 0;
        for (int h0 = 0; h0 < a.group; h0 += 8) {
            const int heads = min(8, a.group - h0);
            if (h0 > 0) {
                load_q(item, h0);
                __syncthreads();
                store_q();
                __syncthreads();
            }
            double sum[4][2];
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j][0] = sum[j][1] = 0.0;
#pragma unroll
            for (int c = 0; c < KB; ++c) {
                dmma(sum[0], (double)m[c].x, s_q[4 * c][lane]);
                dmma(sum[1], (double)m[c].y, s_q[4 * c + 1][lane]);
                dmma(sum[2], (double)m[c].z, s_q[4 * c + 2][lane]);
                dmma(sum[3], (double)m[c].w, s_q[4 * c + 3][lane]);
            }
            // lane (g, t): page g, heads 2 t and 2 t + 1
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const double score = (sum[0][e] + sum[1][e]) + (sum[2][e] + sum[3][e]);
                const unsigned long long key = 2 * t + e < heads ? sort_key(score) : 0ull;
                best = key > best ? key : best;
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            const unsigned long long key = __shfl_xor_sync(0xffffffffu, best, o);
            best = key > best ? key : best;
        }
        if (t == 0 && item.page >= 0)
            a.keys[((size_t)item.b * a.Hkv + item.hk) * a.max_pages + item.page] = item.phys < 0 ? 0ull : best;
    }
}

// ---------------------------------------------------------------- choice

constexpr int kSelectThreads = 256;

// Per (row, key head): the pages always kept, and of the others those with the largest keys.  The smallest key taken is
// found by 8-bit digits, from the highest bit in which the keys differ, each digit's counts in shared memory; then come
// the pages above it and the first ones equal to it, in page order.  The first 2048 pages' keys stay in registers.
// Latency-bound: one CTA per list, three or four digits of two barriers each.  Measured: 16 lists of 2000 pages 7.5 us, 512
// lists of up to 512 pages 9 us.
__global__ void __launch_bounds__(kSelectThreads, 4) attn_select_kernel(const AttnSelectArgs a) {
    constexpr int WARPS = kSelectThreads / 32, C = 8, SPAN = C * kSelectThreads;
    static_assert(kSelectThreads == 256, "one thread per digit");
    __shared__ __align__(16) int s_count[2][256];
    __shared__ int s_part[C * WARPS], s_total, s_digit, s_need;
    __shared__ unsigned s_bits[4];  // OR of the keys' words, and of their complements
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / a.Hkv;
    const unsigned long long* keys = a.keys + (size_t)blockIdx.x * a.max_pages;
    int32_t* out = a.pages + (size_t)blockIdx.x * a.n_sel;
    tc::wait_prerequisites();
    tc::launch_dependents();
    const int len = attn_len(a.lens, b, (long long)a.max_pages * a.page_size);
    const int n = (len + a.page_size - 1) / a.page_size;
    if (n <= a.n_sel) {  // all of them
        for (int i = tid; i < a.n_sel; i += kSelectThreads) out[i] = i < n ? i : -1;
        return;
    }
    auto kept = [&](int i) { return i < a.n_first || i >= n - a.n_last; };
    unsigned long long reg[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int i = c * kSelectThreads + tid;
        reg[c] = i < n && !kept(i) ? keys[i] : 0ull;
    }
    // f(page, key) for this thread's pages that are not kept
    auto each = [&](auto f) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = c * kSelectThreads + tid;
            if (c * kSelectThreads >= n) break;
            if (i < n && !kept(i)) f(i, reg[c]);
        }
        for (int i = SPAN + tid; i < n; i += kSelectThreads)
            if (!kept(i)) f(i, keys[i]);
    };
    const int need_all = a.n_sel - a.n_first - a.n_last;
    if (tid < 4) s_bits[tid] = 0;
    s_count[0][tid] = 0;
    __syncthreads();
    unsigned long long ones = 0, zeros = 0;
    each([&](int, unsigned long long key) {
        ones |= key;
        zeros |= ~key;
    });
    const unsigned bits[4] = {__reduce_or_sync(0xffffffffu, (unsigned)(ones >> 32)), __reduce_or_sync(0xffffffffu, (unsigned)ones),
                              __reduce_or_sync(0xffffffffu, (unsigned)(zeros >> 32)), __reduce_or_sync(0xffffffffu, (unsigned)zeros)};
    if (lane < 4) {
        const unsigned mine = lane == 0 ? bits[0] : lane == 1 ? bits[1] : lane == 2 ? bits[2] : bits[3];
        atomicOr(&s_bits[lane], mine);
    }
    __syncthreads();
    const unsigned long long differ =
        ((unsigned long long)s_bits[0] << 32 | s_bits[1]) & ((unsigned long long)s_bits[2] << 32 | s_bits[3]);
    // `mask`: the bits settled so far, `prefix`: their value in the smallest key taken, `need`: how many are still
    // wanted of the keys that agree in them
    int top = differ == 0 ? -1 : 63 - __clzll((long long)differ);
    unsigned long long mask = top < 0 ? ~0ull : ~((2ull << top) - 1ull);  // top = 63: the shift gives 0, the mask 0
    unsigned long long prefix = ((unsigned long long)s_bits[0] << 32 | s_bits[1]) & mask;
    int need = need_all;
    bool all = need == 0;
    for (int turn = 0; top >= 0 && !all; ++turn) {
        const int shift = top >= 7 ? top - 7 : 0, width = top - shift + 1;
        int* count = s_count[turn & 1];
        each([&](int, unsigned long long key) {
            if ((key & mask) == prefix) atomicAdd(&count[(int)(key >> shift) & ((1 << width) - 1)], 1);
        });
        s_count[(turn & 1) ^ 1][tid] = 0;
        __syncthreads();
        if (warp == 0) {  // lane l: digits 255 - 8 l down to 248 - 8 l
            const int4 hi = reinterpret_cast<const int4*>(count)[63 - 2 * lane], lo = reinterpret_cast<const int4*>(count)[62 - 2 * lane];
            const int v[8] = {hi.w, hi.z, hi.y, hi.x, lo.w, lo.z, lo.y, lo.x};
            int sum = 0;
#pragma unroll
            for (int u = 0; u < 8; ++u) sum += v[u];
            int above = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, above, o);
                if (lane >= o) above += y;
            }
            above -= sum;  // keys with a digit above this lane's
            if (above < need && need <= above + sum) {
                int d = 255 - 8 * lane;
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    if (above < need && need <= above + v[u]) {
                        s_digit = d - u;
                        s_need = need - above;
                        s_total = v[u];
                    }
                    above += v[u];
                }
            }
        }
        __syncthreads();
        need = s_need;
        all = s_total == need;
        prefix |= (unsigned long long)s_digit << shift;
        mask |= ((1ull << width) - 1ull) << shift;
        top = shift - 1;
    }
    // Place of each flagged page among the flagged ones of this span; the number of them.
    auto ranks = [&](const bool (&flag)[C], int (&rank)[C]) -> int {
        unsigned vote[C];
        __syncthreads();
#pragma unroll
        for (int c = 0; c < C; ++c) {
            vote[c] = __ballot_sync(0xffffffffu, flag[c]);
            if (lane == 0) s_part[c * WARPS + warp] = __popc(vote[c]);
        }
        __syncthreads();
        if (warp == 0) {
            constexpr int E = C * WARPS / 32;
            int v[E], sum = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                v[e] = sum;
                sum += s_part[lane * E + e];
            }
            int incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
#pragma unroll
            for (int e = 0; e < E; ++e) s_part[lane * E + e] = v[e] + incl - sum;
            if (lane == 31) s_total = incl;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < C; ++c) rank[c] = s_part[c * WARPS + warp] + __popc(vote[c] & ((1u << lane) - 1u));
        return s_total;
    };
    int written = 0, ties = 0;
    for (int i0 = 0; i0 < n; i0 += SPAN) {
        bool take[C], tie[C];
        int rank[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = i0 + c * kSelectThreads + tid;
            const bool fixed = i < n && kept(i);
            const unsigned long long key = i0 == 0 ? reg[c] : i < n ? keys[i] : 0ull;
            tie[c] = i < n && !fixed && (key & mask) == prefix && need_all > 0;
            take[c] = fixed || (i < n && need_all > 0 && (key & mask) > prefix) || (tie[c] && all);
        }
        if (!all) {  // more equal keys than wanted: the first ones
            const int found = ranks(tie, rank);
#pragma unroll
            for (int c = 0; c < C; ++c) take[c] |= tie[c] && ties + rank[c] < need;
            ties += found;
        }
        const int found = ranks(take, rank);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int i = i0 + c * kSelectThreads + tid, to = written + rank[c];
            if (take[c] && in_bounds(to, a.n_sel)) out[to] = i;
        }
        written += found;
    }
}

}  // namespace gdn
