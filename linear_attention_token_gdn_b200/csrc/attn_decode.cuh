// attn_decode.cuh -- softmax attention of one new token per row over a paged key-value cache, the
// serving step of the attention layer between GDN mixers, over all of a row's keys or over chosen pages.
//
// Per (row, query head), over the row's keys j (key head = query head / group):
//   s_j = scale q . k_j,   y = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m),   m = max_j s_j.
// One pass with a running m, l = sum e^(s - m) and o = sum e^(s - m) v, all fp32.
//
// Bound by HBM: every key and value is read once (4 flop per 2-byte element and query head of the group).
//
// Split.  The rows' lengths live on the device, so the grid is fixed (every CTA resident) and the
// work is cut on the device: the tiles of 16 keys of all (row, key head) pairs stand in one line, and
// each CTA takes an equal stretch of it.  A stretch holds whole pairs, whose results are final, and at
// most two pieces of pairs that neighbours share: o, m and l of those go to the workspace, and a second
// small kernel joins them in the order of the line, so results do not depend on timing.
//
// Tile.  A warp takes 16 keys at a time, S^T = K Q^T and O^T = V^T P^T by mma.sync m16n8k16: the group's
// query heads are the 8 columns (16 in two tiles), so a group of 8 wastes nothing.  Each warp has a ring of its own in
// shared memory, of 3 slots of 16 keys or values, which its lanes fill by 16-byte asynchronous copies, so that two slots
// (8 KB at d = 128) a warp are under way whatever the registers hold, and nothing waits for another warp.  Chunks of
// a row are swizzled by the row, and ldmatrix (transposed for V) delivers the fragments without bank conflicts.  Q lies
// there too: it would take up to 64 registers.  P goes from the accumulators to the B operand by movmatrix.  Places
// behind the row's last key are filled with zeros instead of being read.
// P enters as a 16-bit value and its 16-bit remainder: a single rounding (2^-8 for bf16) would add as much
// error as the output's own rounding, and the tensor pipe has the room (16 % busy).
// m follows the scores lazily: it moves only when a score exceeds it by more than 8 (in log2), so p is at
// most 2^8, and most tiles need one vote instead of a reduction over lanes and a rescale.
//
// Measured: 64 rows of up to 8192 bf16 keys, 32 heads over 8 key heads of 128, 171 to 175 us, 6.2 TB/s, 94 to 96 % of a copy's
// rate; one row of 131,001 fp16 keys, 16 heads over 2 of 256, 51 us, 5.3 TB/s.
#pragma once
#include "attn_prep.cuh"
#include "common.cuh"
#include "warp_mma.cuh"

namespace gdn {

constexpr int kAttnWarps = 4, kAttnThreads = 32 * kAttnWarps;
constexpr int kAttnMaxCtas = 640;  // grid bound: sizes the workspace
constexpr int kAttnMinTiles = 4;   // least tiles per CTA: one per warp

// A place in the line of all rows' work items: row `b`, whose items start at `before`; `total` of all rows.
struct AttnPlace {
    int b;
    long long before, total;
};

__device__ __forceinline__ long long warp_scan(long long x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if ((int)(threadIdx.x & 31) >= o) x += y;
    }
    return x;
}

// Finds the row of item `target(total)` in the line of count(b) items for b < B; all threads of the CTA call
// it and get the same answer.  b = B when the target is not below the total.
template <int THREADS, class Count, class Target>
__device__ __forceinline__ AttnPlace attn_locate(int B, Count count, Target target) {
    if (B <= 32) {  // each warp for itself
        const int lane = threadIdx.x & 31;
        const long long n = lane < B ? count(lane) : 0, incl = warp_scan(n);
        AttnPlace p;
        p.total = __shfl_sync(0xffffffffu, incl, 31);
        const long long want = target(p.total);
        const unsigned hit = __ballot_sync(0xffffffffu, want < incl && want >= incl - n);
        const int src = hit != 0 ? __ffs(hit) - 1 : 0;
        const long long before = __shfl_sync(0xffffffffu, incl - n, src);
        p.b = hit != 0 ? src : B;
        p.before = hit != 0 ? before : p.total;
        return p;
    }
    __shared__ long long s_warp[THREADS / 32];
    __shared__ long long s_before;
    __shared__ int s_b;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long total = 0;
    for (int b = threadIdx.x; b < B; b += THREADS) total += count(b);
    long long first = total;  // this thread's row of the first (often only) chunk, when B <= THREADS
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) s_warp[warp] = total;
    if (threadIdx.x == 0) s_b = B;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) total += s_warp[w];
    const long long want = target(total);
    long long carry = 0;
    if (want < total) {
        for (int base = 0; base < B; base += THREADS) {
            const int b = base + threadIdx.x;
            const long long n = B <= THREADS ? first : (b < B ? count(b) : 0);
            long long incl = warp_scan(n);
            __syncthreads();  // s_warp read by everyone
            if (lane == 31) s_warp[warp] = incl;
            __syncthreads();
            incl += carry;
#pragma unroll
            for (int w = 0; w < THREADS / 32; ++w) {
                if (w < warp) incl += s_warp[w];
                carry += s_warp[w];
            }
            if (b < B && want < incl && want >= incl - n) {
                s_b = b;
                s_before = incl - n;
            }
            if (carry > want) break;  // uniform: carry is the same in all threads
        }
    }
    __syncthreads();
    AttnPlace p;
    p.b = s_b;
    p.before = s_b < B ? s_before : total;
    p.total = total;
    return p;
}

// Length of row b, bounded (and flagged) to what its page table can hold.
__device__ __forceinline__ int attn_len(const int32_t* lens, int b, long long capacity) {
    const int n = lens[b];
    if (n < 0 || n > capacity) {
        raise_error(kErrPage);
        return n < 0 ? 0 : (int)capacity;
    }
    return n;
}

struct AttnDecodeArgs {
    const void *q, *k_cache, *v_cache;
    const int32_t *table, *lens, *pages;        // pages: [B, Hkv, n_sel] logical pages, or NULL (all)
    int B, Hq, Hkv, group, hblocks;             // hblocks: blocks of 8 NT heads per group
    int num_pages, page_size, max_pages, n_sel, tiles_per_page;
    float scale_log2;                           // scale * log2(e)
    int y_dt;
    void* y;
    // meta, where a piece is a CTA's part of a pair, a pair a (row, key head, head block), and a pair's pieces are in
    // CTAs that follow one another.  by_pair: [pair][2], the CTA of the first piece and the number of pieces (1 or 0: no
    // join).  Otherwise [CTA][2], the pair whose first piece the CTA holds (-1: none, or the only one) and their number.
    int* meta;
    int by_pair;
    int alone;                                  // one CTA per pair, no piece
    float* part;                                // [grid][2][8 NT][D + 2]: o, then m and l (log2 scale)
};

// The tiles of a row of `len` keys for one of its (key head, head block) pairs.  With listed pages every row has the
// same number, whatever its length.
template <bool CHOSEN>
__device__ __forceinline__ int attn_tiles(const AttnDecodeArgs& a, int len) {
    return CHOSEN ? a.n_sel * a.tiles_per_page : (len + 15) >> 4;
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// (x0, x1) -> 16-bit pairs hi = round(x), lo = round(x - hi)
template <bool BF>
__device__ __forceinline__ void split16(float x0, float x1, uint32_t& hi, uint32_t& lo) {
    hi = pack2<BF>(x0, x1);
    const float2 f = unpack2<BF>(hi);
    lo = pack2<BF>(x0 - f.x, x1 - f.y);
}

template <int D, int NT>
struct AttnShape {
    static constexpr int MT = D / 16;                    // 16-channel steps of S^T, tiles of O^T
    static constexpr int HB = 8 * NT;                    // heads of a block
    static constexpr int PIECE = HB * (D + 2);           // floats of a piece: o, m, l
    static constexpr int HALF = 16 * D * 2;              // bytes of a slot: 16 keys or values
    static constexpr int SLOTS = 3;                      // keys and values of a tile, and the next tile's keys
    static constexpr int OROW = D + 4;                   // floats of a joined row: 2 OROW = 8 mod 32, no bank conflicts
    static constexpr int RING = kAttnWarps * SLOTS * HALF, JOIN = kAttnWarps * HB * OROW * 4;
    static constexpr int BODY = RING > JOIN ? RING : JOIN;  // the warps' rings, then their results
    static constexpr int SMEM = 512 + BODY + HB * D * 2 + 2 * kAttnWarps * HB * 4;  // 512 to align the rings to a row
    // p is formed 2^7 larger for fp16, at most 2^15: small weights then keep 7 more bits above fp16's smallest step.
    // l carries the same factor, so it drops out.
    __host__ __device__ static constexpr float kLift(bool bf) { return bf ? 0.0f : 7.0f; }
};

// What the 16-byte chunk number of a row in shared memory is combined with (exclusive or).
template <int D>
__host__ __device__ constexpr int attn_swizzle(int row) {
    return D == 32 ? row >> 1 & 3 : row & 7;
}

__device__ __forceinline__ void cp_async16(uint32_t to, const void* from, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}

template <bool BF, int D, int NT, bool CHOSEN>
__global__ void __launch_bounds__(kAttnThreads, D == 256 ? 2 : D == 128 && NT == 2 ? 3 : 4) attn_decode_kernel(const AttnDecodeArgs a) {
    using S = AttnShape<D, NT>;
    extern __shared__ __align__(512) char s_raw[];       // rings or results, Q, then m and l [warp][head]
    char* const s_body = s_raw + ((512u - (tc::smem_u32(s_raw) & 511u)) & 511u);
    float* const s_o = reinterpret_cast<float*>(s_body);
    char* const s_q = s_body + S::BODY;
    float* const s_m = reinterpret_cast<float*>(s_q + S::HB * D * 2);
    float* const s_l = s_m + kAttnWarps * S::HB;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int pairs = a.Hkv * a.hblocks;                 // work rows of a row
    const long long capacity = (long long)a.max_pages * a.page_size;
    const int cta = blockIdx.x;

    tc::wait_prerequisites();
    tc::launch_dependents();  // every CTA is resident: the join's take no place from them

    // rows without a key (with listed pages, their tiles are empty instead)
    for (int b = CHOSEN ? a.B : cta; b < a.B; b += gridDim.x) {
        if (a.lens[b] <= 0) {
            for (int i = tid; i < a.Hq * D; i += kAttnThreads) st1(a.y, a.y_dt, (size_t)b * a.Hq * D + i, 0.0f);
            if (a.by_pair && !a.alone)
                for (int i = tid; i < pairs; i += kAttnThreads) a.meta[2 * (b * pairs + i) + 1] = 0;
        }
    }

    long long share = 1, at, end, row_base;              // row_base: the line's index of b's first tile
    int b;
    if (a.alone) {
        b = cta / pairs;
        const int tiles = attn_tiles<CHOSEN>(a, CHOSEN ? 0 : attn_len(a.lens, b, capacity));
        row_base = 0;
        at = (long long)(cta - b * pairs) * tiles;
        end = at + tiles;
    } else {
        auto cut = [&](long long total) {
            share = (total + gridDim.x - 1) / gridDim.x;
            share = (share + kAttnMinTiles - 1) / kAttnMinTiles * kAttnMinTiles;
            return share * cta;
        };
        long long total;
        if constexpr (CHOSEN) {
            const long long row = (long long)attn_tiles<CHOSEN>(a, 0) * pairs;
            total = row * a.B;
            at = cut(total);
            b = at < total ? (int)(at / row) : a.B;
            row_base = b * row;
        } else {
            const AttnPlace place = attn_locate<kAttnThreads>(
                a.B, [&](int row) { return (long long)attn_tiles<CHOSEN>(a, attn_len(a.lens, row, capacity)) * pairs; }, cut);
            total = place.total;
            at = share * cta;
            b = place.b;
            row_base = place.before;
        }
        end = at + share < total ? at + share : total;
    }
    int starting = -1, pieces = 0;

    while (at < end) {                                   // one (row, key head, head block) piece per turn
        int len = attn_len(a.lens, b, capacity);
        int tiles = attn_tiles<CHOSEN>(a, len);
        while (at >= row_base + (long long)tiles * pairs) {
            row_base += (long long)tiles * pairs;
            ++b;
            len = attn_len(a.lens, b, capacity);
            tiles = attn_tiles<CHOSEN>(a, len);
        }
        const int pair = (int)((at - row_base) / tiles);
        const int hk = pair / a.hblocks, hb = pair - hk * a.hblocks;
        const int first = (int)(at - row_base - (long long)pair * tiles);
        const int last = (int)(end - at < tiles - first ? first + (end - at) : tiles);  // tiles [first, last)
        const int h0 = hk * a.group + hb * S::HB;
        const int heads = min(S::HB, a.group - hb * S::HB);
        const int32_t* table = a.table + (size_t)b * a.max_pages;
        const int32_t* list = CHOSEN ? a.pages + ((size_t)b * a.Hkv + hk) * a.n_sel : nullptr;
        const int row_pages = (len + a.page_size - 1) / a.page_size;

        float o[NT][S::MT][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < S::MT; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.0f;
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.0f;
        }

        // The warp's tiles are first + warp, + kAttnWarps, ...  Their places go through three steps, each a tile ahead of the
        // next, so that no load of the list or of the table is waited for: the logical page, the physical one, the place.
        struct Look {
            int page, off, phys;  // page: -1 when the tile has no key
        };
        struct Tile {
            size_t base;
            int n;
        };
        int tiles_left = (last - first - warp + kAttnWarps - 1) / kAttnWarps;
        int l_slot = (first + warp) / a.tiles_per_page, l_off = first + warp - l_slot * a.tiles_per_page;
        const int step_pages = kAttnWarps / a.tiles_per_page, step_off = kAttnWarps - step_pages * a.tiles_per_page;
        auto list_page = [&](Look& x) {
            x.page = -1;
            x.off = l_off;
            if (tiles_left-- > 0) x.page = CHOSEN ? list[l_slot] : l_slot;
            l_slot += step_pages;
            l_off += step_off;
            if (l_off >= a.tiles_per_page) {
                l_off -= a.tiles_per_page;
                ++l_slot;
            }
        };
        auto look_up = [&](Look& x) {
            if (x.page < 0) return;                      // behind the piece, or padding of the list
            if (CHOSEN && x.page >= row_pages) {
                if (lane == 0) raise_error(kErrPage);
                x.page = -1;
            } else if (len <= x.page * a.page_size + x.off * 16) {
                x.page = -1;
            } else {
                x.phys = table[x.page];
            }
        };
        auto settle = [&](const Look& x) -> Tile {
            if (x.page < 0) return Tile{0, 0};
            if (x.phys < 0 || x.phys >= a.num_pages) {
                if (lane == 0) raise_error(kErrPage);
                return Tile{0, 0};
            }
            const size_t base = (((size_t)x.phys * a.Hkv + hk) * a.page_size + x.off * 16) * D;
            if (!in_bounds((long long)base + 16 * D - 1, (long long)a.num_pages * a.Hkv * a.page_size * D)) return Tile{0, 0};
            return Tile{base, min(16, len - (x.page * a.page_size + x.off * 16))};
        };
        // Slot `slot` of the warp's ring <- the n keys or values from element `base` on; zeros behind them.
        constexpr int CPR = D / 8, RPI = 32 / CPR;       // 16-byte chunks of a row, rows of a copy instruction
        const int r0 = lane / CPR, col = lane % CPR;
        const uint32_t ring = tc::smem_u32(s_body) + warp * (S::SLOTS * S::HALF);
        const uint32_t fill = ring + r0 * (D * 2) + ((col ^ attn_swizzle<D>(r0)) << 4);
        auto copy = [&](const void* cache, size_t base, int n, int slot) {
            if (n > 0) {
                const uint16_t* p = reinterpret_cast<const uint16_t*>(cache) + base + r0 * D + 8 * col;
#pragma unroll
                for (int i = 0; i < 16 / RPI; ++i)
                    cp_async16((fill + slot * S::HALF + i * RPI * (D * 2)) ^ (attn_swizzle<D>(i * RPI) << 4), p + i * RPI * D,
                               r0 + i * RPI < n ? 16 : 0);
            }
            tc::cp_async_commit();
        };

        // Q is asked for before the places, which take two loads that wait for one another
        constexpr int QN = (S::HB * CPR + kAttnThreads - 1) / kAttnThreads;
        uint4 qx[QN];
#pragma unroll
        for (int u = 0; u < QN; ++u) {
            const int i = tid + u * kAttnThreads, h = i / CPR, c = i - h * CPR;
            qx[u] = make_uint4(0, 0, 0, 0);
            if (h < heads)
                qx[u] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.q) + ((size_t)b * a.Hq + h0 + h) * D + 8 * c);
        }
        const int tiles_mine = tiles_left;
        Look look0, look1, look2, look3;
        list_page(look0);
        list_page(look1);
        list_page(look2);
        list_page(look3);
        look_up(look0);
        look_up(look1);
        look_up(look2);
        Tile now = settle(look0);
        copy(a.k_cache, now.base, now.n, 0);
        copy(a.v_cache, now.base, now.n, 1);
        Tile next = settle(look1);
        copy(a.k_cache, next.base, next.n, 2);

#pragma unroll
        for (int u = 0; u < QN; ++u) {
            const int i = tid + u * kAttnThreads, h = i / CPR, c = i - h * CPR;
            if (i < S::HB * CPR) *reinterpret_cast<uint4*>(s_q + h * (D * 2) + ((c ^ attn_swizzle<D>(h)) << 4)) = qx[u];
        }
        __syncthreads();

        // This lane's row and chunk of the first step's matrices; a step on is an exclusive or with 32 bytes, as rows are
        // aligned to their size.
        const int mat = lane >> 3, row = lane & 7;
        const int k_row = row + 8 * (mat & 1), v_row = row + 8 * (mat >> 1), q_row = NT == 2 ? row + 8 * (mat >> 1) : row;
        const uint32_t k_at = ring + k_row * (D * 2) + (((mat >> 1) ^ attn_swizzle<D>(k_row)) << 4);
        const uint32_t v_at = ring + v_row * (D * 2) + (((mat & 1) ^ attn_swizzle<D>(v_row)) << 4);
        const uint32_t q_at = tc::smem_u32(s_q) + q_row * (D * 2) + (((NT == 2 ? mat & 1 : mat) ^ attn_swizzle<D>(q_row)) << 4);

        int slot = 0;
        auto turn = [&]() { slot = slot + 1 == S::SLOTS ? 0 : slot + 1; };
        for (int k = 0; k < tiles_mine; ++k) {
            const int n_now = now.n;
            const Tile after = settle(look2);
            look2 = look3;
            look_up(look2);
            list_page(look3);
            if (n_now == 0) {  // only the ring goes on
                copy(a.v_cache, next.base, next.n, slot);
                turn();
                copy(a.k_cache, after.base, after.n, slot);
                turn();
                now = next;
                next = after;
                continue;
            }
            tc::cp_async_wait<S::SLOTS - 1>();
            __syncwarp();
            float s[NT][4], odd[NT][4];  // the odd steps' part: half as long a chain of dependent products
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] = odd[n][e] = 0.0f;
            }
            uint32_t qf[4];
#pragma unroll
            for (int c = 0; c < S::MT; ++c) {
                uint32_t kf[4];
                wm::ldsm_x4((k_at + slot * S::HALF) ^ (c << 5), kf);
                if constexpr (NT == 2) {
                    wm::ldsm_x4(q_at ^ (c << 5), qf);
                    wm::mma16816x<BF>(c % 2 ? odd[0] : s[0], kf, qf[0], qf[1]);
                    wm::mma16816x<BF>(c % 2 ? odd[NT - 1] : s[NT - 1], kf, qf[2], qf[3]);
                } else {  // two steps' fragments at a time
                    if (c % 2 == 0) wm::ldsm_x4(q_at ^ (c << 5), qf);
                    wm::mma16816x<BF>(c % 2 ? odd[0] : s[0], kf, qf[c % 2 * 2], qf[c % 2 * 2 + 1]);
                }
            }
            __syncwarp();
            copy(a.v_cache, next.base, next.n, slot);
            turn();

            // lane (g, t): keys g (0, 1) and g + 8 (2, 3) of heads 2 t and 2 t + 1
            bool grow = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[n][e] = (s[n][e] + odd[n][e]) * a.scale_log2;
                    if (g + 8 * (e >> 1) >= n_now) s[n][e] = -INFINITY;
                    grow |= s[n][e] > m[n][e & 1] + 8.0f;
                }
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = fmaxf(m[n][e], fmaxf(s[n][e], s[n][e + 2]));
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                        const float f = top == -INFINITY ? 1.0f : exp2f(m[n][e] - top);
                        m[n][e] = top;
                        l[n][e] *= f;
#pragma unroll
                        for (int i = 0; i < S::MT; ++i) {
                            o[n][i][e] *= f;
                            o[n][i][e + 2] *= f;
                        }
                    }
                }
            }
            uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float m0 = (m[n][0] == -INFINITY ? 0.0f : m[n][0]) - S::kLift(BF);
                const float m1 = (m[n][1] == -INFINITY ? 0.0f : m[n][1]) - S::kLift(BF);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float p0 = exp2f(s[n][2 * i] - m0), p1 = exp2f(s[n][2 * i + 1] - m1);
                    l[n][0] += p0;
                    l[n][1] += p1;
                    uint32_t hi, lo;
                    split16<BF>(p0, p1, hi, lo);
                    ph[n][i] = movmatrix(hi);
                    pl[n][i] = movmatrix(lo);
                }
            }
            tc::cp_async_wait<S::SLOTS - 1>();
            __syncwarp();
#pragma unroll
            for (int c = 0; c < S::MT; ++c) {
                uint32_t vt[4];
                wm::ldsm_x4_t((v_at + slot * S::HALF) ^ (c << 5), vt);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    wm::mma16816x<BF>(o[n][c], vt, pl[n][0], pl[n][1]);
                    wm::mma16816x<BF>(o[n][c], vt, ph[n][0], ph[n][1]);
                }
            }
            __syncwarp();
            copy(a.k_cache, after.base, after.n, slot);
            turn();
            now = next;
            next = after;
        }

        // the warps' results side by side, then joined
        __syncthreads();  // every warp is through with its ring
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], x);
                const int h = 8 * n + 2 * t + e;
                float* dst = s_o + (warp * S::HB + h) * S::OROW + g;
#pragma unroll
                for (int c = 0; c < S::MT; ++c) {
                    dst[16 * c] = o[n][c][e];
                    dst[16 * c + 8] = o[n][c][e + 2];
                }
                if (g == 0) {
                    s_m[warp * S::HB + h] = m[n][e];
                    s_l[warp * S::HB + h] = l[n][e];
                }
            }
        }
        __syncthreads();
        const bool whole = first == 0 && last == tiles;
        if (first == 0 && !a.alone) {
            const int last_cta = (int)((row_base + (long long)(pair + 1) * tiles - 1) / share);
            if (!whole) {
                starting = b * pairs + pair;
                pieces = last_cta - cta + 1;
            }
            if (a.by_pair && tid == 0) {
                a.meta[2 * (b * pairs + pair)] = cta;
                a.meta[2 * (b * pairs + pair) + 1] = last_cta - cta + 1;
            }
        }
        float* piece = a.part + ((size_t)cta * 2 + (first == 0 ? 1 : 0)) * S::PIECE;
        for (int i = tid; i < heads * (D / 2); i += kAttnThreads) {
            const int h = i / (D / 2), c = 2 * (i - h * (D / 2));
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, s_m[w * S::HB + h]);
            float sum = 0.0f, y0 = 0.0f, y1 = 0.0f;
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) {
                const float mw = s_m[w * S::HB + h];
                const float f = mw == -INFINITY ? 0.0f : exp2f(mw - top);
                const float2 x = *reinterpret_cast<const float2*>(s_o + (w * S::HB + h) * S::OROW + c);
                sum += f * s_l[w * S::HB + h];
                y0 += f * x.x;
                y1 += f * x.y;
            }
            if (whole) {
                const size_t y = ((size_t)b * a.Hq + h0 + h) * D + c;
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;  // no key left: zeros
                st1(a.y, a.y_dt, y, y0 * inv);
                st1(a.y, a.y_dt, y + 1, y1 * inv);
            } else {
                *reinterpret_cast<float2*>(piece + h * D + c) = make_float2(y0, y1);
                if (c == 0) *reinterpret_cast<float2*>(piece + S::HB * D + 2 * h) = make_float2(top, sum);
            }
        }
        at += last - first;
        if (at < end) __syncthreads();  // the next piece's keys go where the results are
    }
    if (!a.by_pair && !a.alone && tid == 0) {
        a.meta[2 * cta] = starting;
        a.meta[2 * cta + 1] = pieces;
    }
}

// Joins the pieces of a (row, key head, head block) that several CTAs share: y = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,
// M = max m_i.  CTA x takes pair x (by_pair), or the pair whose first piece CTA x of the first kernel held, blockIdx.y
// `per` heads of it, blockIdx.z C channels
// of it, with W / per warps a head, each taking every (W / per)-th piece, BATCH of them loaded together.
// Latency-bound; behind the first kernel it adds 2.3 us for the 64 rows, 4 us for the 296 pieces of the long row (walking from
// piece to piece to find their number: 37).
template <int D, int NT, int W, int C>
__global__ void __launch_bounds__(32 * W) attn_join_kernel(const AttnDecodeArgs a, int ctas, int per) {
    using S = AttnShape<D, NT>;
    constexpr int E = C / 32, V = E < 4 ? E : 4;  // channels of a lane, of one load
    constexpr int BATCH = E <= 2 ? 12 : E < 8 ? 8 : 6;
    __shared__ float s_o[W][C], s_m[W], s_l[W];
    tc::wait_prerequisites();
    const int held = a.meta[2 * blockIdx.x], pieces = a.meta[2 * blockIdx.x + 1];
    const int row = a.by_pair ? blockIdx.x : held, cta0 = a.by_pair ? held : blockIdx.x;
    if (a.by_pair ? pieces <= 1 : row < 0) return;
    if (!in_bounds(cta0 + pieces - 1, ctas)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int hb = row % a.hblocks, hk = row / a.hblocks % a.Hkv, b = row / a.hblocks / a.Hkv;
    const int heads = min(S::HB, a.group - hb * S::HB);
    const int strides = W / per;
    const int h = blockIdx.y * per + warp % per, sub = warp / per;
    const int c0 = blockIdx.z * C;
    const size_t y0 = ((size_t)b * a.Hq + hk * a.group + hb * S::HB + h) * D + c0;
    float top = -INFINITY, sum = 0.0f, y[E];
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = 0.0f;
    if (h < heads) {
        for (int i0 = sub; i0 < pieces; i0 += strides * BATCH) {
            float m[BATCH], lsum[BATCH], o[BATCH][E];
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                const int i = i0 + u * strides;
                m[u] = -INFINITY;
                lsum[u] = 0.0f;
#pragma unroll
                for (int e = 0; e < E; ++e) o[u][e] = 0.0f;
                if (i < pieces) {
                    const float* p = a.part + ((size_t)(cta0 + i) * 2 + (i == 0 ? 1 : 0)) * S::PIECE;
                    const float2 ml = *reinterpret_cast<const float2*>(p + S::HB * D + 2 * h);
                    m[u] = ml.x;
                    lsum[u] = ml.y;
#pragma unroll
                    for (int e = 0; e < E; e += V) {
                        if constexpr (V == 4) *reinterpret_cast<float4*>(&o[u][e]) = *reinterpret_cast<const float4*>(p + h * D + c0 + 32 * e + 4 * lane);
                        else if constexpr (V == 2) *reinterpret_cast<float2*>(&o[u][e]) = *reinterpret_cast<const float2*>(p + h * D + c0 + 2 * lane);
                        else o[u][e] = p[h * D + c0 + lane];
                    }
                }
            }
            float next = top;
#pragma unroll
            for (int u = 0; u < BATCH; ++u) next = fmaxf(next, m[u]);
            const float f0 = top == -INFINITY ? 0.0f : exp2f(top - next);
            sum *= f0;
#pragma unroll
            for (int e = 0; e < E; ++e) y[e] *= f0;
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                const float f = m[u] == -INFINITY ? 0.0f : exp2f(m[u] - next);
                sum = fmaf(f, lsum[u], sum);
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] = fmaf(f, o[u][e], y[e]);
            }
            top = next;
        }
    }
    if (strides == 1) {
        if (h < heads) {
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;  // no key left: zeros
#pragma unroll
            for (int e = 0; e < E; ++e) st1(a.y, a.y_dt, y0 + 32 * (e / V * V) + V * lane + e % V, y[e] * inv);
        }
        return;
    }
    // one head (per = 1): its warps' sums side by side, then one thread a channel
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][32 * (e / V * V) + V * lane + e % V] = y[e];
    if (lane == 0) {
        s_m[warp] = top;
        s_l[warp] = sum;
    }
    __syncthreads();
    const int c = threadIdx.x;
    if (c >= C || blockIdx.y >= heads) return;
    top = s_m[0];
#pragma unroll
    for (int w = 1; w < W; ++w) top = fmaxf(top, s_m[w]);
    float total = 0.0f, yc = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const float f = s_m[w] == -INFINITY ? 0.0f : exp2f(s_m[w] - top);
        total = fmaf(f, s_l[w], total);
        yc = fmaf(f, s_o[w][c], yc);
    }
    st1(a.y, a.y_dt, ((size_t)b * a.Hq + hk * a.group + hb * S::HB + blockIdx.y) * D + c0 + c, total == 0.0f ? 0.0f : yc / total);
}

}  // namespace gdn
