// attn_prep.cuh -- the input side of the attention layer that a stack keeps between its GDN mixers: the
// zero-centred RMSNorm of each query and key head and the position rotation, in one pass over the
// heads, its gradients, and the serving form that puts keys and values into a paged cache.
//
// Forward, per (token, head) row x of d channels with angles theta_i = position * inv_freq_i, i < R/2:
//   n_i = x_i r (1 + w_i),  r = (mean_j x_j^2 + eps)^(-1/2)
//   y_i = n_i cos theta_i - n_{i+R/2} sin theta_i,  y_{i+R/2} = n_{i+R/2} cos theta_i + n_i sin theta_i,
//   y_i = n_i for i >= R.
// Backward, dn = the rotation by -theta of dy, u = x r, gn_i = dn_i (1 + w_i):
//   dx_i = r (gn_i - u_i mean_j(gn_j u_j)),  dw_i = sum over tokens and heads of dn_i u_i.
//
// Bound by HBM: each row is read once and written once (backward: two rows read, one written).  A row
// is shared by d/16 lanes, and a lane holds two chunks of 8 channels: the rotating lanes chunk l of
// both halves of the rotated part, so that both members of a pair are in one lane, the others two
// adjacent chunks behind it.  Every access is then 16 bytes wide, and the only exchange between lanes
// is the sum of squares.  A unit (one token, up to `hps` heads of one of the tensors) computes its
// angles once for its heads.  Angles are reduced in fp64, in revolutions: a position of 2^20 leaves an
// fp32 angle only a few bits behind the point, while position * inv_freq / (2 pi) minus its nearest
// integer is exact in fp64 to 2^-33 of a revolution, and sincospif takes it from there in fp32.
#pragma once
#include "common.cuh"
#include "out_gate.cuh"

namespace gdn {

constexpr int kAttnPrepThreads = 256;

struct AttnPrepArgs {
    const void *q, *k, *v;                      // rows of a token contiguous, tokens *_stride elements apart
    long long q_stride, k_stride, v_stride;
    const float *w_q, *w_k;
    float eps;
    const int32_t* positions;
    const double* inv_freq;
    int rot, N, Hq, Hkv, hps, cq, ck;           // heads per unit; units per token of q, and of k (and of v)
    int out_dt;
    void *q_out, *k_out, *v_out;                // k_out, v_out: the cache when CACHE
    const int32_t *cu, *table;
    int num_seqs, max_pages, num_pages, page_size;
};

// The two chunks of 8 channels that lane `l` of a row holds, and whether they are a rotated pair.
__device__ __forceinline__ bool attn_chunks(int l, int rot, int& i0, int& j0) {
    const int rl = rot >> 4;
    if (l < rl) {
        i0 = 8 * l;
        j0 = i0 + (rot >> 1);
        return true;
    }
    i0 = 16 * l;
    j0 = i0 + 8;
    return false;
}

// cos and sin of position * inv_freq for the lane's 8 pairs.
__device__ __forceinline__ void attn_angles(const double* inv_freq, int i0, bool turns, int position, float (&c)[8],
                                            float (&s)[8]) {
    if (turns) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            double rev = (double)position * (inv_freq[i0 + u] * 0.15915494309189533577);
            rev -= rint(rev);
            sincospif(2.0f * (float)rev, &s[u], &c[u]);
        }
    } else {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            c[u] = 1.0f;
            s[u] = 0.0f;
        }
    }
}

__device__ __forceinline__ void attn_store8(void* p, int dt, size_t i, const float (&x)[8]) {
    if (dt == kBF16) stv<kBF16, 8>(p, i, x);
    else if (dt == kF16) stv<kF16, 8>(p, i, x);
    else stv<kF32, 8>(p, i, x);
}

// Physical page of the logical page `page` of row b; -1 (flagged) when the table names none.
__device__ __forceinline__ int attn_page(const int32_t* table, int max_pages, int num_pages, int b, int page) {
    const int phys = page < max_pages ? table[(size_t)b * max_pages + page] : -1;
    if (phys < 0 || phys >= num_pages) {
        raise_error(kErrPage);
        return -1;
    }
    return phys;
}

// Sequence that token t belongs to, -1 past the last one.  Offsets out of order are flagged by the
// range test of the found sequence.
__device__ __forceinline__ int attn_seq_of(const int32_t* cu, int num_seqs, int N, int t) {
    if (cu == nullptr) return t / (N / num_seqs);
    if (t >= cu[num_seqs]) return -1;
    int lo = 0, hi = num_seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    if (cu[lo] > t || cu[lo + 1] <= t) {
        raise_error(kErrSeqlens);
        return -1;
    }
    return lo;
}

template <int IN, int D, bool CACHE>
__global__ void __launch_bounds__(kAttnPrepThreads) attn_prep_kernel(const AttnPrepArgs a) {
    constexpr int LPR = D / 16;                 // lanes of a row
    constexpr int U = IN == kF32 ? 2 : 4;       // rows in flight
    const int l = threadIdx.x % LPR;
    const int per_token = a.cq + (CACHE ? 2 : 1) * a.ck;
    const unsigned unit = (blockIdx.x * (unsigned)kAttnPrepThreads + threadIdx.x) / LPR;
    int t = (int)(unit / (unsigned)per_token);
    int c = (int)(unit - (unsigned)t * (unsigned)per_token);
    bool live = t < a.N;
    if (!live) t = 0;
    const int part = c < a.cq ? 0 : c < a.cq + a.ck ? 1 : 2;  // q, k, v
    const int heads = part == 0 ? a.Hq : a.Hkv;
    const int h0 = (part == 0 ? c : part == 1 ? c - a.cq : c - a.cq - a.ck) * a.hps;
    const void* x = part == 0 ? a.q : part == 1 ? a.k : a.v;
    const size_t row0 = (size_t)t * (size_t)(part == 0 ? a.q_stride : part == 1 ? a.k_stride : a.v_stride);
    const int position = a.positions[t];

    void* out = part == 0 ? a.q_out : part == 1 ? a.k_out : a.v_out;
    size_t dst0 = (size_t)t * heads * D, dst_step = D;  // of head 0, and from head to head
    if constexpr (CACHE) {
        if (position < 0) live = false;  // a padding token
        if (live) {
            const int seq = attn_seq_of(a.cu, a.num_seqs, a.N, t);
            if (seq < 0) live = false;
            else if (part > 0) {
                const int page = position / a.page_size;
                const int phys = attn_page(a.table, a.max_pages, a.num_pages, seq, page);
                if (phys < 0) live = false;
                else {
                    dst0 = ((size_t)phys * a.Hkv * a.page_size + (position - page * a.page_size)) * D;
                    dst_step = (size_t)a.page_size * D;
                }
            }
        }
    }

    int i0, j0;
    const bool turns = attn_chunks(l, a.rot, i0, j0);
    float cs[8], sn[8], wi[8], wj[8];
    const float* w = part == 0 ? a.w_q : a.w_k;
    attn_angles(a.inv_freq, i0, turns && part < 2, position, cs, sn);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        wi[u] = 1.0f + w[i0 + u];
        wj[u] = 1.0f + w[j0 + u];
    }

    for (int hb = 0; hb < a.hps; hb += U) {
        float xi[U][8], xj[U][8], ss[U];
#pragma unroll
        for (int m = 0; m < U; ++m) {
            const int h = h0 + hb + m;
            const bool ok = live && hb + m < a.hps && h < heads;
            if (ok) {
                ldv<IN, 8>(x, row0 + (size_t)h * D + i0, xi[m]);
                ldv<IN, 8>(x, row0 + (size_t)h * D + j0, xj[m]);
            } else {
#pragma unroll
                for (int u = 0; u < 8; ++u) xi[m][u] = xj[m][u] = 0.0f;
            }
        }
#pragma unroll
        for (int m = 0; m < U; ++m) {
            ss[m] = 0.0f;
#pragma unroll
            for (int u = 0; u < 8; ++u) ss[m] = fmaf(xi[m][u], xi[m][u], fmaf(xj[m][u], xj[m][u], ss[m]));
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) {
#pragma unroll
            for (int m = 0; m < U; ++m) ss[m] += __shfl_xor_sync(0xffffffffu, ss[m], o);
        }
#pragma unroll
        for (int m = 0; m < U; ++m) {
            const int h = h0 + hb + m;
            if (!(live && hb + m < a.hps && h < heads)) continue;
            float yi[8], yj[8];
            const float r = rsqrtf(ss[m] * (1.0f / D) + a.eps);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float ni = xi[m][u] * r * wi[u], nj = xj[m][u] * r * wj[u];
                yi[u] = ni * cs[u] - nj * sn[u];
                yj[u] = nj * cs[u] + ni * sn[u];
                if (CACHE && part == 2) {  // values go as they are
                    yi[u] = xi[m][u];
                    yj[u] = xj[m][u];
                }
            }
            const size_t o = dst0 + (size_t)h * dst_step;
            if constexpr (CACHE) {
                const long long cache = (long long)a.num_pages * a.Hkv * a.page_size * D;
                if (!in_bounds((long long)(o + D - 1), part == 0 ? (long long)a.N * a.Hq * D : cache)) continue;
            }
            attn_store8(out, a.out_dt, o + i0, yi);
            attn_store8(out, a.out_dt, o + j0, yj);
        }
    }
}

// ---------------------------------------------------------------- gradients

struct AttnPrepBwdArgs {
    const void *q, *k, *dyq, *dyk;
    long long q_stride, k_stride;
    const float *w_q, *w_k;
    float eps;
    const int32_t* positions;
    const double* inv_freq;
    int rot, N, Hq, Hkv, hps, cq, ck;
    int gq;                                     // blocks of the queries; the others take the keys
    int dy_dt;
    void *dq, *dk;
    float* partial;                             // [blocks, d]: each block's share of dw
};

template <int IN, int D>
__global__ void __launch_bounds__(kAttnPrepThreads) attn_prep_bwd_kernel(const AttnPrepBwdArgs a) {
    constexpr int LPR = D / 16, SUBS = kAttnPrepThreads / LPR, WARPS = kAttnPrepThreads / 32;
    constexpr int U = IN == kF32 ? 1 : 2;
    __shared__ float s_dw[WARPS][D];
    const int l = threadIdx.x % LPR;
    const bool keys = (int)blockIdx.x >= a.gq;
    const int blk = keys ? blockIdx.x - a.gq : blockIdx.x;
    const int blocks = keys ? gridDim.x - a.gq : a.gq;
    const int heads = keys ? a.Hkv : a.Hq;
    const int per_token = keys ? a.ck : a.cq;
    const void* x = keys ? a.k : a.q;
    const void* dy = keys ? a.dyk : a.dyq;
    void* dx = keys ? a.dk : a.dq;
    const long long stride = keys ? a.k_stride : a.q_stride;
    const float* w = keys ? a.w_k : a.w_q;

    int i0, j0;
    const bool turns = attn_chunks(l, a.rot, i0, j0);
    float wi[8], wj[8], dwi[8], dwj[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        wi[u] = 1.0f + w[i0 + u];
        wj[u] = 1.0f + w[j0 + u];
        dwi[u] = dwj[u] = 0.0f;
    }

    const long long units = (long long)a.N * per_token;  // < 2^31 (host check)
    for (long long base = (long long)blk * SUBS; base < units; base += (long long)blocks * SUBS) {
        const unsigned unit = (unsigned)base + threadIdx.x / LPR;
        const bool live = unit < (unsigned)units;
        const int t = live ? (int)(unit / (unsigned)per_token) : 0;
        const int h0 = live ? (int)(unit - (unsigned)t * (unsigned)per_token) * a.hps : 0;
        float cs[8], sn[8];
        attn_angles(a.inv_freq, i0, turns, a.positions[t], cs, sn);
        for (int hb = 0; hb < a.hps; hb += U) {
            float xi[U][8], xj[U][8], gi[U][8], gj[U][8], ss[U], dot[U];
#pragma unroll
            for (int m = 0; m < U; ++m) {
                const int h = h0 + hb + m;
                if (live && hb + m < a.hps && h < heads) {
                    const size_t r = (size_t)t * (size_t)stride + (size_t)h * D, g = ((size_t)t * heads + h) * D;
                    ldv<IN, 8>(x, r + i0, xi[m]);
                    ldv<IN, 8>(x, r + j0, xj[m]);
                    if (a.dy_dt == kF32) {
                        ldv<kF32, 8>(dy, g + i0, gi[m]);
                        ldv<kF32, 8>(dy, g + j0, gj[m]);
                    } else if (a.dy_dt == kBF16) {
                        ldv<kBF16, 8>(dy, g + i0, gi[m]);
                        ldv<kBF16, 8>(dy, g + j0, gj[m]);
                    } else {
                        ldv<kF16, 8>(dy, g + i0, gi[m]);
                        ldv<kF16, 8>(dy, g + j0, gj[m]);
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < 8; ++u) xi[m][u] = xj[m][u] = gi[m][u] = gj[m][u] = 0.0f;
                }
            }
            // gi, gj become dn, and dot the sum of dn (1 + w) x
#pragma unroll
            for (int m = 0; m < U; ++m) {
                ss[m] = dot[m] = 0.0f;
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float ni = gi[m][u] * cs[u] + gj[m][u] * sn[u], nj = gj[m][u] * cs[u] - gi[m][u] * sn[u];
                    gi[m][u] = ni;
                    gj[m][u] = nj;
                    ss[m] = fmaf(xi[m][u], xi[m][u], fmaf(xj[m][u], xj[m][u], ss[m]));
                    dot[m] = fmaf(ni * wi[u], xi[m][u], fmaf(nj * wj[u], xj[m][u], dot[m]));
                }
            }
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) {
#pragma unroll
                for (int m = 0; m < U; ++m) {
                    ss[m] += __shfl_xor_sync(0xffffffffu, ss[m], o);
                    dot[m] += __shfl_xor_sync(0xffffffffu, dot[m], o);
                }
            }
#pragma unroll
            for (int m = 0; m < U; ++m) {
                const int h = h0 + hb + m;
                if (!(live && hb + m < a.hps && h < heads)) continue;
                const float r = rsqrtf(ss[m] * (1.0f / D) + a.eps);
                const float mean = dot[m] * r * (1.0f / D);  // mean of gn u
                float yi[8], yj[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float ui = xi[m][u] * r, uj = xj[m][u] * r;
                    dwi[u] = fmaf(gi[m][u], ui, dwi[u]);
                    dwj[u] = fmaf(gj[m][u], uj, dwj[u]);
                    yi[u] = r * (gi[m][u] * wi[u] - ui * mean);
                    yj[u] = r * (gj[m][u] * wj[u] - uj * mean);
                }
                const size_t g = ((size_t)t * heads + h) * D;
                stv<IN, 8>(dx, g + i0, yi);
                stv<IN, 8>(dx, g + j0, yj);
            }
        }
    }

    // this block's share of dw: lanes of the same channels, then the warps, in a fixed order
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            dwi[u] += __shfl_xor_sync(0xffffffffu, dwi[u], o);
            dwj[u] += __shfl_xor_sync(0xffffffffu, dwj[u], o);
        }
    }
    if ((threadIdx.x & 31) < LPR) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            s_dw[threadIdx.x >> 5][i0 + u] = dwi[u];
            s_dw[threadIdx.x >> 5][j0 + u] = dwj[u];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += kAttnPrepThreads) {
        float sum = 0.0f;
#pragma unroll
        for (int m = 0; m < WARPS; ++m) sum += s_dw[m][i];
        a.partial[(size_t)blockIdx.x * D + i] = sum;
    }
}

// dw_q, dw_k: the blocks' shares added in fp64, in block order within each of 8 strided sums.
// Grid (2, ceil(d / 32)), block (32, 8).
__global__ void __launch_bounds__(256) attn_prep_dw_kernel(const float* __restrict__ partial, int gq, int blocks, int d,
                                                           float* __restrict__ dw_q, float* __restrict__ dw_k) {
    __shared__ double s[8][32];
    const int i = blockIdx.y * 32 + threadIdx.x;
    const int b0 = blockIdx.x == 0 ? 0 : gq, b1 = blockIdx.x == 0 ? gq : blocks;
    double sum = 0.0;
    if (i < d) {
#pragma unroll 4
        for (int b = b0 + threadIdx.y; b < b1; b += 8) sum += (double)partial[(size_t)b * d + i];
    }
    s[threadIdx.y][threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.y == 0 && i < d) {
#pragma unroll
        for (int m = 1; m < 8; ++m) sum += s[m][threadIdx.x];
        (blockIdx.x == 0 ? dw_q : dw_k)[i] = (float)sum;
    }
}

}  // namespace gdn
