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
// both halves of the rotated part, so that both members of a pair are in one lane, the others of both
// halves of the part behind it.  Every access is then 16 bytes wide and next to its neighbours', and the
// only exchange between lanes is the sum of squares.  A unit (one token, some heads of one of the tensors) computes its
// angles once for its heads, and keeps U rows in flight: a row's registers are loaded again as soon as it
// is unpacked.  Angles are reduced in fp64, in revolutions: a position of 2^20 leaves an fp32 angle
// only a few bits behind the point, while position * inv_freq / (2 pi) minus its nearest integer is exact
// in fp64 to 2^-32 of a revolution.
#pragma once
#include <type_traits>

#include "common.cuh"
#include "out_gate.cuh"
#include "tc_ptx.cuh"

namespace gdn {

constexpr int kAttnPrepThreads = 256;

struct AttnPrepArgs {
    const void *q, *k, *v;                      // rows of a token contiguous, tokens *_stride elements apart
    long long q_stride, k_stride, v_stride;
    const float *w_q, *w_k;
    float eps;
    const int32_t* positions;
    const double* inv_freq;
    int rot, N, Hq, Hkv, cq, ck;                // units per token of q, and of k (with v)
    int out_dt;
    void *q_out, *k_out, *v_out;                // k_out, v_out: the cache when CACHE
    const int32_t *cu, *table;
    int num_seqs, max_pages, num_pages, page_size;
};

// The two chunks of 8 channels that lane `l` of a row of d channels holds: chunk l of both halves of the rotated part,
// or of both halves of the part behind it.
__device__ __forceinline__ void attn_chunks(int l, int d, int rot, int& i0, int& j0) {
    const int rl = rot >> 4;
    if (l < rl) {
        i0 = 8 * l;
        j0 = i0 + (rot >> 1);
    } else {
        i0 = rot + 8 * (l - rl);
        j0 = i0 + ((d - rot) >> 1);
    }
}

// cos and sin of 2 pi phase / 2^32, from the Taylor series about the nearest quarter turn: |x| <= pi / 4, where the
// first terms left out are x^10 / 10! < 2^-25 of the cosine and x^11 / 11! < 2^-28 of the sine.
__device__ __forceinline__ void attn_turn(int phase, float& c, float& s) {
    const unsigned quarter = ((unsigned)phase + 0x20000000u) >> 30;
    const float x = (float)(int)((unsigned)phase - (quarter << 30)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
    const float x2 = x * x;
    const float sx = fmaf(x * x2, fmaf(x2, fmaf(x2, fmaf(x2, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), x);
    const float cx = fmaf(x2, fmaf(x2, fmaf(x2, fmaf(x2, 1.0f / 40320, -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
    const float s0 = quarter & 1 ? cx : sx, c0 = quarter & 1 ? sx : cx;
    s = __uint_as_float(__float_as_uint(s0) ^ (quarter << 30 & 0x80000000u));
    c = __uint_as_float(__float_as_uint(c0) ^ ((quarter + 1) << 30 & 0x80000000u));
}

// cos and sin of position * inv_freq.  Adding and taking away 1.5 * 2^52 rounds to whole revolutions, the fused products
// leave the rest with one rounding, and adding 1.5 * 2^20 puts it, in units of 2^-32, into the low word: three steps of
// the fp64 pipe and no conversion instruction, which run at a quarter of its rate and less.
__device__ __forceinline__ void attn_angle(double position, double f, float& c, float& s) {
    f *= 0.15915494309189533577;
    const double whole = __dadd_rn(__fma_rn(position, f, 0x1.8p52), -0x1.8p52);
    attn_turn(__double2loint(__dadd_rn(__fma_rn(position, f, -whole), 0x1.8p20)), c, s);
}

// The same for the lane's 8 pairs, when only some lanes of the row turn: lane L finds pairs P L .. P L + P - 1, and the
// turning lanes fetch theirs.
template <int LPR, int P>
__device__ __forceinline__ void attn_angles_shared(const double* inv_freq, int pairs, int l, double position, unsigned mask,
                                                   float (&c)[8], float (&s)[8]) {
    float cp[P], sp[P];
#pragma unroll
    for (int j = 0; j < P; ++j) attn_angle(position, l * P + j < pairs ? inv_freq[l * P + j] : 0.0, cp[j], sp[j]);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        c[u] = __shfl_sync(mask, cp[u % P], l * (8 / P) + u / P, LPR);
        s[u] = __shfl_sync(mask, sp[u % P], l * (8 / P) + u / P, LPR);
    }
}

// cos and sin for the lane's 8 pairs (1 and 0 where it does not turn).  All lanes of the row call it.
template <int LPR>
__device__ __forceinline__ void attn_angles(const double* inv_freq, int rot, int l, int position, unsigned mask, float (&c)[8],
                                            float (&s)[8]) {
    const int pairs = rot >> 1;
    const double p = (double)position;
    if (pairs > 4 * LPR) {
#pragma unroll
        for (int u = 0; u < 8; ++u) attn_angle(p, 8 * l + u < pairs ? inv_freq[8 * l + u] : 0.0, c[u], s[u]);
    } else if (pairs > 2 * LPR) {
        attn_angles_shared<LPR, 4>(inv_freq, pairs, l, p, mask, c, s);
    } else if (pairs > 0) {
        attn_angles_shared<LPR, 2>(inv_freq, pairs, l, p, mask, c, s);
    }
    if (8 * l >= pairs) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            c[u] = 1.0f;
            s[u] = 0.0f;
        }
    }
}

// 1 + w for 8 channels.
__device__ __forceinline__ void attn_weights(const float* w, int i0, float2 (&x)[4]) {
#pragma unroll
    for (int u = 0; u < 4; u += 2) {
        const float4 v = *reinterpret_cast<const float4*>(w + i0 + 2 * u);
        x[u] = make_float2(1.0f + v.x, 1.0f + v.y);
        x[u + 1] = make_float2(1.0f + v.z, 1.0f + v.w);
    }
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{.reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n mul.rn.f32x2 rd, ra, rb;\n mov.b64 {%0, %1}, rd;}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{.reg .b64 ra, rb, rc, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n mov.b64 rc, {%6, %7};\n"
        " fma.rn.f32x2 rd, ra, rb, rc;\n mov.b64 {%0, %1}, rd;}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// A lane's 16 channels of a row as they lie in memory.
template <int IN>
struct AttnRow {
    static constexpr int Q = IN == kF32 ? 4 : 2;  // 16-byte words
    uint4 w[Q];
    __device__ __forceinline__ void load(const void* x, size_t row, int i0, int j0) {
        using E = typename std::conditional<IN == kF32, uint32_t, uint16_t>::type;
        const E* p = reinterpret_cast<const E*>(x) + row;
#pragma unroll
        for (int q = 0; q < Q / 2; ++q) {
            w[q] = reinterpret_cast<const uint4*>(p + i0)[q];
            w[Q / 2 + q] = reinterpret_cast<const uint4*>(p + j0)[q];
        }
    }
    __device__ __forceinline__ void get(float2 (&xi)[4], float2 (&xj)[4]) const {
        half(0, xi);
        half(Q / 2, xj);
    }

    __device__ __forceinline__ void get(float (&xi)[8], float (&xj)[8]) const {
        float2 i[4], j[4];
        get(i, j);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            xi[2 * u] = i[u].x, xi[2 * u + 1] = i[u].y;
            xj[2 * u] = j[u].x, xj[2 * u + 1] = j[u].y;
        }
    }

  private:
    __device__ __forceinline__ void half(int q0, float2 (&x)[4]) const {
#pragma unroll
        for (int q = 0; q < Q / 2; ++q) {
            const uint4 v = w[q0 + q];
            if constexpr (IN == kF32) {
                x[2 * q] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
                x[2 * q + 1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
            } else {
                x[0] = unpack2<IN == kBF16>(v.x);
                x[1] = unpack2<IN == kBF16>(v.y);
                x[2] = unpack2<IN == kBF16>(v.z);
                x[3] = unpack2<IN == kBF16>(v.w);
            }
        }
    }
};

// The lanes of this lane's row.
template <int LPR>
__device__ __forceinline__ unsigned attn_row_mask() {
    return (unsigned)((1ull << LPR) - 1) << (threadIdx.x & 31 & ~(LPR - 1));
}

template <int LPR>
__device__ __forceinline__ float attn_row_sum(float x, unsigned mask) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(mask, x, o);
    return x;
}

__device__ __forceinline__ void attn_store8(void* p, int dt, size_t i, const float2 (&x)[4]) {
    const float f[8] = {x[0].x, x[0].y, x[1].x, x[1].y, x[2].x, x[2].y, x[3].x, x[3].y};
    if (dt == kBF16) stv<kBF16, 8>(p, i, f);
    else if (dt == kF16) stv<kF16, 8>(p, i, f);
    else stv<kF32, 8>(p, i, f);
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

// Flags offsets that do not begin at 0, fall, or end behind N; thread `i` of `threads` looks at every threads-th sequence.
// The search for a token's sequence meets a few of the offsets only, and cannot tell that the others are in order.
__device__ __forceinline__ void attn_check_seqlens(const int32_t* cu, int num_seqs, int N, unsigned i, unsigned threads) {
    for (long long s = i; s < num_seqs; s += threads) {
        const int start = cu[s], end = cu[s + 1];
        if (end < start || (s == 0 && start != 0) || (s == num_seqs - 1 && end > N)) raise_error(kErrSeqlens);
    }
}

// Sequence that token t belongs to, -1 past the last one.  Of offsets out of order (attn_check_seqlens flags them) it names
// a sequence that begins at or before t and ends behind it, or none.
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

// Forward.  Measured: 32768 tokens of 40 bf16 heads of 128, half of each rotated, 110 us, 6.1 TB/s read and written, 93 %
// of a copy's rate; into the cache, 17386 tokens of 20 fp16 heads of 256, 68 us, 5.2 TB/s.  Two CTAs an SM with 4 rows of
// each lane under way; one CTA of 141 registers took 318 us.
template <int IN, int D, bool CACHE>
__global__ void __launch_bounds__(kAttnPrepThreads, IN == kF32 ? 1 : 2) attn_prep_kernel(const AttnPrepArgs a) {
    constexpr int LPR = D / 16;                 // lanes of a row
    constexpr int U = IN == kF32 ? 2 : 4;       // rows in flight
    const int l = threadIdx.x % LPR;
    const unsigned mask = attn_row_mask<LPR>();
    // The queries' units, then the keys'.  A token's units stand side by side and take every `step`-th head, so that
    // what is under way at a time is contiguous.
    const unsigned thread = blockIdx.x * (unsigned)kAttnPrepThreads + threadIdx.x;
    unsigned unit = thread / LPR;
    const bool keys = unit >= (unsigned)a.N * (unsigned)a.cq;
    if (keys) unit -= (unsigned)a.N * (unsigned)a.cq;
    const int heads = keys ? a.Hkv : a.Hq, step = keys ? a.ck : a.cq;
    const int t = (int)(unit / (unsigned)step), h0 = (int)(unit - (unsigned)t * (unsigned)step);
    if (t >= a.N) return;
    const int n = (heads - h0 + step - 1) / step;
    const int rows = CACHE && keys ? 2 * n : n;  // keys, then the same heads' values
    const void* x = keys ? a.k : a.q;
    const size_t x0 = (size_t)t * (size_t)(keys ? a.k_stride : a.q_stride) + (size_t)h0 * D;
    const size_t v0 = CACHE && keys ? (size_t)t * (size_t)a.v_stride + (size_t)h0 * D : 0;
    int i0, j0;
    attn_chunks(l, D, a.rot, i0, j0);

    AttnRow<IN> buf[U];
    auto fetch = [&](AttnRow<IN>& to, int m) {
        if (CACHE && m >= n) to.load(a.v, v0 + (size_t)((m - n) * step) * D, i0, j0);
        else to.load(x, x0 + (size_t)(m * step) * D, i0, j0);
    };
#pragma unroll
    for (int m = 0; m < U; ++m) {
        if (m < rows) fetch(buf[m], m);
    }
    const int position = a.positions[t];

    size_t dst0 = ((size_t)t * heads + h0) * D, dst_step = (size_t)step * D;  // of the first head, and to the next
    int page = 0, phys = -1;
    if constexpr (CACHE) {
        // behind the rows' loads and the position's, so that it waits along with them
        if (a.cu != nullptr) attn_check_seqlens(a.cu, a.num_seqs, a.N, thread, (unsigned)a.N * (unsigned)(a.cq + a.ck) * LPR);
        if (position < 0) return;  // a padding token
        const int seq = attn_seq_of(a.cu, a.num_seqs, a.N, t);
        if (seq < 0) return;
        page = position / a.page_size;
        if (keys && page < a.max_pages) phys = a.table[(size_t)seq * a.max_pages + page];  // checked behind the angles
    }
    auto put = [&](void* out, int m, const float2 (&yi)[4], const float2 (&yj)[4]) {
        const size_t o = dst0 + (size_t)m * dst_step;
        if constexpr (CACHE) {
            const long long cache = (long long)a.num_pages * a.Hkv * a.page_size * D;
            if (!in_bounds((long long)(o + D - 1), keys ? cache : (long long)a.N * a.Hq * D)) return;
        }
        attn_store8(out, a.out_dt, o + i0, yi);
        attn_store8(out, a.out_dt, o + j0, yj);
    };

    // y_i = r (x_i ci + x_j mj), y_j = r (x_j cj + x_i si): 1 + w and the rotation in one factor each
    float2 ci[4], cj[4], si[4], mj[4];
    {
        float cs[8], sn[8];
        attn_angles<LPR>(a.inv_freq, a.rot, l, position, mask, cs, sn);
        float2 wi[4], wj[4];
        attn_weights(keys ? a.w_k : a.w_q, i0, wi);
        attn_weights(keys ? a.w_k : a.w_q, j0, wj);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float2 c = make_float2(cs[2 * u], cs[2 * u + 1]), s = make_float2(sn[2 * u], sn[2 * u + 1]);
            ci[u] = mul2(c, wi[u]);
            cj[u] = mul2(c, wj[u]);
            si[u] = mul2(s, wi[u]);
            mj[u] = mul2(make_float2(-s.x, -s.y), wj[u]);
        }
    }
    if (CACHE && keys) {
        if (phys < 0 || phys >= a.num_pages) {
            raise_error(kErrPage);
            return;
        }
        dst0 = (((size_t)phys * a.Hkv + h0) * a.page_size + (position - page * a.page_size)) * D;
        dst_step = (size_t)(step * a.page_size) * D;
    }
    for (int hb = 0; hb < rows; hb += U) {
#pragma unroll
        for (int m = 0; m < U; ++m) {
            if (hb + m >= rows) break;
            float2 xi[4], xj[4];
            buf[m].get(xi, xj);
            if (hb + U + m < rows) fetch(buf[m], hb + U + m);
            if (CACHE && hb + m >= n) {  // values go as they are
                put(a.v_out, hb + m - n, xi, xj);
                continue;
            }
            float2 ss = mul2(xi[0], xi[0]), st = mul2(xj[0], xj[0]);
#pragma unroll
            for (int u = 1; u < 4; ++u) {
                ss = fma2(xi[u], xi[u], ss);
                st = fma2(xj[u], xj[u], st);
            }
            const float2 r = both(rsqrtf(attn_row_sum<LPR>((ss.x + st.x) + (ss.y + st.y), mask) * (1.0f / D) + a.eps));
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float2 yi = mul2(r, fma2(xj[u], mj[u], mul2(xi[u], ci[u])));
                xj[u] = mul2(r, fma2(xi[u], si[u], mul2(xj[u], cj[u])));
                xi[u] = yi;
            }
            put(keys ? a.k_out : a.q_out, hb + m, xi, xj);
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
    int rot, N, Hq, Hkv, hps, cq, ck;           // heads per unit; units per token of q, and of k
    int gq;                                     // blocks of the queries; the others take the keys
    void *dq, *dk;
    float* partial;                             // [blocks, d]: each block's share of dw
    float *dw_q, *dw_k;                         // written by the only block of each tensor; dw_q NULL: shares
};

// Backward, by resident CTAs, so that each writes its share of dw once; those of the queries and of the keys are
// apart, as the weights are.  At the 128 registers of two CTAs an SM the 16-bit forms spill 32 to 72 bytes a thread (d = 128 in
// bf16: 64, 2.4 M local loads and 1.2 M stores of warps over 32768 tokens); the fp32 forms, one CTA an SM, do not.  Measured: the
// 32768 tokens above 195 to 201 us, 5.0 TB/s; 1 + w in registers or in shared memory,
// 4, 8 or 16 heads a unit and rows through shared memory make no difference above 3 %.
template <int IN, int D, int DY>
__global__ void __launch_bounds__(kAttnPrepThreads, IN == kF32 || DY == kF32 ? 1 : 2)
    attn_prep_bwd_kernel(const AttnPrepBwdArgs a) {
    constexpr int LPR = D / 16, SUBS = kAttnPrepThreads / LPR, WARPS = kAttnPrepThreads / 32;
    constexpr int U = IN == kF32 ? 1 : 2;
    __shared__ float s_dw[WARPS][D];
    __shared__ __align__(16) float s_w[4][LPR][4];
    const int l = threadIdx.x % LPR;
    const unsigned mask = attn_row_mask<LPR>();
    const bool keys = (int)blockIdx.x >= a.gq;
    const int blk = keys ? blockIdx.x - a.gq : blockIdx.x;
    const int blocks = keys ? gridDim.x - a.gq : a.gq;
    const int heads = keys ? a.Hkv : a.Hq;
    const void* x = keys ? a.k : a.q;
    const void* dy = keys ? a.dyk : a.dyq;
    void* dx = keys ? a.dk : a.dq;
    const long long stride = keys ? a.k_stride : a.q_stride;
    const float* w = keys ? a.w_k : a.w_q;

    int i0, j0;
    attn_chunks(l, D, a.rot, i0, j0);
    // 1 + w stays in shared memory (its 16 registers would spill as well), in the order that the lanes read it
    float dwi[8], dwj[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) dwi[u] = dwj[u] = 0.0f;
    if (threadIdx.x < LPR) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            s_w[u >> 2][l][u & 3] = 1.0f + w[i0 + u];
            s_w[2 + (u >> 2)][l][u & 3] = 1.0f + w[j0 + u];
        }
    }
    __syncthreads();
    auto weight = [&](int q, float (&x)[8]) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const float4 f = *reinterpret_cast<const float4*>(s_w[2 * q + v][l]);
            x[4 * v] = f.x, x[4 * v + 1] = f.y, x[4 * v + 2] = f.z, x[4 * v + 3] = f.w;
        }
    };

    const unsigned units = (unsigned)a.N * (unsigned)(keys ? a.ck : a.cq);  // < 2^30 (host check)
    for (unsigned unit = (unsigned)blk * SUBS + threadIdx.x / LPR; unit < units; unit += (unsigned)blocks * SUBS) {
        const int c = (int)(unit / (unsigned)a.N), t = (int)(unit - (unsigned)c * (unsigned)a.N);
        const int h0 = c * a.hps, n = min(a.hps, heads - h0);
        const size_t x0 = (size_t)t * (size_t)stride + (size_t)h0 * D, g0 = ((size_t)t * heads + h0) * D;
        AttnRow<IN> xb[U];
        AttnRow<DY> gb[U];
#pragma unroll
        for (int m = 0; m < U; ++m) {
            if (m < n) {
                xb[m].load(x, x0 + (size_t)m * D, i0, j0);
                gb[m].load(dy, g0 + (size_t)m * D, i0, j0);
            }
        }
        float cs[8], sn[8];
        attn_angles<LPR>(a.inv_freq, a.rot, l, a.positions[t], mask, cs, sn);
        for (int hb = 0; hb < n; hb += U) {
#pragma unroll
            for (int m = 0; m < U; ++m) {
                if (hb + m >= n) break;
                float xi[8], xj[8], gi[8], gj[8];
                xb[m].get(xi, xj);
                gb[m].get(gi, gj);
                if (hb + U + m < n) {
                    xb[m].load(x, x0 + (size_t)(hb + U + m) * D, i0, j0);
                    gb[m].load(dy, g0 + (size_t)(hb + U + m) * D, i0, j0);
                }
                // gi, gj become dn, and dot the sum of dn (1 + w) x
                float ss = 0.0f, dot = 0.0f, wi[8], wj[8];
                weight(0, wi);
                weight(1, wj);
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float ni = gi[u] * cs[u] + gj[u] * sn[u], nj = gj[u] * cs[u] - gi[u] * sn[u];
                    gi[u] = ni;
                    gj[u] = nj;
                    ss = fmaf(xi[u], xi[u], fmaf(xj[u], xj[u], ss));
                    dot = fmaf(ni * wi[u], xi[u], fmaf(nj * wj[u], xj[u], dot));
                }
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) {
                    ss += __shfl_xor_sync(mask, ss, o);
                    dot += __shfl_xor_sync(mask, dot, o);
                }
                const float r = rsqrtf(ss * (1.0f / D) + a.eps);
                const float back = r * (r * (dot * r * (1.0f / D)));  // r^2 mean(gn u), of x
                weight(0, wi);
                weight(1, wj);
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    gi[u] *= r;
                    gj[u] *= r;
                    dwi[u] = fmaf(gi[u], xi[u], dwi[u]);
                    dwj[u] = fmaf(gj[u], xj[u], dwj[u]);
                    gi[u] = gi[u] * wi[u] - xi[u] * back;
                    gj[u] = gj[u] * wj[u] - xj[u] * back;
                }
                const size_t g = g0 + (size_t)(hb + m) * D;
                stv<IN, 8>(dx, g + i0, gi);
                stv<IN, 8>(dx, g + j0, gj);
            }
        }
    }
    tc::launch_dependents();

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
        if (a.dw_q != nullptr) (keys ? a.dw_k : a.dw_q)[i] = sum;
        else a.partial[(size_t)blockIdx.x * D + i] = sum;
    }
}

// dw_q, dw_k: the blocks' shares added in fp64, in block order within each of 32 strided sums.
// Grid (2, ceil(d / 32)), block (32, 32).  Measured: 296 blocks of 128 channels, 3.7 us, of which most is the launch.
__global__ void __launch_bounds__(1024) attn_prep_dw_kernel(const float* __restrict__ partial, int gq, int blocks, int d,
                                                            float* __restrict__ dw_q, float* __restrict__ dw_k) {
    __shared__ double s[32][33];
    const int i = blockIdx.y * 32 + threadIdx.x;
    const int b0 = blockIdx.x == 0 ? 0 : gq, b1 = blockIdx.x == 0 ? gq : blocks;
    tc::wait_prerequisites();
    double sum = 0.0;
    if (i < d) {
#pragma unroll 4
        for (int b = b0 + threadIdx.y; b < b1; b += 32) sum += (double)partial[(size_t)b * d + i];
    }
    s[threadIdx.y][threadIdx.x] = sum;
    __syncthreads();
    sum = s[threadIdx.x][threadIdx.y];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int j = blockIdx.y * 32 + threadIdx.y;
    if (threadIdx.x == 0 && j < d) (blockIdx.x == 0 ? dw_q : dw_k)[j] = (float)sum;
}

}  // namespace gdn
