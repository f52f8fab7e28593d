// attn_api.cuh -- the C ABI of the attention operators (declared in include/gdn.h): argument checks and
// launches.  Included by gdn_lib.cu, whose error reporting it uses.
#pragma once
#include <initializer_list>

#include "attn_decode.cuh"
#include "attn_page.cuh"
#include "attn_prep.cuh"

namespace {

struct DeviceInfo {
    int dev = -1, sms = 0;
};

// The current device and its SM count (looked up once per device).
gdn_status_t device_info(DeviceInfo* out) {
    static std::atomic<int> sms[64];
    cudaError_t e = cudaGetDevice(&out->dev);
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
    int n = out->dev < 64 ? sms[out->dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, out->dev);
        if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "SM count: %s", cudaGetErrorString(e));
        if (out->dev < 64) sms[out->dev].store(n, std::memory_order_relaxed);
    }
    out->sms = n;
    return GDN_OK;
}

bool ranges_overlap(const void* a, long long na, const void* b, long long nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a != nullptr && b != nullptr && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

long long elem_size(int dt) { return dt == GDN_F32 ? 4 : 2; }

// Bytes that `n` tokens of `width` elements, `stride` elements apart, span.
long long span_bytes(long long n, long long stride, long long width, int dt) {
    return n > 0 ? ((n - 1) * stride + width) * elem_size(dt) : 0;
}

struct Range {
    const char* name;
    const void* p;
    long long bytes;
};

// No output on an input, nor on another output.
gdn_status_t require_apart(std::initializer_list<Range> outs, std::initializer_list<Range> ins) {
    for (const Range* a = outs.begin(); a != outs.end(); ++a) {
        for (const Range* b = a + 1; b != outs.end(); ++b)
            REQUIRE(!ranges_overlap(a->p, a->bytes, b->p, b->bytes), "%s overlaps %s", a->name, b->name);
        for (const Range& b : ins) REQUIRE(!ranges_overlap(a->p, a->bytes, b.p, b.bytes), "%s overlaps %s", a->name, b.name);
    }
    return GDN_OK;
}

#define REQUIRE_APART(...)                                     \
    do {                                                       \
        const gdn_status_t apart = require_apart(__VA_ARGS__); \
        if (apart != GDN_OK) return apart;                     \
    } while (0)

#define REQUIRE_ATTN_HEADS()                                                                              \
    do {                                                                                                  \
        REQUIRE(Hq >= 1 && Hkv >= 1 && Hq % Hkv == 0, "Hq=%d is not a positive multiple of Hkv=%d", Hq, Hkv); \
        REQUIRE(Hq <= 65536, "Hq=%d too large", Hq);                                                      \
    } while (0)

#define REQUIRE_STRIDE(s, heads, name)                                                                  \
    REQUIRE((s) >= (int64_t)(heads)*d && (s) % 8 == 0 && (s) < (1LL << 31),                               \
            "%s=%lld: not a multiple of 8 of at least heads * d, below 2^31", name, (long long)(s))

#define REQUIRE_PAGES()                                                                                     \
    do {                                                                                                    \
        REQUIRE(num_pages >= 1 && max_pages >= 1, "bad sizes num_pages=%d max_pages=%d", num_pages, max_pages); \
        REQUIRE(page_size >= 1, "page_size=%d < 1", page_size);                                             \
        if (page_size % 16 != 0 || page_size > 1024)                                                        \
            return fail(GDN_ERR_UNSUPPORTED, "page_size=%d is not a multiple of 16 up to 1024", page_size); \
        REQUIRE((long long)max_pages * page_size <= (1LL << 30), "max_pages * page_size above 2^30");       \
    } while (0)

// A launch that may start while the kernel before it on the stream still runs; it waits for that kernel itself.
template <class... P, class... A>
gdn_status_t launch_after(const char* name, void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                          cudaStream_t st, const A&... args) {
    gdn::LaunchScope timed(st, name);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e == cudaSuccess ? GDN_OK : fail(GDN_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
}

// ---------------------------------------------------------------- norm and rotation

// Heads per unit: the most (up to `most`) that still give two CTAs an SM a unit for every group of lanes.  More heads
// share the cost of the angles: 32768 tokens of 40 heads forward take 117 us at 8 heads and 111 at 16; backward, whose
// resident CTAs share out the units, 199 at 8 and 204 at 16.
int attn_heads_per_unit(long long rows, int lanes, int heads, int sms, int most) {
    int hps = 1;
    while (hps < most && hps < heads && rows * lanes / (2 * hps) >= 2LL * sms * gdn::kAttnPrepThreads) hps *= 2;
    return hps;
}

template <int IN, bool CACHE>
gdn_status_t attn_prep_go(int d, const gdn::AttnPrepArgs& a, unsigned grid, cudaStream_t st) {
    const char* name = CACHE ? "attn_prep_cache_kernel" : "attn_prep_kernel";
    gdn::LaunchScope timed(st, name);
    switch (d) {
        case 16: gdn::attn_prep_kernel<IN, 16, CACHE><<<grid, gdn::kAttnPrepThreads, 0, st>>>(a); break;
        case 32: gdn::attn_prep_kernel<IN, 32, CACHE><<<grid, gdn::kAttnPrepThreads, 0, st>>>(a); break;
        case 64: gdn::attn_prep_kernel<IN, 64, CACHE><<<grid, gdn::kAttnPrepThreads, 0, st>>>(a); break;
        case 128: gdn::attn_prep_kernel<IN, 128, CACHE><<<grid, gdn::kAttnPrepThreads, 0, st>>>(a); break;
        default: gdn::attn_prep_kernel<IN, 256, CACHE><<<grid, gdn::kAttnPrepThreads, 0, st>>>(a); break;
    }
    return launched(name);
}

template <bool CACHE>
gdn_status_t attn_prep_launch(gdn::AttnPrepArgs& a, int d, int in_dt, cudaStream_t st) {
    DeviceInfo dev;
    gdn_status_t r = device_info(&dev);
    if (r != GDN_OK) return r;
    const int lanes = d / 16;
    const int hps = attn_heads_per_unit((long long)a.N * (a.Hq + (CACHE ? 2 : 1) * a.Hkv), lanes, a.Hq, dev.sms, 16);
    a.cq = (a.Hq + hps - 1) / hps;
    a.ck = (a.Hkv + hps - 1) / hps;
    const long long threads = (long long)a.N * (a.cq + a.ck) * lanes;
    const long long grid = (threads + gdn::kAttnPrepThreads - 1) / gdn::kAttnPrepThreads;
    REQUIRE(grid * (gdn::kAttnPrepThreads / lanes) < (1LL << 31) && threads < (1LL << 32) - 256, "N=%d with Hq=%d too large",
            a.N, a.Hq);
    if (in_dt == GDN_F32) return attn_prep_go<gdn::kF32, CACHE>(d, a, (unsigned)grid, st);
    if (in_dt == GDN_BF16) return attn_prep_go<gdn::kBF16, CACHE>(d, a, (unsigned)grid, st);
    return attn_prep_go<gdn::kF16, CACHE>(d, a, (unsigned)grid, st);
}

template <int IN, int DY>
gdn_status_t attn_prep_bwd_go(int d, const gdn::AttnPrepBwdArgs& a, unsigned grid, cudaStream_t st) {
    gdn::LaunchScope timed(st, "attn_prep_bwd_kernel");
    switch (d) {
        case 16: gdn::attn_prep_bwd_kernel<IN, 16, DY><<<grid, gdn::kAttnPrepThreads, 0, st>>>(a); break;
        case 32: gdn::attn_prep_bwd_kernel<IN, 32, DY><<<grid, gdn::kAttnPrepThreads, 0, st>>>(a); break;
        case 64: gdn::attn_prep_bwd_kernel<IN, 64, DY><<<grid, gdn::kAttnPrepThreads, 0, st>>>(a); break;
        case 128: gdn::attn_prep_bwd_kernel<IN, 128, DY><<<grid, gdn::kAttnPrepThreads, 0, st>>>(a); break;
        default: gdn::attn_prep_bwd_kernel<IN, 256, DY><<<grid, gdn::kAttnPrepThreads, 0, st>>>(a); break;
    }
    return launched("attn_prep_bwd_kernel");
}

template <int IN>
gdn_status_t attn_prep_bwd_dy(int d, int dy, const gdn::AttnPrepBwdArgs& a, unsigned grid, cudaStream_t st) {
    if (dy == GDN_F32) return attn_prep_bwd_go<IN, gdn::kF32>(d, a, grid, st);
    if (dy == GDN_BF16) return attn_prep_bwd_go<IN, gdn::kBF16>(d, a, grid, st);
    return attn_prep_bwd_go<IN, gdn::kF16>(d, a, grid, st);
}

constexpr int kAttnBwdBlocks = 2048;  // most blocks of the gradient kernel: sizes its workspace

bool attn_head_dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128 || d == 256; }

// ---------------------------------------------------------------- decode

// Whether a pair is left to one CTA, given the most tiles of 16 keys that it can have (by the page table's width: the lengths are
// on the device): up to 256 keys always, up to 512 when there are 64 pairs and more.  Measured in a graph (us, one CTA a pair
// against pieces and a join; bf16, groups of 4, equal rows):
//   rows x key heads    keys     d = 32        64           128          256
//        1 x 2           256   3.9 /  5.7   4.1 /  5.8    5.2 /  6.5    6.7 /  7.3
//                        512   5.3 /  5.9   5.6 /  5.9    7.5 /  6.7   10.0 /  7.7
//        8 x 8           512   7.1 /  9.3   7.5 / 12.5    9.1 / 13.7   11.8 / 16.5
//                       1024  10.8 / 10.1  11.6 / 13.9   14.4 / 16.7   18.9 / 22.3
//       64 x 8           512  10.1 / 15.3  15.2 / 20.8   27.2 / 33.0   47.5 / 52.5
//                       1024  16.2 / 21.0  25.8 / 32.0   45.9 / 53.0   82.3 / 90.9
// Equal rows of 1024 keys would still gain from one CTA a pair at 64 pairs and more; the limit stays below, as one long row among
// short ones would then be alone on its CTA.  Rows of 256 keys under a table for many more are cut: 8 x 8 of 128, 12.0 for 6.4.
bool attn_alone(long long tiles, long long pairs) { return tiles <= (pairs >= 64 ? 32 : 16); }

template <bool BF, int D, int NT, bool CHOSEN>
gdn_status_t attn_decode_run(gdn::AttnDecodeArgs a, const DeviceInfo& dev, cudaStream_t st) {
    using S = gdn::AttnShape<D, NT>;
    static std::atomic<unsigned long long> ready{0};  // devices whose attribute is set
    static std::atomic<int> per_sm{0};
    auto* kernel = gdn::attn_decode_kernel<BF, D, NT, CHOSEN>;
    const unsigned long long bit = dev.dev < 64 ? 1ull << dev.dev : 0;
    if ((ready.load(std::memory_order_acquire) & bit) == 0) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        int n = 0;
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, gdn::kAttnThreads, S::SMEM);
        if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "attn_decode_kernel: %s", cudaGetErrorString(e));
        per_sm.store(n < 1 ? 1 : n, std::memory_order_relaxed);
        ready.fetch_or(bit, std::memory_order_release);
    }
    const long long pairs = (long long)a.B * a.Hkv * a.hblocks;
    // Rows that can hold only a few keys are not cut up: a CTA takes a pair, without looking for its place and without a
    // join behind it.
    const long long most = a.pages != nullptr ? (long long)a.n_sel * a.tiles_per_page : (long long)a.max_pages * a.tiles_per_page;
    a.alone = attn_alone(most, pairs) && pairs < (1LL << 31);
    if (a.alone)
        return launch_after("attn_decode_kernel", kernel, dim3((unsigned)pairs), dim3(gdn::kAttnThreads), S::SMEM, st, a);
    // one resident wave, as far as the workspace reaches (half as far for 16 heads of 256 channels)
    constexpr int reach = D == 256 && NT == 2 ? gdn::kAttnMaxCtas / 2 : gdn::kAttnMaxCtas;
    int fit = per_sm.load(std::memory_order_relaxed);
    if (fit * dev.sms > reach && fit > 1) fit = reach / dev.sms > 1 ? reach / dev.sms : 1;
    const int ctas = fit * dev.sms < reach ? fit * dev.sms : reach;
    // few pairs: many pieces each, so one head per block and sixteen warps over its pieces, and blocks by pair: one per
    // CTA would be mostly blocks without a pair.  Very few: 64 channels of a head per block.
    constexpr int kSlice = D < 64 ? D : 64;
    a.by_pair = pairs * 4 < ctas;
    gdn_status_t r = launch_after("attn_decode_kernel", kernel, dim3((unsigned)ctas), dim3(gdn::kAttnThreads), S::SMEM, st, a);
    if (r != GDN_OK) return r;
    if (a.by_pair && pairs * S::HB * (D / kSlice) <= dev.sms)
        return launch_after("attn_join_kernel", gdn::attn_join_kernel<D, NT, 16, kSlice>, dim3((unsigned)pairs, S::HB, D / kSlice),
                            dim3(512), 0, st, a, ctas, 1);
    if (a.by_pair)
        return launch_after("attn_join_kernel", gdn::attn_join_kernel<D, NT, 16, D>, dim3((unsigned)pairs, S::HB), dim3(512), 0, st,
                            a, ctas, 1);
    return launch_after("attn_join_kernel", gdn::attn_join_kernel<D, NT, 8, D>, dim3((unsigned)ctas, (unsigned)NT), dim3(256), 0, st, a,
                        ctas, 8);
}

template <bool BF, int D>
gdn_status_t attn_decode_d(const gdn::AttnDecodeArgs& a, int nt, const DeviceInfo& dev, cudaStream_t st) {
    if (nt == 2)
        return a.pages == nullptr ? attn_decode_run<BF, D, 2, false>(a, dev, st)
                                  : attn_decode_run<BF, D, 2, true>(a, dev, st);
    return a.pages == nullptr ? attn_decode_run<BF, D, 1, false>(a, dev, st) : attn_decode_run<BF, D, 1, true>(a, dev, st);
}

template <bool BF>
gdn_status_t attn_decode_bf(const gdn::AttnDecodeArgs& a, int d, int nt, const DeviceInfo& dev, cudaStream_t st) {
    switch (d) {
        case 32: return attn_decode_d<BF, 32>(a, nt, dev, st);
        case 64: return attn_decode_d<BF, 64>(a, nt, dev, st);
        case 128: return attn_decode_d<BF, 128>(a, nt, dev, st);
        default: return attn_decode_d<BF, 256>(a, nt, dev, st);
    }
}

bool attn_decode_dim_ok(int d) { return d == 32 || d == 64 || d == 128 || d == 256; }

// Query-head tiles of 8 that a CTA takes together: two for groups above 8, as the keys are then read once for 16.
int attn_head_tiles(int group) { return group > 8 ? 2 : 1; }

constexpr size_t kAttnMetaBytes = (size_t)gdn::kAttnMaxCtas * 2 * sizeof(int);

template <bool BF>
gdn_status_t attn_mean_launch(int d, const gdn::AttnMeanArgs& a, unsigned grid, cudaStream_t st) {
    auto* kernel = d == 32    ? gdn::attn_page_mean_kernel<BF, 32>
                   : d == 64  ? gdn::attn_page_mean_kernel<BF, 64>
                   : d == 128 ? gdn::attn_page_mean_kernel<BF, 128>
                              : gdn::attn_page_mean_kernel<BF, 256>;
    return launch_after("attn_page_mean_kernel", kernel, dim3(grid), dim3(gdn::kMeanThreads), 0, st, a);
}

template <bool BF>
gdn_status_t attn_score_launch(int d, const gdn::AttnSelectArgs& a, unsigned grid, cudaStream_t st) {
    auto* kernel = d == 32    ? gdn::attn_score_kernel<BF, 32>
                   : d == 64  ? gdn::attn_score_kernel<BF, 64>
                   : d == 128 ? gdn::attn_score_kernel<BF, 128>
                              : gdn::attn_score_kernel<BF, 256>;
    return launch_after("attn_score_kernel", kernel, dim3(grid), dim3(gdn::kScoreThreads), 0, st, a);
}

}  // namespace

extern "C" {

gdn_status_t gdn_attn_prep(const void* q, const void* k, int64_t q_stride, int64_t k_stride, const float* w_q,
                           const float* w_k, float eps, const int32_t* positions, const double* inv_freq, int rot_dim,
                           int N, int Hq, int Hkv, int d, gdn_dtype_t in_dtype, gdn_dtype_t out_dtype, void* q_out,
                           void* k_out, gdn_stream_t stream) {
    REQUIRE(N >= 0, "N=%d < 0", N);
    REQUIRE_ATTN_HEADS();
    REQUIRE(attn_head_dim_ok(d), "d=%d not in {16,32,64,128,256}", d);
    REQUIRE(rot_dim >= 0 && rot_dim <= d && rot_dim % 16 == 0, "rot_dim=%d is not a multiple of 16 up to d", rot_dim);
    REQUIRE(dtype_ok(in_dtype) && dtype_ok(out_dtype), "bad dtype");
    REQUIRE(eps >= 0.f, "eps < 0");
    REQUIRE_STRIDE(q_stride, Hq, "q_stride");
    REQUIRE_STRIDE(k_stride, Hkv, "k_stride");
    if (N == 0) return GDN_OK;
    REQUIRE_PTR(q, "q"); REQUIRE_PTR(k, "k"); REQUIRE_PTR(w_q, "w_q"); REQUIRE_PTR(w_k, "w_k");
    REQUIRE_PTR(positions, "positions"); REQUIRE_PTR(q_out, "q_out"); REQUIRE_PTR(k_out, "k_out");
    if (rot_dim > 0) REQUIRE_PTR(inv_freq, "inv_freq");
    const long long nq = (long long)N * Hq * d * elem_size(out_dtype), nk = (long long)N * Hkv * d * elem_size(out_dtype);
    const long long sq = span_bytes(N, q_stride, (long long)Hq * d, in_dtype);
    const long long sk = span_bytes(N, k_stride, (long long)Hkv * d, in_dtype);
    const bool q_in_place = q_out == q && q_stride == (int64_t)Hq * d && in_dtype == out_dtype;
    const bool k_in_place = k_out == k && k_stride == (int64_t)Hkv * d && in_dtype == out_dtype;
    REQUIRE((q_in_place || !ranges_overlap(q_out, nq, q, sq)) && !ranges_overlap(q_out, nq, k, sk) &&
                (k_in_place || !ranges_overlap(k_out, nk, k, sk)) && !ranges_overlap(k_out, nk, q, sq),
            "an output overlaps an input");
    REQUIRE_APART({{"q_out", q_out, nq}, {"k_out", k_out, nk}},
                  {{"w_q", w_q, 4LL * d}, {"w_k", w_k, 4LL * d}, {"positions", positions, 4LL * N},
                   {"inv_freq", inv_freq, 4LL * rot_dim}});
    gdn::AttnPrepArgs a{};
    a.q = q; a.k = k; a.v = nullptr; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = 0;
    a.w_q = w_q; a.w_k = w_k; a.eps = eps; a.positions = positions; a.inv_freq = inv_freq; a.rot = rot_dim;
    a.N = N; a.Hq = Hq; a.Hkv = Hkv; a.out_dt = (int)out_dtype; a.q_out = q_out; a.k_out = k_out;
    return attn_prep_launch<false>(a, d, (int)in_dtype, reinterpret_cast<cudaStream_t>(stream));
}

gdn_status_t gdn_attn_prep_cache(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                                 int64_t v_stride, const float* w_q, const float* w_k, float eps,
                                 const int32_t* positions, const double* inv_freq, int rot_dim,
                                 const int32_t* cu_seqlens, int num_seqs, int N, int Hq, int Hkv, int d,
                                 const int32_t* page_table, int max_pages, int num_pages, int page_size,
                                 gdn_dtype_t in_dtype, gdn_dtype_t out_dtype, void* q_out, void* k_cache, void* v_cache,
                                 gdn_stream_t stream) {
    REQUIRE(N >= 0 && num_seqs >= 1, "bad sizes N=%d num_seqs=%d", N, num_seqs);
    REQUIRE_ATTN_HEADS();
    REQUIRE(attn_head_dim_ok(d), "d=%d not in {16,32,64,128,256}", d);
    REQUIRE(rot_dim >= 0 && rot_dim <= d && rot_dim % 16 == 0, "rot_dim=%d is not a multiple of 16 up to d", rot_dim);
    REQUIRE(dtype_ok(in_dtype) && dtype_ok(out_dtype), "bad dtype");
    REQUIRE(eps >= 0.f, "eps < 0");
    REQUIRE_STRIDE(q_stride, Hq, "q_stride");
    REQUIRE_STRIDE(k_stride, Hkv, "k_stride");
    REQUIRE_STRIDE(v_stride, Hkv, "v_stride");
    REQUIRE(cu_seqlens != nullptr || N % num_seqs == 0, "N=%d not a multiple of num_seqs=%d", N, num_seqs);
    REQUIRE_PAGES();
    if (out_dtype == GDN_F32)
        return fail(GDN_ERR_UNSUPPORTED, "gdn_attn_prep_cache is built for 16-bit caches");
    if (N == 0) return GDN_OK;
    REQUIRE_PTR(q, "q"); REQUIRE_PTR(k, "k"); REQUIRE_PTR(v, "v"); REQUIRE_PTR(w_q, "w_q"); REQUIRE_PTR(w_k, "w_k");
    REQUIRE_PTR(positions, "positions"); REQUIRE_PTR(page_table, "page_table"); REQUIRE_PTR(q_out, "q_out");
    REQUIRE_PTR(k_cache, "k_cache"); REQUIRE_PTR(v_cache, "v_cache"); OPT_PTR(cu_seqlens, "cu_seqlens");
    if (rot_dim > 0) REQUIRE_PTR(inv_freq, "inv_freq");
    const long long nq = (long long)N * Hq * d * 2, nc = (long long)num_pages * Hkv * page_size * d * 2;
    const long long sq = span_bytes(N, q_stride, (long long)Hq * d, in_dtype);
    const long long sk = span_bytes(N, k_stride, (long long)Hkv * d, in_dtype);
    const long long sv = span_bytes(N, v_stride, (long long)Hkv * d, in_dtype);
    const bool in_place = q_out == q && q_stride == (int64_t)Hq * d && in_dtype == out_dtype;
    REQUIRE((in_place || !ranges_overlap(q_out, nq, q, sq)) && !ranges_overlap(q_out, nq, k, sk) &&
                !ranges_overlap(q_out, nq, v, sv),
            "q_out overlaps an input");
    REQUIRE_APART({{"q_out", q_out, nq}, {"k_cache", k_cache, nc}, {"v_cache", v_cache, nc}},
                  {{"w_q", w_q, 4LL * d}, {"w_k", w_k, 4LL * d}, {"positions", positions, 4LL * N},
                   {"inv_freq", inv_freq, 4LL * rot_dim}, {"cu_seqlens", cu_seqlens, 4LL * num_seqs + 4},
                   {"page_table", page_table, 4LL * num_seqs * max_pages}});
    REQUIRE_APART({{"k_cache", k_cache, nc}, {"v_cache", v_cache, nc}}, {{"q", q, sq}, {"k", k, sk}, {"v", v, sv}});
    gdn::AttnPrepArgs a{};
    a.q = q; a.k = k; a.v = v; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.w_q = w_q; a.w_k = w_k; a.eps = eps; a.positions = positions; a.inv_freq = inv_freq; a.rot = rot_dim;
    a.N = N; a.Hq = Hq; a.Hkv = Hkv; a.out_dt = (int)out_dtype; a.q_out = q_out; a.k_out = k_cache; a.v_out = v_cache;
    a.cu = cu_seqlens; a.table = page_table; a.num_seqs = num_seqs; a.max_pages = max_pages; a.num_pages = num_pages;
    a.page_size = page_size;
    return attn_prep_launch<true>(a, d, (int)in_dtype, reinterpret_cast<cudaStream_t>(stream));
}

size_t gdn_attn_prep_bwd_workspace_size(int d) {
    return attn_head_dim_ok(d) ? (size_t)kAttnBwdBlocks * d * sizeof(float) : 0;
}

gdn_status_t gdn_attn_prep_bwd(const void* dq_out, const void* dk_out, const void* q, const void* k, int64_t q_stride,
                               int64_t k_stride, const float* w_q, const float* w_k, float eps,
                               const int32_t* positions, const double* inv_freq, int rot_dim, int N, int Hq, int Hkv,
                               int d, gdn_dtype_t in_dtype, gdn_dtype_t dy_dtype, void* dq, void* dk, float* dw_q,
                               float* dw_k, void* workspace, size_t workspace_bytes, gdn_stream_t stream) {
    REQUIRE(N >= 0, "N=%d < 0", N);
    REQUIRE_ATTN_HEADS();
    REQUIRE(attn_head_dim_ok(d), "d=%d not in {16,32,64,128,256}", d);
    REQUIRE(rot_dim >= 0 && rot_dim <= d && rot_dim % 16 == 0, "rot_dim=%d is not a multiple of 16 up to d", rot_dim);
    REQUIRE(dtype_ok(in_dtype) && dtype_ok(dy_dtype), "bad dtype");
    REQUIRE(eps >= 0.f, "eps < 0");
    REQUIRE_STRIDE(q_stride, Hq, "q_stride");
    REQUIRE_STRIDE(k_stride, Hkv, "k_stride");
    REQUIRE_PTR(dw_q, "dw_q"); REQUIRE_PTR(dw_k, "dw_k");
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (N == 0) {  // no token: zero gradients of the weights
        cudaError_t e = cudaMemsetAsync(dw_q, 0, (size_t)d * 4, st);
        if (e == cudaSuccess) e = cudaMemsetAsync(dw_k, 0, (size_t)d * 4, st);
        return e == cudaSuccess ? GDN_OK : fail(GDN_ERR_CUDA, "memset: %s", cudaGetErrorString(e));
    }
    REQUIRE_PTR(dq_out, "dq_out"); REQUIRE_PTR(dk_out, "dk_out"); REQUIRE_PTR(q, "q"); REQUIRE_PTR(k, "k");
    REQUIRE_PTR(w_q, "w_q"); REQUIRE_PTR(w_k, "w_k"); REQUIRE_PTR(positions, "positions");
    REQUIRE_PTR(dq, "dq"); REQUIRE_PTR(dk, "dk"); REQUIRE_PTR(workspace, "workspace");
    if (rot_dim > 0) REQUIRE_PTR(inv_freq, "inv_freq");
    REQUIRE(workspace_bytes >= gdn_attn_prep_bwd_workspace_size(d), "workspace of %zu bytes, %zu needed", workspace_bytes,
            gdn_attn_prep_bwd_workspace_size(d));
    const long long oq = (long long)N * Hq * d * elem_size(in_dtype), ok = (long long)N * Hkv * d * elem_size(in_dtype);
    const long long gq = (long long)N * Hq * d * elem_size(dy_dtype), gk = (long long)N * Hkv * d * elem_size(dy_dtype);
    const long long sq = span_bytes(N, q_stride, (long long)Hq * d, in_dtype);
    const long long sk = span_bytes(N, k_stride, (long long)Hkv * d, in_dtype);
    REQUIRE_APART({{"dq", dq, oq}, {"dk", dk, ok}, {"dw_q", dw_q, 4LL * d}, {"dw_k", dw_k, 4LL * d},
                   {"workspace", workspace, (long long)gdn_attn_prep_bwd_workspace_size(d)}},
                  {{"dq_out", dq_out, gq}, {"dk_out", dk_out, gk}, {"q", q, sq}, {"k", k, sk}, {"w_q", w_q, 4LL * d},
                   {"w_k", w_k, 4LL * d}, {"positions", positions, 4LL * N}, {"inv_freq", inv_freq, 4LL * rot_dim}});
    DeviceInfo dev;
    gdn_status_t r = device_info(&dev);
    if (r != GDN_OK) return r;
    const int lanes = d / 16, subs = gdn::kAttnPrepThreads / lanes;
    gdn::AttnPrepBwdArgs a{};
    a.q = q; a.k = k; a.dyq = dq_out; a.dyk = dk_out; a.q_stride = q_stride; a.k_stride = k_stride;
    a.w_q = w_q; a.w_k = w_k; a.eps = eps; a.positions = positions; a.inv_freq = inv_freq; a.rot = rot_dim;
    a.N = N; a.Hq = Hq; a.Hkv = Hkv; a.dq = dq; a.dk = dk;
    a.partial = reinterpret_cast<float*>(workspace);
    a.hps = attn_heads_per_unit((long long)N * (Hq + Hkv), lanes, Hq, dev.sms, 8);
    a.cq = (Hq + a.hps - 1) / a.hps;
    a.ck = (Hkv + a.hps - 1) / a.hps;
    const long long uq = (long long)N * a.cq, uk = (long long)N * a.ck;
    REQUIRE(uq < (1LL << 30) && uk < (1LL << 30), "N=%d with Hq=%d too large", N, Hq);
    // resident blocks, shared out between queries and keys by their rows
    const long long want = 2LL * dev.sms < kAttnBwdBlocks ? 2LL * dev.sms : kAttnBwdBlocks;
    long long bq = want * Hq / (Hq + Hkv), bk = want - bq;
    bq = bq < 1 ? 1 : bq;
    bk = bk < 1 ? 1 : bk;
    if (bq > (uq + subs - 1) / subs) bq = (uq + subs - 1) / subs;
    if (bk > (uk + subs - 1) / subs) bk = (uk + subs - 1) / subs;
    // one block of each (it has at most two units per lane group): it writes dw itself
    const bool direct = uq <= 2 * subs && uk <= 2 * subs;
    if (direct) bq = bk = 1;
    a.gq = (int)bq;
    a.dw_q = direct ? dw_q : nullptr;
    a.dw_k = dw_k;
    const unsigned blocks = (unsigned)(bq + bk);
    if (in_dtype == GDN_F32) r = attn_prep_bwd_dy<gdn::kF32>(d, (int)dy_dtype, a, blocks, st);
    else if (in_dtype == GDN_BF16) r = attn_prep_bwd_dy<gdn::kBF16>(d, (int)dy_dtype, a, blocks, st);
    else r = attn_prep_bwd_dy<gdn::kF16>(d, (int)dy_dtype, a, blocks, st);
    if (r != GDN_OK || direct) return r;
    return launch_after("attn_prep_dw_kernel", gdn::attn_prep_dw_kernel, dim3(2, (unsigned)((d + 31) / 32)), dim3(32, 32), 0, st,
                        (const float*)a.partial, a.gq, (int)blocks, d, dw_q, dw_k);
}

size_t gdn_attn_decode_workspace_size(int Hq, int Hkv, int d) {
    if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || !attn_decode_dim_ok(d)) return 0;
    const int nt = attn_head_tiles(Hq / Hkv);
    const size_t ctas = d == 256 && nt == 2 ? gdn::kAttnMaxCtas / 2 : gdn::kAttnMaxCtas;  // as many as are launched
    return kAttnMetaBytes + ctas * 2 * 8 * nt * (d + 2) * sizeof(float);
}

gdn_status_t gdn_attn_decode(const void* q, const void* k_cache, const void* v_cache, const int32_t* page_table,
                             const int32_t* lens, const int32_t* pages, int n_sel, int B, int Hq, int Hkv, int d,
                             int max_pages, int num_pages, int page_size, float scale, gdn_dtype_t dtype,
                             gdn_dtype_t y_dtype, void* y, void* workspace, size_t workspace_bytes, gdn_stream_t stream) {
    REQUIRE(B >= 0, "B=%d < 0", B);
    REQUIRE_ATTN_HEADS();
    REQUIRE(d >= 1, "d=%d < 1", d);
    REQUIRE(dtype_ok(dtype) && dtype_ok(y_dtype), "bad dtype");
    REQUIRE(scale == scale, "scale is NaN");
    if (!attn_decode_dim_ok(d) || dtype == GDN_F32)
        return fail(GDN_ERR_UNSUPPORTED, "gdn_attn_decode is built for d in {32,64,128,256} and 16-bit caches (d=%d)", d);
    REQUIRE_PAGES();
    if (pages != nullptr)
        REQUIRE(n_sel >= 1 && (long long)n_sel * page_size <= (1LL << 30), "bad n_sel=%d", n_sel);
    REQUIRE((long long)B * Hq < (1LL << 31), "B * Hq too large");
    if (B == 0) return GDN_OK;
    REQUIRE_PTR(q, "q"); REQUIRE_PTR(k_cache, "k_cache"); REQUIRE_PTR(v_cache, "v_cache");
    REQUIRE_PTR(page_table, "page_table"); REQUIRE_PTR(lens, "lens"); REQUIRE_PTR(y, "y"); OPT_PTR(pages, "pages");
    REQUIRE_PTR(workspace, "workspace");
    REQUIRE(workspace_bytes >= gdn_attn_decode_workspace_size(Hq, Hkv, d), "workspace of %zu bytes, %zu needed",
            workspace_bytes, gdn_attn_decode_workspace_size(Hq, Hkv, d));
    const long long ny = (long long)B * Hq * d * elem_size(y_dtype), nc = (long long)num_pages * Hkv * page_size * d * 2;
    REQUIRE_APART({{"y", y, ny}, {"workspace", workspace, (long long)gdn_attn_decode_workspace_size(Hq, Hkv, d)}},
                  {{"q", q, (long long)B * Hq * d * 2}, {"k_cache", k_cache, nc}, {"v_cache", v_cache, nc},
                   {"page_table", page_table, 4LL * B * max_pages}, {"lens", lens, 4LL * B},
                   {"pages", pages, 4LL * B * Hkv * n_sel}});
    DeviceInfo dev;
    gdn_status_t r = device_info(&dev);
    if (r != GDN_OK) return r;
    gdn::AttnDecodeArgs a{};
    const int nt = attn_head_tiles(Hq / Hkv);
    a.q = q; a.k_cache = k_cache; a.v_cache = v_cache; a.table = page_table; a.lens = lens; a.pages = pages;
    a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.group = Hq / Hkv; a.hblocks = (a.group + 8 * nt - 1) / (8 * nt);
    a.num_pages = num_pages; a.page_size = page_size; a.max_pages = max_pages; a.n_sel = pages != nullptr ? n_sel : 0;
    a.tiles_per_page = page_size / 16;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.y_dt = (int)y_dtype;
    a.y = y;
    a.meta = reinterpret_cast<int*>(workspace);
    a.part = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + kAttnMetaBytes);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return dtype == GDN_BF16 ? attn_decode_bf<true>(a, d, nt, dev, st) : attn_decode_bf<false>(a, d, nt, dev, st);
}

gdn_status_t gdn_attn_page_mean(const void* k_cache, const int32_t* page_table, const int32_t* lens,
                                const int32_t* starts, int B, int Hkv, int d, int max_pages, int num_pages,
                                int page_size, gdn_dtype_t dtype, float* page_mean, gdn_stream_t stream) {
    REQUIRE(B >= 0 && Hkv >= 1 && Hkv <= 65536, "bad sizes B=%d Hkv=%d", B, Hkv);
    REQUIRE(d >= 1 && dtype_ok(dtype), "bad d=%d or dtype", d);
    if (!attn_decode_dim_ok(d) || dtype == GDN_F32)
        return fail(GDN_ERR_UNSUPPORTED, "gdn_attn_page_mean is built for d in {32,64,128,256} and 16-bit caches (d=%d)", d);
    REQUIRE_PAGES();
    if (B == 0) return GDN_OK;
    REQUIRE_PTR(k_cache, "k_cache"); REQUIRE_PTR(page_table, "page_table"); REQUIRE_PTR(lens, "lens");
    REQUIRE_PTR(page_mean, "page_mean"); OPT_PTR(starts, "starts");
    REQUIRE_APART({{"page_mean", page_mean, (long long)num_pages * Hkv * d * 4}},
                  {{"k_cache", k_cache, (long long)num_pages * Hkv * page_size * d * 2},
                   {"page_table", page_table, 4LL * B * max_pages}, {"lens", lens, 4LL * B}, {"starts", starts, 4LL * B}});
    DeviceInfo dev;
    gdn_status_t r = device_info(&dev);
    if (r != GDN_OK) return r;
    gdn::AttnMeanArgs a{};
    a.k_cache = k_cache; a.table = page_table; a.lens = lens; a.starts = starts; a.B = B; a.Hkv = Hkv;
    a.num_pages = num_pages; a.page_size = page_size; a.max_pages = max_pages; a.mean = page_mean;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const long long most = (long long)B * Hkv * max_pages;  // units at most
    const long long room = (long long)gdn::kMeanPerSm * dev.sms;
    const unsigned grid = (unsigned)(most < room ? most : room);
    return dtype == GDN_BF16 ? attn_mean_launch<true>(d, a, grid, st) : attn_mean_launch<false>(d, a, grid, st);
}

size_t gdn_attn_select_workspace_size(int B, int Hkv, int max_pages) {
    return B < 1 || Hkv < 1 || max_pages < 1 ? 0 : (size_t)B * Hkv * max_pages * sizeof(unsigned long long);
}

gdn_status_t gdn_attn_select(const void* q, const float* page_mean, const int32_t* page_table, const int32_t* lens,
                             int B, int Hq, int Hkv, int d, int max_pages, int num_pages, int page_size, int n_sel,
                             int n_first, int n_last, gdn_dtype_t dtype, int32_t* pages, void* workspace,
                             size_t workspace_bytes, gdn_stream_t stream) {
    REQUIRE(B >= 0, "B=%d < 0", B);
    REQUIRE_ATTN_HEADS();
    REQUIRE(d >= 1 && dtype_ok(dtype), "bad d=%d or dtype", d);
    if (!attn_decode_dim_ok(d) || dtype == GDN_F32)
        return fail(GDN_ERR_UNSUPPORTED, "gdn_attn_select is built for d in {32,64,128,256} and 16-bit queries (d=%d)", d);
    REQUIRE_PAGES();
    REQUIRE(n_sel >= 1 && (long long)n_sel * page_size <= (1LL << 30), "bad n_sel=%d", n_sel);
    REQUIRE(n_first >= 0 && n_last >= 0 && (long long)n_first + n_last <= n_sel, "n_first=%d, n_last=%d: not within n_sel=%d",
            n_first, n_last, n_sel);
    REQUIRE((long long)B * Hkv <= 0x7fffffffLL, "B * Hkv too large");
    if (B == 0) return GDN_OK;
    REQUIRE_PTR(q, "q"); REQUIRE_PTR(page_mean, "page_mean"); REQUIRE_PTR(page_table, "page_table");
    REQUIRE_PTR(lens, "lens"); REQUIRE_PTR(pages, "pages"); REQUIRE_PTR(workspace, "workspace");
    REQUIRE(workspace_bytes >= gdn_attn_select_workspace_size(B, Hkv, max_pages), "workspace of %zu bytes, %zu needed",
            workspace_bytes, gdn_attn_select_workspace_size(B, Hkv, max_pages));
    REQUIRE_APART({{"pages", pages, 4LL * B * Hkv * n_sel},
                   {"workspace", workspace, (long long)gdn_attn_select_workspace_size(B, Hkv, max_pages)}},
                  {{"q", q, (long long)B * Hq * d * 2}, {"page_mean", page_mean, (long long)num_pages * Hkv * d * 4},
                   {"page_table", page_table, 4LL * B * max_pages}, {"lens", lens, 4LL * B}});
    DeviceInfo dev;
    gdn_status_t r = device_info(&dev);
    if (r != GDN_OK) return r;
    gdn::AttnSelectArgs a{};
    a.q = q; a.mean = page_mean; a.table = page_table; a.lens = lens; a.B = B; a.Hq = Hq; a.Hkv = Hkv;
    a.group = Hq / Hkv; a.num_pages = num_pages; a.page_size = page_size; a.max_pages = max_pages; a.n_sel = n_sel;
    a.n_first = n_first; a.n_last = n_last; a.keys = reinterpret_cast<unsigned long long*>(workspace); a.pages = pages;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (max_pages > n_sel) {  // else every row has all its pages chosen
        const long long most = (long long)B * Hkv * ((max_pages + gdn::kScorePages - 1) / gdn::kScorePages);
        const long long room = (long long)gdn::attn_score_per_sm(d) * dev.sms;
        const unsigned grid = (unsigned)(most < room ? most : room);
        r = dtype == GDN_BF16 ? attn_score_launch<true>(d, a, grid, st) : attn_score_launch<false>(d, a, grid, st);
        if (r != GDN_OK) return r;
    }
    return launch_after("attn_select_kernel", gdn::attn_select_kernel, dim3((unsigned)((long long)B * Hkv)),
                        dim3(gdn::kSelectThreads), 0, st, a);
}

}  // extern "C"
