// window_attn.cu -- softmax attention over a sliding window and the first
// `sinks` tokens: forward, backward, the rolling cache's fill and the
// one-token step over that cache.
//
//   visible(t, s) = s <= t and (t - s < window or s < sinks)
//   o_t = sum_s P_ts v_s,  P = softmax over the visible s of scale q_t . k_s
//
// Backward, from lse = log sum exp: P = exp(scale q k^T - lse),
// dS = P (dO v^T - delta), delta_t = dO_t . o_t, dq = scale dS k,
// dk = scale dS^T q, dv = P^T dO.
//
// Forward and backward run on the tensor cores (window_attn_tc.cuh).
#include <math.h>

#include "cla_internal.cuh"
#include "window_attn_tc.cuh"
#include "window_step.cuh"

namespace cla {
namespace {

// One 16-byte piece of a cache slot per thread; it is 5 us of a 32768-token prefill's 528.
__global__ void wa_write_kernel(const char *k, const char *v, const int32_t *lens, char *kc, char *vc, Str3 sk, Str3 sv, int B,
                                int Hkv, int T, long long window, long long sinks, int pieces) {
    const long long S = sinks + window;
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (long long)B * Hkv * S * pieces) return;
    const int piece = (int)(i % pieces);
    const long long slot = i / pieces % S, bh = i / pieces / S;
    const int h = (int)(bh % Hkv), b = (int)(bh / Hkv), n = lens == nullptr ? T : min(max(lens[b], 0), T);
    long long p = slot;  // the last token that falls on the slot
    if (slot >= sinks && slot < n) p += (n - 1 - slot) / window * window;
    if (p >= n) return;
    reinterpret_cast<uint4 *>(kc)[i] = *reinterpret_cast<const uint4 *>(k + 2 * (b * sk.b + h * sk.h + p * sk.t) + 16 * piece);
    reinterpret_cast<uint4 *>(vc)[i] = *reinterpret_cast<const uint4 *>(v + 2 * (b * sv.b + h * sv.h + p * sv.t) + 16 * piece);
}

// ------------------------------------------------------------------ host checks
int wa_check(const char *fn, int64_t B, int64_t H, int64_t Hkv, int64_t T, int64_t d, int64_t window, int64_t sinks,
             int dtype, float scale) {
    if (B < 0 || H < 0 || Hkv < 0 || T < 0) return fail(CLA_ERR_INVALID_ARG, "%s: negative size", fn);
    if (window < 1 || sinks < 0) return fail(CLA_ERR_INVALID_ARG, "%s: window must be at least 1 and sinks 0", fn);
    if (H == 0 || Hkv == 0 ? H != Hkv : H % Hkv != 0)
        return fail(CLA_ERR_INVALID_ARG, "%s: the query heads must be a multiple of the key heads", fn);
    if (!isfinite(scale)) return fail(CLA_ERR_INVALID_ARG, "%s: scale must be finite", fn);
    if (dtype != CLA_BF16 && dtype != CLA_F16) return fail(CLA_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
    if (d != 64 && d != 128) return fail(CLA_ERR_UNSUPPORTED, "%s: head dimension %lld", fn, (long long)d);
    // tiles are numbered in 32 bits, in strides of a grid
    if (!product_below({B, H}, 2e9) || T > kMaxTokens || !product_below({B, H, T, d}, 1e15) ||
        !product_below({B, H, (T + kWT - 1) / kWT}, 2e9))
        return fail(CLA_ERR_UNSUPPORTED, "%s: sizes too large", fn);
    return CLA_OK;
}
int wa_check_cache(const char *fn, int64_t B, int64_t Hkv, int64_t d, int64_t window, int64_t sinks) {
    if (window > kMaxTokens || sinks > kMaxTokens - window || !product_below({B, Hkv, d, sinks + window}, 1e15))
        return fail(CLA_ERR_UNSUPPORTED, "%s: sinks + window must be at most 2^31 - 512, the cache below 10^15 elements", fn);
    return CLA_OK;
}

// The stride triples of a call's tensors: dense where `strides` is NULL.  heads[i]: of tensor i.
int wa_strides(const char *fn, const int64_t *strides, const char *const *names, const int64_t *heads, int n, int64_t B,
               int64_t T, int64_t d, Str3 *out) {
    for (int i = 0; i < n; ++i) {
        if (strides == nullptr) {
            out[i] = Str3{heads[i] * T * d, T * d, d};
            continue;
        }
        const int64_t *s = strides + 3 * i, size[3] = {B, heads[i], T};
        for (int j = 0; j < 3; ++j)
            if (size[j] > 1 && (s[j] <= 0 || s[j] % 8 != 0 || s[j] >= (int64_t)1 << 39))
                return fail(CLA_ERR_INVALID_ARG, "%s: stride %lld of %s: a positive multiple of 8 below 2^39 elements is needed", fn,
                            (long long)s[j], names[i]);
        out[i] = Str3{B > 1 ? s[0] : 0, heads[i] > 1 ? s[1] : 0, T > 1 ? s[2] : 0};
    }
    return CLA_OK;
}

// bh: the heads that a tile's items are dealt out over, key heads forward and query heads for dq.
WaArgs wa_args(const int32_t *lens, float scale, int64_t T, int64_t window, int64_t sinks, int64_t B, int64_t H, int64_t Hkv,
               int64_t bh) {
    const int64_t G = Hkv > 0 ? H / Hkv : 1;
    return WaArgs{lens, scale, (int)T, (int)(window < T ? window : T), (int)(sinks < T ? sinks : T), (int)B, (int)H, (int)Hkv,
                  Div((uint32_t)(G % 2 == 0 ? G / 2 : G)), Div((uint32_t)bh), Div((uint32_t)Hkv), Div((uint32_t)H),
                  Div((uint32_t)G)};
}

int wa_blocks(const char *fn, long long items, unsigned *blocks) {
    int n = 0;
    if (int st = multiprocessors(fn, &n)) return st;
    n = n < kStatusBlocks ? n : kStatusBlocks;
    *blocks = (unsigned)(items < n ? items : n);
    return CLA_OK;
}

long long wa_tiles(long long T) { return (T + kWT - 1) / kWT; }

template <int D, bool BF>
int wa_fwd(const char *fn, const WaMaps &m, void *o, float *lse, const Str3 &so, const WaArgs &g, WsHeader *hdr, cudaStream_t s) {
    static std::atomic<unsigned long long> done{0};
    constexpr int smem = FwdCfg<D>::SMEM;
    static_assert(smem >= kMinSmem, "one block a multiprocessor");
    const long long G = g.H / g.Hkv, tiles = wa_tiles(g.T);
    const long long items = (long long)g.B * g.Hkv * (G % 2 == 0 ? G / 2 * tiles : G * ((tiles + 1) / 2));
    unsigned blocks;
    if (int st = set_max_dynamic_smem(done, (const void *)wa_fwd_kernel<D, BF>, smem)) return st;
    if (int st = wa_blocks(fn, items, &blocks)) return st;
    wa_fwd_kernel<D, BF><<<blocks, FwdCfg<D>::THREADS, smem, s>>>(m, o, lse, so, g, (int)items, hdr);
    return check_launch(fn);
}

// Blocks of the dk/dv kernel: at most one a multiprocessor, and at least 2 steps each.  The partial
// sums are sized for this many whatever the device.
constexpr int kDkvBlocks = 152;
long long wa_dkv_blocks(int64_t B, int64_t H, int64_t T, int64_t window, int64_t sinks) {
    const Lists l((int)T, (int)(window < T ? window : T), (int)(sinks < T ? sinks : T));
    const long long n = (B * H * l.before(l.n) + 1) / 2;
    return n < kDkvBlocks ? n : kDkvBlocks;
}

template <int D, bool BF>
int wa_bwd(const char *fn, const WaMaps &m, const WaMaps &mkv, const void *o, const void *dO, const float *lse, void *dq, void *dk, void *dv,
           const Str3 *r, const WaArgs &g, void *ws, cudaStream_t s) {
    static std::atomic<unsigned long long> done_q{0}, done_kv{0};
    constexpr int smem_q = DqCfg<D>::SMEM, smem_kv = DkvCfg<D>::SMEM;
    static_assert(smem_q >= kMinSmem && smem_kv >= kMinSmem, "one block a multiprocessor");
    char *p = static_cast<char *>(ws);
    WsHeader *hdr = reinterpret_cast<WsHeader *>(p);
    float *delta = reinterpret_cast<float *>(p + sizeof(WsHeader));
    float *parts = reinterpret_cast<float *>(p + sizeof(WsHeader) + align_up((size_t)g.B * g.H * g.T * 4, 16));
    if (int st = set_max_dynamic_smem(done_q, (const void *)wa_dq_kernel<D, BF>, smem_q)) return st;
    if (int st = set_max_dynamic_smem(done_kv, (const void *)wa_dkv_kernel<D, BF>, smem_kv)) return st;
    const long long items = (long long)g.B * g.H * wa_tiles(g.T);
    unsigned blocks;
    if (int st = wa_blocks(fn, items, &blocks)) return st;
    wa_dq_kernel<D, BF><<<blocks, DqCfg<D>::THREADS, smem_q, s>>>(m, o, dO, lse, dq, delta, r[3], r[4], r[5], g, (int)items, hdr);
    if (int st = check_launch(fn)) return st;
    if (int st = wa_blocks(fn, wa_dkv_blocks(g.B, g.H, g.T, g.window, g.sinks), &blocks)) return st;
    CutList *cuts = reinterpret_cast<CutList *>(parts + (size_t)wa_dkv_blocks(g.B, g.H, g.T, g.window, g.sinks) * 4 * kWT * D);
    wa_dkv_kernel<D, BF><<<blocks, DkvCfg<D>::THREADS, smem_kv, s>>>(mkv, lse, delta, dk, dv, parts, cuts, r[6], r[7], g, hdr);
    if (int st = check_launch(fn)) return st;
    if (blocks > 1) {
        wa_join_kernel<D, BF><<<dim3(blocks - 1, kJoinY), 256, 0, s>>>(parts, cuts, dk, dv, r[6], r[7], g.T, (int)blocks);
        return check_launch(fn);
    }
    return CLA_OK;
}

}  // namespace
}  // namespace cla

using namespace cla;

extern "C" int cla_window_attn_fwd(const void *q, const void *k, const void *v, const int32_t *lens, void *o, float *lse,
                                   float scale, int64_t window, int64_t sinks, int dtype, int64_t B, int64_t H,
                                   int64_t Hkv, int64_t T, int64_t d, const int64_t *strides, void *ws,
                                   size_t ws_bytes, void *stream) {
    const char *fn = "cla_window_attn_fwd";
    clear_error();
    if (int st = wa_check(fn, B, H, Hkv, T, d, window, sinks, dtype, scale)) return st;
    if (B * H * T > 0 && (!q || !k || !v || !o || !lse)) return fail(CLA_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (!aligned_or_null({q, k, v, o}, 16) || !aligned_or_null({lse, lens}, 4))
        return fail(CLA_ERR_INVALID_ARG, "%s: a pointer is misaligned", fn);
    if (ws == nullptr || !aligned16(ws) || ws_bytes < sizeof(WsHeader))
        return fail(CLA_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes, sizeof(WsHeader));
    static const char *const names[] = {"q", "k", "v", "o"};
    const int64_t heads[] = {H, Hkv, Hkv, H};
    Str3 r[4];
    if (int st = wa_strides(fn, strides, names, heads, 4, B, T, d, r)) return st;
    const WaArgs g = wa_args(lens, scale, T, window, sinks, B, H, Hkv, B * Hkv);
    cudaStream_t s = (cudaStream_t)stream;
    WsHeader *hdr = static_cast<WsHeader *>(ws);
    if (B * H * T == 0) {
        CLA_CUDA_TRY(cudaMemsetAsync(ws, 0, sizeof(WsHeader), s), fn);
        return CLA_OK;
    }
    const bool bf = dtype == CLA_BF16;
    WaMaps m;
    if (!make_map_bht(&m.q, q, bf, d, T, H, B, r[0]) || !make_map_bht(&m.k, k, bf, d, T, Hkv, B, r[1]) ||
        !make_map_bht(&m.v, v, bf, d, T, Hkv, B, r[2]) || !make_map_bht(&m.x, o, bf, d, T, H, B, r[3]))
        return fail(CLA_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", fn);
    m.g = m.q;
    m.y = m.q;
    if (d == 128) return bf ? wa_fwd<128, true>(fn, m, o, lse, r[3], g, hdr, s) : wa_fwd<128, false>(fn, m, o, lse, r[3], g, hdr, s);
    return bf ? wa_fwd<64, true>(fn, m, o, lse, r[3], g, hdr, s) : wa_fwd<64, false>(fn, m, o, lse, r[3], g, hdr, s);
}

extern "C" size_t cla_window_attn_workspace_size(int64_t B, int64_t H, int64_t Hkv, int64_t T, int64_t d, int64_t window,
                                                 int64_t sinks) {
    return wa_check("cla_window_attn_workspace_size", B, H, Hkv, T, d, window, sinks, CLA_BF16, 1.f) == CLA_OK ? sizeof(WsHeader) : 0;
}

extern "C" size_t cla_window_attn_bwd_workspace_size(int64_t B, int64_t H, int64_t Hkv, int64_t T, int64_t d,
                                                     int64_t window, int64_t sinks) {
    if (wa_check("cla_window_attn_bwd_workspace_size", B, H, Hkv, T, d, window, sinks, CLA_BF16, 1.f) != CLA_OK) return 0;
    return sizeof(WsHeader) + align_up((size_t)(B * H * T) * 4, 16) +
           (size_t)wa_dkv_blocks(B, H, T, window, sinks) * (4 * kWT * d * 4 + sizeof(CutList));
}

extern "C" int cla_window_attn_bwd(const void *q, const void *k, const void *v, const int32_t *lens, const void *o,
                                   const float *lse, const void *dO, void *dq, void *dk, void *dv, float scale,
                                   int64_t window, int64_t sinks, int dtype, int64_t B, int64_t H, int64_t Hkv,
                                   int64_t T, int64_t d, const int64_t *strides, void *ws, size_t ws_bytes, void *stream) {
    const char *fn = "cla_window_attn_bwd";
    clear_error();
    if (int st = wa_check(fn, B, H, Hkv, T, d, window, sinks, dtype, scale)) return st;
    if (B * H * T > 0 && (!q || !k || !v || !o || !lse || !dO || !dq || !dk || !dv))
        return fail(CLA_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (!aligned_or_null({q, k, v, o, dO, dq, dk, dv}, 16) || !aligned_or_null({lse, lens}, 4))
        return fail(CLA_ERR_INVALID_ARG, "%s: a pointer is misaligned", fn);
    const size_t need = cla_window_attn_bwd_workspace_size(B, H, Hkv, T, d, window, sinks);
    if (ws == nullptr || !aligned16(ws) || ws_bytes < need)
        return fail(CLA_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes, need);
    static const char *const names[] = {"q", "k", "v", "o", "dO", "dq", "dk", "dv"};
    const int64_t heads[] = {H, Hkv, Hkv, H, H, H, Hkv, Hkv};
    Str3 r[8];
    if (int st = wa_strides(fn, strides, names, heads, 8, B, T, d, r)) return st;
    const WaArgs g = wa_args(lens, scale, T, window, sinks, B, H, Hkv, B * H);
    cudaStream_t s = (cudaStream_t)stream;
    if (B * H * T == 0) {
        CLA_CUDA_TRY(cudaMemsetAsync(ws, 0, sizeof(WsHeader), s), fn);
        return CLA_OK;
    }
    const bool bf = dtype == CLA_BF16;
    WaMaps m;
    if (!make_map_bht(&m.q, q, bf, d, T, H, B, r[0]) || !make_map_bht(&m.k, k, bf, d, T, Hkv, B, r[1]) ||
        !make_map_bht(&m.v, v, bf, d, T, Hkv, B, r[2]) || !make_map_bht(&m.g, dO, bf, d, T, H, B, r[4]) ||
        !make_map_bht(&m.x, dq, bf, d, T, H, B, r[5]))
        return fail(CLA_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", fn);
    m.y = m.x;
    WaMaps mkv = m;
    if (!make_map_bht(&mkv.x, dk, bf, d, T, Hkv, B, r[6]) || !make_map_bht(&mkv.y, dv, bf, d, T, Hkv, B, r[7]))
        return fail(CLA_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", fn);
    if (d == 128)
        return bf ? wa_bwd<128, true>(fn, m, mkv, o, dO, lse, dq, dk, dv, r, g, ws, s)
                  : wa_bwd<128, false>(fn, m, mkv, o, dO, lse, dq, dk, dv, r, g, ws, s);
    return bf ? wa_bwd<64, true>(fn, m, mkv, o, dO, lse, dq, dk, dv, r, g, ws, s)
              : wa_bwd<64, false>(fn, m, mkv, o, dO, lse, dq, dk, dv, r, g, ws, s);
}

extern "C" int cla_window_cache_write(const void *k, const void *v, const int32_t *lens, void *kcache, void *vcache,
                                      int64_t window, int64_t sinks, int dtype, int64_t B, int64_t Hkv, int64_t T,
                                      int64_t d, const int64_t *strides, void *stream) {
    const char *fn = "cla_window_cache_write";
    clear_error();
    if (int st = wa_check(fn, B, Hkv, Hkv, T, d, window, sinks, dtype, 1.f)) return st;
    if (int st = wa_check_cache(fn, B, Hkv, d, window, sinks)) return st;
    if (B * Hkv * T == 0) return CLA_OK;
    if (!k || !v || !kcache || !vcache) return fail(CLA_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (!aligned_or_null({k, v, kcache, vcache}, 16) || !aligned_or_null({lens}, 4))
        return fail(CLA_ERR_INVALID_ARG, "%s: a pointer is misaligned", fn);
    static const char *const names[] = {"k", "v"};
    const int64_t heads[] = {Hkv, Hkv};
    Str3 r[2];
    if (int st = wa_strides(fn, strides, names, heads, 2, B, T, d, r)) return st;
    const int pieces = (int)(d / 8);
    const long long total = B * Hkv * (sinks + window) * pieces;
    if (total / 256 >= 2147483647ll) return fail(CLA_ERR_UNSUPPORTED, "%s: sizes too large", fn);
    wa_write_kernel<<<(unsigned)((total + 255) / 256), 256, 0, (cudaStream_t)stream>>>(
        (const char *)k, (const char *)v, lens, (char *)kcache, (char *)vcache, r[0], r[1], (int)B, (int)Hkv, (int)T, window, sinks,
        pieces);
    return check_launch(fn);
}

namespace cla {
namespace {

constexpr int kMaxSplits = 16;  // blocks of a cluster; above 8 with the kernel's leave

void step_config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute &at, long long clusters, int splits, cudaStream_t s) {
    cfg.gridDim = dim3((unsigned)(clusters * splits));
    cfg.blockDim = dim3(kStepWarps * 32);
    cfg.stream = s;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)splits;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
}

// Clusters of each size that the current device runs at once (0: none), asked for once per device.
template <int D, bool BF, int NG>
int step_resident(const char *fn, int (&n)[kMaxSplits + 1]) {
    static std::atomic<int> known[64][kMaxSplits + 1];  // the number and 1
    int dev = 0;
    CLA_CUDA_TRY(cudaGetDevice(&dev), fn);
    const bool keep = dev < 64;
    for (int s = 1; s <= kMaxSplits; ++s) {
        n[s] = keep ? known[dev][s].load(std::memory_order_relaxed) - 1 : -1;
        if (n[s] >= 0) continue;
        if (s > 8)
            CLA_CUDA_TRY(cudaFuncSetAttribute((const void *)wa_step_kernel<D, BF, NG>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1), fn);
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute at;
        step_config(cfg, at, 1, s, nullptr);
        CLA_CUDA_TRY(cudaOccupancyMaxActiveClusters(&n[s], wa_step_kernel<D, BF, NG>, &cfg), fn);
        if (keep) known[dev][s].store(n[s] + 1, std::memory_order_relaxed);
    }
    return CLA_OK;
}

// Splits the slots of a (sequence, key head) over as many blocks as give the least rounds of clusters
// times the 16-slot tiles of a warp; a round's latency and join count as 3 tiles.  Measured (us; 4
// warps a block, d = 128, key heads in all x slots; 1, 2, 3, 4, 6, 8, 16 blocks a cluster):
//   8 x 32772   604 307 209 160 111  86  54      256 x 4100  104 124  98 110 110 121 177
//   64 x 2052    47  31  27  23  23  31  44      512 x 4100  230 202 190 187 194 221 335
//   128 x 4100   88  57  53  70  59  66  96
template <int D, bool BF, int NG>
int wa_step(const char *fn, const void *q, const void *k, const void *v, void *kc, void *vc, const int32_t *pos, void *o,
            const Str3 *r, StepArgs g, cudaStream_t s) {
    const int G = g.H / g.Hkv;
    g.groups = (G + 8 * NG - 1) / (8 * NG);
    const long long units = (long long)g.B * g.Hkv * g.groups, tiles = (g.slots + 15) / 16;
    int resident[kMaxSplits + 1];
    if (int st = step_resident<D, BF, NG>(fn, resident)) return st;
    g.splits = 1;
    long long least = -1;
    for (int n = 1; n <= kMaxSplits && (n - 1) * kStepWarps < tiles; ++n) {
        if (resident[n] == 0) continue;
        const long long cost = (units + resident[n] - 1) / resident[n] * ((tiles + n * kStepWarps - 1) / (n * kStepWarps) + 3);
        if (least < 0 || cost < least) least = cost, g.splits = n;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at;
    step_config(cfg, at, units, g.splits, s);
    CLA_CUDA_TRY(cudaLaunchKernelEx(&cfg, wa_step_kernel<D, BF, NG>, (const uint16_t *)q, (const uint16_t *)k, (const uint16_t *)v,
                                    (uint16_t *)kc, (uint16_t *)vc, pos, (uint16_t *)o, r[0], r[1], r[2], g),
                 fn);
    return check_launch(fn);
}

}  // namespace
}  // namespace cla

extern "C" int cla_window_attn_step(const void *q, const void *k, const void *v, void *kcache, void *vcache,
                                    const int32_t *pos, void *o, float scale, int64_t window, int64_t sinks, int dtype,
                                    int64_t B, int64_t H, int64_t Hkv, int64_t d, const int64_t *strides, void *stream) {
    const char *fn = "cla_window_attn_step";
    clear_error();
    if (int st = wa_check(fn, B, H, Hkv, 1, d, window, sinks, dtype, scale)) return st;
    if (int st = wa_check_cache(fn, B, Hkv, d, window, sinks)) return st;
    if (!product_below({B, H}, 1 << 27)) return fail(CLA_ERR_UNSUPPORTED, "%s: B * H must be below 2^27", fn);
    if (B * H == 0) return CLA_OK;
    if (!q || !k || !v || !kcache || !vcache || !pos || !o)
        return fail(CLA_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (!aligned_or_null({q, k, v, kcache, vcache, o}, 16) || !aligned_or_null({pos}, 4))
        return fail(CLA_ERR_INVALID_ARG, "%s: a pointer is misaligned", fn);
    static const char *const names[] = {"q", "k", "v"};
    const int64_t heads[] = {H, Hkv, Hkv};
    Str3 r[3];
    int64_t full[9];
    if (strides != nullptr)
        for (int i = 0; i < 3; ++i) full[3 * i] = strides[2 * i], full[3 * i + 1] = strides[2 * i + 1], full[3 * i + 2] = d;
    if (int st = wa_strides(fn, strides ? full : nullptr, names, heads, 3, B, 1, d, r)) return st;
    const StepArgs g{scale * 1.4426950408889634f, window, sinks + window, (int)sinks, (int)B, (int)H, (int)Hkv, 1, 1};
    cudaStream_t s = (cudaStream_t)stream;
    // 16 heads a block read the cache once for up to 16 heads of a group (64 x 2 x 4100 x 128, 16 heads a
    // group: 64 us against 78 with two blocks of 8) in 240 registers; 8 or fewer take 161
    const bool bf = dtype == CLA_BF16, wide = H / Hkv > 8;
#define CLA_STEP(D, BF) \
    (wide ? wa_step<D, BF, 2>(fn, q, k, v, kcache, vcache, pos, o, r, g, s) : wa_step<D, BF, 1>(fn, q, k, v, kcache, vcache, pos, o, r, g, s))
    if (d == 128) return bf ? CLA_STEP(128, true) : CLA_STEP(128, false);
    return bf ? CLA_STEP(64, true) : CLA_STEP(64, false);
#undef CLA_STEP
}
