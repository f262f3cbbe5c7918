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
// One warp walks the visible tokens of one row (forward, dq) or the tokens
// that see one key (dk, dv); a lane holds d / 32 columns.
#include <math.h>

#include "cla_internal.cuh"
#include "elem_io.cuh"

namespace cla {
namespace {

struct Str3 {
    long long b, h, t;
};

struct WaArgs {
    const int32_t *lens;
    float scale;
    long long T, window, sinks;
    int B, H, Hkv;
};

__device__ __forceinline__ long long wa_len(const WaArgs &g, int b) {
    if (g.lens == nullptr) return g.T;
    const long long n = g.lens[b];
    return n < 0 ? 0 : (n > g.T ? g.T : n);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename E, int N>
__device__ __forceinline__ void row_ld(const E *p, float (&v)[N]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = to_f32(p[lane * N + i]);
}
template <typename E, int N>
__device__ __forceinline__ void row_st(E *p, const float (&v)[N]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < N; ++i) p[lane * N + i] = from_f32<E>(v[i]);
}
template <int N>
__device__ __forceinline__ float dot(const float (&a)[N], const float (&b)[N]) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) s = fmaf(a[i], b[i], s);
    return warp_sum(s);
}

template <typename E, int N>
__global__ void wa_fwd_kernel(const E *q, const E *k, const E *v, E *o, float *lse, Str3 sq, Str3 sk, Str3 sv, Str3 so,
                              WaArgs g) {
    const long long row = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (row >= (long long)g.B * g.H * g.T) return;
    const long long t = row % g.T;
    const int h = (int)(row / g.T % g.H), b = (int)(row / g.T / g.H), hk = h / (g.H / g.Hkv);
    float acc[N], qv[N], kv[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
    float m = -INFINITY, l = 0.f;
    if (t < wa_len(g, b)) {
        row_ld(q + b * sq.b + h * sq.h + t * sq.t, qv);
        const long long lo = t - g.window + 1 > 0 ? t - g.window + 1 : 0;
        for (long long s = 0; s <= t; s = (s + 1 >= g.sinks && s + 1 < lo) ? lo : s + 1) {
            if (s < lo && s >= g.sinks) continue;
            row_ld(k + b * sk.b + hk * sk.h + s * sk.t, kv);
            const float x = dot(qv, kv) * g.scale;
            const float mn = fmaxf(m, x), f = expf(m - mn), p = expf(x - mn);
            row_ld(v + b * sv.b + hk * sv.h + s * sv.t, kv);
            l = l * f + p;
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = fmaf(p, kv[i], acc[i] * f);
            m = mn;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] /= l;
    }
    row_st(o + b * so.b + h * so.h + t * so.t, acc);
    if ((threadIdx.x & 31) == 0) lse[row] = l > 0.f ? m + logf(l) : -INFINITY;
}

template <typename E, int N>
__global__ void wa_dq_kernel(const E *q, const E *k, const E *v, const E *o, const float *lse, const E *dO, E *dq,
                             float *delta, Str3 sq, Str3 sk, Str3 sv, Str3 so, Str3 sd, Str3 sdq, WaArgs g) {
    const long long row = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (row >= (long long)g.B * g.H * g.T) return;
    const long long t = row % g.T;
    const int h = (int)(row / g.T % g.H), b = (int)(row / g.T / g.H), hk = h / (g.H / g.Hkv);
    float acc[N], qv[N], gv[N], kv[N], vv[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
    if (t < wa_len(g, b)) {
        row_ld(q + b * sq.b + h * sq.h + t * sq.t, qv);
        row_ld(dO + b * sd.b + h * sd.h + t * sd.t, gv);
        row_ld(o + b * so.b + h * so.h + t * so.t, vv);
        const float dl = dot(gv, vv), e = lse[row];
        if ((threadIdx.x & 31) == 0) delta[row] = dl;
        const long long lo = t - g.window + 1 > 0 ? t - g.window + 1 : 0;
        for (long long s = 0; s <= t; s = (s + 1 >= g.sinks && s + 1 < lo) ? lo : s + 1) {
            if (s < lo && s >= g.sinks) continue;
            row_ld(k + b * sk.b + hk * sk.h + s * sk.t, kv);
            row_ld(v + b * sv.b + hk * sv.h + s * sv.t, vv);
            const float p = expf(dot(qv, kv) * g.scale - e);
            const float ds = p * (dot(gv, vv) - dl) * g.scale;
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = fmaf(ds, kv[i], acc[i]);
        }
    }
    row_st(dq + b * sdq.b + h * sdq.h + t * sdq.t, acc);
}

template <typename E, int N>
__global__ void wa_dkv_kernel(const E *q, const E *k, const E *v, const float *lse, const float *delta, const E *dO,
                              E *dk, E *dv, Str3 sq, Str3 sk, Str3 sv, Str3 sd, Str3 sdk, Str3 sdv, WaArgs g) {
    const long long row = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (row >= (long long)g.B * g.Hkv * g.T) return;
    const long long s = row % g.T;
    const int hk = (int)(row / g.T % g.Hkv), b = (int)(row / g.T / g.Hkv), G = g.H / g.Hkv;
    float ak[N], av[N], qv[N], gv[N], kv[N], vv[N];
#pragma unroll
    for (int i = 0; i < N; ++i) ak[i] = av[i] = 0.f;
    const long long n = wa_len(g, b);
    if (s < n) {
        row_ld(k + b * sk.b + hk * sk.h + s * sk.t, kv);
        row_ld(v + b * sv.b + hk * sv.h + s * sv.t, vv);
        const long long end = s < g.sinks || g.window > n - s ? n : s + g.window;
        for (int h = hk * G; h < (hk + 1) * G; ++h)
            for (long long t = s; t < end; ++t) {
                const long long at = ((long long)b * g.H + h) * g.T + t;
                row_ld(q + b * sq.b + h * sq.h + t * sq.t, qv);
                row_ld(dO + b * sd.b + h * sd.h + t * sd.t, gv);
                const float p = expf(dot(qv, kv) * g.scale - lse[at]);
                const float ds = p * (dot(gv, vv) - delta[at]) * g.scale;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    ak[i] = fmaf(ds, qv[i], ak[i]);
                    av[i] = fmaf(p, gv[i], av[i]);
                }
            }
    }
    row_st(dk + b * sdk.b + hk * sdk.h + s * sdk.t, ak);
    row_st(dv + b * sdv.b + hk * sdv.h + s * sdv.t, av);
}

// One 16-byte piece of a cache slot per thread.
__global__ void wa_write_kernel(const char *k, const char *v, char *kc, char *vc, Str3 sk, Str3 sv, WaArgs g, int pieces) {
    const long long S = g.sinks + g.window;
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (long long)g.B * g.Hkv * S * pieces) return;
    const int piece = (int)(i % pieces);
    const long long slot = i / pieces % S, bh = i / pieces / S;
    const int h = (int)(bh % g.Hkv), b = (int)(bh / g.Hkv);
    const long long n = wa_len(g, b);
    long long p = slot;
    if (slot >= g.sinks && slot < n) p += (n - 1 - slot) / g.window * g.window;
    if (p >= n) return;
    reinterpret_cast<uint4 *>(kc)[i] = *reinterpret_cast<const uint4 *>(k + 2 * (b * sk.b + h * sk.h + p * sk.t) + 16 * piece);
    reinterpret_cast<uint4 *>(vc)[i] = *reinterpret_cast<const uint4 *>(v + 2 * (b * sv.b + h * sv.h + p * sv.t) + 16 * piece);
}

// A warp per (b, query head) walks the cache; the new token comes from k and v themselves, and
// the first query head of a key head writes it into its slot.
template <typename E, int N>
__global__ void wa_step_kernel(const E *q, const E *k, const E *v, E *kc, E *vc, const int32_t *pos, E *o, Str3 sq,
                               Str3 sk, Str3 sv, WaArgs g) {
    const long long row = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (row >= (long long)g.B * g.H) return;
    const int h = (int)(row % g.H), b = (int)(row / g.H), G = g.H / g.Hkv, hk = h / G;
    const long long S = g.sinks + g.window, p = pos[b];
    float acc[N], qv[N], kn[N], vn[N], x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
    if (p >= 0) {
        const long long mine = p < g.sinks ? p : g.sinks + (p - g.sinks) % g.window, n = p + 1 < S ? p + 1 : S;
        row_ld(q + b * sq.b + h * sq.h, qv);
        row_ld(k + b * sk.b + hk * sk.h, kn);
        row_ld(v + b * sv.b + hk * sv.h, vn);
        E *kb = kc + ((long long)b * g.Hkv + hk) * S * (32 * N), *vb = vc + ((long long)b * g.Hkv + hk) * S * (32 * N);
        float m = dot(qv, kn) * g.scale, l = 1.f;
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = vn[i];
        for (long long s = 0; s < n; ++s) {
            if (s == mine) continue;
            row_ld(kb + s * (32 * N), x);
            const float z = dot(qv, x) * g.scale;
            const float mn = fmaxf(m, z), f = expf(m - mn), e = expf(z - mn);
            row_ld(vb + s * (32 * N), x);
            l = l * f + e;
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = fmaf(e, x[i], acc[i] * f);
            m = mn;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] /= l;
        if (h == hk * G) {
            row_st(kb + mine * (32 * N), kn);
            row_st(vb + mine * (32 * N), vn);
        }
    }
    row_st(o + row * (32 * N), acc);
}

// ------------------------------------------------------------------ host checks
int wa_check(const char *fn, int64_t B, int64_t H, int64_t Hkv, int64_t T, int64_t d, int64_t window, int64_t sinks,
             int dtype, float scale) {
    if (B < 0 || H < 0 || Hkv < 0 || T < 0) return fail(CLA_ERR_INVALID_ARG, "%s: negative size", fn);
    if (window < 1 || sinks < 0) return fail(CLA_ERR_INVALID_ARG, "%s: window must be at least 1 and sinks 0", fn);
    if (Hkv == 0 ? H != 0 : H % Hkv != 0)
        return fail(CLA_ERR_INVALID_ARG, "%s: the query heads must be a multiple of the key heads", fn);
    if (!isfinite(scale)) return fail(CLA_ERR_INVALID_ARG, "%s: scale must be finite", fn);
    if (dtype != CLA_BF16 && dtype != CLA_F16) return fail(CLA_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
    if (d != 64 && d != 128) return fail(CLA_ERR_UNSUPPORTED, "%s: head dimension %lld", fn, (long long)d);
    if (!product_below({B, H}, 2147483648.0) || T > kMaxTokens || !product_below({B, H, T, d}, 1e15) ||
        !product_below({B, Hkv, d, window}, 1e15) || !product_below({B, Hkv, d, sinks}, 1e15))
        return fail(CLA_ERR_UNSUPPORTED, "%s: sizes too large", fn);
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
            if (size[j] > 1 && (s[j] <= 0 || s[j] % 8 != 0 || s[j] > (int64_t)1e15 / size[j]))
                return fail(CLA_ERR_INVALID_ARG, "%s: stride %lld of %s: a positive multiple of 8 elements is needed", fn,
                            (long long)s[j], names[i]);
        out[i] = Str3{B > 1 ? s[0] : 0, heads[i] > 1 ? s[1] : 0, T > 1 ? s[2] : 0};
    }
    return CLA_OK;
}

unsigned warps_grid(long long warps) { return (unsigned)((warps + 3) / 4); }

}  // namespace
}  // namespace cla

using namespace cla;

#define WA_DISPATCH(kernel, grid, ...)                                                                              \
    do {                                                                                                            \
        if (dtype == CLA_BF16) {                                                                                    \
            using E = __nv_bfloat16;                                                                                \
            if (d == 64) kernel<E, 2><<<grid, 128, 0, s>>>(__VA_ARGS__);                                            \
            else kernel<E, 4><<<grid, 128, 0, s>>>(__VA_ARGS__);                                                    \
        } else {                                                                                                    \
            using E = __half;                                                                                       \
            if (d == 64) kernel<E, 2><<<grid, 128, 0, s>>>(__VA_ARGS__);                                            \
            else kernel<E, 4><<<grid, 128, 0, s>>>(__VA_ARGS__);                                                    \
        }                                                                                                           \
        if (int st = check_launch(fn)) return st;                                                                   \
    } while (0)

extern "C" int cla_window_attn_fwd(const void *q, const void *k, const void *v, const int32_t *lens, void *o, float *lse,
                                   float scale, int64_t window, int64_t sinks, int dtype, int64_t B, int64_t H,
                                   int64_t Hkv, int64_t T, int64_t d, const int64_t *strides, void *stream) {
    const char *fn = "cla_window_attn_fwd";
    clear_error();
    if (int st = wa_check(fn, B, H, Hkv, T, d, window, sinks, dtype, scale)) return st;
    if (B * H * T == 0) return CLA_OK;
    if (!q || !k || !v || !o || !lse) return fail(CLA_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (!aligned_or_null({q, k, v, o}, 16) || !aligned_or_null({lse, lens}, 4))
        return fail(CLA_ERR_INVALID_ARG, "%s: a pointer is misaligned", fn);
    static const char *const names[] = {"q", "k", "v", "o"};
    const int64_t heads[] = {H, Hkv, Hkv, H};
    Str3 r[4];
    if (int st = wa_strides(fn, strides, names, heads, 4, B, T, d, r)) return st;
    const WaArgs g{lens, scale, T, window < T ? window : T, sinks < T ? sinks : T, (int)B, (int)H, (int)Hkv};
    cudaStream_t s = (cudaStream_t)stream;
    WA_DISPATCH(wa_fwd_kernel, warps_grid(B * H * T), (const E *)q, (const E *)k, (const E *)v, (E *)o, lse, r[0], r[1],
                r[2], r[3], g);
    return CLA_OK;
}

extern "C" size_t cla_window_attn_bwd_workspace_size(int64_t B, int64_t H, int64_t Hkv, int64_t T, int64_t d,
                                                     int64_t window, int64_t sinks) {
    if (wa_check("cla_window_attn_bwd_workspace_size", B, H, Hkv, T, d, window, sinks, CLA_BF16, 1.f) != CLA_OK) return 0;
    return sizeof(WsHeader) + align_up((size_t)(B * H * T) * 4, 16);
}

extern "C" int cla_window_attn_bwd(const void *q, const void *k, const void *v, const int32_t *lens, const void *o,
                                   const float *lse, const void *dO, void *dq, void *dk, void *dv, float scale,
                                   int64_t window, int64_t sinks, int dtype, int64_t B, int64_t H, int64_t Hkv,
                                   int64_t T, int64_t d, const int64_t *strides, void *ws, size_t ws_bytes, void *stream) {
    const char *fn = "cla_window_attn_bwd";
    clear_error();
    if (int st = wa_check(fn, B, H, Hkv, T, d, window, sinks, dtype, scale)) return st;
    if (B * H * T == 0) return CLA_OK;
    if (!q || !k || !v || !o || !lse || !dO || !dq || !dk || !dv)
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
    const WaArgs g{lens, scale, T, window < T ? window : T, sinks < T ? sinks : T, (int)B, (int)H, (int)Hkv};
    cudaStream_t s = (cudaStream_t)stream;
    CLA_CUDA_TRY(cudaMemsetAsync(ws, 0, sizeof(WsHeader), s), fn);
    float *delta = reinterpret_cast<float *>(static_cast<char *>(ws) + sizeof(WsHeader));
    WA_DISPATCH(wa_dq_kernel, warps_grid(B * H * T), (const E *)q, (const E *)k, (const E *)v, (const E *)o, lse,
                (const E *)dO, (E *)dq, delta, r[0], r[1], r[2], r[3], r[4], r[5], g);
    WA_DISPATCH(wa_dkv_kernel, warps_grid(B * Hkv * T), (const E *)q, (const E *)k, (const E *)v, lse, delta,
                (const E *)dO, (E *)dk, (E *)dv, r[0], r[1], r[2], r[4], r[6], r[7], g);
    return CLA_OK;
}

extern "C" int cla_window_cache_write(const void *k, const void *v, const int32_t *lens, void *kcache, void *vcache,
                                      int64_t window, int64_t sinks, int dtype, int64_t B, int64_t Hkv, int64_t T,
                                      int64_t d, const int64_t *strides, void *stream) {
    const char *fn = "cla_window_cache_write";
    clear_error();
    if (int st = wa_check(fn, B, Hkv, Hkv, T, d, window, sinks, dtype, 1.f)) return st;
    if (B * Hkv * T == 0) return CLA_OK;
    if (!k || !v || !kcache || !vcache) return fail(CLA_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (!aligned_or_null({k, v, kcache, vcache}, 16) || !aligned_or_null({lens}, 4))
        return fail(CLA_ERR_INVALID_ARG, "%s: a pointer is misaligned", fn);
    static const char *const names[] = {"k", "v"};
    const int64_t heads[] = {Hkv, Hkv};
    Str3 r[2];
    if (int st = wa_strides(fn, strides, names, heads, 2, B, T, d, r)) return st;
    const int pieces = (int)(d / 8);
    const WaArgs g{lens, 1.f, T, window, sinks, (int)B, (int)Hkv, (int)Hkv};
    const long long total = B * Hkv * (sinks + window) * pieces;
    if (total / 256 >= 2147483647ll) return fail(CLA_ERR_UNSUPPORTED, "%s: sizes too large", fn);
    wa_write_kernel<<<(unsigned)((total + 255) / 256), 256, 0, (cudaStream_t)stream>>>(
        (const char *)k, (const char *)v, (char *)kcache, (char *)vcache, r[0], r[1], g, pieces);
    return check_launch(fn);
}

extern "C" size_t cla_window_attn_step_workspace_size(int64_t B, int64_t H, int64_t Hkv, int64_t d, int64_t window,
                                                      int64_t sinks) {
    if (wa_check("cla_window_attn_step_workspace_size", B, H, Hkv, 1, d, window, sinks, CLA_BF16, 1.f) != CLA_OK) return 0;
    return sizeof(WsHeader);
}

extern "C" int cla_window_attn_step(const void *q, const void *k, const void *v, void *kcache, void *vcache,
                                    const int32_t *pos, void *o, float scale, int64_t window, int64_t sinks, int dtype,
                                    int64_t B, int64_t H, int64_t Hkv, int64_t d, const int64_t *strides, void *ws,
                                    size_t ws_bytes, void *stream) {
    const char *fn = "cla_window_attn_step";
    clear_error();
    if (int st = wa_check(fn, B, H, Hkv, 1, d, window, sinks, dtype, scale)) return st;
    if (B * H == 0) return CLA_OK;
    if (!q || !k || !v || !kcache || !vcache || !pos || !o)
        return fail(CLA_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (!aligned_or_null({q, k, v, kcache, vcache, o}, 16) || !aligned_or_null({pos}, 4))
        return fail(CLA_ERR_INVALID_ARG, "%s: a pointer is misaligned", fn);
    const size_t need = cla_window_attn_step_workspace_size(B, H, Hkv, d, window, sinks);
    if (ws == nullptr || !aligned16(ws) || ws_bytes < need)
        return fail(CLA_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes, need);
    static const char *const names[] = {"q", "k", "v"};
    const int64_t heads[] = {H, Hkv, Hkv};
    Str3 r[3];
    int64_t full[9];
    if (strides != nullptr)
        for (int i = 0; i < 3; ++i) full[3 * i] = strides[2 * i], full[3 * i + 1] = strides[2 * i + 1], full[3 * i + 2] = d;
    if (int st = wa_strides(fn, strides ? full : nullptr, names, heads, 3, B, 1, d, r)) return st;
    const WaArgs g{nullptr, scale, 1, window, sinks, (int)B, (int)H, (int)Hkv};
    cudaStream_t s = (cudaStream_t)stream;
    WA_DISPATCH(wa_step_kernel, warps_grid(B * H), (const E *)q, (const E *)k, (const E *)v, (E *)kcache, (E *)vcache, pos,
                (E *)o, r[0], r[1], r[2], g);
    return CLA_OK;
}
