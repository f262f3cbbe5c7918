// qk_norm_rope.cu -- root-mean-square norm of every query and key head and the
// rotation by its token's position, in one pass; and the adjoint.
//
//   r = 1 / sqrt(mean(x^2) + eps),  n = r x,  y = w n,
//   o = y with the pairs (y_i, y_i+rot/2), i < rot / 2 (interleaved: (y_2i, y_2i+1)),
//       turned by the angle pos freq_i
// Backward, with g the gradient on o turned back:
//   dw = sum over rows of g n,  dx = r (g w - n mean(g w n))
//     = r (g w - x r^2 mean(g w x)):  both of a row's sums are taken at once.
//
// What bounds them is memory: a row is read once and written once (backward:
// two reads, one write).  A row is handled by the fewest lanes, a power of two,
// that take 16 of its values each, as the two 8-value pieces whose pairs turn
// into one another, so the rotation stays within a lane.  A group of such lanes
// takes a token and walks over its heads: the sines and cosines are formed once
// for all of them.
//
// Angles: positions reach 2^31 and an angle's 24 bits of fp32 would leave
// nothing of its fraction of a turn.  freq / 2 pi is formed as a 64-bit
// fraction of a turn from the integer product of freq's 24 bits and 2^64 / 2 pi;
// its product with the position wraps around as turns do.  What is left of the
// angle is off by less than 2^-33 (1 + |freq|) turns and is rounded to 24 bits.
#include <math.h>

#include "cla_internal.cuh"
#include "elem_io.cuh"
#include "strided.cuh"

namespace cla {
namespace {

constexpr int kQnThreads = 256;
constexpr int kQnBlocks = 456;  // of the backward: 3 for each of 152 multiprocessors

struct QnArgs {
    const float *w[2], *freq;  // of queries and keys
    const int32_t *pos, *lens;
    float eps, inv_d;
    int B, T, heads[2], d, rot, span, spans;  // span: heads that a group of lanes walks over
    long long items;
};

// freq / 2 pi as a signed fraction of a turn in 64 bits
__device__ __forceinline__ unsigned long long turns(float f) {
    const unsigned int u = __float_as_uint(f) & 0x7fffffffu;
    const int e = max((int)(u >> 23), 1) - 150;  // |f| = m 2^e
    const unsigned long long m = (u & 0x7fffffu) | (u >= 0x800000u ? 0x800000u : 0u), K = 0x28be60db9391054aull;
    const unsigned long long lo = m * K, hi = __umul64hi(m, K);
    unsigned long long t;
    if (e >= 0) t = e < 64 ? lo << e : 0ull;
    else if (e > -64) t = lo >> -e | hi << (64 + e);
    else t = e > -128 ? hi >> (-e - 64) : 0ull;
    return f < 0.f ? 0ull - t : t;
}
__device__ __forceinline__ void sincos_at(float f, int pos, float &s, float &c) {
    const unsigned long long phase = turns(f) * (unsigned long long)(long long)pos;
    sincospif((float)(int)(unsigned int)(phase >> 32) * 0x1p-31f, &s, &c);
}

// 8 values as they lie in memory
template <typename E>
struct Piece {
    uint4 v;
};
template <>
struct Piece<float> {
    uint4 v, w;
};
template <typename E>
__device__ __forceinline__ Piece<E> load_piece(const E *p) {
    Piece<E> r;
    r.v = __ldcs(reinterpret_cast<const uint4 *>(p));
    if constexpr (sizeof(E) == 4) r.w = __ldcs(reinterpret_cast<const uint4 *>(p) + 1);
    return r;
}
__device__ __forceinline__ float2 pair_f32(uint32_t u, __nv_bfloat16) { return __bfloat1622float2(reinterpret_cast<__nv_bfloat162 &>(u)); }
__device__ __forceinline__ float2 pair_f32(uint32_t u, __half) { return __half22float2(reinterpret_cast<__half2 &>(u)); }
__device__ __forceinline__ uint32_t pair_of(float a, float b, __nv_bfloat16) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return reinterpret_cast<uint32_t &>(v);
}
__device__ __forceinline__ uint32_t pair_of(float a, float b, __half) {
    __half2 v = __floats2half2_rn(a, b);
    return reinterpret_cast<uint32_t &>(v);
}
template <typename E>
__device__ __forceinline__ void unpack(const Piece<E> &p, float *x) {
    if constexpr (sizeof(E) == 4) {
        const uint32_t u[8] = {p.v.x, p.v.y, p.v.z, p.v.w, p.w.x, p.w.y, p.w.z, p.w.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(u[i]);
    } else {
        const uint32_t u[4] = {p.v.x, p.v.y, p.v.z, p.v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = pair_f32(u[i], E());
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
}
template <typename E>
__device__ __forceinline__ void store_piece(E *p, const float *x) {
    if constexpr (sizeof(E) == 4) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pair_of(x[0], x[1], E()), pair_of(x[2], x[3], E()), pair_of(x[4], x[5], E()),
                                                   pair_of(x[6], x[7], E()));
    }
}

// What a lane has of a row: values 8 c0.. and 8 c1.., x[0..7] and x[8..15]; the 8 frequencies from 8 sub on.
template <int G, bool IL>
struct Lane {
    int sub, c0, c1;
    bool in, turned;
    __device__ Lane(const QnArgs &g) {
        sub = threadIdx.x % G;
        in = 16 * sub < g.d;
        turned = 16 * sub < g.rot;
        c0 = turned && !IL ? 8 * sub : 16 * sub;
        c1 = turned && !IL ? 8 * sub + g.rot / 2 : 16 * sub + 8;
    }
    __device__ void angles(const QnArgs &g, int pos, float *s, float *c) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s[i] = 0.f, c[i] = 1.f;
            if (turned) sincos_at(g.freq[8 * sub + i], pos, s[i], c[i]);
        }
    }
    __device__ void weights(const float *w, float *x) const {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = w != nullptr && in ? w[i < 8 ? c0 + i : c1 + i - 8] : 1.f;
    }
    // the 16 values turned by (s, c)
    static __device__ __forceinline__ void turn(float *x, const float *s, const float *c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float &a = x[IL ? 2 * i : i], &b = x[IL ? 2 * i + 1 : 8 + i];
            const float t = a * c[i] - b * s[i];
            b = b * c[i] + a * s[i];
            a = t;
        }
    }
};

template <int G>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int x = 1; x < G; x <<= 1) v += __shfl_xor_sync(~0u, v, x);
    return v;
}

struct QnFwd {
    const void *x[2];
    void *o[2];
    Triple sx[2], so[2];
};

// Every lane stays for the shuffles; `on` says whether its group has a token.
template <typename E, int G, bool IL>
__global__ void __launch_bounds__(kQnThreads) qn_fwd_kernel(QnFwd p, QnArgs g) {
    constexpr int U = 4;  // rows in flight
    const Lane<G, IL> l(g);
    const long long item = (long long)blockIdx.x * (kQnThreads / G) + threadIdx.x / G;
    const bool on = item < g.items;
    const long long token = on ? item / g.spans : 0;
    const int b = (int)(token / g.T), t = (int)(token % g.T), first = on ? (int)(item % g.spans) * g.span : 0;
    const bool live = on && (g.lens == nullptr || t < g.lens[b]);
    float s[8], c[8], w[16];
    l.angles(g, live ? (g.pos != nullptr ? g.pos[token] : t) : 0, s, c);
    const int all = g.heads[0] + g.heads[1];
    for (int which = 0; which < 2; ++which) {
        const int base = which == 0 ? 0 : g.heads[0];
        const int lo = max(first, base), hi = min(min(first + g.span, base + g.heads[which]), all);
        const E *x = static_cast<const E *>(p.x[which]) + b * p.sx[which].b + t * p.sx[which].t;
        E *o = static_cast<E *>(p.o[which]) + b * p.so[which].b + t * p.so[which].t;
        l.weights(g.w[which], w);
        const int n = on ? hi - lo : 0;
        for (int h = 0; __any_sync(~0u, h < n); h += U) {
            Piece<E> a[U], z[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                a[u] = z[u] = Piece<E>{};
                if (h + u < n && live && l.in) {
                    const E *row = x + (lo - base + h + u) * p.sx[which].h;
                    a[u] = load_piece(row + l.c0);
                    z[u] = load_piece(row + l.c1);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float v[16], q = 0.f;
                unpack(a[u], v);
                unpack(z[u], v + 8);
#pragma unroll
                for (int i = 0; i < 16; ++i) q = fmaf(v[i], v[i], q);
                const float r = rsqrtf(row_sum<G>(q) * g.inv_d + g.eps);
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = v[i] * r * w[i];
                if (l.turned) l.turn(v, s, c);
                if (h + u < n && l.in) {
                    E *row = o + (lo - base + h + u) * p.so[which].h;
                    if (!live)
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = 0.f;
                    store_piece(row + l.c0, v);
                    store_piece(row + l.c1, v + 8);
                }
            }
        }
    }
}

struct QnBwd {
    const void *x[2], *g[2];
    void *dx[2];
    Triple sx[2], sg[2], sdx[2];
};

// A persistent block leaves its rows' sums of dw in parts[block][2][d].
template <typename E, int G, bool IL>
__global__ void __launch_bounds__(kQnThreads) qn_bwd_kernel(QnBwd p, QnArgs g, float *parts) {
    __shared__ float s_w[kQnThreads / 32][2][G * 16];
    const Lane<G, IL> l(g);
    float acc[2][16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[0][i] = acc[1][i] = 0.f;
    for (long long at = (long long)blockIdx.x * (kQnThreads / G); at < g.items; at += (long long)gridDim.x * (kQnThreads / G)) {
        const long long item = at + threadIdx.x / G;
        const bool on = item < g.items;
        const long long token = on ? item / g.spans : 0;
        const int b = (int)(token / g.T), t = (int)(token % g.T), first = on ? (int)(item % g.spans) * g.span : 0;
        const bool live = on && (g.lens == nullptr || t < g.lens[b]);
        float s[8], c[8];
        l.angles(g, live ? (g.pos != nullptr ? g.pos[token] : t) : 0, s, c);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = -s[i];
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const int base = which == 0 ? 0 : g.heads[0];
            const int lo = max(first, base), hi = min(first + g.span, base + g.heads[which]);
            const E *x = static_cast<const E *>(p.x[which]) + b * p.sx[which].b + t * p.sx[which].t;
            const E *y = static_cast<const E *>(p.g[which]) + b * p.sg[which].b + t * p.sg[which].t;
            E *dx = static_cast<E *>(p.dx[which]) + b * p.sdx[which].b + t * p.sdx[which].t;
            float w[16];
            l.weights(g.w[which], w);
            const int n = on ? hi - lo : 0;
            for (int h = 0; __any_sync(~0u, h < n); ++h) {
                const long long row = lo - base + h;
                const bool here = h < n && live && l.in;
                float v[16], u[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = u[i] = 0.f;
                if (here) {
                    unpack(load_piece(x + row * p.sx[which].h + l.c0), v);
                    unpack(load_piece(x + row * p.sx[which].h + l.c1), v + 8);
                    unpack(load_piece(y + row * p.sg[which].h + l.c0), u);
                    unpack(load_piece(y + row * p.sg[which].h + l.c1), u + 8);
                }
                if (l.turned) l.turn(u, s, c);
                float q = 0.f, m = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) q = fmaf(v[i], v[i], q), m = fmaf(u[i] * w[i], v[i], m);
                q = row_sum<G>(q);
                m = row_sum<G>(m);
                const float r = rsqrtf(q * g.inv_d + g.eps), k = m * g.inv_d * r * r;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    acc[which][i] = fmaf(u[i] * r, v[i], acc[which][i]);
                    v[i] = r * (u[i] * w[i] - v[i] * k);
                }
                if (h < n && l.in) {
                    E *to = dx + row * p.sdx[which].h;
                    store_piece(to + l.c0, v);
                    store_piece(to + l.c1, v + 8);
                }
            }
        }
    }
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float v = acc[which][i];
#pragma unroll
            for (int x = G; x < 32; x <<= 1) v += __shfl_xor_sync(~0u, v, x);
            if (lane < G && l.in) s_w[warp][which][i < 8 ? l.c0 + i : l.c1 + i - 8] = v;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * g.d; i += kQnThreads) {
        float v = 0.f;
#pragma unroll
        for (int x = 0; x < kQnThreads / 32; ++x) v += s_w[x][i / g.d][i % g.d];
        parts[(long long)blockIdx.x * 2 * g.d + i] = v;
    }
}

// dw = the blocks' parts, in a fixed order: 8 threads take every eighth of a column's
__global__ void __launch_bounds__(256) qn_join_kernel(const float *__restrict__ parts, float *dwq, float *dwk, int d, int blocks) {
    __shared__ float s[8][32];
    const int col = blockIdx.x * 32 + threadIdx.x % 32, y = threadIdx.x / 32;
    float v = 0.f;
    if (col < 2 * d)
        for (int i = y; i < blocks; i += 8) v += parts[(long long)i * 2 * d + col];
    s[y][threadIdx.x % 32] = v;
    __syncthreads();
    if (y == 0 && col < 2 * d) {
#pragma unroll
        for (int i = 1; i < 8; ++i) v += s[i][threadIdx.x];
        float *to = col < d ? dwq : dwk;
        if (to != nullptr) to[col < d ? col : col - d] = v;
    }
}

// ------------------------------------------------------------------ host
int qn_check(const char *fn, int64_t B, int64_t H, int64_t Hkv, int64_t T, int64_t d, int64_t rot, float eps, int dtype) {
    if (B < 0 || H < 0 || Hkv < 0 || T < 0 || d < 0 || rot < 0) return fail(CLA_ERR_INVALID_ARG, "%s: negative size", fn);
    if (!(eps > 0.f) || !isfinite(eps)) return fail(CLA_ERR_INVALID_ARG, "%s: eps must be a positive finite number", fn);
    if (rot > d) return fail(CLA_ERR_INVALID_ARG, "%s: %lld rotated values of a head of %lld", fn, (long long)rot, (long long)d);
    if (dtype_bytes(dtype) == 0) return fail(CLA_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
    if (d < 16 || d > 256 || d % 16 != 0 || rot % 16 != 0)
        return fail(CLA_ERR_UNSUPPORTED, "%s: head dimension %lld with %lld rotated: multiples of 16 up to 256 are needed", fn, (long long)d,
                    (long long)rot);
    if (!product_below({B, T}, 2147483648.0) || !product_below({H + Hkv}, 1 << 20) || !product_below({B, T, H + Hkv}, 68719476736.0))
        return fail(CLA_ERR_UNSUPPORTED, "%s: sizes too large", fn);
    return CLA_OK;
}

int qn_lanes(int64_t d) {
    int n = 1;
    while (16 * n < d) n *= 2;
    return n;
}

// Heads that a group of lanes walks over: all, or as few as it takes to have 8 groups of lanes for every thread slot
// of 64 multiprocessors.
QnArgs qn_args(const float *wq, const float *wk, const float *freq, const int32_t *pos, const int32_t *lens, float eps, int64_t rot,
               int64_t B, int64_t H, int64_t Hkv, int64_t T, int64_t d) {
    QnArgs g = {};
    g.w[0] = wq, g.w[1] = wk, g.freq = freq, g.pos = pos, g.lens = lens;
    g.eps = eps, g.inv_d = 1.f / (float)d;
    g.B = (int)B, g.T = (int)T, g.heads[0] = (int)H, g.heads[1] = (int)Hkv, g.d = (int)d, g.rot = (int)rot;
    g.span = (int)(H + Hkv);
    const long long enough = 152ll * 1024 / qn_lanes(d);
    while (g.span > 1 && B * T * ((H + Hkv + g.span - 1) / g.span) < enough) g.span = (g.span + 1) / 2;
    g.spans = (int)((H + Hkv + g.span - 1) / g.span);
    g.items = B * T * g.spans;
    return g;
}

template <typename E, bool IL>
int qn_fwd(const char *fn, const QnFwd &p, const QnArgs &g, cudaStream_t s) {
    const int G = qn_lanes(g.d), per = kQnThreads / G;
    const unsigned grid = (unsigned)((g.items + per - 1) / per);
    switch (G) {
        case 1: qn_fwd_kernel<E, 1, IL><<<grid, kQnThreads, 0, s>>>(p, g); break;
        case 2: qn_fwd_kernel<E, 2, IL><<<grid, kQnThreads, 0, s>>>(p, g); break;
        case 4: qn_fwd_kernel<E, 4, IL><<<grid, kQnThreads, 0, s>>>(p, g); break;
        case 8: qn_fwd_kernel<E, 8, IL><<<grid, kQnThreads, 0, s>>>(p, g); break;
        default: qn_fwd_kernel<E, 16, IL><<<grid, kQnThreads, 0, s>>>(p, g);
    }
    return check_launch(fn);
}

unsigned qn_bwd_blocks(const QnArgs &g) {
    const long long per = kQnThreads / qn_lanes(g.d), n = (g.items + per - 1) / per;
    return (unsigned)(n < kQnBlocks ? n : kQnBlocks);
}

template <typename E, bool IL>
int qn_bwd(const char *fn, const QnBwd &p, const QnArgs &g, float *dwq, float *dwk, float *parts, cudaStream_t s) {
    const unsigned grid = qn_bwd_blocks(g);
    switch (qn_lanes(g.d)) {
        case 1: qn_bwd_kernel<E, 1, IL><<<grid, kQnThreads, 0, s>>>(p, g, parts); break;
        case 2: qn_bwd_kernel<E, 2, IL><<<grid, kQnThreads, 0, s>>>(p, g, parts); break;
        case 4: qn_bwd_kernel<E, 4, IL><<<grid, kQnThreads, 0, s>>>(p, g, parts); break;
        case 8: qn_bwd_kernel<E, 8, IL><<<grid, kQnThreads, 0, s>>>(p, g, parts); break;
        default: qn_bwd_kernel<E, 16, IL><<<grid, kQnThreads, 0, s>>>(p, g, parts);
    }
    if (int st = check_launch(fn)) return st;
    if (dwq == nullptr && dwk == nullptr) return CLA_OK;
    qn_join_kernel<<<(unsigned)((2 * g.d + 31) / 32), 256, 0, s>>>(parts, dwq, dwk, g.d, (int)grid);
    return check_launch(fn);
}

}  // namespace
}  // namespace cla

using namespace cla;

extern "C" int cla_qk_norm_rope_fwd(const void *q, const void *k, const float *wq, const float *wk, const float *freq,
                                    const int32_t *pos, const int32_t *lens, void *qo, void *ko, float eps, int64_t rot,
                                    int interleaved, int dtype, int64_t B, int64_t H, int64_t Hkv, int64_t T, int64_t d,
                                    const int64_t *strides, void *stream) {
    const char *fn = "cla_qk_norm_rope_fwd";
    clear_error();
    if (int st = qn_check(fn, B, H, Hkv, T, d, rot, eps, dtype)) return st;
    const bool any_q = B * T * H > 0, any_k = B * T * Hkv > 0;
    if ((any_q && (!q || !qo)) || (any_k && (!k || !ko)) || ((any_q || any_k) && rot > 0 && !freq))
        return fail(CLA_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (!aligned_or_null({q, k, qo, ko}, 16) || !aligned_or_null({wq, wk, freq, pos, lens}, 4))
        return fail(CLA_ERR_INVALID_ARG, "%s: a pointer is misaligned", fn);
    static const char *const names[] = {"q", "k", "qo", "ko"};
    const int64_t heads[] = {H, Hkv, H, Hkv}, ds[] = {d, d, d, d};
    Triple r[4];
    if (int st = view_strides(fn, strides, names, heads, ds, 4, B, T, (int64_t)(16 / dtype_bytes(dtype)), r)) return st;
    if (!any_q && !any_k) return CLA_OK;
    const QnArgs g = qn_args(wq, wk, freq, pos, lens, eps, rot, B, H, Hkv, T, d);
    const QnFwd p = {{q, k}, {qo, ko}, {r[0], r[1]}, {r[2], r[3]}};
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == CLA_F32) return interleaved ? qn_fwd<float, true>(fn, p, g, s) : qn_fwd<float, false>(fn, p, g, s);
    if (dtype == CLA_BF16) return interleaved ? qn_fwd<__nv_bfloat16, true>(fn, p, g, s) : qn_fwd<__nv_bfloat16, false>(fn, p, g, s);
    return interleaved ? qn_fwd<__half, true>(fn, p, g, s) : qn_fwd<__half, false>(fn, p, g, s);
}

extern "C" size_t cla_qk_norm_rope_bwd_workspace_size(int64_t B, int64_t H, int64_t Hkv, int64_t T, int64_t d) {
    if (qn_check("cla_qk_norm_rope_bwd_workspace_size", B, H, Hkv, T, d, 0, 1.f, CLA_F32) != CLA_OK) return 0;
    return (size_t)kQnBlocks * 2 * d * 4;
}

extern "C" int cla_qk_norm_rope_bwd(const void *q, const void *k, const float *wq, const float *wk, const float *freq,
                                    const int32_t *pos, const int32_t *lens, const void *dqo, const void *dko, void *dq, void *dk,
                                    float *dwq, float *dwk, float eps, int64_t rot, int interleaved, int dtype, int64_t B,
                                    int64_t H, int64_t Hkv, int64_t T, int64_t d, const int64_t *strides, void *ws,
                                    size_t ws_bytes, void *stream) {
    const char *fn = "cla_qk_norm_rope_bwd";
    clear_error();
    if (int st = qn_check(fn, B, H, Hkv, T, d, rot, eps, dtype)) return st;
    const bool any_q = B * T * H > 0, any_k = B * T * Hkv > 0;
    if ((any_q && (!q || !dqo || !dq)) || (any_k && (!k || !dko || !dk)) || ((any_q || any_k) && rot > 0 && !freq))
        return fail(CLA_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (!aligned_or_null({q, k, dqo, dko, dq, dk}, 16) || !aligned_or_null({wq, wk, freq, pos, lens, dwq, dwk}, 4))
        return fail(CLA_ERR_INVALID_ARG, "%s: a pointer is misaligned", fn);
    const size_t need = cla_qk_norm_rope_bwd_workspace_size(B, H, Hkv, T, d);
    if (ws == nullptr || !aligned16(ws) || ws_bytes < need)
        return fail(CLA_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes, need);
    static const char *const names[] = {"q", "k", "dqo", "dko", "dq", "dk"};
    const int64_t heads[] = {H, Hkv, H, Hkv, H, Hkv}, ds[] = {d, d, d, d, d, d};
    Triple r[6];
    if (int st = view_strides(fn, strides, names, heads, ds, 6, B, T, (int64_t)(16 / dtype_bytes(dtype)), r)) return st;
    cudaStream_t s = (cudaStream_t)stream;
    if (!any_q && !any_k) {
        if (dwq) CLA_CUDA_TRY(cudaMemsetAsync(dwq, 0, d * 4, s), fn);
        if (dwk) CLA_CUDA_TRY(cudaMemsetAsync(dwk, 0, d * 4, s), fn);
        return CLA_OK;
    }
    const QnArgs g = qn_args(wq, wk, freq, pos, lens, eps, rot, B, H, Hkv, T, d);
    const QnBwd p = {{q, k}, {dqo, dko}, {dq, dk}, {r[0], r[1]}, {r[2], r[3]}, {r[4], r[5]}};
    float *parts = static_cast<float *>(ws);
    if (dtype == CLA_F32)
        return interleaved ? qn_bwd<float, true>(fn, p, g, dwq, dwk, parts, s) : qn_bwd<float, false>(fn, p, g, dwq, dwk, parts, s);
    if (dtype == CLA_BF16)
        return interleaved ? qn_bwd<__nv_bfloat16, true>(fn, p, g, dwq, dwk, parts, s)
                           : qn_bwd<__nv_bfloat16, false>(fn, p, g, dwq, dwk, parts, s);
    return interleaved ? qn_bwd<__half, true>(fn, p, g, dwq, dwk, parts, s) : qn_bwd<__half, false>(fn, p, g, dwq, dwk, parts, s);
}
