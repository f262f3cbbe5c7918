// gated_scan.cu -- the gated linear recurrence whose decays and inputs are
// formed from gates inside the kernel: forward, backward and the one-token
// step.
//
//   r = sigmoid(rgate), i = sigmoid(igate), L = -c softplus(lam) r, a = e^L,
//   m = sqrt(1 - a^2),  h_t = a_t h_{t-1} + m_t i_t x_t
//
// The factor m keeps the state's variance where the inputs' is.  The adjoint
// is hbar_t = dh_t + a_{t+1} hbar_{t+1}, and with u = i x
//   dx = hbar m i,   digate = hbar m u (1 - i),
//   G  = dL L = hbar L a (h_{t-1} - a u / m),
//   drgate = G (1 - r),   dlam = sum G sigmoid(lam) / softplus(lam),
// where L / m -> 0 as L -> 0: writing the gradients with dL L instead of dL
// leaves no division by a vanishing m.
#include <math.h>

#include "cla_internal.cuh"
#include "elem_io.cuh"

namespace cla {
namespace {

constexpr int kGsChunk = CLA_GATED_SCAN_CKPT_CHUNK;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct Gate {
    float r1, i, i1, a, m, rm, y;  // 1 - r, i, 1 - i, a, m, 1/m, log2 a
};

__device__ __forceinline__ float softplus(float v) { return v > 20.f ? v : log1pf(expf(v)); }

__device__ __forceinline__ Gate gate(float rg, float ig, float nl2) {
    const float er = exp2f(-fabsf(rg) * kLog2e), ei = exp2f(-fabsf(ig) * kLog2e);
    const float R = 1.f / ((1.f + er) * (1.f + ei));
    const float ir = R * (1.f + ei), ii = R * (1.f + er);
    Gate q;
    const float r = rg >= 0.f ? ir : er * ir;
    q.r1 = rg >= 0.f ? er * ir : ir;
    q.i = ig >= 0.f ? ii : ei * ii;
    q.i1 = ig >= 0.f ? ei * ii : ii;
    float y = nl2 * r;
    y = y < -126.f ? -126.f : y;
    q.y = y;
    q.a = exp2f(y);
    const float om = fmaxf(-expm1f(2.f * y * kLn2), 1e-37f);
    q.rm = rsqrtf(om);
    q.m = om * q.rm;
    return q;
}

struct GsArgs {
    const uint8_t *reset;
    const int32_t *lens;
    long long T;
    int B, D;
    float c;
};

__device__ __forceinline__ long long seq_len(const GsArgs &g, int b) {
    if (g.lens == nullptr) return g.T;
    const long long n = g.lens[b];
    return n < 0 ? 0 : (n > g.T ? g.T : n);
}

template <typename E, bool STATES>
__global__ void gated_fwd_kernel(const E *x, const E *rg, const E *ig, const float *lam, const float *h0, E *h,
                                 float *hT, float *ckpt, GsArgs g) {
    const long long u = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (u >= (long long)g.B * g.D) return;
    const int b = (int)(u / g.D), d = (int)(u % g.D);
    const long long n = seq_len(g, b), nc = (g.T + kGsChunk - 1) / kGsChunk;
    const float nl2 = -g.c * softplus(lam[d]) * kLog2e;
    float s = h0 != nullptr ? h0[u] : 0.f;
    for (long long t = 0; t < g.T; ++t) {
        if (ckpt != nullptr && t % kGsChunk == 0) ckpt[((long long)b * nc + t / kGsChunk) * g.D + d] = s;
        const size_t at = ((size_t)b * g.T + t) * g.D + d;
        if (t < n) {
            const Gate q = gate(to_f32(rg[at]), to_f32(ig[at]), nl2);
            const float w = q.i * to_f32(x[at]);
            s = (g.reset != nullptr && g.reset[(size_t)b * g.T + t]) ? w : fmaf(q.a, s, q.m * w);
        }
        if constexpr (!STATES) h[at] = from_f32<E>(t < n ? s : 0.f);
    }
    if (hT != nullptr) hT[u] = s;
}

template <typename E>
__global__ void gated_bwd_kernel(const E *x, const E *rg, const E *ig, const float *lam, const float *ckpt,
                                 const E *dh, const float *dhT, E *dx, E *drg, E *dig, float *part, float *dh0,
                                 GsArgs g) {
    const long long u = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (u >= (long long)g.B * g.D) return;
    const int b = (int)(u / g.D), d = (int)(u % g.D);
    const long long n = seq_len(g, b), nc = (g.T + kGsChunk - 1) / kGsChunk;
    const float nl2 = -g.c * softplus(lam[d]) * kLog2e;
    float hb = dhT != nullptr ? dhT[u] : 0.f;  // a_{t+1} hbar_{t+1}
    double sum = 0.0;
    float hs[kGsChunk];
    for (long long ch = nc - 1; ch >= 0; --ch) {
        const long long t0 = ch * kGsChunk;
        const int m = (int)(g.T - t0 < kGsChunk ? g.T - t0 : kGsChunk);
        float s = ckpt[((long long)b * nc + ch) * g.D + d];
        for (int j = 0; j < m; ++j) {
            hs[j] = s;
            const size_t at = ((size_t)b * g.T + t0 + j) * g.D + d;
            if (t0 + j < n) {
                const Gate q = gate(to_f32(rg[at]), to_f32(ig[at]), nl2);
                const float w = q.i * to_f32(x[at]);
                s = (g.reset != nullptr && g.reset[(size_t)b * g.T + t0 + j]) ? w : fmaf(q.a, s, q.m * w);
            }
        }
        for (int j = m - 1; j >= 0; --j) {
            const size_t at = ((size_t)b * g.T + t0 + j) * g.D + d;
            float ox = 0.f, orr = 0.f, oi = 0.f;
            if (t0 + j < n) {
                const Gate q = gate(to_f32(rg[at]), to_f32(ig[at]), nl2);
                const float xv = to_f32(x[at]), w = q.i * xv;
                const bool rs = g.reset != nullptr && g.reset[(size_t)b * g.T + t0 + j];
                hb += to_f32(dh[at]);
                const float mm = rs ? 1.f : q.m;
                ox = hb * mm * q.i;
                oi = hb * mm * w * q.i1;
                const float G = rs ? 0.f : hb * (q.y * kLn2) * q.a * (hs[j] - q.a * q.rm * w);
                orr = G * q.r1;
                sum += (double)G;
                hb = rs ? 0.f : hb * q.a;
            }
            dx[at] = from_f32<E>(ox);
            drg[at] = from_f32<E>(orr);
            dig[at] = from_f32<E>(oi);
        }
    }
    part[u] = (float)sum;
    if (dh0 != nullptr) dh0[u] = hb;
}

// dlam_d = sigmoid(lam) / softplus(lam) * sum of the partial rows, in their order.  The ratio
// tends to 1 as lam -> -inf (both tend to e^lam).
__global__ void gated_dlam_kernel(const float *part, const float *lam, float *dlam, long long rows, int D) {
    const int d = blockIdx.x * blockDim.x + threadIdx.x;
    if (d >= D) return;
    float s = 0.f;
    for (long long i = 0; i < rows; ++i) s += part[i * D + d];
    const float l = lam[d];
    dlam[d] = l < -20.f ? s : s * (1.f / (1.f + expf(-l))) / softplus(l);
}

template <typename E>
__global__ void gated_step_kernel(const E *x, const E *rg, const E *ig, const float *lam, const uint8_t *reset,
                                  float *h, E *y, int B, int D, float c) {
    const long long u = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (u >= (long long)B * D) return;
    const int b = (int)(u / D), d = (int)(u % D);
    const Gate q = gate(to_f32(rg[u]), to_f32(ig[u]), -c * softplus(lam[d]) * kLog2e);
    const float w = q.i * to_f32(x[u]);
    const float s = (reset != nullptr && reset[b]) ? w : fmaf(q.a, h[u], q.m * w);
    h[u] = s;
    y[u] = from_f32<E>(s);
}

size_t gs_chunks(int64_t T) { return (size_t)((T + kGsChunk - 1) / kGsChunk); }

int gs_check(const char *fn, int64_t B, int64_t T, int64_t D, int dtype, float c) {
    if (B < 0 || T < 0 || D < 0) return fail(CLA_ERR_INVALID_ARG, "%s: negative size", fn);
    if (!(c > 0.f) || !isfinite(c)) return fail(CLA_ERR_INVALID_ARG, "%s: c must be positive and finite", fn);
    if (dtype_bytes(dtype) == 0) return fail(CLA_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
    if (!product_below({B, D}, 2147483648.0) || !product_below({B, T, D}, 1e15) || T > kMaxTokens)
        return fail(CLA_ERR_UNSUPPORTED, "%s: B * D must be below 2^31, T at most 2^31 - 512", fn);
    return CLA_OK;
}

}  // namespace
}  // namespace cla

using namespace cla;

extern "C" size_t cla_gated_scan_ckpt_elems(int64_t B, int64_t T, int64_t D) {
    if (B < 0 || T < 0 || D < 0 || T > kMaxTokens || !product_below({B, T, D}, 1e15)) return 0;
    return gs_chunks(T) * (size_t)B * (size_t)D;
}

extern "C" size_t cla_gated_scan_workspace_size(int64_t B, int64_t T, int64_t D) {
    if (B < 0 || T < 0 || D < 0 || T > kMaxTokens || !product_below({B, T, D}, 1e15)) return 0;
    return sizeof(WsHeader) + (cla_gated_scan_ckpt_elems(B, T, D) + (size_t)B * D) * 4;
}

template <typename E>
static int gs_fwd(const void *x, const void *rg, const void *ig, const float *lam, const float *h0, void *h, float *hT,
                  float *ckpt, const GsArgs &g, cudaStream_t s) {
    const unsigned grid = (unsigned)(((long long)g.B * g.D + 127) / 128);
    if (grid == 0) return CLA_OK;
    if (h != nullptr)
        gated_fwd_kernel<E, false><<<grid, 128, 0, s>>>((const E *)x, (const E *)rg, (const E *)ig, lam, h0, (E *)h, hT, ckpt, g);
    else
        gated_fwd_kernel<E, true><<<grid, 128, 0, s>>>((const E *)x, (const E *)rg, (const E *)ig, lam, h0, nullptr, hT, ckpt, g);
    return check_launch("cla_gated_scan_fwd");
}

extern "C" int cla_gated_scan_fwd(const void *x, const void *rgate, const void *igate, const float *lam, const float *h0,
                                  const uint8_t *reset, const int32_t *lens, void *h, float *hT, float *ckpt, float c,
                                  int dtype, int64_t B, int64_t T, int64_t D, void *ws, size_t ws_bytes, void *stream) {
    const char *fn = "cla_gated_scan_fwd";
    clear_error();
    if (int st = gs_check(fn, B, T, D, dtype, c)) return st;
    if (B * D == 0) return CLA_OK;
    if (lam == nullptr || (T > 0 && (!x || !rgate || !igate || !h)))
        return fail(CLA_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (!aligned_or_null({x, rgate, igate, h}, dtype_bytes(dtype)) || !aligned_or_null({lam, h0, hT, ckpt, lens}, 4))
        return fail(CLA_ERR_INVALID_ARG, "%s: a pointer is misaligned", fn);
    if (ws == nullptr || !aligned16(ws) || ws_bytes < cla_gated_scan_workspace_size(B, T, D))
        return fail(CLA_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes,
                    cla_gated_scan_workspace_size(B, T, D));
    const GsArgs g{reset, lens, T, (int)B, (int)D, c};
    cudaStream_t s = (cudaStream_t)stream;
    CLA_CUDA_TRY(cudaMemsetAsync(ws, 0, sizeof(WsHeader), s), fn);
    if (dtype == CLA_F32) return gs_fwd<float>(x, rgate, igate, lam, h0, h, hT, ckpt, g, s);
    if (dtype == CLA_BF16) return gs_fwd<__nv_bfloat16>(x, rgate, igate, lam, h0, h, hT, ckpt, g, s);
    return gs_fwd<__half>(x, rgate, igate, lam, h0, h, hT, ckpt, g, s);
}

template <typename E>
static int gs_bwd(const void *x, const void *rg, const void *ig, const float *lam, const float *h0, const float *ckpt,
                  const void *dh, const float *dhT, void *dx, void *drg, void *dig, float *dlam, float *dh0,
                  const GsArgs &g, void *ws, cudaStream_t s) {
    float *states = reinterpret_cast<float *>(static_cast<char *>(ws) + sizeof(WsHeader));
    float *part = states + gs_chunks(g.T) * (size_t)g.B * g.D;
    if (ckpt == nullptr && g.T > 0) {
        if (int st = gs_fwd<E>(x, rg, ig, lam, h0, nullptr, nullptr, states, g, s)) return st;
        ckpt = states;
    }
    const unsigned grid = (unsigned)(((long long)g.B * g.D + 127) / 128);
    if (grid > 0) {
        gated_bwd_kernel<E><<<grid, 128, 0, s>>>((const E *)x, (const E *)rg, (const E *)ig, lam, ckpt, (const E *)dh,
                                                 dhT, (E *)dx, (E *)drg, (E *)dig, part, dh0, g);
        if (int st = check_launch("cla_gated_scan_bwd")) return st;
    }
    if (dlam != nullptr && g.D > 0) {
        gated_dlam_kernel<<<(g.D + 127) / 128, 128, 0, s>>>(part, lam, dlam, g.B, g.D);
        return check_launch("cla_gated_scan_bwd");
    }
    return CLA_OK;
}

extern "C" int cla_gated_scan_bwd(const void *x, const void *rgate, const void *igate, const float *lam, const float *h0,
                                  const uint8_t *reset, const int32_t *lens, const float *ckpt, const void *dh,
                                  const float *dhT, void *dx, void *drgate, void *digate, float *dlam, float *dh0,
                                  float c, int dtype, int64_t B, int64_t T, int64_t D, void *ws, size_t ws_bytes,
                                  void *stream) {
    const char *fn = "cla_gated_scan_bwd";
    clear_error();
    if (int st = gs_check(fn, B, T, D, dtype, c)) return st;
    if (D == 0) return CLA_OK;
    if (lam == nullptr || (B * T > 0 && (!x || !rgate || !igate || !dh || !dx || !drgate || !digate)))
        return fail(CLA_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (!aligned_or_null({x, rgate, igate, dh, dx, drgate, digate}, dtype_bytes(dtype)) ||
        !aligned_or_null({lam, h0, dhT, ckpt, dlam, dh0, lens}, 4))
        return fail(CLA_ERR_INVALID_ARG, "%s: a pointer is misaligned", fn);
    if (ws == nullptr || !aligned16(ws) || ws_bytes < cla_gated_scan_workspace_size(B, T, D))
        return fail(CLA_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes,
                    cla_gated_scan_workspace_size(B, T, D));
    const GsArgs g{reset, lens, T, (int)B, (int)D, c};
    cudaStream_t s = (cudaStream_t)stream;
    CLA_CUDA_TRY(cudaMemsetAsync(ws, 0, sizeof(WsHeader), s), fn);
    if (dtype == CLA_F32)
        return gs_bwd<float>(x, rgate, igate, lam, h0, ckpt, dh, dhT, dx, drgate, digate, dlam, dh0, g, ws, s);
    if (dtype == CLA_BF16)
        return gs_bwd<__nv_bfloat16>(x, rgate, igate, lam, h0, ckpt, dh, dhT, dx, drgate, digate, dlam, dh0, g, ws, s);
    return gs_bwd<__half>(x, rgate, igate, lam, h0, ckpt, dh, dhT, dx, drgate, digate, dlam, dh0, g, ws, s);
}

extern "C" int cla_gated_scan_step(const void *x, const void *rgate, const void *igate, const float *lam,
                                   const uint8_t *reset, float *h, void *y, float c, int dtype, int64_t B, int64_t D,
                                   void *stream) {
    const char *fn = "cla_gated_scan_step";
    clear_error();
    if (int st = gs_check(fn, B, 1, D, dtype, c)) return st;
    if (B * D == 0) return CLA_OK;
    if (!x || !rgate || !igate || !lam || !h || !y) return fail(CLA_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (!aligned_or_null({x, rgate, igate, y}, dtype_bytes(dtype)) || !aligned_or_null({lam, h}, 4))
        return fail(CLA_ERR_INVALID_ARG, "%s: a pointer is misaligned", fn);
    cudaStream_t s = (cudaStream_t)stream;
    const unsigned grid = (unsigned)((B * D + 127) / 128);
    if (dtype == CLA_F32)
        gated_step_kernel<float><<<grid, 128, 0, s>>>((const float *)x, (const float *)rgate, (const float *)igate, lam, reset, h, (float *)y, (int)B, (int)D, c);
    else if (dtype == CLA_BF16)
        gated_step_kernel<__nv_bfloat16><<<grid, 128, 0, s>>>((const __nv_bfloat16 *)x, (const __nv_bfloat16 *)rgate, (const __nv_bfloat16 *)igate, lam, reset, h, (__nv_bfloat16 *)y, (int)B, (int)D, c);
    else
        gated_step_kernel<__half><<<grid, 128, 0, s>>>((const __half *)x, (const __half *)rgate, (const __half *)igate, lam, reset, h, (__half *)y, (int)B, (int)D, c);
    return check_launch(fn);
}
