// delta_step.cu -- the delta rule with a decay per head, token by token on a
// state that is updated in place:
//
//   u = beta (v - a S^T k),  S' = a S + k u^T,  o = S'^T q = a S^T q + (q . k) u
//
// The second form of o lets one pass over the old state give both S^T k and
// S^T q, so a token takes one sum over the state's rows.
//
// What bounds it is reading and writing the state once, for however many tokens
// a call brings.  A block holds 32 columns of a head's state in registers: a
// thread 4 neighbouring columns of every 16th row, so that a warp's accesses
// are whole 128-byte lines.  The sums over rows go through shuffles and shared
// memory, with one barrier a token; four tokens' inputs are fetched together, a
// warp for each.
//
// Measured on GB300: one token for 64 x 32 states of 128 x 128: 43 us for 271 MB
// (6.3 TB/s, 92% of the measured copy rate); 8 tokens for 32 x 32 states: 49 us
// where the states' traffic is 20: the chain of a token (sums, exchange, update)
// at 24 warps a multiprocessor.
#include <math.h>

#include "cla_internal.cuh"
#include "elem_io.cuh"
#include "strided.cuh"

namespace cla {
namespace {

constexpr int kDsThreads = 128, kDsCols = 32, kDsTokens = 4;  // tokens whose inputs are fetched together

struct DsArgs {
    const void *q, *k, *v;
    const float *log_decay, *beta;
    const int32_t *lens;
    float *S, *o;
    Triple sq, sk, sv, sl, sb;
    int B, H, Hk, T, dv, slices;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

template <typename E, int DK>
__global__ void __launch_bounds__(kDsThreads) delta_step_kernel(DsArgs g) {
    constexpr int R = DK / 16, W = kDsThreads / 32;  // rows of a thread
    __shared__ __align__(16) float4 s_kq[kDsTokens][DK];  // k twice, q twice: operands of paired products as they are read
    __shared__ __align__(16) float s_v[kDsTokens][kDsCols];
    __shared__ float s_a[kDsTokens], s_b[kDsTokens];
    __shared__ __align__(16) float2 s_part[2][W][2][8][2];  // the warps' sums: S^T k and S^T q of 4 columns, two and two
    __shared__ float s_qk[kDsTokens];
    static_assert(kDsTokens <= W && kDsCols == 32, "a warp for every token");
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, cg = lane % 8, rg = warp * 4 + lane / 8;
    const unsigned bh = blockIdx.x / (unsigned)g.slices;
    const int slice = (int)(blockIdx.x - bh * (unsigned)g.slices);
    const int b = (int)(bh / (unsigned)g.H), h = (int)(bh - (unsigned)b * (unsigned)g.H);
    const int col = slice * kDsCols + 4 * cg;
    const bool in = col < g.dv;
    const int n = g.lens == nullptr ? g.T : min(max(g.lens[b], 0), g.T);
    float *S = g.S + ((long long)bh * DK + rg) * g.dv + col;
    float2 x[R][2];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float4 f = in && n > 0 ? __ldcs(reinterpret_cast<const float4 *>(S + 16ll * i * g.dv)) : make_float4(0.f, 0.f, 0.f, 0.f);
        x[i][0] = make_float2(f.x, f.y), x[i][1] = make_float2(f.z, f.w);
    }
    const int hk = (int)((unsigned)h / (unsigned)(g.H / g.Hk));
    float *o = g.o + (long long)bh * g.T * g.dv + col;
    const E *q = static_cast<const E *>(g.q) + b * g.sq.b + hk * g.sq.h + lane;
    const E *k = static_cast<const E *>(g.k) + b * g.sk.b + hk * g.sk.h + lane;
    const E *v = static_cast<const E *>(g.v) + b * g.sv.b + h * g.sv.h + slice * kDsCols + lane;
    const float *ld = g.log_decay + b * g.sl.b + h * g.sl.h, *be = g.beta + b * g.sb.b + h * g.sb.h;
    for (int t0 = 0; t0 < n; t0 += kDsTokens) {
        const int nt = min(kDsTokens, n - t0);
        if (t0 > 0) __syncthreads();  // the tokens before have been used
        if (warp < nt) {  // a token's inputs by a warp
            const long long t = t0 + warp;
            float qk = 0.f, kk[DK / 32], qq[DK / 32];
#pragma unroll
            for (int i = 0; i < DK / 32; ++i) kk[i] = to_f32(k[t * g.sk.t + 32 * i]), qq[i] = to_f32(q[t * g.sq.t + 32 * i]);
            s_v[warp][lane] = slice * kDsCols + lane < g.dv ? to_f32(v[t * g.sv.t]) : 0.f;
            if (lane == 0) {
                const float l = ld[t * g.sl.t];
                s_a[warp] = l == -INFINITY ? -1.f : expf(l);  // -1: a reset, which a decay that underflows is not
                s_b[warp] = be[t * g.sb.t];
            }
#pragma unroll
            for (int i = 0; i < DK / 32; ++i) {
                s_kq[warp][lane + 32 * i] = make_float4(kk[i], kk[i], qq[i], qq[i]);
                qk = fmaf(kk[i], qq[i], qk);
            }
#pragma unroll
            for (int w = 1; w < 32; w <<= 1) qk += __shfl_xor_sync(~0u, qk, w);
            if (lane == 0) s_qk[warp] = qk;
        }
        __syncthreads();
        for (int t = 0; t < nt; ++t) {
            float a = s_a[t];
            if (a < 0.f) {  // whatever the state holds
                a = 0.f;
#pragma unroll
                for (int i = 0; i < R; ++i) x[i][0] = x[i][1] = both(0.f);
            }
            float2 sk[2] = {both(0.f), both(0.f)}, sq[2] = {both(0.f), both(0.f)};
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float4 kq = s_kq[t][rg + 16 * i];
                const float2 kk = make_float2(kq.x, kq.y), qq = make_float2(kq.z, kq.w);
                sk[0] = fma2(kk, x[i][0], sk[0]), sk[1] = fma2(kk, x[i][1], sk[1]);
                sq[0] = fma2(qq, x[i][0], sq[0]), sq[1] = fma2(qq, x[i][1], sq[1]);
            }
            // the four lanes of a column group add up: one half of the sums goes to either pair of them, a half of that to each
            const bool hi = lane & 16, odd = lane & 8;
            float2 keep[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float2 give = hi ? sk[e] : sq[e];
                keep[e] = hi ? sq[e] : sk[e];
                keep[e].x += __shfl_xor_sync(~0u, give.x, 16), keep[e].y += __shfl_xor_sync(~0u, give.y, 16);
            }
            const float2 give = odd ? keep[0] : keep[1];
            float2 sum = odd ? keep[1] : keep[0];
            sum.x += __shfl_xor_sync(~0u, give.x, 8), sum.y += __shfl_xor_sync(~0u, give.y, 8);
            float2(*part)[2][8][2] = s_part[t & 1];  // the other one may still be read
            part[warp][hi][cg][odd] = sum;
            __syncthreads();
            const float qk = s_qk[t];
            float4 p = *reinterpret_cast<const float4 *>(part[0][0][cg]), y = *reinterpret_cast<const float4 *>(part[0][1][cg]);
#pragma unroll
            for (int w = 1; w < W; ++w) {
                const float4 f = *reinterpret_cast<const float4 *>(part[w][0][cg]), e = *reinterpret_cast<const float4 *>(part[w][1][cg]);
                p.x += f.x, p.y += f.y, p.z += f.z, p.w += f.w;
                y.x += e.x, y.y += e.y, y.z += e.z, y.w += e.w;
            }
            const float4 vv = *reinterpret_cast<const float4 *>(&s_v[t][4 * cg]);
            const float beta = s_b[t];
            const float2 u0 = make_float2(beta * fmaf(-a, p.x, vv.x), beta * fmaf(-a, p.y, vv.y));
            const float2 u1 = make_float2(beta * fmaf(-a, p.z, vv.z), beta * fmaf(-a, p.w, vv.w));
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float2 kk = *reinterpret_cast<const float2 *>(&s_kq[t][rg + 16 * i]);
                x[i][0] = fma2(kk, u0, mul2(both(a), x[i][0]));
                x[i][1] = fma2(kk, u1, mul2(both(a), x[i][1]));
            }
            if (rg == 0 && in)
                *reinterpret_cast<float4 *>(o + (long long)(t0 + t) * g.dv) =
                    make_float4(fmaf(qk, u0.x, a * y.x), fmaf(qk, u0.y, a * y.y), fmaf(qk, u1.x, a * y.z), fmaf(qk, u1.y, a * y.w));
        }
    }
    if (in && n > 0) {
#pragma unroll
        for (int i = 0; i < R; ++i)
            __stcs(reinterpret_cast<float4 *>(S + 16ll * i * g.dv), make_float4(x[i][0].x, x[i][0].y, x[i][1].x, x[i][1].y));
    }
    if (in)
        for (int t = n + rg; t < g.T; t += 16) *reinterpret_cast<float4 *>(o + (long long)t * g.dv) = make_float4(0.f, 0.f, 0.f, 0.f);
}

template <typename E>
int ds_launch(const char *fn, int64_t dk, const DsArgs &g, unsigned grid, cudaStream_t s) {
    if (dk == 128) delta_step_kernel<E, 128><<<grid, kDsThreads, 0, s>>>(g);
    else delta_step_kernel<E, 64><<<grid, kDsThreads, 0, s>>>(g);
    return check_launch(fn);
}

}  // namespace
}  // namespace cla

using namespace cla;

extern "C" int cla_delta_step(const void *q, const void *k, const void *v, const float *log_decay, const float *beta,
                              const int32_t *lens, float *S, float *o, int dtype, int64_t B, int64_t H, int64_t Hk, int64_t T,
                              int64_t dim_k, int64_t dim_v, const int64_t *strides, void *stream) {
    const char *fn = "cla_delta_step";
    clear_error();
    if (B < 0 || H < 0 || Hk < 0 || T < 0 || dim_k < 0 || dim_v < 0) return fail(CLA_ERR_INVALID_ARG, "%s: negative size", fn);
    if (H == 0 || Hk == 0 ? H != Hk : H % Hk != 0)
        return fail(CLA_ERR_INVALID_ARG, "%s: the value heads must be a multiple of the key heads", fn);
    const int64_t bytes = (int64_t)dtype_bytes(dtype);
    if (bytes == 0) return fail(CLA_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
    if ((dim_k != 64 && dim_k != 128) || dim_v % 4 != 0 || dim_v == 0)
        return fail(CLA_ERR_UNSUPPORTED, "%s: head dimensions %lld, %lld: dim_k of 64 or 128 and dim_v a multiple of 4 are needed", fn,
                    (long long)dim_k, (long long)dim_v);
    const int64_t slices = (dim_v + kDsCols - 1) / kDsCols;
    if (!product_below({B, H, slices}, 2147483648.0) || T > 65536 || !product_below({B, H, T, dim_v}, 1e15))
        return fail(CLA_ERR_UNSUPPORTED, "%s: sizes too large", fn);
    const bool any = B * H * T > 0;
    if (any && (!q || !k || !v || !log_decay || !beta || !S || !o)) return fail(CLA_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (!aligned_or_null({q, k, v}, (uintptr_t)bytes) || !aligned_or_null({log_decay, beta, lens}, 4) || !aligned_or_null({S, o}, 16))
        return fail(CLA_ERR_INVALID_ARG, "%s: a pointer is misaligned", fn);
    static const char *const names[] = {"q", "k", "v", "log_decay", "beta"};
    const int64_t heads[] = {Hk, Hk, H, H, H}, ds[] = {dim_k, dim_k, dim_v, 1, 1};
    Triple r[5];
    if (int st = view_strides(fn, strides, names, heads, ds, 5, B, T, 1, r)) return st;
    if (!any) return CLA_OK;
    const DsArgs g = {q, k, v, log_decay, beta, lens, S, o, r[0], r[1], r[2], r[3], r[4], (int)B, (int)H, (int)Hk, (int)T, (int)dim_v,
                      (int)slices};
    const unsigned grid = (unsigned)(B * H * slices);
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == CLA_F32) return ds_launch<float>(fn, dim_k, g, grid, s);
    if (dtype == CLA_BF16) return ds_launch<__nv_bfloat16>(fn, dim_k, g, grid, s);
    return ds_launch<__half>(fn, dim_k, g, grid, s);
}
