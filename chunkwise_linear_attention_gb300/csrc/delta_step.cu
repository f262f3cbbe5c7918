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
// memory.
#include "cla_internal.cuh"
#include "elem_io.cuh"
#include "strided.cuh"

namespace cla {
namespace {

constexpr int kDsThreads = 128, kDsCols = 32;

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

template <typename E, int DK>
__global__ void __launch_bounds__(kDsThreads) delta_step_kernel(DsArgs g) {
    constexpr int R = DK / 16;  // rows of a thread
    __shared__ float s_q[DK], s_k[DK], s_part[kDsThreads / 32][3][kDsCols];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, cg = lane % 8, rg = warp * 4 + lane / 8;
    const int slice = blockIdx.x % g.slices;
    const long long bh = blockIdx.x / g.slices;
    const int b = (int)(bh / g.H), h = (int)(bh % g.H), hk = h / (g.H / g.Hk);
    const int col = slice * kDsCols + 4 * cg;
    const bool in = col < g.dv;
    const int n = g.lens == nullptr ? g.T : min(max(g.lens[b], 0), g.T);
    float *S = g.S + bh * DK * g.dv + col, *o = g.o + bh * g.T * g.dv + col;
    const E *q = static_cast<const E *>(g.q) + b * g.sq.b + hk * g.sq.h, *k = static_cast<const E *>(g.k) + b * g.sk.b + hk * g.sk.h;
    const E *v = static_cast<const E *>(g.v) + b * g.sv.b + h * g.sv.h + col;
    const float *ld = g.log_decay + b * g.sl.b + h * g.sl.h, *be = g.beta + b * g.sb.b + h * g.sb.h;

    float4 x[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
        x[i] = in && n > 0 ? __ldcs(reinterpret_cast<const float4 *>(S + (long long)(rg + 16 * i) * g.dv)) : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int t = 0; t < n; ++t) {
        for (int i = threadIdx.x; i < DK; i += kDsThreads) {
            s_q[i] = to_f32(q[t * g.sq.t + i]);
            s_k[i] = to_f32(k[t * g.sk.t + i]);
        }
        const float a = expf(ld[t * g.sl.t]), beta = be[t * g.sb.t];
        float vv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) vv[e] = in ? to_f32(v[t * g.sv.t + e]) : 0.f;
        __syncthreads();
        float sk[4] = {0.f, 0.f, 0.f, 0.f}, sq[4] = {0.f, 0.f, 0.f, 0.f}, qk = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float kk = s_k[rg + 16 * i], qq = s_q[rg + 16 * i];
            x[i].x = a == 0.f ? 0.f : a * x[i].x;
            x[i].y = a == 0.f ? 0.f : a * x[i].y;
            x[i].z = a == 0.f ? 0.f : a * x[i].z;
            x[i].w = a == 0.f ? 0.f : a * x[i].w;
            sk[0] = fmaf(kk, x[i].x, sk[0]), sk[1] = fmaf(kk, x[i].y, sk[1]), sk[2] = fmaf(kk, x[i].z, sk[2]), sk[3] = fmaf(kk, x[i].w, sk[3]);
            sq[0] = fmaf(qq, x[i].x, sq[0]), sq[1] = fmaf(qq, x[i].y, sq[1]), sq[2] = fmaf(qq, x[i].z, sq[2]), sq[3] = fmaf(qq, x[i].w, sq[3]);
            qk = fmaf(qq, kk, qk);
        }
#pragma unroll
        for (int w = 8; w < 32; w <<= 1) {
#pragma unroll
            for (int e = 0; e < 4; ++e) sk[e] += __shfl_xor_sync(~0u, sk[e], w), sq[e] += __shfl_xor_sync(~0u, sq[e], w);
            qk += __shfl_xor_sync(~0u, qk, w);
        }
        if (lane < 8) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s_part[warp][0][4 * cg + e] = sk[e], s_part[warp][1][4 * cg + e] = sq[e];
            s_part[warp][2][cg] = qk;
        }
        __syncthreads();
        float u[4], y[4];
        qk = 0.f;
#pragma unroll
        for (int w = 0; w < kDsThreads / 32; ++w) qk += s_part[w][2][cg];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float p = 0.f, r = 0.f;
#pragma unroll
            for (int w = 0; w < kDsThreads / 32; ++w) p += s_part[w][0][4 * cg + e], r += s_part[w][1][4 * cg + e];
            u[e] = beta * (vv[e] - p);
            y[e] = fmaf(qk, u[e], r);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float kk = s_k[rg + 16 * i];
            x[i].x = fmaf(kk, u[0], x[i].x), x[i].y = fmaf(kk, u[1], x[i].y), x[i].z = fmaf(kk, u[2], x[i].z), x[i].w = fmaf(kk, u[3], x[i].w);
        }
        if (rg == 0 && in) *reinterpret_cast<float4 *>(o + (long long)t * g.dv) = make_float4(y[0], y[1], y[2], y[3]);
        __syncthreads();
    }
    if (in && n > 0) {
#pragma unroll
        for (int i = 0; i < R; ++i) __stcs(reinterpret_cast<float4 *>(S + (long long)(rg + 16 * i) * g.dv), x[i]);
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
    if (!product_below({B, H, slices}, 2147483648.0) || T >= (int64_t)1 << 31 || !product_below({B, H, T, dim_v}, 1e15))
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
