// window_cache8.cu -- the rolling cache of window_attn.cu held in 8 bits: its
// fill from prompts and the one-token step over it.
//
// Slots go in blocks of 64.  What a block of a key head holds is e4m3 numbers
// times the block's factor, the smallest power of two (2^-64 at least) under
// which the largest of them stays within 448.  A power of two costs e4m3 none
// of its relative accuracy, makes a number's rounding depend on the number
// alone (above the subnormal end), and lets a block change its factor without
// rounding again, save what becomes subnormal.
//
// A step puts its token into its slot.  The block's factor becomes that of what
// the block then holds; where that differs from the one it had, the block's
// other numbers are written anew.
//
// The step is bound by reading the cache once.  As in window_step.cuh, the
// blocks of threads of a cluster share the slots of a (sequence, key head), and
// a warp takes 16 slots at a time from memory into the operands of m16n8k16
// products:
//   scores^T [16 slots x 8 heads] = K Q^T,  o^T [16 columns x 8 heads] += V^T P^T.
// e4m3 numbers turn into fp16 exactly, two with one instruction.  Queries turn
// into fp16 too, each head's by a power of two of its own under which its
// largest lies in [1, 2): exact for bf16 down to 2^-14 of that, and off by less
// than 2^-25 of it below.  The factors of v's blocks go into the exponent: with
// t = s + log2 f, the weights are 2^(t - m) with m the running maximum of t, and
// the sum that divides takes each with 1 / f.  Weights are in [0, 2^15]
// (2^7 at the maximum, 8 above before the maximum moves) as fp16 for their
// product: rounded by 2^-12 of themselves, or 2^-32 of the largest.
#include <math.h>

#include <type_traits>

#include "cla_internal.cuh"
#include "elem_io.cuh"
#include "strided.cuh"
#include "window_step.cuh"

namespace cla {
namespace {

constexpr int kC8Block = CLA_WINDOW_CACHE8_BLOCK;
static_assert(kC8Block == 64, "a block is a tile of four warps");

// two fp32 to e4m3 (a to the low byte), rounded to nearest even, 448 beyond it
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t f16x2_of(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
    return r;
}
// the factor of a block whose largest number is `top`
__device__ __forceinline__ float factor_of(float top) {
    // the exponent of top / 448 = top / (1.75 2^8), one up where top's mantissa is above 1.75
    const int e = (int)((__float_as_uint(top) + 0x1fffffu) >> 23) - 8;
    return __uint_as_float((uint32_t)min(max(e, 127 - 64), 127 + 120) << 23);
}
__device__ __forceinline__ float inverse(float f) { return __uint_as_float((254u << 23) - __float_as_uint(f)); }  // of a power of two

template <typename E>
__device__ __forceinline__ void load16(const E *p, float (&x)[16]) {
    const uint4 a[2] = {reinterpret_cast<const uint4 *>(p)[0], reinterpret_cast<const uint4 *>(p)[1]};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t w[4] = {a[i].x, a[i].y, a[i].z, a[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = unpack16<std::is_same<E, __nv_bfloat16>::value>(w[j]);
            x[8 * i + 2 * j] = f.x, x[8 * i + 2 * j + 1] = f.y;
        }
    }
}
__device__ __forceinline__ uint4 code16(const float (&x)[16], float by) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        w[j] = e4m3x2(x[4 * j] * by, x[4 * j + 1] * by) | e4m3x2(x[4 * j + 2] * by, x[4 * j + 3] * by) << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void decode16(const uint4 &c, float (&x)[16]) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t h = f16x2_of(w[j / 2] >> 16 * (j & 1));
        const float2 f = unpack16<false>(h);
        x[2 * j] = f.x, x[2 * j + 1] = f.y;
    }
}

// ------------------------------------------------------------------ prompts
// A block of threads per block of slots, of k or of v; every thread 16 values at a time.
template <typename E, int D>
__global__ void __launch_bounds__(128) c8_write_kernel(const E *k, const E *v, const int32_t *lens, uint8_t *kc, uint8_t *vc, float *kf,
                                                       float *vf, Triple sk, Triple sv, int Hkv, int T, long long window, long long sinks,
                                                       int blocks) {
    constexpr int P = D / 16, N = kC8Block * P / 128;  // pieces of a slot, of a thread
    __shared__ float s_top[4];
    const long long S = sinks + window;
    const long long bh = blockIdx.x / blocks, first = (long long)(blockIdx.x % blocks) * kC8Block;
    const int h = (int)(bh % Hkv), b = (int)(bh / Hkv), n = lens == nullptr ? T : min(max(lens[b], 0), T);
    if (first >= n) return;  // no token reaches the block
    const bool of_v = blockIdx.y != 0;
    const Triple st = of_v ? sv : sk;
    const E *x = (of_v ? v : k) + b * st.b + h * st.h;
    float val[N][16], top = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int at = threadIdx.x + 128 * i;
        const long long slot = first + at / P;
        long long p = slot;  // the last token that falls on the slot
        if (slot >= sinks && slot < n) p += (n - 1 - slot) / window * window;
#pragma unroll
        for (int j = 0; j < 16; ++j) val[i][j] = 0.f;
        if (slot < S && p < n) load16(x + p * st.t + 16 * (at % P), val[i]);
#pragma unroll
        for (int j = 0; j < 16; ++j) top = fmaxf(top, fabsf(val[i][j]));
    }
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, w));
    if (threadIdx.x % 32 == 0) s_top[threadIdx.x / 32] = top;
    __syncthreads();
    const float f = factor_of(fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]))), by = inverse(f);
    uint8_t *to = (of_v ? vc : kc) + (bh * S + first) * D;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int at = threadIdx.x + 128 * i;
        const long long slot = first + at / P;
        if (slot < S && slot < n) reinterpret_cast<uint4 *>(to)[at] = code16(val[i], by);
    }
    if (threadIdx.x == 0) (of_v ? vf : kf)[blockIdx.x] = f;
}

// ------------------------------------------------------------------ one token
struct Step8Args {
    const int32_t *pos;
    float c;  // scale log2 e
    long long window, sinks, slots;
    int H, Hkv, splits, blocks;  // blocks: of slots, of a sequence and key head
    Triple sq, sk, sv;
};

// The token's values into slot `mine` of its block (of n held slots in all), by all threads; what comes
// after a barrier sees it.
template <typename E, int D>
__device__ __forceinline__ void put_token(uint8_t *cache, float *factor, const E *x, long long first, long long mine, long long n,
                                          float *s_top) {
    constexpr int P = D / 16, N = kC8Block * P / 128;
    uint4 code[N];
    uint32_t most = 0u;
    float val[16], top = 0.f;
    int own = -1;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int at = threadIdx.x + 128 * i;
        const long long slot = first + at / P;
        code[i] = make_uint4(0u, 0u, 0u, 0u);
        if (slot == mine) {
            own = i;
            load16(x + 16 * (at % P), val);
#pragma unroll
            for (int j = 0; j < 16; ++j) top = fmaxf(top, fabsf(val[j]));
        } else if (slot < n) {
            code[i] = reinterpret_cast<const uint4 *>(cache + first * D)[at];
        }
        most = __vmaxu4(most, __vmaxu4(__vmaxu4(code[i].x & 0x7f7f7f7fu, code[i].y & 0x7f7f7f7fu),
                                       __vmaxu4(code[i].z & 0x7f7f7f7fu, code[i].w & 0x7f7f7f7fu)));
    }
    most = __vmaxu4(most, most >> 16);
    most = min(max(most & 0xffu, most >> 8 & 0xffu), 0x7eu);  // a NaN counts as the largest number
    const float old = *factor;
    if (most != 0u) top = fmaxf(top, unpack16<false>(f16x2_of(most)).x * old);
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, w));
    if (threadIdx.x % 32 == 0) s_top[threadIdx.x / 32] = top;
    __syncthreads();
    const float f = factor_of(fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]))), by = inverse(f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int at = threadIdx.x + 128 * i;
        const long long slot = first + at / P;
        uint4 *to = reinterpret_cast<uint4 *>(cache + first * D) + at;
        if (i == own) {
            *to = code16(val, by);
        } else if (slot < n && f != old) {
            float y[16];
            decode16(code[i], y);
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] *= old;
            *to = code16(y, by);
        }
    }
    __syncthreads();  // the old factor has been read, and s_top is free
    if (threadIdx.x == 0) *factor = f;
}

template <typename E, int D, int NG>
__global__ void __launch_bounds__(128) c8_step_kernel(const E *__restrict__ q, const E *__restrict__ k, const E *__restrict__ v,
                                                      uint8_t *kc, uint8_t *vc, float *kf, float *vf, E *__restrict__ o, Step8Args g) {
    constexpr int NH = 8 * NG, KC = D / 64, M = D / 16;  // 64-column pieces; products of 16 columns of o
    constexpr bool BF = std::is_same<E, __nv_bfloat16>::value;
    __shared__ float s_o[kStepWarps][NH][D], s_m[kStepWarps][NH], s_l[kStepWarps][NH], s_top[4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
    const int split = blockIdx.x % g.splits;
    const long long unit = blockIdx.x / g.splits;
    const int hk = (int)(unit % g.Hkv), b = (int)(unit / g.Hkv), G = g.H / g.Hkv;
    E *ob = o + ((long long)b * g.H + hk * G) * D;
    const long long p = g.pos[b];
    if (p < 0) {  // the whole cluster leaves
        if (split == 0)
            for (int i = threadIdx.x; i < G * D / 2; i += blockDim.x) reinterpret_cast<uint32_t *>(ob)[i] = 0u;
        return;
    }
    const long long mine = p < g.sinks ? p : g.sinks + (p - g.sinks) % g.window, n = min(p + 1, g.slots);
    uint8_t *kb = kc + unit * g.slots * D, *vb = vc + unit * g.slots * D;
    float *kfb = kf + unit * g.blocks, *vfb = vf + unit * g.blocks;
    const long long used = (n + kC8Block - 1) / kC8Block, share = (used + g.splits - 1) / g.splits;
    const long long first = split * share, end = min(used, first + share);
    if (mine / kC8Block >= first && mine / kC8Block < end) {
        const long long at = mine / kC8Block;
        put_token<E, D>(kb, kfb + at, k + b * g.sk.b + hk * g.sk.h, at * kC8Block, mine, n, s_top);
        put_token<E, D>(vb, vfb + at, v + b * g.sv.b + hk * g.sv.h, at * kC8Block, mine, n, s_top);
        __syncthreads();
    }
    for (int h0 = 0; h0 < G; h0 += NH) {  // 16 heads at most, or the cache again (from L2)
        const int nh = min(NH, G - h0);
        uint32_t qf[NG][KC][8];
        float fac[NG][2];
#pragma unroll
        for (int a = 0; a < NG; ++a) {
            float x[KC][16], top = 0.f;
#pragma unroll
            for (int c = 0; c < KC; ++c) {
#pragma unroll
                for (int i = 0; i < 16; ++i) x[c][i] = 0.f;
                if (8 * a + r < nh) load16(q + b * g.sq.b + (hk * G + h0 + 8 * a + r) * g.sq.h + 64 * c + 16 * j, x[c]);
#pragma unroll
                for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[c][i]));
            }
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
            const uint32_t e = min(max(__float_as_uint(top) >> 23, 1u), 253u);  // 2^(e - 127) <= top
            const float up = __uint_as_float(e << 23), down = __uint_as_float((254u - e) << 23);
#pragma unroll
            for (int c = 0; c < KC; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) qf[a][c][i] = pack16<false>(make_float2(x[c][2 * i] * down, x[c][2 * i + 1] * down));
            fac[a][0] = __shfl_sync(~0u, up, 8 * j) * g.c;  // of heads 2j, 2j + 1
            fac[a][1] = __shfl_sync(~0u, up, 8 * j + 4) * g.c;
        }
        float acc[NG][M][4], m[NG][2], l[NG][2];
#pragma unroll
        for (int a = 0; a < NG; ++a) {
            m[a][0] = m[a][1] = -INFINITY;
            l[a][0] = l[a][1] = 0.f;
#pragma unroll
            for (int y = 0; y < M; ++y) acc[a][y][0] = acc[a][y][1] = acc[a][y][2] = acc[a][y][3] = 0.f;
        }
        uint4 kx[2][KC];
        uint32_t vx[4][D / 32];
        float kfac = 0.f, vfac = 0.f;
        auto load = [&](long long blk) {
            const long long s0 = blk * kC8Block + 16 * warp;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    const long long s = s0 + r + 8 * i;
                    kx[i][c] = s < n ? __ldcs(reinterpret_cast<const uint4 *>(kb + s * D + 64 * c + 16 * j)) : make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const long long s = s0 + 2 * j + (i & 1) + 8 * (i >> 1);
                if constexpr (D == 128) {
                    const uint4 w = s < n ? __ldcs(reinterpret_cast<const uint4 *>(vb + s * D + 16 * r)) : make_uint4(0u, 0u, 0u, 0u);
                    vx[i][0] = w.x, vx[i][1] = w.y, vx[i][2] = w.z, vx[i][3] = w.w;
                } else {
                    const uint2 w = s < n ? __ldcs(reinterpret_cast<const uint2 *>(vb + s * D + 8 * r)) : make_uint2(0u, 0u);
                    vx[i][0] = w.x, vx[i][1] = w.y;
                }
            }
            kfac = kfb[blk], vfac = fmaxf(vfb[blk], 0x1p-64f);
        };
        if (first < end) load(first);
        for (long long blk = first; blk < end; ++blk) {
            const long long s0 = blk * kC8Block + 16 * warp;
            const bool in0 = s0 + r < n, in1 = s0 + r + 8 < n;
            const float lift = __log2f(vfac), less = __frcp_rn(vfac);
            uint32_t pw[NG][2];
#pragma unroll
            for (int a = 0; a < NG; ++a) {
                float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    const uint32_t w0[4] = {kx[0][c].x, kx[0][c].y, kx[0][c].z, kx[0][c].w};
                    const uint32_t w1[4] = {kx[1][c].x, kx[1][c].y, kx[1][c].z, kx[1][c].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mma16x8<false>(s, f16x2_of(w0[i]), f16x2_of(w1[i]), f16x2_of(w0[i] >> 16), f16x2_of(w1[i] >> 16), qf[a][c][2 * i],
                                       qf[a][c][2 * i + 1]);
                }
                // s: (slot r, heads 2j, 2j + 1), (slot r + 8, the same heads)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[i] = (i < 2 ? in0 : in1) ? fmaf(s[i], fac[a][i & 1] * kfac, lift) : -INFINITY;
                float top[2] = {fmaxf(s[0], s[2]), fmaxf(s[1], s[3])};
                if (__any_sync(~0u, top[0] > m[a][0] + 8.f || top[1] > m[a][1] + 8.f)) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int x = 4; x < 32; x <<= 1) top[e] = fmaxf(top[e], __shfl_xor_sync(~0u, top[e], x));
                        const float mn = fmaxf(m[a][e], top[e]), f = mn == -INFINITY ? 1.f : ex2(m[a][e] - mn);
                        m[a][e] = mn;
                        l[a][e] *= f;
#pragma unroll
                        for (int y = 0; y < M; ++y) acc[a][y][e] *= f, acc[a][y][2 + e] *= f;
                    }
                }
                const float mu[2] = {m[a][0] == -INFINITY ? 0.f : m[a][0] - 7.f, m[a][1] == -INFINITY ? 0.f : m[a][1] - 7.f};
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 e = make_float2(ex2(s[2 * i] - mu[0]), ex2(s[2 * i + 1] - mu[1]));
                    l[a][0] = fmaf(e.x, less, l[a][0]);
                    l[a][1] = fmaf(e.y, less, l[a][1]);
                    pw[a][i] = transpose8x8(pack16<false>(e));
                }
            }
#pragma unroll
            for (int y = 0; y < D / 32; ++y) {
                // two columns of d a product: 4 y + 0, 1 and 4 y + 2, 3 of this lane's
                const uint32_t a0 = __byte_perm(vx[0][y], vx[1][y], 0x5140), a1 = __byte_perm(vx[0][y], vx[1][y], 0x7362);
                const uint32_t b0 = __byte_perm(vx[2][y], vx[3][y], 0x5140), b1 = __byte_perm(vx[2][y], vx[3][y], 0x7362);
                const uint32_t f0 = f16x2_of(a0), f1 = f16x2_of(a0 >> 16), f2 = f16x2_of(b0), f3 = f16x2_of(b0 >> 16);
                const uint32_t h0_ = f16x2_of(a1), h1 = f16x2_of(a1 >> 16), h2 = f16x2_of(b1), h3 = f16x2_of(b1 >> 16);
#pragma unroll
                for (int a = 0; a < NG; ++a) {
                    mma16x8<false>(acc[a][2 * y], f0, f1, f2, f3, pw[a][0], pw[a][1]);
                    mma16x8<false>(acc[a][2 * y + 1], h0_, h1, h2, h3, pw[a][0], pw[a][1]);
                }
            }
            if (blk + 1 < end) load(blk + 1);
        }
        // product y, row r: column (D / 8) r + 2 y, row r + 8: the next one
#pragma unroll
        for (int a = 0; a < NG; ++a)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[a][e] += __shfl_xor_sync(~0u, l[a][e], x);
                const int h = 8 * a + 2 * j + e;
                if (r == 0) s_m[warp][h] = m[a][e], s_l[warp][h] = l[a][e];
#pragma unroll
                for (int y = 0; y < M; ++y)
                    *reinterpret_cast<float2 *>(&s_o[warp][h][D / 8 * r + 2 * y]) = make_float2(acc[a][y][e], acc[a][y][2 + e]);
            }
        __syncthreads();
        // the warps' parts into the first's
        for (int i = threadIdx.x; i < NH * D; i += blockDim.x) {
            const int h = i / D, d = i % D;
            float mm = s_m[0][h];
#pragma unroll
            for (int w = 1; w < kStepWarps; ++w) mm = fmaxf(mm, s_m[w][h]);
            const float mu = mm == -INFINITY ? 0.f : mm;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kStepWarps; ++w) s += s_o[w][h][d] * ex2(s_m[w][h] - mu);
            s_o[0][h][d] = s;
        }
        __syncthreads();
        if (threadIdx.x < NH) {
            const int h = threadIdx.x;
            float mm = s_m[0][h], s = 0.f;
#pragma unroll
            for (int w = 1; w < kStepWarps; ++w) mm = fmaxf(mm, s_m[w][h]);
            const float mu = mm == -INFINITY ? 0.f : mm;
#pragma unroll
            for (int w = 0; w < kStepWarps; ++w) s += s_l[w][h] * ex2(s_m[w][h] - mu);
            s_m[0][h] = mm;
            s_l[0][h] = s;
        }
        if (g.splits > 1) cluster_sync();
        else __syncthreads();
        // each block of the cluster finishes its share of the outputs
        const uint32_t ao = smem_u32(&s_o[0][0][0]), am = smem_u32(&s_m[0][0]), al = smem_u32(&s_l[0][0]);
        for (int i = split * blockDim.x + threadIdx.x; i < nh * D / 2; i += g.splits * blockDim.x) {
            const int h = i / (D / 2), d = i % (D / 2) * 2;
            float mm = -INFINITY;
            for (int w = 0; w < g.splits; ++w) mm = fmaxf(mm, ld_cluster(map_rank(am + 4 * h, w)));
            float lt = 0.f, x = 0.f, y = 0.f;
            for (int w = 0; w < g.splits; ++w) {
                const float f = ex2(ld_cluster(map_rank(am + 4 * h, w)) - mm);
                const uint32_t at = map_rank(ao + 4 * (h * D + d), w);
                lt += f * ld_cluster(map_rank(al + 4 * h, w));
                x += f * ld_cluster(at);
                y += f * ld_cluster(at + 4);
            }
            reinterpret_cast<uint32_t *>(ob + (long long)h0 * D)[i] = pack16<BF>(make_float2(x / lt, y / lt));
        }
        if (g.splits > 1) cluster_sync();  // no block leaves, or starts anew, while its part is being read
        else __syncthreads();
    }
}

// ------------------------------------------------------------------ host
int c8_check(const char *fn, int64_t B, int64_t H, int64_t Hkv, int64_t T, int64_t d, int64_t window, int64_t sinks, int dtype,
             float scale) {
    if (B < 0 || H < 0 || Hkv < 0 || T < 0) return fail(CLA_ERR_INVALID_ARG, "%s: negative size", fn);
    if (window < 1 || sinks < 0) return fail(CLA_ERR_INVALID_ARG, "%s: window must be at least 1 and sinks 0", fn);
    if (H == 0 || Hkv == 0 ? H != Hkv : H % Hkv != 0)
        return fail(CLA_ERR_INVALID_ARG, "%s: the query heads must be a multiple of the key heads", fn);
    if (!isfinite(scale)) return fail(CLA_ERR_INVALID_ARG, "%s: scale must be finite", fn);
    if (dtype != CLA_BF16 && dtype != CLA_F16) return fail(CLA_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
    if (d != 64 && d != 128) return fail(CLA_ERR_UNSUPPORTED, "%s: head dimension %lld", fn, (long long)d);
    if (window > kMaxTokens || sinks > kMaxTokens - window || !product_below({B, Hkv, d, sinks + window}, 1e15))
        return fail(CLA_ERR_UNSUPPORTED, "%s: sinks + window must be at most 2^31 - 512, the cache below 10^15 elements", fn);
    if (T > kMaxTokens || !product_below({B, H}, 1 << 27) || !product_below({B, Hkv, (sinks + window + kC8Block - 1) / kC8Block}, 2147483648.0))
        return fail(CLA_ERR_UNSUPPORTED, "%s: sizes too large", fn);
    return CLA_OK;
}

constexpr int kC8Splits = 16;  // blocks of a cluster; above 8 with the kernel's leave

void c8_config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute &at, long long clusters, int splits, cudaStream_t s) {
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
template <typename E, int D, int NG>
int c8_resident(const char *fn, int (&n)[kC8Splits + 1]) {
    static std::atomic<int> known[64][kC8Splits + 1];  // the number and 1
    int dev = 0;
    CLA_CUDA_TRY(cudaGetDevice(&dev), fn);
    const bool keep = dev < 64;
    for (int s = 1; s <= kC8Splits; ++s) {
        n[s] = keep ? known[dev][s].load(std::memory_order_relaxed) - 1 : -1;
        if (n[s] >= 0) continue;
        if (s > 8)
            CLA_CUDA_TRY(cudaFuncSetAttribute((const void *)c8_step_kernel<E, D, NG>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1), fn);
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute at;
        c8_config(cfg, at, 1, s, nullptr);
        CLA_CUDA_TRY(cudaOccupancyMaxActiveClusters(&n[s], c8_step_kernel<E, D, NG>, &cfg), fn);
        if (keep) known[dev][s].store(n[s] + 1, std::memory_order_relaxed);
    }
    return CLA_OK;
}

// Splits the slots of a (sequence, key head) over as many blocks as give the least rounds of clusters times the blocks
// of slots of each; a round's latency and join count as 4.
template <typename E, int D, int NG>
int c8_step(const char *fn, const void *q, const void *k, const void *v, void *kc, void *vc, float *kf, float *vf, void *o, int64_t B,
            Step8Args g, cudaStream_t s) {
    int resident[kC8Splits + 1];
    if (int st = c8_resident<E, D, NG>(fn, resident)) return st;
    const long long units = B * g.Hkv;
    g.splits = 1;
    long long least = -1;
    for (int n = 1; n <= kC8Splits && n <= g.blocks; ++n) {
        if (resident[n] == 0 || units * n >= 2147483648ll) continue;
        const long long cost = (units + resident[n] - 1) / resident[n] * ((g.blocks + n - 1) / n + 4);
        if (least < 0 || cost < least) least = cost, g.splits = n;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at;
    c8_config(cfg, at, units, g.splits, s);
    CLA_CUDA_TRY(cudaLaunchKernelEx(&cfg, c8_step_kernel<E, D, NG>, (const E *)q, (const E *)k, (const E *)v, (uint8_t *)kc, (uint8_t *)vc, kf,
                                    vf, (E *)o, g),
                 fn);
    return check_launch(fn);
}

}  // namespace
}  // namespace cla

using namespace cla;

extern "C" int cla_window_cache8_write(const void *k, const void *v, const int32_t *lens, void *kcache, void *vcache, float *kscale,
                                       float *vscale, int64_t window, int64_t sinks, int dtype, int64_t B, int64_t Hkv, int64_t T,
                                       int64_t d, const int64_t *strides, void *stream) {
    const char *fn = "cla_window_cache8_write";
    clear_error();
    if (int st = c8_check(fn, B, Hkv, Hkv, T, d, window, sinks, dtype, 1.f)) return st;
    if (B * Hkv * T == 0) return CLA_OK;
    if (!k || !v || !kcache || !vcache || !kscale || !vscale) return fail(CLA_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (!aligned_or_null({k, v, kcache, vcache}, 16) || !aligned_or_null({lens, kscale, vscale}, 4))
        return fail(CLA_ERR_INVALID_ARG, "%s: a pointer is misaligned", fn);
    static const char *const names[] = {"k", "v"};
    const int64_t heads[] = {Hkv, Hkv}, ds[] = {d, d};
    Triple r[2];
    if (int st = view_strides(fn, strides, names, heads, ds, 2, B, T, 8, r)) return st;
    const int blocks = (int)((sinks + window + kC8Block - 1) / kC8Block);
    const dim3 grid((unsigned)(B * Hkv * blocks), 2);
    cudaStream_t s = (cudaStream_t)stream;
#define CLA_C8_WRITE(E, D)                                                                                                       \
    c8_write_kernel<E, D><<<grid, 128, 0, s>>>((const E *)k, (const E *)v, lens, (uint8_t *)kcache, (uint8_t *)vcache, kscale, vscale, \
                                               r[0], r[1], (int)Hkv, (int)T, window, sinks, blocks)
    if (dtype == CLA_BF16) {
        if (d == 128) CLA_C8_WRITE(__nv_bfloat16, 128);
        else CLA_C8_WRITE(__nv_bfloat16, 64);
    } else {
        if (d == 128) CLA_C8_WRITE(__half, 128);
        else CLA_C8_WRITE(__half, 64);
    }
#undef CLA_C8_WRITE
    return check_launch(fn);
}

extern "C" int cla_window_attn_step8(const void *q, const void *k, const void *v, void *kcache, void *vcache, float *kscale,
                                     float *vscale, const int32_t *pos, void *o, float scale, int64_t window, int64_t sinks, int dtype,
                                     int64_t B, int64_t H, int64_t Hkv, int64_t d, const int64_t *strides, void *stream) {
    const char *fn = "cla_window_attn_step8";
    clear_error();
    if (int st = c8_check(fn, B, H, Hkv, 1, d, window, sinks, dtype, scale)) return st;
    if (B * H == 0) return CLA_OK;
    if (!q || !k || !v || !kcache || !vcache || !kscale || !vscale || !pos || !o)
        return fail(CLA_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (!aligned_or_null({q, k, v, kcache, vcache, o}, 16) || !aligned_or_null({pos, kscale, vscale}, 4))
        return fail(CLA_ERR_INVALID_ARG, "%s: a pointer is misaligned", fn);
    static const char *const names[] = {"q", "k", "v"};
    const int64_t heads[] = {H, Hkv, Hkv}, ds[] = {d, d, d};
    Triple r[3];
    int64_t full[9];
    if (strides != nullptr)
        for (int i = 0; i < 3; ++i) full[3 * i] = strides[2 * i], full[3 * i + 1] = strides[2 * i + 1], full[3 * i + 2] = d;
    if (int st = view_strides(fn, strides ? full : nullptr, names, heads, ds, 3, B, 1, 8, r)) return st;
    const Step8Args g{pos,    scale * 1.4426950408889634f, window, sinks, sinks + window, (int)H, (int)Hkv, 1,
                      (int)((sinks + window + kC8Block - 1) / kC8Block), r[0], r[1], r[2]};
    cudaStream_t s = (cudaStream_t)stream;
    const bool bf = dtype == CLA_BF16, wide = H / Hkv > 8;
#define CLA_STEP8(E, D)                                                                             \
    (wide ? c8_step<E, D, 2>(fn, q, k, v, kcache, vcache, kscale, vscale, o, B, g, s) \
          : c8_step<E, D, 1>(fn, q, k, v, kcache, vcache, kscale, vscale, o, B, g, s))
    if (d == 128) return bf ? CLA_STEP8(__nv_bfloat16, 128) : CLA_STEP8(__half, 128);
    return bf ? CLA_STEP8(__nv_bfloat16, 64) : CLA_STEP8(__half, 64);
#undef CLA_STEP8
}
