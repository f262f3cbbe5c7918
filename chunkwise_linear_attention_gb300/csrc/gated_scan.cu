// gated_scan.cu -- the gated linear recurrence whose decays and inputs are
// formed from gates inside the kernel: forward, backward and the one-token
// step.
//
//   r = sigmoid(rgate), i = sigmoid(igate), L = -c softplus(lam) r, a = e^L,
//   m = sqrt(1 - a^2),  h_t = a_t h_{t-1} + m_t i_t x_t
//
// The factor m keeps the state's variance where the inputs' is.  With
// c_t = a_t hbar_t the adjoint is hbar_t = dh_t + c_{t+1}, and with u = i x
//   dx = hbar m i,   digate = hbar m u (1 - i),
//   G  = dL L = hbar L a (h_{t-1} - a u / m),
//   drgate = G (1 - r),   dlam = sum G sigmoid(lam) / softplus(lam),
// where L / m -> 0 as L -> 0: writing the gradients with dL L instead of dL
// leaves no division by a vanishing m.
//
// Decomposition (one warp = one chunk of 8 L steps x 16 channels): lane =
// (sub, cg), cg in 0..3 picks 4 adjacent channels and sub in 0..7 a run of L
// steps.  Every input is read once; a lane keeps its run's decays and inputs
// in registers, composes them, composes across the 8 runs by shuffles, and
// publishes the chunk's pair.  The state entering a chunk is folded from the
// published pairs of its group's earlier chunks (32 chunks a group, eight
// lanes at a time) and the state at the end of the group before.  That order
// is fixed by the chunk's place alone, so the result does not depend on which
// block came first, and only one wait per 32 chunks is on the serial path.
#include <math.h>

#include "cla_internal.cuh"
#include "elem_io.cuh"

namespace cla {
namespace {

constexpr int kGsCkpt = CLA_GATED_SCAN_CKPT_CHUNK;
constexpr int kGsGroup = 32;  // chunks of a group
constexpr int kGsWarps = 4;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float softplus(float v) { return v > 20.f ? v : log1pf(expf(v)); }
__device__ __forceinline__ float ex2a(float v) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
}
__device__ __forceinline__ float rcpa(float v) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
}
__device__ __forceinline__ float rsqa(float v) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
}
__device__ __forceinline__ float2 f2(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

struct Gate2 {
    float2 a, y, m, rm, r1, i, i1;  // a, log2 a, m, 1 / m, 1 - r, i, 1 - i
};

// The gates of two channels at once (the paired fp32 instructions round each lane as the scalar
// ones do).  Both sigmoids share one reciprocal, of (1 + e^-|rgate|)(1 + e^-igate): a closed
// rgate keeps its relative accuracy down to the smallest float, since m grows with the root of
// it, and igate does not close below 2^-120.  a = 2^y and 1 - a come from one
// split y = k + f, 2^f = 1 + t: a = 2^k + 2^k t and 1 - a = (1 - 2^k) - 2^k t, which for decays
// near 1 (k = 0) is -t itself, with no digits lost, where 1 - a^2 from a rounded a would keep
// only those above 2^-24 / (1 - a).  The polynomial is a least-maximum-error fit of 2^f on
// [-1/2, 1/2] with p(0) = 1 (Lawson's reweighted least squares, degree 6, 2e-9).  NaN passes
// through: the clamps are comparisons that a NaN fails.
__device__ __forceinline__ Gate2 gate2(float2 rg, float2 ig, float2 nl2) {
    constexpr float kP1 = 6.931471825e-01f, kP2 = 2.402264774e-01f, kP3 = 5.550332367e-02f, kP4 = 9.618437849e-03f,
                    kP5 = 1.339887269e-03f, kP6 = 1.535334159e-04f, kMagic = 12582912.0f;
    Gate2 q;
    float2 pi = mul2(ig, f2(-kLog2e));
    pi.x = pi.x > 120.f ? 120.f : pi.x;
    pi.y = pi.y > 120.f ? 120.f : pi.y;
    const float2 er = make_float2(ex2a(-fabsf(rg.x) * kLog2e), ex2a(-fabsf(rg.y) * kLog2e));
    const float2 ei = make_float2(ex2a(pi.x), ex2a(pi.y));
    const float2 br = add2(er, f2(1.f)), bi = add2(ei, f2(1.f));
    const float2 pp = mul2(br, bi);
    const float2 R = make_float2(rcpa(pp.x), rcpa(pp.y));
    const float2 big = mul2(R, bi), small = mul2(er, big);  // sigmoid(|rgate|) and 1 - it
    const float2 r = make_float2(rg.x >= 0.f ? big.x : small.x, rg.y >= 0.f ? big.y : small.y);
    q.r1 = make_float2(rg.x >= 0.f ? small.x : big.x, rg.y >= 0.f ? small.y : big.y);
    q.i = mul2(R, br);
    q.i1 = mul2(ei, q.i);
    float2 y = mul2(nl2, r);
    y.x = y.x < -126.f ? -126.f : y.x;
    y.y = y.y < -126.f ? -126.f : y.y;
    q.y = y;
    const float2 km = add2(y, f2(kMagic));
    const float2 k = add2(km, f2(-kMagic));
    const float2 f = fma2(k, f2(-1.f), y);
    float2 t = fma2(f2(kP6), f, f2(kP5));
    t = fma2(t, f, f2(kP4));
    t = fma2(t, f, f2(kP3));
    t = fma2(t, f, f2(kP2));
    t = fma2(t, f, f2(kP1));
    t = mul2(t, f);
    const float2 sc = make_float2(__int_as_float((__float_as_int(km.x) << 23) + 0x3f800000),
                                  __int_as_float((__float_as_int(km.y) << 23) + 0x3f800000));
    q.a = fma2(sc, t, sc);
    const float2 ns = mul2(sc, f2(-1.f));
    float2 om = fma2(ns, t, add2(ns, f2(1.f)));  // 1 - a
    om = mul2(om, add2(q.a, f2(1.f)));           // 1 - a^2
    om = make_float2(fmaxf(om.x, 1e-37f), fmaxf(om.y, 1e-37f));
    q.rm = make_float2(rsqa(om.x), rsqa(om.y));
    q.m = mul2(om, q.rm);
    return q;
}

struct GsArgs {
    const uint8_t *reset;
    const int32_t *lens;
    long long T, chunks;
    int B, D, n_cw;  // n_cw: groups of 16 channels
    float c;
};

__device__ __forceinline__ long long seq_len(const GsArgs &g, int b) {
    if (g.lens == nullptr) return g.T;
    const long long n = g.lens[b];
    return n < 0 ? 0 : (n > g.T ? g.T : n);
}

// Four adjacent elements as they lie in memory; VEC: with one access, else one by one (rows that
// are not aligned), those below `n` only.
template <typename E>
struct Raw4 {
    uint2 w;
};
template <>
struct Raw4<float> {
    float4 w;
};
template <typename E, bool VEC>
__device__ __forceinline__ Raw4<E> ld4(const E *p, int n) {
    Raw4<E> r;
    if constexpr (VEC) {
        r.w = __ldcs(reinterpret_cast<const decltype(r.w) *>(p));
    } else if constexpr (sizeof(E) == 4) {
        r.w = make_float4(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f, n > 3 ? p[3] : 0.f);
    } else {
        const unsigned short *s = reinterpret_cast<const unsigned short *>(p);
        const unsigned int a = n > 0 ? s[0] : 0, b = n > 1 ? s[1] : 0, c = n > 2 ? s[2] : 0, d = n > 3 ? s[3] : 0;
        r.w = make_uint2(a | b << 16, c | d << 16);
    }
    return r;
}
__device__ __forceinline__ float2 unpack2(unsigned int u, __nv_bfloat16) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack2(unsigned int u, __half) {
    return __half22float2(*reinterpret_cast<__half2 *>(&u));
}
template <typename E>
__device__ __forceinline__ void cvt4(const Raw4<E> &r, float2 (&v)[2]) {
    if constexpr (sizeof(E) == 4) {
        v[0] = make_float2(r.w.x, r.w.y);
        v[1] = make_float2(r.w.z, r.w.w);
    } else {
        v[0] = unpack2(r.w.x, E());
        v[1] = unpack2(r.w.y, E());
    }
}
__device__ __forceinline__ unsigned int pack2(float2 v, __nv_bfloat16) {
    __nv_bfloat162 h = __float22bfloat162_rn(v);
    return *reinterpret_cast<unsigned int *>(&h);
}
__device__ __forceinline__ unsigned int pack2(float2 v, __half) {
    __half2 h = __float22half2_rn(v);
    return *reinterpret_cast<unsigned int *>(&h);
}
template <typename E, bool VEC>
__device__ __forceinline__ void st4(E *p, const float2 (&v)[2], int n) {
    if constexpr (VEC) {
        if constexpr (sizeof(E) == 4)
            __stcs(reinterpret_cast<float4 *>(p), make_float4(v[0].x, v[0].y, v[1].x, v[1].y));
        else
            __stcs(reinterpret_cast<uint2 *>(p), make_uint2(pack2(v[0], E()), pack2(v[1], E())));
    } else {
        if (n > 0) p[0] = from_f32<E>(v[0].x);
        if (n > 1) p[1] = from_f32<E>(v[0].y);
        if (n > 2) p[2] = from_f32<E>(v[1].x);
        if (n > 3) p[3] = from_f32<E>(v[1].y);
    }
}
__device__ __forceinline__ void ldf4(const float *p, float2 (&v)[2], int n) {
    v[0] = make_float2(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f);
    v[1] = make_float2(n > 2 ? p[2] : 0.f, n > 3 ? p[3] : 0.f);
}
__device__ __forceinline__ void stf4(float *p, const float2 (&v)[2], int n) {
    if (n > 0) p[0] = v[0].x;
    if (n > 1) p[1] = v[0].y;
    if (n > 2) p[2] = v[1].x;
    if (n > 3) p[3] = v[1].y;
}

// (A, B) after (pa, pb): B <- A pb + B, A <- A pa.  RST: a decay of exactly 0 (a reset; no other
// decay is below 2^-126) drops what came before, NaN and infinity included.
template <bool RST>
__device__ __forceinline__ void after(float2 &A, float2 &B, float2 pa, float2 pb) {
    if constexpr (RST) {
        if (A.x == 0.f) pa.x = pb.x = 0.f;
        if (A.y == 0.f) pa.y = pb.y = 0.f;
    }
    B = fma2(A, pb, B);
    A = mul2(A, pa);
}
template <bool RST>
__device__ __forceinline__ float2 apply(float2 A, float2 s, float2 B) {
    if constexpr (RST) {
        if (A.x == 0.f) s.x = 0.f;
        if (A.y == 0.f) s.y = 0.f;
    }
    return fma2(A, s, B);
}
__device__ __forceinline__ float2 shfl_up2(float2 v, int d) {
    return make_float2(__shfl_up_sync(~0u, v.x, d), __shfl_up_sync(~0u, v.y, d));
}
__device__ __forceinline__ float2 shfl_down2(float2 v, int d) {
    return make_float2(__shfl_down_sync(~0u, v.x, d), __shfl_down_sync(~0u, v.y, d));
}
__device__ __forceinline__ float2 shfl2(float2 v, int l) {
    return make_float2(__shfl_sync(~0u, v.x, l), __shfl_sync(~0u, v.y, l));
}

// Inclusive pairs across the 8 runs, earlier runs at lower (REV: higher) lanes.
template <bool RST, bool REV>
__device__ __forceinline__ void scan_runs(float2 (&A)[2], float2 (&B)[2], int sub) {
#pragma unroll
    for (int off = 1; off < 8; off <<= 1)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const float2 pa = REV ? shfl_down2(A[v], 4 * off) : shfl_up2(A[v], 4 * off);
            const float2 pb = REV ? shfl_down2(B[v], 4 * off) : shfl_up2(B[v], 4 * off);
            if (REV ? sub + off < 8 : sub >= off) after<RST>(A[v], B[v], pa, pb);
        }
}

// Published values: 32-bit words, 0 until written (the launch clears them); +0.0 goes out as
// -0.0.  Each element of a 16-byte relaxed access is single-copy atomic: a reader that sees a
// nonzero word sees the value, without fences.
__device__ __forceinline__ unsigned int pub(float v) {
    const unsigned int b = __float_as_uint(v);
    return b != 0u ? b : 0x80000000u;
}
__device__ __forceinline__ void publish4(unsigned int *p, const float2 (&v)[2]) {
    asm volatile("st.relaxed.gpu.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(pub(v[0].x)), "r"(pub(v[0].y)),
                 "r"(pub(v[1].x)), "r"(pub(v[1].y))
                 : "memory");
}
__device__ __forceinline__ bool peek4(const unsigned int *p, float2 (&v)[2]) {
    unsigned int a, b, c, d;
    asm volatile("ld.relaxed.gpu.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "l"(p) : "memory");
    v[0] = make_float2(__uint_as_float(a), __uint_as_float(b));
    v[1] = make_float2(__uint_as_float(c), __uint_as_float(d));
    return a != 0u && b != 0u && c != 0u && d != 0u;
}
// Polls until the four words are there, a bounded number of times; then records the timeout and
// carries on with what it saw.
__device__ __forceinline__ void wait4(const unsigned int *p, float2 (&v)[2], WsHeader *hdr, unsigned int where) {
    for (unsigned int it = 0; it < kSpinLimit; ++it) {
        if (peek4(p, v)) return;
        if (it >= 8) __nanosleep(64);
    }
    atomicOr(&hdr->error, kErrTimeout);
    atomicExch(&hdr->where, where);
}

struct GsWords {
    WsHeader *hdr;
    unsigned int *pairs;   // [chunk][b][cw][cg][A, B][4], chunks in the scan's order
    unsigned int *states;  // [group][b][cw][cg][4]
};

// The state entering chunk `idx` (of `per` units a chunk; this warp's is `rem`): the pairs of
// the group's chunks before it, eight lanes folding contiguous shares and then each other's, on
// the state at the end of the group before, or `s0`.  Publishes this chunk's pair (held by the
// lanes with `pubs`) and, at the end of a group, the state behind it.
template <bool RST>
__device__ __forceinline__ void carry_in(const GsWords &w, long long idx, long long chunks, long long per, long long rem,
                                         int sub, int cg, bool pubs, const float2 (&A)[2], const float2 (&B)[2],
                                         const float2 (&s0)[2], float2 (&s)[2], unsigned int where) {
    const int n = (int)(idx % kGsGroup);
    const long long first = idx - n;
    const bool last_of_group = n == kGsGroup - 1;
    if (pubs && !last_of_group && idx + 1 < chunks) {
        unsigned int *p = w.pairs + ((idx * per + rem) * 4 + cg) * 8;
        publish4(p, A);
        publish4(p + 4, B);
    }
    float2 PA[2] = {f2(1.f), f2(1.f)}, PB[2] = {f2(0.f), f2(0.f)};
    if (n > 0) {
        const int share = (n + 7) / 8, k0 = sub * share, k1 = k0 + share < n ? k0 + share : n;
        for (int k = k0; k < k1; ++k) {
            const unsigned int *p = w.pairs + (((first + k) * per + rem) * 4 + cg) * 8;
            float2 a[2], b[2];
            wait4(p, a, w.hdr, where);
            wait4(p + 4, b, w.hdr, where);
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                after<RST>(a[v], b[v], PA[v], PB[v]);
                PA[v] = a[v];
                PB[v] = b[v];
            }
        }
        __syncwarp();
        scan_runs<RST, false>(PA, PB, sub);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            PA[v] = shfl2(PA[v], 28 + cg);
            PB[v] = shfl2(PB[v], 28 + cg);
        }
    }
    float2 S[2] = {s0[0], s0[1]};
    if (first > 0) {
        wait4(w.states + (((first / kGsGroup - 1) * per + rem) * 4 + cg) * 4, S, w.hdr, where + 1);
        __syncwarp();
    }
#pragma unroll
    for (int v = 0; v < 2; ++v) s[v] = apply<RST>(PA[v], S[v], PB[v]);
    if (pubs && last_of_group && idx + 1 < chunks) {
        const float2 e[2] = {apply<RST>(A[0], s[0], B[0]), apply<RST>(A[1], s[1], B[1])};
        publish4(w.states + ((idx / kGsGroup * per + rem) * 4 + cg) * 4, e);
    }
}

// Blocks take their units in the order in which they start, so that every unit a warp waits for
// belongs to a warp that runs already.
__device__ __forceinline__ long long take_unit(WsHeader *hdr, int which) {
    __shared__ unsigned int ticket;
    if (threadIdx.x == 0) ticket = atomicAdd(&hdr->ticket[which], 1u);
    __syncthreads();
    return (long long)ticket * kGsWarps + (threadIdx.x >> 5);
}

// ------------------------------------------------------------------ forward
// L = 8 steps a lane for 2-byte elements, 4 for fp32 (the raw inputs of a run are held in
// registers until they are used).  h may be NULL: only the checkpoint is written then.
template <typename E, bool VEC, bool RST, int L>
__global__ void __launch_bounds__(kGsWarps * 32, 4)
gated_fwd_kernel(const E *__restrict__ x, const E *__restrict__ rg, const E *__restrict__ ig, const float *__restrict__ lam,
                 const float *__restrict__ h0, E *__restrict__ h, float *__restrict__ hT, float *__restrict__ ckpt, GsArgs g,
                 GsWords w) {
    const long long per = (long long)g.B * g.n_cw, unit = take_unit(w.hdr, 0);
    const long long chunk = unit / per, rem = unit - chunk * per;
    if (chunk >= g.chunks) return;
    const int b = (int)(rem / g.n_cw), lane = threadIdx.x & 31, sub = lane >> 2, cg = lane & 3;
    const int c0 = (int)(rem % g.n_cw) * 16 + cg * 4, nv = g.D - c0;
    const long long n = nv > 0 ? seq_len(g, b) : 0, t0 = chunk * (8 * L) + sub * L;
    const size_t at0 = ((size_t)b * g.T + t0) * g.D + c0;

    Raw4<E> rx[L], rr[L], ri[L];
    bool rs[L];
#pragma unroll
    for (int j = 0; j < L; ++j) {
        if (t0 + j < n) {
            const size_t at = at0 + (size_t)j * g.D;
            rr[j] = ld4<E, VEC>(rg + at, nv);
            ri[j] = ld4<E, VEC>(ig + at, nv);
            rx[j] = ld4<E, VEC>(x + at, nv);
            if constexpr (RST) rs[j] = g.reset[(size_t)b * g.T + t0 + j] != 0;
        }
    }
    float2 nl2[2], s0[2] = {f2(0.f), f2(0.f)};
    ldf4(lam + (nv > 0 ? c0 : 0), nl2, nv);
#pragma unroll
    for (int v = 0; v < 2; ++v)
        nl2[v] = make_float2(-g.c * softplus(nl2[v].x) * kLog2e, -g.c * softplus(nl2[v].y) * kLog2e);
    if (h0 != nullptr && nv > 0) ldf4(h0 + (size_t)b * g.D + c0, s0, nv);

    float2 a[L][2], u[L][2], A[2] = {f2(1.f), f2(1.f)}, B[2] = {f2(0.f), f2(0.f)};
#pragma unroll
    for (int j = 0; j < L; ++j) {
        const bool on = t0 + j < n;
        float2 xv[2], rv[2], iv[2];
        cvt4<E>(rx[j], xv);
        cvt4<E>(rr[j], rv);
        cvt4<E>(ri[j], iv);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            if (on) {
                const Gate2 q = gate2(rv[v], iv[v], nl2[v]);
                a[j][v] = q.a;
                u[j][v] = mul2(mul2(q.m, q.i), xv[v]);
                if constexpr (RST)
                    if (rs[j]) {
                        a[j][v] = f2(0.f);
                        u[j][v] = mul2(q.i, xv[v]);
                    }
            } else {
                a[j][v] = f2(1.f);
                u[j][v] = f2(0.f);
            }
            const float2 pa = A[v], pb = B[v];
            A[v] = a[j][v];
            B[v] = u[j][v];
            after<RST>(A[v], B[v], pa, pb);
        }
    }
    scan_runs<RST, false>(A, B, sub);
    float2 Ax[2], Bx[2], s[2];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        Ax[v] = shfl_up2(A[v], 4);
        Bx[v] = shfl_up2(B[v], 4);
        if (sub == 0) Ax[v] = f2(1.f), Bx[v] = f2(0.f);
    }
    carry_in<RST>(w, chunk, g.chunks, per, rem, sub, cg, sub == 7, A, B, s0, s, 11u);
    if (nv <= 0) return;
#pragma unroll
    for (int v = 0; v < 2; ++v) s[v] = apply<RST>(Ax[v], s[v], Bx[v]);
    if (ckpt != nullptr && (sub * L) % kGsCkpt == 0 && t0 < g.T)
        stf4(ckpt + ((size_t)b * ((g.T + kGsCkpt - 1) / kGsCkpt) + t0 / kGsCkpt) * g.D + c0, s, nv);
#pragma unroll
    for (int j = 0; j < L; ++j) {
#pragma unroll
        for (int v = 0; v < 2; ++v) s[v] = apply<RST>(a[j][v], s[v], u[j][v]);
        if (t0 + j < g.T) {
            if (h != nullptr) {
                const bool on = t0 + j < n;
                const float2 z[2] = {on ? s[0] : f2(0.f), on ? s[1] : f2(0.f)};
                st4<E, VEC>(h + at0 + (size_t)j * g.D, z, nv);
            }
            if (hT != nullptr && t0 + j == g.T - 1) stf4(hT + (size_t)b * g.D + c0, s, nv);
        }
    }
}

// ------------------------------------------------------------------ backward
// Chunks of 32 steps, the last first, 4 steps a lane: the states before each step are rebuilt
// from the checkpoint at the chunk's start, the adjoint's carry c_t = a_t (dh_t + c_{t+1}) is
// scanned as the forward's state is, and every gradient is written once.  Each chunk leaves its
// sums of G for dlam in a row of `part`.
template <typename E, bool VEC, bool RST>
__global__ void __launch_bounds__(kGsWarps * 32, 3)
gated_bwd_kernel(const E *__restrict__ x, const E *__restrict__ rg, const E *__restrict__ ig, const float *__restrict__ lam,
                 const float *__restrict__ ckpt, const E *__restrict__ dh, const float *__restrict__ dhT,
                 E *__restrict__ dx, E *__restrict__ drg, E *__restrict__ dig, float *__restrict__ part,
                 float *__restrict__ dh0, GsArgs g, GsWords w) {
    constexpr int L = 4;
    static_assert(8 * L == kGsCkpt, "a chunk of the backward starts at a checkpoint");
    const long long per = (long long)g.B * g.n_cw, unit = take_unit(w.hdr, 1);
    const long long idx = unit / per, rem = unit - idx * per, chunk = g.chunks - 1 - idx;
    if (chunk < 0) return;
    const int b = (int)(rem / g.n_cw), lane = threadIdx.x & 31, sub = lane >> 2, cg = lane & 3;
    const int c0 = (int)(rem % g.n_cw) * 16 + cg * 4, nv = g.D - c0;
    const long long n = nv > 0 ? seq_len(g, b) : 0, t0 = chunk * (8 * L) + sub * L;
    const size_t at0 = ((size_t)b * g.T + t0) * g.D + c0;

    Raw4<E> rx[L], rr[L], ri[L], rd[L];
    bool rs[L];
#pragma unroll
    for (int j = 0; j < L; ++j) {
        if (t0 + j < n) {
            const size_t at = at0 + (size_t)j * g.D;
            rr[j] = ld4<E, VEC>(rg + at, nv);
            ri[j] = ld4<E, VEC>(ig + at, nv);
            rx[j] = ld4<E, VEC>(x + at, nv);
            rd[j] = ld4<E, VEC>(dh + at, nv);
            if constexpr (RST) rs[j] = g.reset[(size_t)b * g.T + t0 + j] != 0;
        }
    }
    float2 nl2[2], s0[2] = {f2(0.f), f2(0.f)}, hs[2] = {f2(0.f), f2(0.f)};
    ldf4(lam + (nv > 0 ? c0 : 0), nl2, nv);
#pragma unroll
    for (int v = 0; v < 2; ++v)
        nl2[v] = make_float2(-g.c * softplus(nl2[v].x) * kLog2e, -g.c * softplus(nl2[v].y) * kLog2e);
    if (nv > 0) {
        if (dhT != nullptr) ldf4(dhT + (size_t)b * g.D + c0, s0, nv);
        ldf4(ckpt + ((size_t)b * g.chunks + chunk) * g.D + c0, hs, nv);
    }

    // per step: a, L a, 1 - r, a u / m, m i, x (1 - i), dh, and b = m i x, then h_{t-1}
    float2 a[L][2], La[L][2], r1[L][2], w2[L][2], mi[L][2], xi[L][2], gd[L][2], hp[L][2];
    float2 A[2] = {f2(1.f), f2(1.f)}, B[2] = {f2(0.f), f2(0.f)};
#pragma unroll
    for (int j = 0; j < L; ++j) {
        const bool on = t0 + j < n;
        float2 xv[2], rv[2], iv[2];
        cvt4<E>(rx[j], xv);
        cvt4<E>(rr[j], rv);
        cvt4<E>(ri[j], iv);
        cvt4<E>(rd[j], gd[j]);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            if (on) {
                const Gate2 q = gate2(rv[v], iv[v], nl2[v]);
                a[j][v] = q.a;
                La[j][v] = mul2(mul2(q.y, f2(kLn2)), q.a);
                r1[j][v] = q.r1;
                w2[j][v] = mul2(mul2(q.a, q.rm), mul2(q.i, xv[v]));
                mi[j][v] = mul2(q.m, q.i);
                if constexpr (RST)
                    if (rs[j]) a[j][v] = La[j][v] = w2[j][v] = f2(0.f), mi[j][v] = q.i;
                xi[j][v] = mul2(xv[v], q.i1);
                hp[j][v] = mul2(mi[j][v], xv[v]);
            } else {
                a[j][v] = f2(1.f);
                La[j][v] = r1[j][v] = w2[j][v] = mi[j][v] = xi[j][v] = hp[j][v] = gd[j][v] = f2(0.f);
            }
            const float2 pa = A[v], pb = B[v];
            A[v] = a[j][v];
            B[v] = hp[j][v];
            after<RST>(A[v], B[v], pa, pb);
        }
    }
    scan_runs<RST, false>(A, B, sub);
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        const float2 pa = shfl_up2(A[v], 4), pb = shfl_up2(B[v], 4);
        if (sub > 0) hs[v] = apply<RST>(pa, hs[v], pb);
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const float2 next = apply<RST>(a[j][v], hs[v], hp[j][v]);
            hp[j][v] = hs[v];
            hs[v] = next;
        }
        A[v] = f2(1.f);
        B[v] = f2(0.f);
#pragma unroll
        for (int j = L - 1; j >= 0; --j) {
            const float2 pa = A[v], pb = B[v];
            A[v] = a[j][v];
            B[v] = apply<RST>(a[j][v], gd[j][v], f2(0.f));
            after<RST>(A[v], B[v], pa, pb);
        }
    }
    scan_runs<RST, true>(A, B, sub);
    float2 Ax[2], Bx[2], s[2];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        Ax[v] = shfl_down2(A[v], 4);
        Bx[v] = shfl_down2(B[v], 4);
        if (sub == 7) Ax[v] = f2(1.f), Bx[v] = f2(0.f);
    }
    carry_in<RST>(w, idx, g.chunks, per, rem, sub, cg, sub == 0, A, B, s0, s, 13u);
    float2 sum[2] = {f2(0.f), f2(0.f)};
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        s[v] = apply<RST>(Ax[v], s[v], Bx[v]);
#pragma unroll
        for (int j = L - 1; j >= 0; --j) {
            const float2 hb = add2(gd[j][v], s[v]);
            s[v] = apply<RST>(a[j][v], hb, f2(0.f));
            float2 before = hp[j][v];
            if constexpr (RST) {
                if (a[j][v].x == 0.f) before = f2(0.f);
            }
            const float2 G = mul2(mul2(hb, La[j][v]), fma2(w2[j][v], f2(-1.f), before));
            sum[v] = add2(sum[v], G);
            const float2 ox = mul2(hb, mi[j][v]);
            mi[j][v] = ox;
            xi[j][v] = mul2(ox, xi[j][v]);
            r1[j][v] = mul2(G, r1[j][v]);
        }
    }
    if (nv > 0) {
#pragma unroll
        for (int j = 0; j < L; ++j)
            if (t0 + j < g.T) {
                const size_t at = at0 + (size_t)j * g.D;
                st4<E, VEC>(dx + at, mi[j], nv);
                st4<E, VEC>(dig + at, xi[j], nv);
                st4<E, VEC>(drg + at, r1[j], nv);
            }
        if (dh0 != nullptr && chunk == 0 && sub == 0) stf4(dh0 + (size_t)b * g.D + c0, s, nv);
    }
#pragma unroll
    for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int off = 16; off >= 4; off >>= 1)
            sum[v] = add2(sum[v], make_float2(__shfl_xor_sync(~0u, sum[v].x, off), __shfl_xor_sync(~0u, sum[v].y, off)));
    if (nv > 0 && sub == 0) stf4(part + ((size_t)chunk * g.B + b) * g.D + c0, sum, nv);
}

// Sums of rows: block (x, y) adds its share of the rows of 32 channels, in a fixed order, into
// row y of `out`.  With one share the result is dlam: sigmoid(lam) / softplus(lam) times the sum
// (the ratio tends to 1 as lam -> -inf, where both tend to e^lam).
__global__ void __launch_bounds__(1024) gated_dlam_kernel(const float *__restrict__ part, const float *__restrict__ lam,
                                                          float *__restrict__ out, long long rows, int D) {
    __shared__ float s[32][33];
    const int c = threadIdx.x & 31, r = threadIdx.x >> 5, d = blockIdx.x * 32 + c;
    const long long share = (rows + gridDim.y - 1) / gridDim.y, r0 = share * blockIdx.y, r1 = min(rows, r0 + share);
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (d < D)
        for (long long i = r0 + r; i < r1; i += 128)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + 32 * k < r1) v[k] += part[(i + 32 * k) * D + d];
    s[r][c] = (v[0] + v[1]) + (v[2] + v[3]);
    __syncthreads();
    if (r != 0 || d >= D) return;
    float t[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) t[i] = s[i][c];
#pragma unroll
    for (int k = 16; k > 0; k >>= 1)
#pragma unroll
        for (int i = 0; i < k; ++i) t[i] += t[i + k];
    float z = t[0];
    if (gridDim.y == 1) {
        const float l = lam[d];
        if (l >= -20.f) z *= 1.f / (1.f + expf(-l)) / softplus(l);
    }
    out[(size_t)blockIdx.y * D + d] = z;
}

// ------------------------------------------------------------------ one token
template <typename E>
__global__ void gated_step_kernel(const E *x, const E *rg, const E *ig, const float *lam, const uint8_t *reset,
                                  float *h, E *y, int B, int D, float c) {
    const long long u = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (u >= (long long)B * D) return;
    const int b = (int)(u / D), d = (int)(u % D);
    const Gate2 q = gate2(f2(to_f32(rg[u])), f2(to_f32(ig[u])), f2(-c * softplus(lam[d]) * kLog2e));
    const float w = q.i.x * to_f32(x[u]);
    const float s = (reset != nullptr && reset[b]) ? w : fmaf(q.a.x, h[u], q.m.x * w);
    h[u] = s;
    y[u] = from_f32<E>(s);
}

// ------------------------------------------------------------------ host side
int gs_check(const char *fn, int64_t B, int64_t T, int64_t D, int dtype, float c) {
    if (B < 0 || T < 0 || D < 0) return fail(CLA_ERR_INVALID_ARG, "%s: negative size", fn);
    if (!(c > 0.f) || !isfinite(c)) return fail(CLA_ERR_INVALID_ARG, "%s: c must be positive and finite", fn);
    if (dtype_bytes(dtype) == 0) return fail(CLA_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
    if (!product_below({B, D}, 2147483648.0) || !product_below({B, T, D}, 1e12) || T > kMaxTokens)
        return fail(CLA_ERR_UNSUPPORTED, "%s: B * D must be below 2^31, B * T * D below 10^12, T at most 2^31 - 512", fn);
    return CLA_OK;
}

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// The workspace: header, the words of the published pairs and states (sized for the backward's
// chunks of 32 steps, twice the forward's at most), the rebuilt checkpoint, the rows of dlam's
// sums and the rows that these are reduced to.
struct GsLayout {
    size_t words, clear, states, ckpt, part, part2, total;
};
constexpr long long kDlamRows = 1024;  // above these many rows, dlam's sums go in two steps
constexpr int kDlamShares = 64;

GsLayout gs_layout(int64_t B, int64_t T, int64_t D) {
    GsLayout l;
    const size_t units = (size_t)B * ceil_div(D, 16), ch = (size_t)ceil_div(T, kGsCkpt);
    l.words = sizeof(WsHeader);
    l.states = l.words + ch * units * 4 * 8 * 4;
    l.clear = l.states + (size_t)ceil_div(ch, kGsGroup) * units * 4 * 4 * 4;
    l.ckpt = l.clear;
    l.part = l.ckpt + align_up(ch * (size_t)B * D * 4, 16);
    l.part2 = l.part + align_up(ch * (size_t)B * D * 4, 16);
    l.total = l.part2 + (ch * B > (size_t)kDlamRows ? align_up((size_t)kDlamShares * D * 4, 16) : 0);
    return l;
}

bool gs_sizes_ok(int64_t B, int64_t T, int64_t D) {
    return B >= 0 && T >= 0 && D >= 0 && T <= kMaxTokens && product_below({B, D}, 2147483648.0) && product_below({B, T, D}, 1e12);
}

template <typename E>
bool vec_ok(int64_t D, std::initializer_list<const void *> ps) {
    return D % 4 == 0 && aligned_or_null(ps, 4 * sizeof(E));
}

GsWords gs_words(void *ws, const GsLayout &l) {
    char *p = static_cast<char *>(ws);
    return GsWords{reinterpret_cast<WsHeader *>(p), reinterpret_cast<unsigned int *>(p + l.words),
                   reinterpret_cast<unsigned int *>(p + l.states)};
}

// Clears the header and the words, which lie one behind the other from the start of `ws`.
int gs_clear(const char *fn, void *ws, const GsLayout &l, cudaStream_t s) {
    CLA_CUDA_TRY(cudaMemsetAsync(ws, 0, l.clear, s), fn);
    return CLA_OK;
}

template <typename E>
int gs_fwd(const char *fn, const void *x, const void *rg, const void *ig, const float *lam, const float *h0, void *h,
           float *hT, float *ckpt, GsArgs g, void *ws, const GsLayout &l, cudaStream_t s) {
    constexpr int L = sizeof(E) == 2 ? 8 : 4;
    g.chunks = ceil_div(g.T, 8 * L);
    const long long blocks = ceil_div(g.chunks * g.B * g.n_cw, kGsWarps);
    const bool vec = vec_ok<E>(g.D, {x, rg, ig, h});
    const GsWords w = gs_words(ws, l);
#define CLA_GS_FWD(V, R)                                                                                             \
    gated_fwd_kernel<E, V, R, L><<<(unsigned)blocks, kGsWarps * 32, 0, s>>>((const E *)x, (const E *)rg, (const E *)ig, \
                                                                            lam, h0, (E *)h, hT, ckpt, g, w)
    if (vec && g.reset == nullptr) CLA_GS_FWD(true, false);
    else if (vec) CLA_GS_FWD(true, true);
    else if (g.reset == nullptr) CLA_GS_FWD(false, false);
    else CLA_GS_FWD(false, true);
#undef CLA_GS_FWD
    return check_launch(fn);
}

template <typename E>
int gs_bwd(const char *fn, const void *x, const void *rg, const void *ig, const float *lam, const float *h0,
           const float *ckpt, const void *dh, const float *dhT, void *dx, void *drg, void *dig, float *dlam, float *dh0,
           GsArgs g, void *ws, const GsLayout &l, cudaStream_t s) {
    char *p = static_cast<char *>(ws);
    if (int st = gs_clear(fn, ws, l, s)) return st;
    if (ckpt == nullptr) {
        float *states = reinterpret_cast<float *>(p + l.ckpt);
        if (int st = gs_fwd<E>(fn, x, rg, ig, lam, h0, nullptr, nullptr, states, g, ws, l, s)) return st;
        // the words again, but not the header, which holds the scan's status
        CLA_CUDA_TRY(cudaMemsetAsync(p + l.words, 0, l.clear - l.words, s), fn);
        ckpt = states;
    }
    g.chunks = ceil_div(g.T, kGsCkpt);
    const long long blocks = ceil_div(g.chunks * g.B * g.n_cw, kGsWarps);
    const bool vec = vec_ok<E>(g.D, {x, rg, ig, dh, dx, drg, dig});
    const GsWords w = gs_words(ws, l);
    float *part = reinterpret_cast<float *>(p + l.part);
#define CLA_GS_BWD(V, R)                                                                                              \
    gated_bwd_kernel<E, V, R><<<(unsigned)blocks, kGsWarps * 32, 0, s>>>((const E *)x, (const E *)rg, (const E *)ig, lam, \
                                                                         ckpt, (const E *)dh, dhT, (E *)dx, (E *)drg,   \
                                                                         (E *)dig, part, dh0, g, w)
    if (vec && g.reset == nullptr) CLA_GS_BWD(true, false);
    else if (vec) CLA_GS_BWD(true, true);
    else if (g.reset == nullptr) CLA_GS_BWD(false, false);
    else CLA_GS_BWD(false, true);
#undef CLA_GS_BWD
    if (int st = check_launch(fn)) return st;
    if (dlam != nullptr) {
        long long rows = g.chunks * g.B;
        if (rows > kDlamRows) {
            float *part2 = reinterpret_cast<float *>(p + l.part2);
            gated_dlam_kernel<<<dim3((unsigned)ceil_div(g.D, 32), kDlamShares), 1024, 0, s>>>(part, lam, part2, rows, g.D);
            if (int st = check_launch(fn)) return st;
            part = part2;
            rows = kDlamShares;
        }
        gated_dlam_kernel<<<dim3((unsigned)ceil_div(g.D, 32), 1), 1024, 0, s>>>(part, lam, dlam, rows, g.D);
        return check_launch(fn);
    }
    return CLA_OK;
}

}  // namespace
}  // namespace cla

using namespace cla;

extern "C" size_t cla_gated_scan_ckpt_elems(int64_t B, int64_t T, int64_t D) {
    return gs_sizes_ok(B, T, D) ? (size_t)ceil_div(T, kGsCkpt) * (size_t)B * (size_t)D : 0;
}

extern "C" size_t cla_gated_scan_workspace_size(int64_t B, int64_t T, int64_t D) {
    return gs_sizes_ok(B, T, D) ? gs_layout(B, T, D).total : 0;
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
    const GsArgs g{reset, lens, T, 0, (int)B, (int)D, (int)ceil_div(D, 16), c};
    const GsLayout l = gs_layout(B, T, D);
    cudaStream_t s = (cudaStream_t)stream;
    if (int st = gs_clear(fn, ws, l, s)) return st;
    if (T == 0) {
        if (hT == nullptr) return CLA_OK;
        if (h0 != nullptr) CLA_CUDA_TRY(cudaMemcpyAsync(hT, h0, (size_t)(B * D) * 4, cudaMemcpyDeviceToDevice, s), fn);
        else CLA_CUDA_TRY(cudaMemsetAsync(hT, 0, (size_t)(B * D) * 4, s), fn);
        return CLA_OK;
    }
    if (dtype == CLA_F32) return gs_fwd<float>(fn, x, rgate, igate, lam, h0, h, hT, ckpt, g, ws, l, s);
    if (dtype == CLA_BF16) return gs_fwd<__nv_bfloat16>(fn, x, rgate, igate, lam, h0, h, hT, ckpt, g, ws, l, s);
    return gs_fwd<__half>(fn, x, rgate, igate, lam, h0, h, hT, ckpt, g, ws, l, s);
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
    const GsArgs g{reset, lens, T, 0, (int)B, (int)D, (int)ceil_div(D, 16), c};
    const GsLayout l = gs_layout(B, T, D);
    cudaStream_t s = (cudaStream_t)stream;
    if (B * T == 0) {
        if (dlam != nullptr) CLA_CUDA_TRY(cudaMemsetAsync(dlam, 0, (size_t)D * 4, s), fn);
        if (dh0 != nullptr && B > 0) {
            if (dhT != nullptr) CLA_CUDA_TRY(cudaMemcpyAsync(dh0, dhT, (size_t)(B * D) * 4, cudaMemcpyDeviceToDevice, s), fn);
            else CLA_CUDA_TRY(cudaMemsetAsync(dh0, 0, (size_t)(B * D) * 4, s), fn);
        }
        return gs_clear(fn, ws, l, s);
    }
    if (dtype == CLA_F32)
        return gs_bwd<float>(fn, x, rgate, igate, lam, h0, ckpt, dh, dhT, dx, drgate, digate, dlam, dh0, g, ws, l, s);
    if (dtype == CLA_BF16)
        return gs_bwd<__nv_bfloat16>(fn, x, rgate, igate, lam, h0, ckpt, dh, dhT, dx, drgate, digate, dlam, dh0, g, ws, l, s);
    return gs_bwd<__half>(fn, x, rgate, igate, lam, h0, ckpt, dh, dhT, dx, drgate, digate, dlam, dh0, g, ws, l, s);
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
