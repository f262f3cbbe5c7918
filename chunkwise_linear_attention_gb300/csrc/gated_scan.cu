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
// Decomposition.  A warp takes 8 L steps x 16 channels: lane = (sub, cg), cg in
// 0..3 picks 4 adjacent channels and sub in 0..7 a run of L steps.  Every
// input is read once; a lane keeps its run's decays and inputs in registers,
// composes them, then the 8 runs compose by shuffles, the block's warps (most
// of them one behind the other in time) in shared memory, and the blocks
// through pairs that they publish.  The state entering a block's steps is
// folded from the published pairs of its group's earlier blocks (8 a group,
// one a sub) and the state at the end of the group before.  That order is
// fixed by the place in the sequence alone, so the result does not depend on
// which block came first, and only one wait per 8 blocks is on the serial path.
//
// Measured at 8 x 4096 x 1024 bf16 (GB300): forward 93 us (8 bytes a step and
// channel: 2.9 TB/s, 43% of the measured copy rate), backward 187 us (14
// bytes: 2.5 TB/s, 37%).  What bounds both is latency at 16 and 12 warps a
// multiprocessor: 44 and 94 instructions a step and channel issue on 45% of
// the cycles.  Of a forward block's 12000 cycles the counter takes 2300, the
// loads and gates 4200, the scan and the block's exchange 1700, the look at
// the blocks before 1850, the second pass and the stores 1150.  Persistent
// blocks that ask for their next unit early (335 us for both passes) and five
// backward blocks a multiprocessor with part of their registers in shared
// memory (339 us) were slower: the first spills, the second has more blocks
// than a row of chunks in flight, which then wait for each other.
#include <math.h>

#include "cla_internal.cuh"
#include "elem_io.cuh"

namespace cla {
namespace {

constexpr int kGsCkpt = CLA_GATED_SCAN_CKPT_CHUNK;
constexpr int kGsGroup = 8;  // block chunks of a group: a lane looks at one pair, all at once
constexpr int kFwdWarps = 4, kFwdBlocks = 4;  // warps a block and blocks a multiprocessor
constexpr int kBwdWarps = 4, kBwdBlocks = 3;
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
__device__ __forceinline__ float sqra(float v) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(v));
    return y;
}
__device__ __forceinline__ float2 f2(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

struct Gate2 {
    float2 a, y, m, rm, r1, i, i1;  // a, log2 a, m, 1 / m, 1 - r, i, 1 - i
};

__device__ __forceinline__ float min_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// The gates of two channels at once (the paired fp32 instructions round each lane as the scalar
// ones do).  e^-g is held at 2^126, so that 1 - sigmoid(g) = e^-g sigmoid(g) stays finite: a gate
// does not close below 2^-126.  a = 2^y and 1 - a come from one split y = k + f, 2^f = 1 + t:
// a = 2^k + 2^k t and 1 - a = (1 - 2^k) - 2^k t, which for decays near 1 (k = 0) is -t itself,
// with no digits lost, where 1 - a^2 from a rounded a would keep only those above
// 2^-24 / (1 - a).  The polynomial is a least-maximum-error fit of 2^f on [-1/2, 1/2] with
// p(0) = 1 (Lawson's reweighted least squares, degree 6, 2e-9).  NaN passes through.
//
// BWD: with the factors that the gradients need (rm, r1, i1); without them nothing has to be held
// in range for 1 - sigmoid(g), and m is one square root.
template <bool BWD>
__device__ __forceinline__ Gate2 gate2(float2 rg, float2 ig, float2 nl2) {
    constexpr float kP1 = 6.931471825e-01f, kP2 = 2.402264774e-01f, kP3 = 5.550332367e-02f, kP4 = 9.618437849e-03f,
                    kP5 = 1.339887269e-03f, kP6 = 1.535334159e-04f, kMagic = 12582912.0f;
    Gate2 q;
    const float2 pr = mul2(rg, f2(-kLog2e)), pi = mul2(ig, f2(-kLog2e));
    const float2 er = BWD ? make_float2(ex2a(min_nan(pr.x, 126.f)), ex2a(min_nan(pr.y, 126.f))) : make_float2(ex2a(pr.x), ex2a(pr.y));
    const float2 ei = BWD ? make_float2(ex2a(min_nan(pi.x, 126.f)), ex2a(min_nan(pi.y, 126.f))) : make_float2(ex2a(pi.x), ex2a(pi.y));
    const float2 br = add2(er, f2(1.f)), bi = add2(ei, f2(1.f));
    const float2 r = make_float2(rcpa(br.x), rcpa(br.y));
    q.i = make_float2(rcpa(bi.x), rcpa(bi.y));
    if constexpr (BWD) {
        q.r1 = mul2(er, r);
        q.i1 = mul2(ei, q.i);
    }
    float2 y = mul2(nl2, r);
    y = make_float2(max_nan(y.x, -126.f), max_nan(y.y, -126.f));
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
    // 2^k: the low bits of km are k
    const float2 sc = make_float2(__uint_as_float(__float_as_uint(km.x) * (1u << 23) + 0x3f800000u),
                                  __uint_as_float(__float_as_uint(km.y) * (1u << 23) + 0x3f800000u));
    t = mul2(sc, t);
    q.a = add2(sc, t);
    float2 om = fma2(t, f2(-1.f), fma2(sc, f2(-1.f), f2(1.f)));  // 1 - a
    om = mul2(om, add2(q.a, f2(1.f)));                            // 1 - a^2
    if constexpr (BWD) {
        om = make_float2(fmaxf(om.x, 1e-37f), fmaxf(om.y, 1e-37f));
        q.rm = make_float2(rsqa(om.x), rsqa(om.y));
        q.m = mul2(om, q.rm);
    } else {
        q.m = make_float2(sqra(om.x), sqra(om.y));
    }
    return q;
}

struct GsArgs {
    const uint8_t *reset;
    const int32_t *lens;
    const float *rate;  // -c softplus(lam) log2 e
    int T, B, D;
    int tw, n_cw, chunks;  // warps of a block in time; groups of 16 channels (whole blocks); block chunks
    float c;
};

__device__ __forceinline__ int seq_len(const GsArgs &g, int b) {
    return g.lens == nullptr ? g.T : min(max(__ldg(g.lens + b), 0), g.T);
}

// Four adjacent elements as they lie in memory.
template <typename E>
struct Raw4 {
    uint2 w;
};
template <>
struct Raw4<float> {
    float4 w;
};
// VEC: with one access, else one by one (rows that are not aligned), those below `n` only.
template <typename E, bool VEC>
__device__ __forceinline__ Raw4<E> ld4(const E *p, int n) {
    Raw4<E> r;
    if constexpr (VEC) {
        r.w = __ldcs(reinterpret_cast<const decltype(r.w) *>(p));
    } else if constexpr (sizeof(E) == 4) {
        r.w = make_float4(n > 0 ? __ldg(p) : 0.f, n > 1 ? __ldg(p + 1) : 0.f, n > 2 ? __ldg(p + 2) : 0.f, n > 3 ? __ldg(p + 3) : 0.f);
    } else {
        const unsigned short *s = reinterpret_cast<const unsigned short *>(p);
        const unsigned int a = n > 0 ? __ldg(s) : 0, b = n > 1 ? __ldg(s + 1) : 0, c = n > 2 ? __ldg(s + 2) : 0, d = n > 3 ? __ldg(s + 3) : 0;
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

// A reset's decay is -0: no other is negative, so a product of decays is -0 where a reset is among
// them (two of them are kept apart below) and +0 only where decays ran out of range.
// One step's decay (ONE) is at least 2^-126 otherwise, and a plain comparison tells.
template <bool ONE>
__device__ __forceinline__ bool is_reset(float a) { return ONE ? a == 0.f : __float_as_uint(a) == 0x80000000u; }
constexpr float kReset = -0.0f;

// (A, B) after (pa, pb): B <- A pb + B, A <- A pa.  RST: behind a reset, what came before it is
// dropped, NaN and infinity included; a product that only underflowed drops neither.
template <bool RST, bool ONE = false>
__device__ __forceinline__ void after(float2 &A, float2 &B, float2 pa, float2 pb) {
    if constexpr (RST) {
        if (is_reset<ONE>(A.x)) pa.x = pb.x = 0.f;
        if (is_reset<ONE>(A.y)) pa.y = pb.y = 0.f;
    }
    B = fma2(A, pb, B);
    A = mul2(A, pa);
}
template <bool RST, bool ONE = false>
__device__ __forceinline__ float2 apply(float2 A, float2 s, float2 B) {
    if constexpr (RST) {
        if (is_reset<ONE>(A.x)) s.x = 0.f;
        if (is_reset<ONE>(A.y)) s.y = 0.f;
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
// -0.0, of a decay, where that is a reset, as the smallest number.  Each element of a 16-byte relaxed access is single-copy atomic: a reader that sees a
// nonzero word sees the value, without fences.
__device__ __forceinline__ unsigned int pub(float v) {
    const unsigned int b = __float_as_uint(v);
    return b != 0u ? b : 0x80000000u;
}
__device__ __forceinline__ unsigned int pub_decay(float v) { return max(__float_as_uint(v), 1u); }
template <bool DECAY>
__device__ __forceinline__ void publish4(unsigned int *p, const float2 (&v)[2]) {
    auto word = [](float x) { return DECAY ? pub_decay(x) : pub(x); };
    asm volatile("st.relaxed.gpu.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(word(v[0].x)), "r"(word(v[0].y)),
                 "r"(word(v[1].x)), "r"(word(v[1].y))
                 : "memory");
}
__device__ __forceinline__ bool peek4(const unsigned int *p, float2 (&v)[2]) {
    unsigned int a, b, c, d;
    asm volatile("ld.relaxed.gpu.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "l"(p) : "memory");
    v[0] = make_float2(__uint_as_float(a), __uint_as_float(b));
    v[1] = make_float2(__uint_as_float(c), __uint_as_float(d));
    return a != 0u && b != 0u && c != 0u && d != 0u;
}
// Polls until the words that a lane asks for are there (p: a pair, q: a state; either may be NULL),
// a bounded number of times; then records the timeout and carries on with what it saw.
__device__ __forceinline__ void wait_words(const unsigned int *p, float2 (&a)[2], float2 (&b)[2], const unsigned int *q,
                                           float2 (&s)[2], WsHeader *hdr, unsigned int where) {
    for (unsigned int it = 0; it < kSpinLimit; ++it) {
        bool ok = true;
        if (p != nullptr) {
            const bool x = peek4(p, a), y = peek4(p + 4, b);
            ok = x && y;
        }
        if (q != nullptr) ok = peek4(q, s) && ok;
        if (ok) return;
        if (it >= 8) __nanosleep(64);
    }
    atomicOr(&hdr->error, kErrTimeout);
    atomicExch(&hdr->where, where);
}

struct GsWords {
    WsHeader *hdr;
    unsigned int *pairs;   // [block chunk][b][cw][cg][A, B][4], chunks in the scan's order
    unsigned int *states;  // [group][b][cw][cg][4]
};

// By one warp: publishes the pair (A, B) of block chunk `idx` for 16 channels (`rem` of the `per`
// groups of them; every lane holds its cg's), and returns the state entering it: the pairs of the
// group's chunks before it, one a sub, on the state at the end of the group before, or `s0`.  The
// last chunk of a group publishes the state behind it.
template <bool RST>
__device__ __forceinline__ void carry_in(const GsWords &w, int idx, int chunks, int per, int rem, const float2 (&A)[2],
                                         const float2 (&B)[2], const float2 (&s0)[2], float2 (&s)[2], unsigned int where) {
    const int lane = threadIdx.x & 31, sub = lane >> 2, cg = lane & 3;
    const int n = idx % kGsGroup, first = idx - n;
    const bool last_of_group = n == kGsGroup - 1, more = idx + 1 < chunks && sub == 0;
    if (more && !last_of_group) {
        unsigned int *p = w.pairs + (((size_t)idx * per + rem) * 4 + cg) * 8;
        publish4<true>(p, A);
        publish4<false>(p + 4, B);
    }
    float2 PA[2] = {f2(1.f), f2(1.f)}, PB[2] = {f2(0.f), f2(0.f)}, S[2] = {s0[0], s0[1]};
    wait_words(sub < n ? w.pairs + (((size_t)(first + sub) * per + rem) * 4 + cg) * 8 : nullptr, PA, PB,
               first > 0 ? w.states + (((size_t)(first / kGsGroup - 1) * per + rem) * 4 + cg) * 4 : nullptr, S, w.hdr, where);
    __syncwarp();
    if (n > 0) {
        scan_runs<RST, false>(PA, PB, sub);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            PA[v] = shfl2(PA[v], 28 + cg);
            PB[v] = shfl2(PB[v], 28 + cg);
        }
    }
#pragma unroll
    for (int v = 0; v < 2; ++v) s[v] = apply<RST>(PA[v], S[v], PB[v]);
    if (more && last_of_group) {
        const float2 e[2] = {apply<RST>(A[0], s[0], B[0]), apply<RST>(A[1], s[1], B[1])};
        publish4<false>(w.states + (((size_t)(idx / kGsGroup) * per + rem) * 4 + cg) * 4, e);
    }
}

// What the warps of a block exchange: each warp's pair, the state entering the block's steps for
// each group of channels, the block's unit.
template <int NW>
struct Exchange {
    float4 pair[NW][4][2];
    float4 in[NW][4];
    unsigned int ticket;
    __device__ __forceinline__ static float4 pack(const float2 (&v)[2]) { return make_float4(v[0].x, v[0].y, v[1].x, v[1].y); }
    __device__ __forceinline__ static void unpack(float4 r, float2 (&v)[2]) {
        v[0] = make_float2(r.x, r.y);
        v[1] = make_float2(r.z, r.w);
    }
};

// The block's part of the scan.  A, B: this warp's whole pair, in the lanes of `holder` (the sub
// whose run is last in the scan's order).  Returns the state entering this warp's steps.
template <bool RST, int NW>
__device__ __forceinline__ void block_carry(Exchange<NW> &ex, const GsArgs &g, const GsWords &w, int idx, int per, int rem,
                                            int holder, const float2 (&A)[2], const float2 (&B)[2], const float2 (&s0)[2],
                                            float2 (&s)[2], unsigned int where) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane >> 2, cg = lane & 3;
    const int cb = NW / g.tw, wt = warp / cb, wc = warp - wt * cb;
    if (sub == holder) {
        ex.pair[warp][cg][0] = ex.pack(A);
        ex.pair[warp][cg][1] = ex.pack(B);
    }
    __syncthreads();
    // the pairs of the warps before this one; the first warp: of all of them
    float2 PA[2] = {f2(1.f), f2(1.f)}, PB[2] = {f2(0.f), f2(0.f)};
    for (int k = 0; k < (wt == 0 ? g.tw : wt); ++k) {
        float2 a[2], b[2];
        ex.unpack(ex.pair[k * cb + wc][cg][0], a);
        ex.unpack(ex.pair[k * cb + wc][cg][1], b);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            after<RST>(a[v], b[v], PA[v], PB[v]);
            PA[v] = a[v];
            PB[v] = b[v];
        }
    }
    if (wt == 0) {
        carry_in<RST>(w, idx, g.chunks, per, rem, PA, PB, s0, s, where);
        if (sub == 0) ex.in[wc][cg] = ex.pack(s);
    }
    __syncthreads();
    if (wt > 0) {
        ex.unpack(ex.in[wc][cg], s);
#pragma unroll
        for (int v = 0; v < 2; ++v) s[v] = apply<RST>(PA[v], s[v], PB[v]);
    }
}

// Blocks take units from a counter, in the order in which they start: every unit that a block waits
// for was taken by a block that runs already, whatever else the GPU does.
template <int NW>
__device__ __forceinline__ int take_unit(Exchange<NW> &ex, WsHeader *hdr, int which) {
    if (threadIdx.x == 0) ex.ticket = atomicAdd(&hdr->ticket[which], 1u);
    __syncthreads();
    return (int)ex.ticket;
}

// What a unit is: block chunk, sequence, channels, and this lane's run of steps in it.
struct Unit {
    int idx, rem, chunk, t0, b, c0, nv, n, rows;  // channels from c0 (nv of them exist); n: steps of the run in the sequence, rows: in T
    size_t at;
    template <int L, int NW, bool REV>
    static __device__ __forceinline__ Unit make(const GsArgs &g, int unit) {
        const int warp = threadIdx.x >> 5, sub = (threadIdx.x >> 2) & 7, cg = threadIdx.x & 3;
        const int cb = NW / g.tw, wt = warp / cb, cbs = g.n_cw / cb, per = g.B * cbs;
        Unit u;
        u.idx = unit / per;
        const int r = unit - u.idx * per;
        u.b = r / cbs;
        const int cw = (r - u.b * cbs) * cb + warp - wt * cb;
        u.rem = u.b * g.n_cw + cw;
        u.chunk = REV ? (g.chunks - u.idx) * g.tw - 1 - wt : u.idx * g.tw + wt;  // of 8 L steps
        u.c0 = cw * 16 + cg * 4;
        u.nv = g.D - u.c0;
        u.t0 = u.chunk * (8 * L) + sub * L;
        u.n = u.nv <= 0 ? 0 : min(max(seq_len(g, u.b) - u.t0, 0), L);
        u.rows = u.nv <= 0 ? 0 : min(max(g.T - u.t0, 0), L);
        u.at = ((size_t)u.b * g.T + u.t0) * g.D + u.c0;
        return u;
    }
};

// Clears the words that are waited for, and the header, and forms the channels' rates
// -c softplus(lam) log2 e (padded to whole units): once here instead of in every unit, where they
// cost 5 instructions a step and channel.
__global__ void gated_setup_kernel(uint4 *ws, long long words, float *rate, const float *__restrict__ lam, int D, int padded, float c) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    for (long long k = i; k < words; k += (long long)gridDim.x * blockDim.x) ws[k] = make_uint4(0u, 0u, 0u, 0u);
    for (long long k = i; k < padded; k += (long long)gridDim.x * blockDim.x) rate[k] = k < D ? -c * softplus(lam[k]) * kLog2e : 0.f;
}
__device__ __forceinline__ void load_rate(const float *rate, int c0, float2 (&v)[2]) {
    const float4 r = __ldg(reinterpret_cast<const float4 *>(rate + c0));
    v[0] = make_float2(r.x, r.y);
    v[1] = make_float2(r.z, r.w);
}

// ------------------------------------------------------------------ forward
// L = 8 steps a lane for 2-byte elements, 4 for fp32 (whose raw rows take twice the registers).
// h may be NULL: only the checkpoint is written then.
template <typename E, bool VEC, bool RST, int L>
__global__ void __launch_bounds__(kFwdWarps * 32, kFwdBlocks)
gated_fwd_kernel(const E *__restrict__ x, const E *__restrict__ rg, const E *__restrict__ ig,
                 const float *__restrict__ h0, E *__restrict__ h, float *__restrict__ hT, float *__restrict__ ckpt, GsArgs g,
                 GsWords w) {
    __shared__ Exchange<kFwdWarps> ex;
    const Unit q = Unit::make<L, kFwdWarps, false>(g, take_unit(ex, w.hdr, 0));
    const int sub = (threadIdx.x >> 2) & 7;
    Raw4<E> rx[L], rr[L], ri[L];
    bool rs[L];
#pragma unroll
    for (int j = 0; j < L; ++j)
        if (j < q.n) {
            const size_t at = q.at + (size_t)j * g.D;
            rr[j] = ld4<E, VEC>(rg + at, q.nv);
            ri[j] = ld4<E, VEC>(ig + at, q.nv);
            rx[j] = ld4<E, VEC>(x + at, q.nv);
            if constexpr (RST) rs[j] = g.reset[(size_t)q.b * g.T + q.t0 + j] != 0;
        }
    float2 nl2[2], s0[2] = {f2(0.f), f2(0.f)};
    load_rate(g.rate, q.c0, nl2);
    if (h0 != nullptr && q.nv > 0) ldf4(h0 + (size_t)q.b * g.D + q.c0, s0, q.nv);
    const bool full = __all_sync(~0u, q.n == L);

    float2 a[L][2], u[L][2], A[2] = {f2(1.f), f2(1.f)}, B[2] = {f2(0.f), f2(0.f)};
#pragma unroll
    for (int j = 0; j < L; ++j) {
        float2 xv[2], rv[2], iv[2];
        cvt4<E>(rr[j], rv);
        cvt4<E>(ri[j], iv);
        cvt4<E>(rx[j], xv);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const Gate2 e = gate2<false>(rv[v], iv[v], nl2[v]);
            a[j][v] = e.a;
            u[j][v] = mul2(mul2(e.m, e.i), xv[v]);
            if constexpr (RST)
                if (j < q.n && rs[j]) {
                    a[j][v] = f2(kReset);
                    u[j][v] = mul2(e.i, xv[v]);
                }
        }
    }
    if (!full) {  // behind the sequence
#pragma unroll
        for (int j = 0; j < L; ++j)
            if (j >= q.n) a[j][0] = a[j][1] = f2(1.f), u[j][0] = u[j][1] = f2(0.f);
    }
#pragma unroll
    for (int j = 0; j < L; ++j)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const float2 pa = A[v], pb = B[v];
            A[v] = a[j][v];
            B[v] = u[j][v];
            after<RST, true>(A[v], B[v], pa, pb);
        }
    scan_runs<RST, false>(A, B, sub);
    float2 Ax[2], Bx[2], s[2];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        Ax[v] = shfl_up2(A[v], 4);
        Bx[v] = shfl_up2(B[v], 4);
        if (sub == 0) Ax[v] = f2(1.f), Bx[v] = f2(0.f);
    }
    block_carry<RST, kFwdWarps>(ex, g, w, q.idx, g.B * g.n_cw, q.rem, 7, A, B, s0, s, 11u);
    if (q.nv <= 0) return;
#pragma unroll
    for (int v = 0; v < 2; ++v) s[v] = apply<RST>(Ax[v], s[v], Bx[v]);
    if (ckpt != nullptr && (sub * L) % kGsCkpt == 0 && q.rows > 0)
        stf4(ckpt + ((size_t)q.b * ((g.T + kGsCkpt - 1) / kGsCkpt) + q.t0 / kGsCkpt) * g.D + q.c0, s, q.nv);
#pragma unroll
    for (int j = 0; j < L; ++j) {
#pragma unroll
        for (int v = 0; v < 2; ++v) s[v] = apply<RST, true>(a[j][v], s[v], u[j][v]);
        if (j < q.rows && h != nullptr) {
            float2 z[2] = {s[0], s[1]};
            if (!full && j >= q.n) z[0] = z[1] = f2(0.f);
            st4<E, VEC>(h + q.at + (size_t)j * g.D, z, q.nv);
        }
    }
    // the steps behind T keep the state, so the run's last one is T's
    if (hT != nullptr && q.rows > 0 && q.t0 + q.rows == g.T) stf4(hT + (size_t)q.b * g.D + q.c0, s, q.nv);
}

// ------------------------------------------------------------------ backward
// Chunks of 32 steps, the last first, 4 steps a lane: the states before each step are rebuilt
// from the checkpoint at the chunk's start, the adjoint's carry c_t = a_t (dh_t + c_{t+1}) is
// scanned as the forward's state is, and every gradient is written once.  Each chunk leaves its
// sums of G for dlam in a row of `part`.
template <typename E, bool VEC, bool RST>
__global__ void __launch_bounds__(kBwdWarps * 32, kBwdBlocks)
gated_bwd_kernel(const E *__restrict__ x, const E *__restrict__ rg, const E *__restrict__ ig,
                 const float *__restrict__ ckpt, const E *__restrict__ dh, const float *__restrict__ dhT,
                 E *__restrict__ dx, E *__restrict__ drg, E *__restrict__ dig, float *__restrict__ part,
                 float *__restrict__ dh0, GsArgs g, GsWords w) {
    constexpr int L = 4;
    static_assert(8 * L == kGsCkpt, "a warp's steps start at a checkpoint");
    __shared__ Exchange<kBwdWarps> ex;
    const Unit q = Unit::make<L, kBwdWarps, true>(g, take_unit(ex, w.hdr, 1));
    const int sub = (threadIdx.x >> 2) & 7, ckpts = (g.T + kGsCkpt - 1) / kGsCkpt;
    Raw4<E> rx[L], rr[L], ri[L], rd[L];
    bool rs[L];
#pragma unroll
    for (int j = 0; j < L; ++j)
        if (j < q.n) {
            const size_t at = q.at + (size_t)j * g.D;
            rr[j] = ld4<E, VEC>(rg + at, q.nv);
            ri[j] = ld4<E, VEC>(ig + at, q.nv);
            rx[j] = ld4<E, VEC>(x + at, q.nv);
            rd[j] = ld4<E, VEC>(dh + at, q.nv);
            if constexpr (RST) rs[j] = g.reset[(size_t)q.b * g.T + q.t0 + j] != 0;
        }
    float2 nl2[2], s0[2] = {f2(0.f), f2(0.f)}, hs[2] = {f2(0.f), f2(0.f)};
    load_rate(g.rate, q.c0, nl2);
    if (q.nv > 0) {
        if (dhT != nullptr) ldf4(dhT + (size_t)q.b * g.D + q.c0, s0, q.nv);
        if (q.chunk < ckpts) ldf4(ckpt + ((size_t)q.b * ckpts + q.chunk) * g.D + q.c0, hs, q.nv);
    }
    const bool full = __all_sync(~0u, q.n == L);

    // per step: a, L a, 1 - r, a u / m, m i, x (1 - i), and b = m i x, then h_{t-1}
    float2 a[L][2], La[L][2], r1[L][2], w2[L][2], mi[L][2], xi[L][2], hp[L][2];
    float2 A[2] = {f2(1.f), f2(1.f)}, B[2] = {f2(0.f), f2(0.f)};
#pragma unroll
    for (int j = 0; j < L; ++j) {
        float2 xv[2], rv[2], iv[2];
        cvt4<E>(rr[j], rv);
        cvt4<E>(ri[j], iv);
        cvt4<E>(rx[j], xv);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const Gate2 e = gate2<true>(rv[v], iv[v], nl2[v]);
            a[j][v] = e.a;
            La[j][v] = mul2(mul2(e.y, f2(kLn2)), e.a);
            r1[j][v] = e.r1;
            w2[j][v] = mul2(mul2(e.a, e.rm), mul2(e.i, xv[v]));
            mi[j][v] = mul2(e.m, e.i);
            if constexpr (RST)
                if (j < q.n && rs[j])
                    a[j][v] = f2(kReset), La[j][v] = w2[j][v] = f2(0.f), mi[j][v] = e.i;
            xi[j][v] = mul2(xv[v], e.i1);
            hp[j][v] = mul2(mi[j][v], xv[v]);
        }
    }
    if (!full) {  // behind the sequence
#pragma unroll
        for (int j = 0; j < L; ++j)
            if (j >= q.n)
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    a[j][v] = f2(1.f);
                    La[j][v] = r1[j][v] = w2[j][v] = mi[j][v] = xi[j][v] = hp[j][v] = f2(0.f);
                }
    }
#pragma unroll
    for (int j = 0; j < L; ++j)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const float2 pa = A[v], pb = B[v];
            A[v] = a[j][v];
            B[v] = hp[j][v];
            after<RST, true>(A[v], B[v], pa, pb);
        }
    scan_runs<RST, false>(A, B, sub);
    auto grad = [&](int j, float2 (&v)[2]) {  // dh_t of the run's step j
        cvt4<E>(rd[j], v);
        if (!full && j >= q.n) v[0] = v[1] = f2(0.f);
    };
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        const float2 pa = shfl_up2(A[v], 4), pb = shfl_up2(B[v], 4);
        if (sub > 0) hs[v] = apply<RST>(pa, hs[v], pb);
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const float2 next = apply<RST, true>(a[j][v], hs[v], hp[j][v]);
            hp[j][v] = hs[v];
            hs[v] = next;
        }
        A[v] = f2(1.f);
        B[v] = f2(0.f);
    }
#pragma unroll
    for (int j = L - 1; j >= 0; --j) {
        float2 gd[2];
        grad(j, gd);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const float2 pa = A[v], pb = B[v];
            A[v] = a[j][v];
            B[v] = apply<RST, true>(a[j][v], gd[v], f2(0.f));
            after<RST, true>(A[v], B[v], pa, pb);
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
    block_carry<RST, kBwdWarps>(ex, g, w, q.idx, g.B * g.n_cw, q.rem, 0, A, B, s0, s, 13u);
    float2 sum[2] = {f2(0.f), f2(0.f)};
#pragma unroll
    for (int v = 0; v < 2; ++v) s[v] = apply<RST>(Ax[v], s[v], Bx[v]);
#pragma unroll
    for (int j = L - 1; j >= 0; --j) {
        float2 gd[2], ox[2], oi[2], orr[2];
        grad(j, gd);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const float2 hb = add2(gd[v], s[v]);
            s[v] = apply<RST, true>(a[j][v], hb, f2(0.f));
            float2 before = hp[j][v];
            if constexpr (RST)
                if (is_reset<true>(a[j][v].x)) before = f2(0.f);  // a reset is one of all channels
            const float2 G = mul2(mul2(hb, La[j][v]), fma2(w2[j][v], f2(-1.f), before));
            sum[v] = add2(sum[v], G);
            ox[v] = mul2(hb, mi[j][v]);
            oi[v] = mul2(ox[v], xi[j][v]);
            orr[v] = mul2(G, r1[j][v]);
        }
        if (j < q.rows) {
            const size_t at = q.at + (size_t)j * g.D;
            st4<E, VEC>(dx + at, ox, q.nv);
            st4<E, VEC>(dig + at, oi, q.nv);
            st4<E, VEC>(drg + at, orr, q.nv);
        }
    }
    if (q.nv > 0 && dh0 != nullptr && q.chunk == 0 && sub == 0) stf4(dh0 + (size_t)q.b * g.D + q.c0, s, q.nv);
#pragma unroll
    for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int off = 16; off >= 4; off >>= 1)
            sum[v] = add2(sum[v], make_float2(__shfl_xor_sync(~0u, sum[v].x, off), __shfl_xor_sync(~0u, sum[v].y, off)));
    if (q.nv > 0 && sub == 0 && q.chunk < ckpts) stf4(part + ((size_t)q.chunk * g.B + q.b) * g.D + q.c0, sum, q.nv);
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
// A thread takes 4 adjacent channels (VEC: with one access a tensor): at 512 x 4096 bf16 12 us against
// 20 us with one channel a thread, at 1024 x 8192 31 (4.4 TB/s, 64% of the measured copy rate) against
// 61.  Four rows a thread, which share their channels' rates, gave 29 at the latter and nothing below.
template <typename E, bool VEC>
__global__ void __launch_bounds__(128) gated_step_kernel(const E *x, const E *rg, const E *ig, const float *lam, const uint8_t *reset,
                                                         float *h, E *y, int B, int D, float c) {
    const int quads = (D + 3) / 4;
    const long long u = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const int b = (int)(u / quads), d = (int)(u % quads) * 4, n = D - d;
    if (b >= B) return;
    const size_t at = (size_t)b * D + d;
    float2 xv[2], rv[2], iv[2], hv[2], l[2], s[2];
    cvt4<E>(ld4<E, VEC>(rg + at, n), rv);
    cvt4<E>(ld4<E, VEC>(ig + at, n), iv);
    cvt4<E>(ld4<E, VEC>(x + at, n), xv);
    if constexpr (VEC) {
        const float4 r = *reinterpret_cast<const float4 *>(h + at);
        hv[0] = make_float2(r.x, r.y);
        hv[1] = make_float2(r.z, r.w);
    } else {
        ldf4(h + at, hv, n);
    }
    ldf4(lam + d, l, n);
    const bool fresh = reset != nullptr && reset[b] != 0;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
        const Gate2 q = gate2<false>(rv[v], iv[v], make_float2(-c * softplus(l[v].x) * kLog2e, -c * softplus(l[v].y) * kLog2e));
        const float2 w = mul2(q.i, xv[v]);
        s[v] = fresh ? w : fma2(q.a, hv[v], mul2(q.m, w));
    }
    if constexpr (VEC) *reinterpret_cast<float4 *>(h + at) = make_float4(s[0].x, s[0].y, s[1].x, s[1].y);
    else stf4(h + at, s, n);
    st4<E, VEC>(y + at, s, n);
}

template <typename E>
int gs_step(const char *fn, const void *x, const void *rg, const void *ig, const float *lam, const uint8_t *reset, float *h, void *y,
            float c, int64_t B, int64_t D, cudaStream_t s) {
    const unsigned grid = (unsigned)((B * ((D + 3) / 4) + 127) / 128);
    auto go = [&](auto kernel) {
        kernel<<<grid, 128, 0, s>>>((const E *)x, (const E *)rg, (const E *)ig, lam, reset, h, (E *)y, (int)B, (int)D, c);
    };
    if (D % 4 == 0 && aligned_or_null({x, rg, ig, y}, 4 * sizeof(E)) && aligned16(h)) go(gated_step_kernel<E, true>);
    else go(gated_step_kernel<E, false>);
    return check_launch(fn);
}

// ------------------------------------------------------------------ host side
// 10^12 elements, rounded up to whole units, are fewer than 2^31 units of 32 steps x 16 channels.
bool gs_sizes_ok(int64_t B, int64_t T, int64_t D) {
    return B >= 0 && T >= 0 && D >= 0 && T <= kMaxTokens && product_below({B, D}, 2147483648.0) &&
           product_below({B, T + 511, D / 128 + 1, 128}, 1e12);
}

int gs_check(const char *fn, int64_t B, int64_t T, int64_t D, int dtype, float c) {
    if (B < 0 || T < 0 || D < 0) return fail(CLA_ERR_INVALID_ARG, "%s: negative size", fn);
    if (!(c > 0.f) || !isfinite(c)) return fail(CLA_ERR_INVALID_ARG, "%s: c must be positive and finite", fn);
    if (dtype_bytes(dtype) == 0) return fail(CLA_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
    if (!gs_sizes_ok(B, T, D))
        return fail(CLA_ERR_UNSUPPORTED, "%s: B * D must be below 2^31, B * T * D well below 10^12, T at most 2^31 - 512", fn);
    return CLA_OK;
}

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// The workspace: header, the words of the published pairs and states (blocks that have a
// successor cover at least 4 warps x 32 steps), the channels' rates, the rebuilt checkpoint, the
// rows of dlam's sums and the rows that these are reduced to.
struct GsLayout {
    size_t words, clear, states, rate, ckpt, part, part2, total;
};
// Above these many rows dlam's sums go in two steps, of enough shares to fill the GPU (1024 rows of
// 1024 channels: 19 us in one step, 8 + 4 us in two).
constexpr long long kDlamRows = 128;
constexpr int kDlamShares = 64;

// Groups of 16 channels, in whole blocks whatever their shape.
int64_t gs_groups(int64_t D) { return ceil_div(D, 16 * kFwdWarps) * kFwdWarps; }
static_assert(kFwdWarps >= kBwdWarps, "groups in whole blocks");

GsLayout gs_layout(int64_t B, int64_t T, int64_t D) {
    GsLayout l;
    const size_t units = (size_t)B * gs_groups(D), ch = (size_t)ceil_div(T, kGsCkpt);
    const size_t blocks = (size_t)ceil_div(T, kGsCkpt * (kFwdWarps < kBwdWarps ? kFwdWarps : kBwdWarps));
    l.words = sizeof(WsHeader);
    l.states = l.words + blocks * units * 4 * 8 * 4;
    l.clear = l.states + (size_t)ceil_div(blocks, kGsGroup) * units * 4 * 4 * 4;
    l.rate = l.clear;
    l.ckpt = l.rate + (size_t)gs_groups(D) * 64;
    l.part = l.ckpt + align_up(ch * (size_t)B * D * 4, 16);
    l.part2 = l.part + align_up(ch * (size_t)B * D * 4, 16);
    l.total = l.part2 + (ch * B > (size_t)kDlamRows ? align_up((size_t)kDlamShares * D * 4, 16) : 0);
    return l;
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

// The header and the words lie one behind the other from the start of `ws`; `from`: the first byte
// that is cleared.
int gs_setup(const char *fn, void *ws, const GsLayout &l, size_t from, const float *lam, int64_t D, float c, cudaStream_t s) {
    char *p = static_cast<char *>(ws);
    const long long words = (long long)((l.clear - from) / 16), padded = gs_groups(D) * 16, most = words > padded ? words : padded;
    const long long blocks = ceil_div(most, 256);
    gated_setup_kernel<<<(unsigned)(blocks < 608 ? blocks : 608), 256, 0, s>>>(
        reinterpret_cast<uint4 *>(p + from), words, reinterpret_cast<float *>(p + l.rate), lam, (int)D, (int)padded, c);
    return check_launch(fn);
}

// A block's warps lie one behind the other in time, as far as T fills them (a power of two), and
// the rest of them side by side in the channels.
template <int NW>
unsigned gs_grid(GsArgs &g, int steps) {
    g.tw = 1;
    while (g.tw < NW && (long long)g.tw * steps < g.T) g.tw *= 2;
    g.chunks = (int)ceil_div(g.T, (long long)steps * g.tw);
    const int cb = NW / g.tw;
    g.n_cw = (int)(ceil_div(ceil_div(g.D, 16), cb) * cb);
    return (unsigned)(g.chunks * g.B * (g.n_cw / cb));
}

template <typename E, bool V, bool R>
int gs_fwd_launch(const char *fn, const void *x, const void *rg, const void *ig, const float *h0, void *h,
                  float *hT, float *ckpt, GsArgs g, const GsWords &w, cudaStream_t s) {
    constexpr int L = sizeof(E) == 2 ? 8 : 4;
    const unsigned blocks = gs_grid<kFwdWarps>(g, 8 * L);
    gated_fwd_kernel<E, V, R, L><<<blocks, kFwdWarps * 32, 0, s>>>((const E *)x, (const E *)rg, (const E *)ig, h0, (E *)h, hT, ckpt, g, w);
    return check_launch(fn);
}

template <typename E>
int gs_fwd(const char *fn, const void *x, const void *rg, const void *ig, const float *h0, void *h,
           float *hT, float *ckpt, const GsArgs &g, void *ws, const GsLayout &l, cudaStream_t s) {
    const bool vec = vec_ok<E>(g.D, {x, rg, ig, h});
    const GsWords w = gs_words(ws, l);
    if (vec && g.reset == nullptr) return gs_fwd_launch<E, true, false>(fn, x, rg, ig, h0, h, hT, ckpt, g, w, s);
    if (vec) return gs_fwd_launch<E, true, true>(fn, x, rg, ig, h0, h, hT, ckpt, g, w, s);
    if (g.reset == nullptr) return gs_fwd_launch<E, false, false>(fn, x, rg, ig, h0, h, hT, ckpt, g, w, s);
    return gs_fwd_launch<E, false, true>(fn, x, rg, ig, h0, h, hT, ckpt, g, w, s);
}

template <typename E, bool V, bool R>
int gs_bwd_launch(const char *fn, const void *x, const void *rg, const void *ig, const float *ckpt,
                  const void *dh, const float *dhT, void *dx, void *drg, void *dig, float *part, float *dh0, GsArgs g,
                  const GsWords &w, cudaStream_t s) {
    const unsigned blocks = gs_grid<kBwdWarps>(g, 32);
    gated_bwd_kernel<E, V, R><<<blocks, kBwdWarps * 32, 0, s>>>((const E *)x, (const E *)rg, (const E *)ig, ckpt, (const E *)dh, dhT,
                                                                  (E *)dx, (E *)drg, (E *)dig, part, dh0, g, w);
    return check_launch(fn);
}

template <typename E>
int gs_bwd(const char *fn, const void *x, const void *rg, const void *ig, const float *lam, const float *h0,
           const float *ckpt, const void *dh, const float *dhT, void *dx, void *drg, void *dig, float *dlam, float *dh0,
           GsArgs g, void *ws, const GsLayout &l, cudaStream_t s) {
    char *p = static_cast<char *>(ws);
    g.rate = reinterpret_cast<const float *>(p + l.rate);
    if (int st = gs_setup(fn, ws, l, 0, lam, g.D, g.c, s)) return st;
    if (ckpt == nullptr) {
        float *states = reinterpret_cast<float *>(p + l.ckpt);
        if (int st = gs_fwd<E>(fn, x, rg, ig, h0, nullptr, nullptr, states, g, ws, l, s)) return st;
        // the words again, but not the header, which holds the scan's status
        if (int st = gs_setup(fn, ws, l, l.words, lam, g.D, g.c, s)) return st;
        ckpt = states;
    }
    const bool vec = vec_ok<E>(g.D, {x, rg, ig, dh, dx, drg, dig});
    const GsWords w = gs_words(ws, l);
    float *part = reinterpret_cast<float *>(p + l.part);
    int st;
    if (vec && g.reset == nullptr) st = gs_bwd_launch<E, true, false>(fn, x, rg, ig, ckpt, dh, dhT, dx, drg, dig, part, dh0, g, w, s);
    else if (vec) st = gs_bwd_launch<E, true, true>(fn, x, rg, ig, ckpt, dh, dhT, dx, drg, dig, part, dh0, g, w, s);
    else if (g.reset == nullptr) st = gs_bwd_launch<E, false, false>(fn, x, rg, ig, ckpt, dh, dhT, dx, drg, dig, part, dh0, g, w, s);
    else st = gs_bwd_launch<E, false, true>(fn, x, rg, ig, ckpt, dh, dhT, dx, drg, dig, part, dh0, g, w, s);
    if (st) return st;
    if (dlam != nullptr) {
        long long rows = ceil_div(g.T, kGsCkpt) * g.B;
        if (rows > kDlamRows) {
            float *part2 = reinterpret_cast<float *>(p + l.part2);
            const long long columns = ceil_div(g.D, 32), want = ceil_div(320, columns), shares = want < kDlamShares ? want : kDlamShares;
            gated_dlam_kernel<<<dim3((unsigned)columns, (unsigned)(shares > 1 ? shares : 2)), 1024, 0, s>>>(part, lam, part2, rows, g.D);
            if (int st = check_launch(fn)) return st;
            part = part2;
            rows = shares > 1 ? shares : 2;
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
    const GsLayout l = gs_layout(B, T, D);
    const GsArgs g{reset, lens, reinterpret_cast<const float *>(static_cast<char *>(ws) + l.rate), (int)T, (int)B, (int)D, 1, 0, 0, c};
    cudaStream_t s = (cudaStream_t)stream;
    if (int st = gs_setup(fn, ws, l, 0, lam, D, c, s)) return st;
    if (T == 0) {
        if (hT == nullptr) return CLA_OK;
        if (h0 != nullptr) CLA_CUDA_TRY(cudaMemcpyAsync(hT, h0, (size_t)(B * D) * 4, cudaMemcpyDeviceToDevice, s), fn);
        else CLA_CUDA_TRY(cudaMemsetAsync(hT, 0, (size_t)(B * D) * 4, s), fn);
        return CLA_OK;
    }
    if (dtype == CLA_F32) return gs_fwd<float>(fn, x, rgate, igate, h0, h, hT, ckpt, g, ws, l, s);
    if (dtype == CLA_BF16) return gs_fwd<__nv_bfloat16>(fn, x, rgate, igate, h0, h, hT, ckpt, g, ws, l, s);
    return gs_fwd<__half>(fn, x, rgate, igate, h0, h, hT, ckpt, g, ws, l, s);
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
    const GsArgs g{reset, lens, nullptr, (int)T, (int)B, (int)D, 1, 0, 0, c};
    const GsLayout l = gs_layout(B, T, D);
    cudaStream_t s = (cudaStream_t)stream;
    if (B * T == 0) {
        if (dlam != nullptr) CLA_CUDA_TRY(cudaMemsetAsync(dlam, 0, (size_t)D * 4, s), fn);
        if (dh0 != nullptr && B > 0) {
            if (dhT != nullptr) CLA_CUDA_TRY(cudaMemcpyAsync(dh0, dhT, (size_t)(B * D) * 4, cudaMemcpyDeviceToDevice, s), fn);
            else CLA_CUDA_TRY(cudaMemsetAsync(dh0, 0, (size_t)(B * D) * 4, s), fn);
        }
        CLA_CUDA_TRY(cudaMemsetAsync(ws, 0, sizeof(WsHeader), s), fn);
        return CLA_OK;
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
    if (dtype == CLA_F32) return gs_step<float>(fn, x, rgate, igate, lam, reset, h, y, c, B, D, s);
    if (dtype == CLA_BF16) return gs_step<__nv_bfloat16>(fn, x, rgate, igate, lam, reset, h, y, c, B, D, s);
    return gs_step<__half>(fn, x, rgate, igate, lam, reset, h, y, c, B, D, s);
}
