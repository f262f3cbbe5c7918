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
// that take 16 of its values each, both of each pair, so the rotation stays
// within a lane, and in 16-byte pieces beside the neighbouring lanes', so every
// access moves whole sectors.  A block's groups of such lanes take neighbouring
// tokens and walk over their heads together: the sines and cosines are formed
// once for all of them.  Queries come first and
// keys after them, so that one set of weights and sums is held at a time.  Rows
// come through asynchronous copies into a lane's own column of shared memory,
// several rows ahead and without registers.  Arithmetic is on pairs of fp32.
//
// Measured on GB300 (bf16, every pass on other inputs): prefill 1 x 32/8 x
// 32768 x 128 out of a fused projection 105 us for 671 MB (6.4 TB/s, 94% of the
// measured copy rate; loads into registers four rows at a time 147), with
// neighbours as pairs 105 too (147 where a lane's 32 bytes lay in one piece) and
// half of each head rotated 106 (125); training pass 4 x 16/16 x 8192 x 64 115 us
// for 671 MB (5.8 TB/s, 86%): backward 62 of a floor of 59, forward 47 of 40,
// join and the gaps between launches the rest.
//
// Angles: positions reach 2^31 and an angle's 24 bits of fp32 would leave
// nothing of its fraction of a turn.  freq / 2 pi is formed as a 64-bit
// fraction of a turn from the integer product of freq's 24 bits and 2^64 / 2 pi;
// its product with the position wraps around as turns do, and its upper 32 bits
// are the angle: off by less than 2^-31 (1 + |freq|) turns.
#include <float.h>
#include <math.h>

#include "cla_internal.cuh"
#include "elem_io.cuh"
#include "strided.cuh"

namespace cla {
namespace {

// Blocks, chosen for a part with 152 multiprocessors, on which they all run at once: forward 2 for each, backward one (its lanes
// hold 16 sums of dw as well, up to 159 registers; with 128 they went to local memory and the backward took some 100 us where
// it takes 62).  Numbers of their own, not asked of the device: dw's sums are in an order that the sizes alone fix, and a part
// with fewer multiprocessors takes two rounds.
constexpr int kFwdThreads = 256, kFwdBlocks = 304, kBwdThreads = 384, kBwdBlocks = 152;

struct QnArgs {
    const float *w[2], *freq;  // of queries and keys
    const int32_t *pos, *lens;
    float eps, inv_d;
    int T, heads[2], d, rot;
    long long tokens, groups;  // groups: of as many tokens as a block has groups of lanes
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
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 minus(float2 a) { return make_float2(-a.x, -a.y); }

// Sines and cosines of two angles: the nearest quarter turn is taken off the 32-bit fraction of a turn exactly, what is left,
// at most an eighth, goes through the Taylor series (terms up to x^9 and x^8: off by 2e-9 and 2.5e-8), and the quarters say
// which of the two is which and with what sign.
__device__ __forceinline__ void sincos_at(const unsigned long long *turn, int pos, float2 &s, float2 &c) {
    unsigned q[2];
    float left[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const unsigned phase = (unsigned)(turn[i] * (unsigned long long)(long long)pos >> 32);
        q[i] = (phase + 0x20000000u) >> 30;
        left[i] = (float)(int)(phase - (q[i] << 30));
    }
    const float2 x = mul2(make_float2(left[0], left[1]), both(6.283185307179586f * 0x1p-32f)), y = mul2(x, x);
    float2 p = fma2(y, both(1.f / 362880.f), both(-1.f / 5040.f));
    p = fma2(fma2(p, y, both(1.f / 120.f)), y, both(-1.f / 6.f));
    p = fma2(mul2(p, y), x, x);
    float2 r = fma2(y, both(1.f / 40320.f), both(-1.f / 720.f));
    r = fma2(fma2(r, y, both(1.f / 24.f)), y, both(-0.5f));
    r = fma2(r, y, both(1.f));
    const float2 a = make_float2(q[0] & 1u ? r.x : p.x, q[1] & 1u ? r.y : p.y), b = make_float2(q[0] & 1u ? p.x : r.x, q[1] & 1u ? p.y : r.y);
    s = make_float2(__uint_as_float(__float_as_uint(a.x) ^ (q[0] & 2u) << 30), __uint_as_float(__float_as_uint(a.y) ^ (q[1] & 2u) << 30));
    c = make_float2(__uint_as_float(__float_as_uint(b.x) ^ (q[0] + 1u & 2u) << 30),
                    __uint_as_float(__float_as_uint(b.y) ^ (q[1] + 1u & 2u) << 30));
}

__device__ __forceinline__ float2 pair_f32(uint32_t u, __nv_bfloat16) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ float2 pair_f32(uint32_t u, __half) { return __half22float2(reinterpret_cast<__half2 &>(u)); }
__device__ __forceinline__ uint32_t pair_of(float2 v, __nv_bfloat16) {
    const __nv_bfloat162 h = __float22bfloat162_rn(v);
    return reinterpret_cast<const uint32_t &>(h);
}
__device__ __forceinline__ uint32_t pair_of(float2 v, __half) {
    const __half2 h = __float22half2_rn(v);
    return reinterpret_cast<const uint32_t &>(h);
}

// A lane's 16 values of a row: the two that turn into one another are a[i] and b[i], in either half of the rotated values
// or, interleaved, side by side.  v[0 ..]: 16-byte pieces as they lie in memory, the half of them from c0 on, then from c1.
template <typename E, bool IL>
struct Row {
    static constexpr int N = sizeof(E);  // pieces
    float2 a[4], b[4];
    __device__ __forceinline__ void unpack(const uint4 *v) {
        float x[16];
        if constexpr (N == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[4 * i] = __uint_as_float(v[i].x), x[4 * i + 1] = __uint_as_float(v[i].y);
                x[4 * i + 2] = __uint_as_float(v[i].z), x[4 * i + 3] = __uint_as_float(v[i].w);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = pair_f32(u[j], E());
                    x[8 * i + 2 * j] = f.x, x[8 * i + 2 * j + 1] = f.y;
                }
            }
        }
        set(x);
    }
    __device__ __forceinline__ void set(const float *x) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = IL ? make_float2(x[4 * i], x[4 * i + 2]) : make_float2(x[2 * i], x[2 * i + 1]);
            b[i] = IL ? make_float2(x[4 * i + 1], x[4 * i + 3]) : make_float2(x[8 + 2 * i], x[9 + 2 * i]);
        }
    }
    __device__ __forceinline__ void get(float *x) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            (IL ? x[4 * i] : x[2 * i]) = a[i].x, (IL ? x[4 * i + 2] : x[2 * i + 1]) = a[i].y;
            (IL ? x[4 * i + 1] : x[8 + 2 * i]) = b[i].x, (IL ? x[4 * i + 3] : x[9 + 2 * i]) = b[i].y;
        }
    }
    // live: else zeros, whatever the weights have made of the row
    __device__ __forceinline__ void store(E *p, int gap, int apart, bool live) const {
        float x[16];
        get(x);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            uint4 v;
            if constexpr (N == 4) {
                const float *y = x + 4 * i;
                v = make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3]));
            } else {
                const float *y = x + 8 * i;
                v = make_uint4(pair_of(make_float2(y[0], y[1]), E()), pair_of(make_float2(y[2], y[3]), E()),
                               pair_of(make_float2(y[4], y[5]), E()), pair_of(make_float2(y[6], y[7]), E()));
            }
            *reinterpret_cast<uint4 *>(p + (i < N / 2 ? 0 : apart) + (N == 4 && i % 2 ? gap : 0)) = live ? v : make_uint4(0u, 0u, 0u, 0u);
        }
    }
};

// What a lane has of a row: 8 values from c0 on and 8 from c0 + apart on, in fp32 four and four with a gap, so that
// neighbouring lanes' 16-byte pieces lie side by side (32 bytes in a row a lane would make two half sectors of each in
// every access).  Halves as pairs: the lanes of the rotated values have both of a pair, the others equal parts of the rest.
// Neighbours as pairs: equal parts of the row.
template <typename E, int G, bool IL>
struct Lane {
    int sub, c0, gap, apart;
    bool in;
    __device__ Lane(const QnArgs &g) {
        const bool turned = IL || 16 * (threadIdx.x % G) < g.rot;
        const int from = turned ? 0 : g.rot, n = IL ? g.d : turned ? g.rot : g.d - g.rot;  // the values that such lanes share
        sub = threadIdx.x % G;
        in = 16 * sub < g.d;
        c0 = from + (sub - from / 16) * (sizeof(E) == 4 ? 4 : 8);
        gap = sizeof(E) == 4 ? n / 4 : 4;
        apart = n / 2;
    }
    // where the lane's i-th value lies
    __device__ __forceinline__ int at(int i) const { return c0 + (i / 4 % 2) * gap + i / 8 * apart + i % 4; }
    // the frequency of the first of its pairs 2 i and 2 i + 1
    __device__ __forceinline__ int frequency(int i) const { return IL ? at(4 * i) / 2 : at(2 * i); }
    __device__ __forceinline__ void weights(const float *w, Row<E, IL> &x) const {
        float y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = w != nullptr && in ? w[at(i)] : 1.f;
        x.set(y);
    }
};

template <int G>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int x = 1; x < G; x <<= 1) v += __shfl_xor_sync(~0u, v, x);
    return v;
}

// Where a lane is in its block's list of rows: token (b, t), head.  The list has the groups of neighbouring tokens, one for
// every group of lanes of the block, one behind the other, and in each its heads.
template <int G>
struct At {
    long long group;
    int head, b, t;
    bool on, live;  // there is such a token; it is of its sequence
    __device__ void token(const QnArgs &g, bool ahead) {  // ahead: of the group before, b and t are known
        const int step = blockDim.x / G;
        const long long n = group * step + threadIdx.x / G;
        on = n < g.tokens;
        if (ahead && step <= g.T) {
            if (t >= g.T - step) t -= g.T - step, ++b;
            else t += step;
        } else {
            b = (int)((unsigned)n / (unsigned)g.T), t = (int)((unsigned)n % (unsigned)g.T);
        }
        if (!on) b = 0, t = 0;  // and stays so: what follows is not on either
        live = on && (g.lens == nullptr || t < g.lens[b]);
    }
    __device__ At(const QnArgs &g, long long unit, int heads) : group(unit / heads), head((int)(unit % heads)) { token(g, false); }
    // to the next row: true where that is of another group
    __device__ __forceinline__ bool next(const QnArgs &g, int heads) {
        if (++head < heads) return false;
        head = 0, ++group;
        token(g, true);
        return true;
    }
};

// Rows on their way to a lane: 16-byte pieces in shared memory, in the lane's own column of a stage.
template <int THREADS, int STAGES, int PIECES>
struct Queue {
    static constexpr int BYTES = STAGES * PIECES * THREADS * 16;
    uint32_t base;
    __device__ __forceinline__ Queue(const void *smem) : base((uint32_t)__cvta_generic_to_shared(smem) + 16 * threadIdx.x) {}
    __device__ __forceinline__ uint32_t at(int stage, int piece) const { return base + (stage * PIECES + piece) * (THREADS * 16); }
    template <typename E>
    __device__ __forceinline__ void put(int stage, int first, const E *p, int gap, int apart, bool in) const {  // zeros where it is not in
#pragma unroll
        for (int i = 0; i < (int)sizeof(E); ++i)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at(stage, first + i)),
                         "l"(p + (i < (int)sizeof(E) / 2 ? 0 : apart) + (sizeof(E) == 4 && i % 2 ? gap : 0)), "r"(in ? 16 : 0)
                         : "memory");
    }
    __device__ __forceinline__ static void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    __device__ __forceinline__ static void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory"); }
    __device__ __forceinline__ uint4 get(int stage, int piece) const {
        uint4 v;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(at(stage, piece))
                     : "memory");
        return v;
    }
};

template <typename T>
__device__ __forceinline__ T pick(const T (&a)[2], int which) { return which == 0 ? a[0] : a[1]; }

// Sines and cosines of the lane's 8 angles at its token.
template <typename E, int G, bool IL>
__device__ __forceinline__ void angles(const QnArgs &g, const Lane<E, G, IL> &l, const At<G> &a, const unsigned long long *s_turn,
                                       float2 *s, float2 *c) {
    const int pos = !a.live ? 0 : g.pos != nullptr ? g.pos[(long long)a.b * g.T + a.t] : a.t;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s[i] = both(0.f), c[i] = both(1.f);
        const int f = l.frequency(i);
        if (2 * f < g.rot) sincos_at(s_turn + f, pos, s[i], c[i]);
    }
}

// The block's equal share of the list of all rows, queries before keys.
struct Share {
    long long at, end;
    __device__ Share(long long all) {
        const long long w = blockIdx.x, n = gridDim.x;
        at = all / n * w + (all % n) * w / n;
        end = all / n * (w + 1) + (all % n) * (w + 1) / n;
    }
};

struct QnFwd {
    const void *x[2];
    void *o[2];
    Triple sx[2], so[2];
};

template <typename E>
constexpr int qn_fwd_stages() { return sizeof(E) == 4 ? 4 : 8; }
template <typename E>
constexpr int qn_bwd_stages() { return 2; }

template <typename E, int G, bool IL>
__global__ void __launch_bounds__(kFwdThreads, 2) qn_fwd_kernel(QnFwd p, QnArgs g) {
    constexpr int S = qn_fwd_stages<E>(), N = Row<E, IL>::N;
    extern __shared__ __align__(16) char smem[];
    __shared__ unsigned long long s_turn[128];
    const Queue<kFwdThreads, S, N> queue(smem);
    const Lane<E, G, IL> l(g);
    for (int i = threadIdx.x; i < g.rot / 2; i += kFwdThreads) s_turn[i] = turns(g.freq[i]);
    const Share share(g.groups * (g.heads[0] + g.heads[1]));
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const int heads = pick(g.heads, which);
        const long long base = which == 0 ? 0 : g.groups * g.heads[0];
        const long long lo = max(share.at, base), hi = min(share.end, base + g.groups * heads);
        if (lo >= hi) continue;
        const Triple sx = pick(p.sx, which), so = pick(p.so, which);
        const E *x = static_cast<const E *>(pick(p.x, which)) + l.c0;
        E *o = static_cast<E *>(pick(p.o, which)) + l.c0;
        At<G> f(g, lo - base, heads), c = f;
        const E *xf = x + f.b * sx.b + f.t * sx.t + f.head * sx.h;
        E *oc = o + c.b * so.b + c.t * so.t + c.head * so.h;
        int left = (int)(hi - lo), coming = left;  // rows to be finished, to be asked for
        auto fetch = [&](int stage) {
            if (coming > 0) {
                queue.put(stage, 0, xf, l.gap, l.apart, f.live && l.in);
                xf += sx.h;
                if (--coming > 0 && f.next(g, heads)) xf = x + f.b * sx.b + f.t * sx.t;
            }
            queue.commit();
        };
#pragma unroll 1
        for (int i = 0; i < S; ++i) fetch(i);
        // w_a cos, w_b sin, w_b cos, w_a sin
        float2 wac[4], wbs[4], wbc[4], was[4];
        Row<E, IL> w;
        l.weights(pick(g.w, which), w);
        auto coefficients = [&]() {
            angles(g, l, c, s_turn, was, wac);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                wbs[i] = mul2(w.b[i], minus(was[i])), wbc[i] = mul2(w.b[i], wac[i]);
                was[i] = mul2(w.a[i], was[i]), wac[i] = mul2(w.a[i], wac[i]);
            }
        };
        int stage = 0;
        Row<E, IL> y, z;
        float r = 0.f, r1 = 0.f;
        auto begin = [&](Row<E, IL> &v, float &r) {  // the next row, and its reciprocal root
            queue.wait();
            uint4 u[N];
#pragma unroll
            for (int i = 0; i < N; ++i) u[i] = queue.get(stage, i);
            fetch(stage);
            stage = stage + 1 == S ? 0 : stage + 1;
            v.unpack(u);
            float2 q = both(0.f), q1 = both(0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) q = fma2(v.a[i], v.a[i], q), q1 = fma2(v.b[i], v.b[i], q1);
            r = rsqrtf(row_sum<G>(q.x + q.y + (q1.x + q1.y)) * g.inv_d + g.eps);
        };
        begin(y, r);
        __syncthreads();  // s_turn is there
        coefficients();
        auto finish = [&](Row<E, IL> &v, float r) {  // true behind the last row
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 a = mul2(v.a[i], both(r)), b = mul2(v.b[i], both(r));
                v.a[i] = fma2(a, wac[i], mul2(b, wbs[i]));
                v.b[i] = fma2(b, wbc[i], mul2(a, was[i]));
            }
            if (c.on && l.in) v.store(oc, l.gap, l.apart, c.live);
            if (--left == 0) return true;
            oc += so.h;
            if (c.next(g, heads)) {
                oc = o + c.b * so.b + c.t * so.t;
                coefficients();
            }
            return false;
        };
        // a row begins beside the end of the one before it; behind the last, with what an old stage holds
#pragma unroll 1
        while (true) {
            begin(z, r1);
            if (finish(y, r)) break;
            begin(y, r);
            if (finish(z, r1)) break;
        }
    }
}

struct QnBwd {
    const void *x[2], *g[2];
    void *dx[2];
    Triple sx[2], sg[2], sdx[2];
};

// Sums of many rows go to pairs of fp32, 48 bits: x the sum, y what its roundings have left.
__device__ __forceinline__ void add(float2 &s, float v) {
    const float t = __fadd_rn(s.x, v), b = __fsub_rn(t, s.x);
    s.y = __fadd_rn(s.y, __fadd_rn(__fsub_rn(s.x, __fsub_rn(t, b)), __fsub_rn(v, b)));
    s.x = t;
}
__device__ __forceinline__ void add(float2 &s, float2 v) {
    add(s, v.x);
    s.y = __fadd_rn(s.y, v.y);
}
__device__ __forceinline__ float total(float2 s) { return fabsf(s.x) <= FLT_MAX ? s.x + s.y : s.x; }  // an infinity stays one

// The sums of 16 values over the lanes of a warp that have the same columns (lane % G alike), scattered: a lane is left with
// those of its values first, first + 1, ... in v[0 .. N), with G = 1 two lanes with the same one.
template <int G>
struct Scatter {
    static constexpr int N = G > 2 ? G / 2 : 1;
    static __device__ __forceinline__ int first(int lane) {
        int at = 0;
#pragma unroll
        for (int x = 16, n = 8; x >= G && n > 0; x >>= 1, n >>= 1) at += lane & x ? n : 0;
        return at;
    }
    static __device__ __forceinline__ void sum(float (&v)[16], int lane) {
#pragma unroll
        for (int x = 16, n = 8; x >= G; x >>= 1, n >>= 1) {
            const bool up = lane & x;
            if (n == 0) v[0] += __shfl_xor_sync(~0u, v[0], x);
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float give = up ? v[i] : v[i + n];
                v[i] = (up ? v[i + n] : v[i]) + __shfl_xor_sync(~0u, give, x);
            }
        }
    }
};

// A block leaves its rows' sums of dw in parts[block][2][d].  A lane adds kBwdRows rows at most in fp32, one after the other;
// the warp's sums of them, the warps' and the blocks' go to pairs of fp32 (fp64 runs at a small share of fp32's rate here).  All
// in fp32, 2300 rows a lane that are alike left 6 times what 64 rows can.
constexpr int kBwdRows = 64;
template <typename E, int G, bool IL>
__global__ void __launch_bounds__(kBwdThreads, 1) qn_bwd_kernel(QnBwd p, QnArgs g, float2 *parts, WsHeader *hdr) {
    constexpr int S = qn_bwd_stages<E>(), N = Row<E, IL>::N, W = kBwdThreads / 32;
    extern __shared__ __align__(16) char smem[];
    __shared__ unsigned long long s_turn[128];
    __shared__ float2 s_w[W][G * 16];
    const Queue<kBwdThreads, S, 2 * N> queue(smem);
    const Lane<E, G, IL> l(g);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, first = Scatter<G>::first(lane);
    const bool owner = l.in && (G > 1 || lane % 2 == 0);  // of the sums that it is left with
    if (blockIdx.x == 0 && threadIdx.x < (int)sizeof(WsHeader) / 4) reinterpret_cast<uint32_t *>(hdr)[threadIdx.x] = 0u;  // nothing waits
    for (int i = threadIdx.x; i < g.rot / 2; i += kBwdThreads) s_turn[i] = turns(g.freq[i]);
    const Share share(g.groups * (g.heads[0] + g.heads[1]));
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const int heads = pick(g.heads, which);
        const long long base = which == 0 ? 0 : g.groups * g.heads[0];
        const long long lo = max(share.at, base), hi = min(share.end, base + g.groups * heads);
#pragma unroll
        for (int i = 0; i < Scatter<G>::N; ++i)
            if (owner) s_w[warp][l.at(first + i)] = both(0.f);
        if (lo < hi) {
            const Triple sx = pick(p.sx, which), sg = pick(p.sg, which), sd = pick(p.sdx, which);
            const E *x = static_cast<const E *>(pick(p.x, which)) + l.c0, *y = static_cast<const E *>(pick(p.g, which)) + l.c0;
            E *d = static_cast<E *>(pick(p.dx, which)) + l.c0;
            At<G> f(g, lo - base, heads), c = f;
            const E *xf = x + f.b * sx.b + f.t * sx.t + f.head * sx.h, *yf = y + f.b * sg.b + f.t * sg.t + f.head * sg.h;
            E *dc = d + c.b * sd.b + c.t * sd.t + c.head * sd.h;
            int left = (int)(hi - lo), coming = left;
            auto fetch = [&](int stage) {
                if (coming > 0) {
                    queue.put(stage, 0, xf, l.gap, l.apart, f.live && l.in);
                    queue.put(stage, N, yf, l.gap, l.apart, f.live && l.in);
                    xf += sx.h, yf += sg.h;
                    if (--coming > 0 && f.next(g, heads)) xf = x + f.b * sx.b + f.t * sx.t, yf = y + f.b * sg.b + f.t * sg.t;
                }
                queue.commit();
            };
#pragma unroll 1
            for (int i = 0; i < S; ++i) fetch(i);
            Row<E, IL> w;
            l.weights(pick(g.w, which), w);
            float2 sn[4], cs[4];
            __syncthreads();  // s_turn is there
            angles(g, l, c, s_turn, sn, cs);
            int stage = 0;
#pragma unroll 1
            while (left > 0) {
                Row<E, IL> acc;
#pragma unroll
                for (int i = 0; i < 4; ++i) acc.a[i] = acc.b[i] = both(0.f);
#pragma unroll 1
                for (const int end = max(left - kBwdRows, 0); left > end; --left) {
                    queue.wait();
                    uint4 v[N], u[N];
#pragma unroll
                    for (int i = 0; i < N; ++i) v[i] = queue.get(stage, i), u[i] = queue.get(stage, N + i);
                    fetch(stage);
                    stage = stage + 1 == S ? 0 : stage + 1;
                    Row<E, IL> z, e;
                    z.unpack(v);
                    e.unpack(u);
                    float2 q = both(0.f), m = both(0.f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 t = e.a[i];  // turned back
                        e.a[i] = fma2(t, cs[i], mul2(e.b[i], sn[i]));
                        e.b[i] = fma2(e.b[i], cs[i], mul2(t, minus(sn[i])));
                        q = fma2(z.a[i], z.a[i], q), q = fma2(z.b[i], z.b[i], q);
                        m = fma2(mul2(e.a[i], w.a[i]), z.a[i], m), m = fma2(mul2(e.b[i], w.b[i]), z.b[i], m);
                    }
                    const float r = rsqrtf(row_sum<G>(q.x + q.y) * g.inv_d + g.eps), k = row_sum<G>(m.x + m.y) * g.inv_d * r * r;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acc.a[i] = fma2(mul2(e.a[i], both(r)), z.a[i], acc.a[i]);
                        acc.b[i] = fma2(mul2(e.b[i], both(r)), z.b[i], acc.b[i]);
                        z.a[i] = mul2(both(r), fma2(z.a[i], both(-k), mul2(e.a[i], w.a[i])));
                        z.b[i] = mul2(both(r), fma2(z.b[i], both(-k), mul2(e.b[i], w.b[i])));
                    }
                    if (c.on && l.in) z.store(dc, l.gap, l.apart, c.live);
                    dc += sd.h;
                    if (left > 1 && c.next(g, heads)) {
                        dc = d + c.b * sd.b + c.t * sd.t;
                        angles(g, l, c, s_turn, sn, cs);
                    }
                }
                float v[16];
                acc.get(v);
                Scatter<G>::sum(v, lane);
#pragma unroll
                for (int i = 0; i < Scatter<G>::N; ++i)
                    if (owner) add(s_w[warp][l.at(first + i)], v[i]);
            }
        }
        // the join may take its place; it waits for this grid's end
        if (which == 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        __syncthreads();
        for (int i = threadIdx.x; i < g.d; i += kBwdThreads) {
            float2 v = s_w[0][i];
#pragma unroll
            for (int x = 1; x < W; ++x) add(v, s_w[x][i]);
            parts[((long long)blockIdx.x * 2 + which) * g.d + i] = v;
        }
        __syncthreads();  // the warps' sums have been read
    }
}

// dw = the blocks' parts, in a fixed order: 16 threads take every 16th of a column's.  It starts while the backward still
// writes them, so they are no memory that stays as it is for the kernel's life: no __restrict__.
__global__ void __launch_bounds__(256) qn_join_kernel(const float2 *parts, float *dwq, float *dwk, int d, int blocks) {
    __shared__ float2 s[16][16];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int x = threadIdx.x % 16, col = blockIdx.x * 16 + x, y = threadIdx.x / 16;
    float2 v = both(0.f);
#pragma unroll 5
    for (int i = y; i < blocks; i += 16) add(v, parts[(long long)i * 2 * d + col]);
    s[y][x] = v;
    __syncthreads();
    if (y == 0) {
#pragma unroll
        for (int i = 1; i < 16; ++i) add(v, s[i][x]);
        float *to = col < d ? dwq : dwk;
        if (to != nullptr) to[col < d ? col : col - d] = total(v);
    }
}

// ------------------------------------------------------------------ host
int qn_check(const char *fn, int64_t B, int64_t H, int64_t Hkv, int64_t T, int64_t d, int64_t rot, float eps, int dtype) {
    if (B < 0 || H < 0 || Hkv < 0 || T < 0 || d < 0 || rot < 0) return fail(CLA_ERR_INVALID_ARG, "%s: negative size", fn);
    if (!(eps > 0.f) || !isfinite(eps)) return fail(CLA_ERR_INVALID_ARG, "%s: eps must be a positive finite number", fn);
    if (rot > d) return fail(CLA_ERR_INVALID_ARG, "%s: %lld rotated values of a head of %lld", fn, (long long)rot, (long long)d);
    if (dtype_bytes(dtype) == 0) return fail(CLA_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
    if (d < 16 || d > 256 || d % 16 != 0 || rot % 16 != 0)
        return fail(CLA_ERR_UNSUPPORTED, "%s: head dimension %lld with %lld rotated: multiples of 16 up to 256 are needed", fn,
                    (long long)d, (long long)rot);
    if (!product_below({B, T}, 2147483648.0) || !product_below({H + Hkv}, 1 << 20) || !product_below({B, T, H + Hkv}, 68719476736.0))
        return fail(CLA_ERR_UNSUPPORTED, "%s: sizes too large", fn);
    return CLA_OK;
}

int qn_lanes(int64_t d) {
    int n = 1;
    while (16 * n < d) n *= 2;
    return n;
}

QnArgs qn_args(const float *wq, const float *wk, const float *freq, const int32_t *pos, const int32_t *lens, float eps, int64_t rot,
               int64_t B, int64_t H, int64_t Hkv, int64_t T, int64_t d, int threads) {
    QnArgs g = {};
    g.w[0] = wq, g.w[1] = wk, g.freq = freq, g.pos = pos, g.lens = lens;
    g.eps = eps, g.inv_d = 1.f / (float)d;
    g.T = (int)T, g.heads[0] = (int)H, g.heads[1] = (int)Hkv, g.d = (int)d, g.rot = (int)rot;
    g.tokens = B * T;
    const long long per = threads / qn_lanes(d);
    g.groups = (g.tokens + per - 1) / per;
    return g;
}

// Blocks that run at once, each with one row of each of its lanes' at least; forward as many rounds of them as give each
// 16, so that multiprocessors that are further from memory take fewer (1 x 32/8 x 32768 x 128: 105 us with 8 rounds against
// 116 with one, 107 with 4 or 16, 143 with 33; 4/1 heads x 65536 x 128 with the backward: 99 with 2, 105 with one, 103 with 4).
unsigned qn_fwd_blocks(const QnArgs &g) {
    const long long n = g.groups * (g.heads[0] + g.heads[1]), rounds = n / (16 * kFwdBlocks);
    return (unsigned)(n < kFwdBlocks ? n : rounds < 1 ? kFwdBlocks : rounds < 4096 ? rounds * kFwdBlocks : 4096 * kFwdBlocks);
}

unsigned qn_bwd_blocks(const QnArgs &g) {
    const long long n = g.groups * (g.heads[0] + g.heads[1]);
    return (unsigned)(n < kBwdBlocks ? n : kBwdBlocks);
}

template <typename E, int G, bool IL>
int qn_fwd_g(const char *fn, const QnFwd &p, const QnArgs &g, cudaStream_t s) {
    static std::atomic<unsigned long long> done{0};
    constexpr int smem = Queue<kFwdThreads, qn_fwd_stages<E>(), Row<E, IL>::N>::BYTES;
    if (int st = set_max_dynamic_smem(done, (const void *)qn_fwd_kernel<E, G, IL>, smem)) return st;
    qn_fwd_kernel<E, G, IL><<<qn_fwd_blocks(g), kFwdThreads, smem, s>>>(p, g);
    return check_launch(fn);
}

template <typename E, bool IL>
int qn_fwd(const char *fn, const QnFwd &p, const QnArgs &g, cudaStream_t s) {
    switch (qn_lanes(g.d)) {
        case 1: return qn_fwd_g<E, 1, IL>(fn, p, g, s);
        case 2: return qn_fwd_g<E, 2, IL>(fn, p, g, s);
        case 4: return qn_fwd_g<E, 4, IL>(fn, p, g, s);
        case 8: return qn_fwd_g<E, 8, IL>(fn, p, g, s);
        default: return qn_fwd_g<E, 16, IL>(fn, p, g, s);
    }
}

template <typename E, int G, bool IL>
int qn_bwd_g(const char *fn, const QnBwd &p, const QnArgs &g, float2 *parts, cudaStream_t s) {
    static std::atomic<unsigned long long> done{0};
    constexpr int smem = Queue<kBwdThreads, qn_bwd_stages<E>(), 2 * Row<E, IL>::N>::BYTES;
    if (int st = set_max_dynamic_smem(done, (const void *)qn_bwd_kernel<E, G, IL>, smem)) return st;
    qn_bwd_kernel<E, G, IL><<<qn_bwd_blocks(g), kBwdThreads, smem, s>>>(p, g, parts, reinterpret_cast<WsHeader *>(parts) - 1);
    return check_launch(fn);
}

template <typename E, bool IL>
int qn_bwd(const char *fn, const QnBwd &p, const QnArgs &g, float *dwq, float *dwk, float2 *parts, cudaStream_t s) {
    int st;
    switch (qn_lanes(g.d)) {
        case 1: st = qn_bwd_g<E, 1, IL>(fn, p, g, parts, s); break;
        case 2: st = qn_bwd_g<E, 2, IL>(fn, p, g, parts, s); break;
        case 4: st = qn_bwd_g<E, 4, IL>(fn, p, g, parts, s); break;
        case 8: st = qn_bwd_g<E, 8, IL>(fn, p, g, parts, s); break;
        default: st = qn_bwd_g<E, 16, IL>(fn, p, g, parts, s);
    }
    if (st != CLA_OK || (dwq == nullptr && dwk == nullptr)) return st;
    // the join's launch goes beside the backward's end
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at;
    cfg.gridDim = dim3((unsigned)(2 * g.d / 16));  // d is a multiple of 16
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    CLA_CUDA_TRY(cudaLaunchKernelEx(&cfg, qn_join_kernel, (const float2 *)parts, dwq, dwk, g.d, (int)qn_bwd_blocks(g)), fn);
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
    const QnArgs g = qn_args(wq, wk, freq, pos, lens, eps, rot, B, H, Hkv, T, d, kFwdThreads);
    const QnFwd p = {{q, k}, {qo, ko}, {r[0], r[1]}, {r[2], r[3]}};
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == CLA_F32) return interleaved ? qn_fwd<float, true>(fn, p, g, s) : qn_fwd<float, false>(fn, p, g, s);
    if (dtype == CLA_BF16) return interleaved ? qn_fwd<__nv_bfloat16, true>(fn, p, g, s) : qn_fwd<__nv_bfloat16, false>(fn, p, g, s);
    return interleaved ? qn_fwd<__half, true>(fn, p, g, s) : qn_fwd<__half, false>(fn, p, g, s);
}

extern "C" size_t cla_qk_norm_rope_bwd_workspace_size(int64_t B, int64_t H, int64_t Hkv, int64_t T, int64_t d) {
    if (qn_check("cla_qk_norm_rope_bwd_workspace_size", B, H, Hkv, T, d, 0, 1.f, CLA_F32) != CLA_OK) return 0;
    return sizeof(WsHeader) + (size_t)kBwdBlocks * 2 * d * sizeof(float2);
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
        CLA_CUDA_TRY(cudaMemsetAsync(ws, 0, sizeof(WsHeader), s), fn);
        if (dwq) CLA_CUDA_TRY(cudaMemsetAsync(dwq, 0, d * 4, s), fn);
        if (dwk) CLA_CUDA_TRY(cudaMemsetAsync(dwk, 0, d * 4, s), fn);
        return CLA_OK;
    }
    const QnArgs g = qn_args(wq, wk, freq, pos, lens, eps, rot, B, H, Hkv, T, d, kBwdThreads);
    const QnBwd p = {{q, k}, {dqo, dko}, {dq, dk}, {r[0], r[1]}, {r[2], r[3]}, {r[4], r[5]}};
    float2 *parts = reinterpret_cast<float2 *>(static_cast<WsHeader *>(ws) + 1);
    if (dtype == CLA_F32)
        return interleaved ? qn_bwd<float, true>(fn, p, g, dwq, dwk, parts, s) : qn_bwd<float, false>(fn, p, g, dwq, dwk, parts, s);
    if (dtype == CLA_BF16)
        return interleaved ? qn_bwd<__nv_bfloat16, true>(fn, p, g, dwq, dwk, parts, s)
                           : qn_bwd<__nv_bfloat16, false>(fn, p, g, dwq, dwk, parts, s);
    return interleaved ? qn_bwd<__half, true>(fn, p, g, dwq, dwk, parts, s) : qn_bwd<__half, false>(fn, p, g, dwq, dwk, parts, s);
}
