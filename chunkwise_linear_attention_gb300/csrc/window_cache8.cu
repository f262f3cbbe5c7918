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
// The step is bound by reading the cache once.  The list of all blocks of slots
// that hold tokens, over sequences and key heads, is cut into equal shares, one
// for every thread block that runs at once, whatever the lengths: shares by
// whole pairs left a third of the GPU idle at 512 pairs (146 us against 91).  A
// warp takes 16 slots of each block of its thread block's share, which come
// through a ring of asynchronous copies, into the operands of m16n8k16 products:
//   scores^T [16 slots x 8 heads] = K Q^T,  o^T [16 columns x 8 heads] += V^T P^T.
// A pair that lies within a share is finished by its thread block; the parts of
// one that is cut go to the workspace and are added by a second kernel, which is
// launched beside the first and waits for its end.
//
// e4m3 numbers turn into fp16 exactly, two with one instruction.  Queries turn
// into fp16 too, each head's by a power of two of its own under which its
// largest lies in [1, 2): exact for bf16 down to 2^-14 of that, and off by less
// than 2^-25 of it below.
//
// The factors of v's blocks may lie 2^184 apart, so no weight is taken together
// with one.  The total is held against the running maximum m of the scores
// alone.  A tile's weights go into its product as 2^(s - t + 15), t the largest
// score of its 16 slots, in two fp16 parts: off by 2^-22 of themselves at most,
// or 2^-40 of the tile's largest, and no number of the tile is 2^18 above
// another that e4m3 has not rounded to zero.  (One part would leave 2^-11.)  Up
// to four heads leave columns 4 to 7 of the product free: the second parts go
// there, and one product does for both.  The product is added to the sums in
// fp32 times f 2^(t - m - 15); the sums are held at 2^-32 of their value, so that
// they stay finite whatever the number of slots.  Weights below 2^-110 of the
// largest may count as nothing, much as in any fp32 softmax, and 2^-90 of a sum
// may be lost for every tile, where what is added leaves fp32's normal range.
//
// Measured on GB300: 64 x 32/8 x 128, window 4096, sinks 4, bf16: 92 us for 539
// MB (5.9 TB/s, 87% of the measured copy rate); 2 x 32/4 x 128, window 65536:
// 33 us, of which the stream of 134 MB is 20 and the rest the start, the parts
// and the join; 4 x 16/4, window 1024: 12 us; 64 x 64/4 x 128, window 4096: 71
// us for 269 MB, where the products of 16 heads in two parts bound it.
//   Against the first case's 91 us with weights in one part and the factors in
// their exponents: two thread blocks a multiprocessor and tiles four deep; three
// with three or four deep 95 and 97 us, two of five and six deep 93 and 94.
// Scores formed a block ahead of their weights changed nothing (92 us), more
// shares than blocks that run at once cost their starts (97 us at twice as many).
#include <float.h>
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
// A block of threads per block of slots, of k or of v, its values in registers as they come: 8 pieces a thread on their way.
template <bool BF>
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
    if constexpr (BF) {
        const __nv_bfloat162 m = __hmax2(reinterpret_cast<__nv_bfloat162 &>(a), __habs2(reinterpret_cast<__nv_bfloat162 &>(b)));
        return reinterpret_cast<const uint32_t &>(m);
    } else {
        const __half2 m = __hmax2(reinterpret_cast<__half2 &>(a), __habs2(reinterpret_cast<__half2 &>(b)));
        return reinterpret_cast<const uint32_t &>(m);
    }
}
template <typename E, int D>
__global__ void __launch_bounds__(128) c8_write_kernel(const E *k, const E *v, const int32_t *lens, uint8_t *kc, uint8_t *vc, float *kf,
                                                       float *vf, Triple sk, Triple sv, int Hkv, int T, unsigned window, int sinks,
                                                       int blocks) {
    constexpr bool BF = std::is_same<E, __nv_bfloat16>::value;
    constexpr int P = D / 16, N = kC8Block * P / 128;  // pieces of 16 values of a slot, of a thread
    __shared__ float s_top[4];
    const long long S = (long long)sinks + window;
    const unsigned bh = blockIdx.x / (unsigned)blocks;
    const int first = (int)(blockIdx.x % (unsigned)blocks) * kC8Block;
    const int h = (int)(bh % (unsigned)Hkv), b = (int)(bh / (unsigned)Hkv), n = lens == nullptr ? T : min(max(lens[b], 0), T);
    if (first >= n) return;  // no token reaches the block
    const bool of_v = blockIdx.y != 0;
    const Triple st = of_v ? sv : sk;
    const E *x = (of_v ? v : k) + b * st.b + h * st.h;
    uint4 val[N][2];
    bool held[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int at = threadIdx.x + 128 * i, slot = first + at / P;
        long long p = slot;  // the last token that falls on the slot
        if (slot >= sinks && slot < n) p += (unsigned)(n - 1 - slot) / window * (long long)window;
        held[i] = slot < S && slot < n;
        const uint4 *row = reinterpret_cast<const uint4 *>(x + p * st.t) + 2 * (at % P);
        val[i][0] = held[i] ? __ldcs(row) : make_uint4(0u, 0u, 0u, 0u);
        val[i][1] = held[i] ? __ldcs(row + 1) : make_uint4(0u, 0u, 0u, 0u);
    }
    uint32_t most = 0u;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint4 w = val[i][e];
            most = max_abs2<BF>(max_abs2<BF>(max_abs2<BF>(max_abs2<BF>(most, w.x), w.y), w.z), w.w);
        }
    const float2 two = unpack16<BF>(most);
    float top = fmaxf(two.x, two.y);
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, w));
    if (threadIdx.x % 32 == 0) s_top[threadIdx.x / 32] = top;
    __syncthreads();
    const float f = factor_of(fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]))), by = inverse(f);
    uint4 *to = reinterpret_cast<uint4 *>((of_v ? vc : kc) + (bh * S + first) * D) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint4 y = val[i][e / 2];
            const float2 p = unpack16<BF>(e % 2 ? y.z : y.x), q = unpack16<BF>(e % 2 ? y.w : y.y);
            w[e] = e4m3x2(p.x * by, p.y * by) | e4m3x2(q.x * by, q.y * by) << 16;
        }
        if (held[i]) to[128 * i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (threadIdx.x == 0) (of_v ? vf : kf)[blockIdx.x] = f;
}

// ------------------------------------------------------------------ one token
// A thread block's share of the work is an equal piece of the list of all blocks of slots that hold tokens, (sequence,
// key head, block) in this order: segments of (sequence, key head) pairs, of which at most the first and the last are cut.
constexpr int kC8MaxBlocks = 608;  // thread blocks of the step at most: 4 for each of 152 multiprocessors

struct Step8Args {
    const int32_t *pos;
    float c;  // scale log2 e
    long long window, sinks, slots;
    int B, H, Hkv, blocks;  // blocks: of slots, of a sequence and key head
    Triple sq, sk, sv;
};

// What the join has to do for a thread block's last segment: add to its part those of the blocks up to `last`.
struct Cut8 {
    int unit, slot, last, all;  // unit: sequence Hkv + key head, or -1: nothing to do; all: blocks of slots in the list
};
// Where thread block `c`'s share of the list begins: all c / blocks, rounded down (c is at most 608).
__device__ __forceinline__ unsigned share_of(unsigned all, unsigned c) { return all / gridDim.x * c + all % gridDim.x * c / gridDim.x; }

__device__ __forceinline__ long long held_slots(const Step8Args &g, int b) { return max(0ll, min((long long)g.pos[b] + 1, g.slots)); }
__device__ __forceinline__ int held_blocks(const Step8Args &g, int b) { return (int)((held_slots(g, b) + kC8Block - 1) / kC8Block); }

// Sum over a block's threads, and what the threads before this one add to it.
__device__ __forceinline__ unsigned block_scan(unsigned v, unsigned &before, unsigned *s_sum) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    unsigned up = v;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const unsigned y = __shfl_up_sync(~0u, up, x);
        if (lane >= x) up += y;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = up;
    __syncthreads();
    unsigned all = 0;
    before = up - v;
#pragma unroll
    for (int w = 0; w < kStepWarps; ++w) {
        if (w < warp) before += s_sum[w];
        all += s_sum[w];
    }
    return all;
}

// Where 16-byte piece c of slot s lies in a warp's tile.  K's reads take pieces j (or 4 + j) of slots 2i, 2i + 1 at
// once, V's piece r of four even (or odd) slots: the exclusive or with these keeps either apart in the banks.
template <int D>
__device__ __forceinline__ uint32_t tile_at(int s, int c) {
    return D == 128 ? s * 128 + ((c ^ (s & 6) ^ ((s & 1) << 2)) << 4) : s * 64 + ((c ^ (s >> 1 & 3)) << 4);
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}

// four e4m3 numbers without their signs; 0 for a NaN
__device__ __forceinline__ uint32_t size4(uint32_t w) {
    w &= 0x7f7f7f7fu;
    return w & ~__vcmpeq4(w, 0x7f7f7f7fu);
}
// The token into the block of slots that the warps' tiles (K's 16 slots, then V's) hold, and into the caches: `row` of this
// warp's 16 slots is its own, where that is one of them, and the first n of them hold tokens.  All threads of the block
// call it together.  kfac, vfac: the block's factors, before and after.
template <typename E, int D>
__device__ __forceinline__ void put_token(uint32_t tile, uint8_t *kc, uint8_t *vc, float *kf, float *vf, const E (*s_new)[D], int row,
                                          int n, float &kfac, float &vfac, float (*s_top)[kStepWarps]) {
    constexpr int P = D / 16, R = 32 / P;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, c = lane % P;
    __syncthreads();  // s_new is there
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        uint32_t most = 0u;
#pragma unroll
        for (int x = 0; x < 16 / R; ++x) {
            const int s = lane / P + R * x;
            const uint4 w = lds16(tile + which * 16 * D + tile_at<D>(s, c));
            if (s != row) most = __vmaxu4(most, __vmaxu4(__vmaxu4(size4(w.x), size4(w.y)), __vmaxu4(size4(w.z), size4(w.w))));
        }
        most = __vmaxu4(most, most >> 16);
        most = max(most & 0xffu, most >> 8 & 0xffu);
        float val[16], top = 0.f;
        load16(s_new[which] + 16 * c, val);
#pragma unroll
        for (int j = 0; j < 16; ++j) top = fmaxf(top, fabsf(val[j]));
        if (most != 0u) top = fmaxf(top, unpack16<false>(f16x2_of(most)).x * (which == 0 ? kfac : vfac));
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
        if (lane == 0) s_top[which][warp] = top;
    }
    __syncthreads();
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const float *tops = s_top[which];
        const float old = which == 0 ? kfac : vfac, f = factor_of(fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]))), by = inverse(f);
        uint8_t *to = which == 0 ? kc : vc;
#pragma unroll 1
        for (int s = lane / P; s < 16; s += R) {
            if (s != row && (s >= n || f == old)) continue;
            float val[16];
            if (s == row) {
                load16(s_new[which] + 16 * c, val);
            } else {
                decode16(lds16(tile + which * 16 * D + tile_at<D>(s, c)), val);
#pragma unroll
                for (int j = 0; j < 16; ++j) val[j] *= old;
            }
            const uint4 code = code16(val, by);
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(tile + which * 16 * D + tile_at<D>(s, c)), "r"(code.x),
                         "r"(code.y), "r"(code.z), "r"(code.w)
                         : "memory");
            *reinterpret_cast<uint4 *>(to + s * D + 16 * c) = code;
        }
        if (threadIdx.x == 0) *(which == 0 ? kf : vf) = f;
        (which == 0 ? kfac : vfac) = f;
    }
    __syncwarp();
}

// acc += x times what belongs to its column
__device__ __forceinline__ void add_times(float (&acc)[4], const float (&x)[4], float2 by) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const float2 v = __ffma2_rn(make_float2(x[i], x[i + 1]), by, make_float2(acc[i], acc[i + 1]));
        acc[i] = v.x, acc[i + 1] = v.y;
    }
}

constexpr int kC8Stages = 4;  // tiles of a warp on their way

// NH query heads at once are the columns of NG products; four are in either half of one's.
template <int NH>
constexpr int c8_groups() { return NH <= 8 ? 1 : NH / 8; }
template <int D, int NH>
constexpr int c8_smem() {
    return kStepWarps * (kC8Stages * 32 * D + 8 * c8_groups<NH>() * (D + 2) * 4);  // the ring of tiles, the parts of the result
}
template <int D>
constexpr size_t c8_part(size_t G) {  // floats of a part: G heads' sums, their maxima and totals
    return G * (D + 2);
}

template <typename E, int D, int NH>
__global__ void __launch_bounds__(128, 2) c8_step_kernel(const E *__restrict__ q, const E *__restrict__ k, const E *__restrict__ v,
                                                         uint8_t *kc, uint8_t *vc, float *kf, float *vf, E *__restrict__ o,
                                                         float *__restrict__ parts, Cut8 *__restrict__ cuts, WsHeader *hdr, Step8Args g) {
    constexpr int NG = c8_groups<NH>(), N = 8 * NG;  // columns
    constexpr int KC = D / 64, M = D / 16, P = D / 16;  // 64-column pieces; products of 16 columns of o; pieces of a slot
    constexpr bool HALVES = NH == 4;  // columns 4 to 7: the same heads, whose products take the weights' second parts
    constexpr bool BF = std::is_same<E, __nv_bfloat16>::value;
    extern __shared__ __align__(128) char smem[];
    __shared__ __align__(16) E s_new[2][D];
    __shared__ float s_top[2][kStepWarps];
    __shared__ unsigned s_sum[kStepWarps], s_at[2];
    char *const s_parts = smem + kStepWarps * kC8Stages * 32 * D;
    float(*s_o)[N][D] = reinterpret_cast<float(*)[N][D]>(s_parts);
    float(*s_m)[N] = reinterpret_cast<float(*)[N]>(s_parts + kStepWarps * N * D * 4);
    float(*s_l)[N] = s_m + kStepWarps;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3, G = g.H / g.Hkv;

    if (blockIdx.x == 0 && threadIdx.x < (int)sizeof(WsHeader) / 4) reinterpret_cast<uint32_t *>(hdr)[threadIdx.x] = 0u;  // nothing waits
    // this block's share, and the pair in which it starts (all counts of blocks of slots are below 2^31)
    unsigned all = 0, before = 0, held = 0;
    for (int b0 = 0; b0 < g.B; b0 += 128) {
        held = b0 + (int)threadIdx.x < g.B ? (unsigned)held_blocks(g, b0 + threadIdx.x) * g.Hkv : 0u;
        all += block_scan(held, before, s_sum);
    }
    unsigned at = share_of(all, blockIdx.x);
    const unsigned start = at, end = share_of(all, blockIdx.x + 1);
    if (threadIdx.x == 0) cuts[blockIdx.x].unit = -1;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may take its place; it waits for this grid's end
    unsigned seen = 0;
    for (int b0 = 0; b0 < g.B && at < end && seen <= at; b0 += 128) {
        if (g.B > 128) {
            held = b0 + (int)threadIdx.x < g.B ? (unsigned)held_blocks(g, b0 + threadIdx.x) * g.Hkv : 0u;
            const unsigned more = block_scan(held, before, s_sum);
            before += seen;
            seen += more;
        }
        if (before <= at && at < before + held) s_at[0] = b0 + threadIdx.x, s_at[1] = at - before;
    }
    __syncthreads();
    int b = 0, used = 1, hk = 0, first = 0;
    if (at < end) b = (int)s_at[0], used = held_blocks(g, b), hk = (int)(s_at[1] / (unsigned)used), first = (int)(s_at[1] % (unsigned)used);

    const uint32_t ring = smem_u32(smem) + warp * (kC8Stages * 32 * D), ring_end = ring + kC8Stages * 32 * D;
    // where this lane's pieces go in a tile: the x-th 512 x bytes on, with the keys of tile_at the same for every other x
    uint32_t at_lane[2] = {tile_at<D>(lane / P, lane % P), tile_at<D>(lane / P + 32 / P, lane % P) - 512u};
    // the segment: blocks [first, first + cnt) of pair (b, hk), whose n first slots hold tokens
    int n = 0, cnt = 0, own = 0, mine = 0;
    uint8_t *kb = nullptr, *vb = nullptr;
    const uint8_t *kl = nullptr, *vl = nullptr;
    auto locate = [&]() {
        const long long p = g.pos[b], unit = (long long)b * g.Hkv + hk, from = ((long long)first * kC8Block + 16 * warp) * D + 16 * lane;
        // positions and slots are below 2^31
        mine = (int)(p < g.sinks ? p : g.sinks + (unsigned)(p - g.sinks) % (unsigned)g.window), n = (int)min(p + 1, g.slots);
        cnt = min(used - first, (int)(end - at));
        own = mine / kC8Block - first;  // the token's block, where that is of this segment
        kb = kc + unit * g.slots * D, vb = vc + unit * g.slots * D;
        kl = kb + from, vl = vb + from;
    };
    // the warp's 16 slots of block i, which lie one behind the other; zeros behind the last that holds a token
    auto fetch = [&](int i, uint32_t to) {
        constexpr int R = 32 / P;
        const int s0 = (first + i) * kC8Block + 16 * warp;
        const long long from = (long long)i * (kC8Block * D);
        if (s0 + 16 <= n) {
#pragma unroll
            for (int x = 0; x < 16 / R; ++x) {
                cp_async16(to + at_lane[x & 1] + 512 * x, kl + from + 512 * x, 16u);
                cp_async16(to + 16 * D + at_lane[x & 1] + 512 * x, vl + from + 512 * x, 16u);
            }
        } else {
#pragma unroll 1
            for (int x = 0; x < 16 / R; ++x) {
                const bool in = s0 + lane / P + R * x < n;
                cp_async16(to + at_lane[x & 1] + 512 * x, in ? kl + from + 512 * x : kb, in ? 16u : 0u);
                cp_async16(to + 16 * D + at_lane[x & 1] + 512 * x, in ? vl + from + 512 * x : vb, in ? 16u : 0u);
            }
        }
    };
    auto prefetch = [&]() {
        __syncwarp();  // the warp has read its tiles, and written its part of the token's block
#pragma unroll 1
        for (int i = 0; i < kC8Stages; ++i) {
            if (i < cnt) fetch(i, ring + i * (32 * D));
            cp_async_commit();
        }
    };
    if (at < end) locate(), prefetch();
    while (at < end) {
        float *kfb = kf + ((long long)b * g.Hkv + hk) * g.blocks + first, *vfb = vf + ((long long)b * g.Hkv + hk) * g.blocks + first;
        for (int h0 = 0; h0 < G; h0 += NH) {  // NH heads at most, or the segment again (from L2)
            const int nh = min(NH, G - h0);
            if (h0 == 0 && threadIdx.x < 2 * P * 2) {  // the token's key and value
                const int which = threadIdx.x / (2 * P), c = threadIdx.x % (2 * P);
                const E *x = which == 0 ? k + b * g.sk.b + hk * g.sk.h : v + b * g.sv.b + hk * g.sv.h;
                reinterpret_cast<uint4 *>(s_new[which])[c] = reinterpret_cast<const uint4 *>(x)[c];
            }
            uint32_t qf[NG][KC][8];
            float fac[NG][2];
#pragma unroll
            for (int a = 0; a < NG; ++a) {
                float x[KC][16], top = 0.f;
#pragma unroll
                for (int c = 0; c < KC; ++c) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[c][i] = 0.f;
                    const int h = HALVES ? r & 3 : 8 * a + r;
                    if (h < nh) load16(q + b * g.sq.b + (hk * G + h0 + h) * g.sq.h + 64 * c + 16 * j, x[c]);
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
            // per head: the running maximum (8 less than the maximum at most; finite from the start, so that a score of -inf
            // weighs nothing wherever it comes) and the total; acc: 2^-32 of the sums
            float acc[NG][M][4], mu[NG][2], l[NG][2];
#pragma unroll
            for (int a = 0; a < NG; ++a) {
                mu[a][0] = mu[a][1] = -FLT_MAX;
                l[a][0] = l[a][1] = 0.f;
#pragma unroll
                for (int y = 0; y < M; ++y) acc[a][y][0] = acc[a][y][1] = acc[a][y][2] = acc[a][y][3] = 0.f;
            }
            float kfs = 0.f, vfs = 0.f;  // the factors of 32 blocks, one in each lane
            uint32_t tile = ring;
#pragma unroll 1
            for (int i = 0; i < cnt; ++i) {
                if (i % 32 == 0 && i + lane < cnt) kfs = __ldcg(kfb + i + lane), vfs = __ldcg(vfb + i + lane);
                float kfac = __shfl_sync(~0u, kfs, i % 32), vfac = __shfl_sync(~0u, vfs, i % 32);
                cp_async_wait<kC8Stages - 1>();
                __syncwarp();
                const int left = n - (first + i) * kC8Block - 16 * warp;  // slots from the warp's first that hold a token
                if (h0 == 0 && i == own) {
                    const int s0 = n - left;
                    put_token<E, D>(tile, kb + (long long)s0 * D, vb + (long long)s0 * D, kfb + i, vfb + i, s_new, mine - s0, left, kfac,
                                    vfac, s_top);
                }
                const float part = vfac * 0x1p-32f;
                uint4 kx[2][KC];
                uint32_t vx[4][D / 32];
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int c = 0; c < KC; ++c) kx[x][c] = lds16(tile + tile_at<D>(r, 4 * c + j) + 8 * x * D);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    if constexpr (D == 128) {
                        const uint4 w = lds16(tile + 16 * D + tile_at<D>(2 * j + (x & 1), r) + 8 * (x >> 1) * D);
                        vx[x][0] = w.x, vx[x][1] = w.y, vx[x][2] = w.z, vx[x][3] = w.w;
                    } else {
                        const uint2 w = lds8(tile + 16 * D + tile_at<D>(2 * j + (x & 1), r >> 1) + 8 * (r & 1) + 8 * (x >> 1) * D);
                        vx[x][0] = w.x, vx[x][1] = w.y;
                    }
                }
                __syncwarp();
                if (i + kC8Stages < cnt) fetch(i + kC8Stages, tile);
                cp_async_commit();
                tile = tile + 32 * D == ring_end ? ring : tile + 32 * D;
                uint32_t pw[NG][2], pl[NG][2];
                float2 by[NG];  // what the products of heads 2j, 2j + 1 are added with
                float most[NG][2], all[NG][2];  // the tile's largest score and its weights' sum
#pragma unroll
                for (int a = 0; a < NG; ++a) {
                    float s[2][4] = {};  // two sums, so that products wait half as long for one another
#pragma unroll
                    for (int c = 0; c < KC; ++c) {
                        const uint32_t w0[4] = {kx[0][c].x, kx[0][c].y, kx[0][c].z, kx[0][c].w};
                        const uint32_t w1[4] = {kx[1][c].x, kx[1][c].y, kx[1][c].z, kx[1][c].w};
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            mma16x8<false>(s[x & 1], f16x2_of(w0[x]), f16x2_of(w1[x]), f16x2_of(w0[x] >> 16), f16x2_of(w1[x] >> 16),
                                           qf[a][c][2 * x], qf[a][c][2 * x + 1]);
                    }
                    // z: (slot r, heads 2j, 2j + 1), (slot r + 8, the same heads); top: the tile's largest
                    const float f0 = fac[a][0] * kfac, f1 = fac[a][1] * kfac;
                    float z[4] = {(s[0][0] + s[1][0]) * f0, (s[0][1] + s[1][1]) * f1, (s[0][2] + s[1][2]) * f0, (s[0][3] + s[1][3]) * f1};
                    if (left < 16) {
                        if (r >= left) z[0] = z[1] = -INFINITY;
                        if (r + 8 >= left) z[2] = z[3] = -INFINITY;
                    }
                    float(&top)[2] = most[a];
                    top[0] = fmaxf(z[0], z[2]), top[1] = fmaxf(z[1], z[3]);
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) {
                        top[0] = fmaxf(top[0], __shfl_xor_sync(~0u, top[0], x));
                        top[1] = fmaxf(top[1], __shfl_xor_sync(~0u, top[1], x));
                    }
                    const float t0 = fmaxf(top[0], -FLT_MAX) - 15.f, t1 = fmaxf(top[1], -FLT_MAX) - 15.f;
                    z[0] = ex2(z[0] - t0), z[1] = ex2(z[1] - t1), z[2] = ex2(z[2] - t0), z[3] = ex2(z[3] - t1);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t h = pack16<false>(make_float2(z[2 * x], z[2 * x + 1]));
                        const float2 e = unpack16<false>(h);
                        const uint32_t rest = pack16<false>(make_float2(z[2 * x] - e.x, z[2 * x + 1] - e.y));
                        pw[a][x] = transpose8x8(HALVES && j >= 2 ? rest : h);
                        if constexpr (!HALVES) pl[a][x] = transpose8x8(rest);
                    }
                    all[a][0] = z[0] + z[2], all[a][1] = z[1] + z[3];
                }
                // behind the weights, which do not wait for it: the running maximum
                bool up = false;
#pragma unroll
                for (int a = 0; a < NG; ++a) up = up || most[a][0] - mu[a][0] > 8.f || most[a][1] - mu[a][1] > 8.f;
                if (__any_sync(~0u, up)) {
#pragma unroll
                    for (int a = 0; a < NG; ++a) {
                        const float(&top)[2] = most[a];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float mn = fmaxf(mu[a][e], top[e]), f = ex2(mu[a][e] - mn);
                            mu[a][e] = mn;
                            l[a][e] *= f;
#pragma unroll
                            for (int y = 0; y < M; ++y) acc[a][y][e] *= f, acc[a][y][2 + e] *= f;
                        }
                    }
                }
#pragma unroll
                for (int a = 0; a < NG; ++a) {
                    const float(&top)[2] = most[a];
                    const float e0 = ex2(fmaxf(top[0], -FLT_MAX) - 15.f - mu[a][0]), e1 = ex2(fmaxf(top[1], -FLT_MAX) - 15.f - mu[a][1]);
                    l[a][0] = fmaf(all[a][0], e0, l[a][0]);
                    l[a][1] = fmaf(all[a][1], e1, l[a][1]);
                    by[a] = make_float2(e0 * part, e1 * part);
                }
#pragma unroll
                for (int y = 0; y < D / 32; ++y) {
                    // two columns of d a product: 4 y + 0, 1 and 4 y + 2, 3 of this lane's
                    const uint32_t a0 = __byte_perm(vx[0][y], vx[1][y], 0x5140), a1 = __byte_perm(vx[0][y], vx[1][y], 0x7362);
                    const uint32_t b0 = __byte_perm(vx[2][y], vx[3][y], 0x5140), b1 = __byte_perm(vx[2][y], vx[3][y], 0x7362);
                    const uint32_t f0 = f16x2_of(a0), f1 = f16x2_of(a0 >> 16), f2 = f16x2_of(b0), f3 = f16x2_of(b0 >> 16);
                    const uint32_t f4 = f16x2_of(a1), f5 = f16x2_of(a1 >> 16), f6 = f16x2_of(b1), f7 = f16x2_of(b1 >> 16);
#pragma unroll
                    for (int a = 0; a < NG; ++a) {
                        float u[4] = {0.f, 0.f, 0.f, 0.f}, w[4] = {0.f, 0.f, 0.f, 0.f};
                        if constexpr (!HALVES) {
                            mma16x8<false>(u, f0, f1, f2, f3, pl[a][0], pl[a][1]);
                            mma16x8<false>(w, f4, f5, f6, f7, pl[a][0], pl[a][1]);
                        }
                        mma16x8<false>(u, f0, f1, f2, f3, pw[a][0], pw[a][1]);
                        mma16x8<false>(w, f4, f5, f6, f7, pw[a][0], pw[a][1]);
                        add_times(acc[a][2 * y], u, by[a]);
                        add_times(acc[a][2 * y + 1], w, by[a]);
                    }
                }
            }
            // the next segment, or this one for more heads, is on its way while the parts meet
            const long long unit = (long long)b * g.Hkv + hk;
            const int slot = 2 * blockIdx.x + (at != start);
            const bool whole = cnt == used;
            if (h0 + NH >= G) {
                if (!whole && first == 0 && threadIdx.x == 0) {
                    // the thread block that has the pair's last block of slots: the least c with share_of(c + 1) >= at + used
                    const unsigned long long x = at + (unsigned)used;
                    cuts[blockIdx.x] = Cut8{(int)unit, slot, (int)((x * gridDim.x + all - 1) / all) - 1, (int)all};
                }
                at += cnt;
                first = 0;
                if (at < end && ++hk == g.Hkv) {
                    hk = 0;
                    do used = held_blocks(g, ++b);
                    while (used == 0);
                }
                if (at < end) locate(), prefetch();
            } else {
                prefetch();
            }
            // product y, row r: column (D / 8) r + 2 y, row r + 8: the next one
#pragma unroll
            for (int a = 0; a < NG; ++a)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) l[a][e] += __shfl_xor_sync(~0u, l[a][e], x);
                    const int h = 8 * a + 2 * j + e;
                    if (r == 0) s_m[warp][h] = mu[a][e], s_l[warp][h] = l[a][e];
#pragma unroll
                    for (int y = 0; y < M; ++y)
                        *reinterpret_cast<float2 *>(&s_o[warp][h][D / 8 * r + 2 * y]) = make_float2(acc[a][y][e], acc[a][y][2 + e]);
                }
            __syncthreads();
            // the warps' parts together: the outputs of a whole segment, or a part for the join
            float *part = parts + slot * c8_part<D>(G);
            for (int i = threadIdx.x; i < nh * D / 2; i += blockDim.x) {
                const int h = i / (D / 2), d = i % (D / 2) * 2;
                float mm = s_m[0][h];
#pragma unroll
                for (int w = 1; w < kStepWarps; ++w) mm = fmaxf(mm, s_m[w][h]);
                float lt = 0.f, x = 0.f, y = 0.f;
#pragma unroll
                for (int w = 0; w < kStepWarps; ++w) {
                    const float f = ex2(s_m[w][h] - mm);
                    float2 e = *reinterpret_cast<const float2 *>(&s_o[w][h][d]);
                    if constexpr (HALVES) {
                        const float2 rest = *reinterpret_cast<const float2 *>(&s_o[w][h + 4][d]);
                        e.x += rest.x, e.y += rest.y;
                    }
                    lt = fmaf(f, s_l[w][h], lt), x = fmaf(f, e.x, x), y = fmaf(f, e.y, y);
                }
                if (whole) {
                    reinterpret_cast<uint32_t *>(o + (unit * G + h0) * D)[i] = pack16<BF>(make_float2(x / lt * 0x1p32f, y / lt * 0x1p32f));
                } else {
                    reinterpret_cast<float2 *>(part + h0 * D)[i] = make_float2(x, y);
                    if (d == 0) reinterpret_cast<float2 *>(part + G * D)[h0 + h] = make_float2(mm, lt);
                }
            }
            __syncthreads();  // the parts have been read
        }
    }
    // rows without a sequence
    for (b = blockIdx.x; b < g.B; b += gridDim.x)
        if (g.pos[b] < 0)
            for (long long i = threadIdx.x; i < (long long)g.H * D / 2; i += blockDim.x)
                reinterpret_cast<uint32_t *>(o + (long long)b * g.H * D)[i] = 0u;
}

// Adds the parts of a cut (sequence, key head), for a query head of the group, in a fixed order: their common maximum first,
// then every eighth part by a warp.  A block of it fits beside the step's two (34 registers; with 59 it did not, and the
// step took 2 us more).  It starts while the step still writes parts and cuts, so these are no memory that stays as it is
// for the kernel's life: no __restrict__, and the wait keeps the loads behind it.
template <typename E, int D>
__global__ void __launch_bounds__(256) c8_join_kernel(const float *parts, const Cut8 *cuts, E *o, int G) {
    constexpr int W = 8, N = D / 32;
    __shared__ float s_o[W][D], s_f[kC8MaxBlocks], s_m[W], s_l[W];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Cut8 cut = cuts[blockIdx.x];
    if (cut.unit < 0) return;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, h = blockIdx.y, n = cut.last - (int)blockIdx.x + 1;
    auto part_of = [&](int i) { return parts + (i == 0 ? cut.slot : 2 * ((int)blockIdx.x + i)) * c8_part<D>(G); };
    constexpr int K = (kC8MaxBlocks + 255) / 256;
    float2 ml[K];
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = threadIdx.x + 256 * k;
        const unsigned c = blockIdx.x + i;
        ml[k] = make_float2(-INFINITY, 0.f);
        if (i < n && share_of(cut.all, c) < share_of(cut.all, c + 1))  // else: more thread blocks than blocks of slots
            ml[k] = reinterpret_cast<const float2 *>(part_of(i) + G * D)[h];
        m = fmaxf(m, ml[k].x);
    }
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, x));
    if (lane == 0) s_m[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) m = fmaxf(m, s_m[w]);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const bool there = ml[k].x != -INFINITY;
        const float f = there ? ex2(ml[k].x - m) : 0.f;
        if (threadIdx.x + 256 * k < kC8MaxBlocks) s_f[threadIdx.x + 256 * k] = there ? f : -1.f;
        l += f * ml[k].y;
    }
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) l += __shfl_xor_sync(~0u, l, x);
    if (lane == 0) s_l[warp] = l;
    __syncthreads();
    float x[N];
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = 0.f;
#pragma unroll 4
    for (int i = warp; i < n; i += W) {
        const float f = s_f[i], *part = part_of(i) + h * D + lane;
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (f != -1.f) x[e] = fmaf(f, part[32 * e], x[e]);  // of a part that is there, were its weight 0: it may hold a NaN
    }
#pragma unroll
    for (int e = 0; e < N; ++e) s_o[warp][32 * e + lane] = x[e];
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += 256) {
        float lt = 0.f, y = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) lt += s_l[w], y += s_o[w][d];
        o[((long long)cut.unit * G + h) * D + d] = from_f32<E>(y / lt * 0x1p32f);
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
    if (T > kMaxTokens || !product_below({B, H}, 1 << 27) ||
        !product_below({B, Hkv, (sinks + window + kC8Block - 1) / kC8Block}, 2147483648.0))
        return fail(CLA_ERR_UNSUPPORTED, "%s: sizes too large", fn);
    return CLA_OK;
}

// Blocks of the step that the current device runs at once, asked for once per device.
template <typename E, int D, int NH>
int c8_resident(const char *fn, int *n) {
    static std::atomic<int> known[64];
    static std::atomic<unsigned long long> done{0};
    constexpr int smem = c8_smem<D, NH>();
    int dev = 0, sms = 0;
    CLA_CUDA_TRY(cudaGetDevice(&dev), fn);
    *n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (*n != 0) return CLA_OK;
    if (int st = set_max_dynamic_smem(done, (const void *)c8_step_kernel<E, D, NH>, smem)) return st;
    if (int st = multiprocessors(fn, &sms)) return st;
    CLA_CUDA_TRY(cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, c8_step_kernel<E, D, NH>, kStepWarps * 32, smem), fn);
    *n = *n * sms < kC8MaxBlocks ? *n * sms : kC8MaxBlocks;
    if (dev < 64) known[dev].store(*n, std::memory_order_relaxed);
    return CLA_OK;
}

template <typename E, int D, int NH>
int c8_step(const char *fn, const void *q, const void *k, const void *v, void *kc, void *vc, float *kf, float *vf, void *o,
            const Step8Args &g, void *ws, cudaStream_t s) {
    int n = 0;
    if (int st = c8_resident<E, D, NH>(fn, &n)) return st;
    const long long most = (long long)g.B * g.Hkv * g.blocks;
    const unsigned grid = (unsigned)(most < n ? most : n);
    WsHeader *hdr = static_cast<WsHeader *>(ws);
    Cut8 *cuts = reinterpret_cast<Cut8 *>(hdr + 1);
    float *parts = reinterpret_cast<float *>(cuts + kC8MaxBlocks);
    c8_step_kernel<E, D, NH><<<grid, kStepWarps * 32, c8_smem<D, NH>(), s>>>(
        (const E *)q, (const E *)k, (const E *)v, (uint8_t *)kc, (uint8_t *)vc, kf, vf, (E *)o, parts, cuts, hdr, g);
    if (int st = check_launch(fn)) return st;
    if (g.blocks == 1) return CLA_OK;  // nothing is cut
    // the join's launch goes beside the step's end
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at;
    cfg.gridDim = dim3(grid, (unsigned)(g.H / g.Hkv));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    CLA_CUDA_TRY(cudaLaunchKernelEx(&cfg, c8_join_kernel<E, D>, (const float *)parts, (const Cut8 *)cuts, (E *)o, g.H / g.Hkv), fn);
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
                                               r[0], r[1], (int)Hkv, (int)T, (unsigned)window, (int)sinks, blocks)
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

extern "C" size_t cla_window_attn_step8_workspace_size(int64_t B, int64_t H, int64_t Hkv, int64_t d, int64_t window, int64_t sinks) {
    if (c8_check("cla_window_attn_step8_workspace_size", B, H, Hkv, 1, d, window, sinks, CLA_BF16, 1.f) != CLA_OK) return 0;
    const int64_t most = B * Hkv * ((sinks + window + kC8Block - 1) / kC8Block);  // a thread block has one block of slots at least
    const int64_t parts = 2 * (most < kC8MaxBlocks ? most : kC8MaxBlocks);
    return sizeof(WsHeader) + sizeof(Cut8) * kC8MaxBlocks + (size_t)(parts * (Hkv ? H / Hkv : 0) * (d + 2) * 4);
}

extern "C" int cla_window_attn_step8(const void *q, const void *k, const void *v, void *kcache, void *vcache, float *kscale,
                                     float *vscale, const int32_t *pos, void *o, float scale, int64_t window, int64_t sinks, int dtype,
                                     int64_t B, int64_t H, int64_t Hkv, int64_t d, const int64_t *strides, void *ws, size_t ws_bytes,
                                     void *stream) {
    const char *fn = "cla_window_attn_step8";
    clear_error();
    if (int st = c8_check(fn, B, H, Hkv, 1, d, window, sinks, dtype, scale)) return st;
    if (H > 0 && H / Hkv > 65535) return fail(CLA_ERR_UNSUPPORTED, "%s: %lld query heads of a key head", fn, (long long)(H / Hkv));
    if (B * H > 0 && (!q || !k || !v || !kcache || !vcache || !kscale || !vscale || !pos || !o))
        return fail(CLA_ERR_INVALID_ARG, "%s: a required pointer is NULL", fn);
    if (!aligned_or_null({q, k, v, kcache, vcache, o}, 16) || !aligned_or_null({pos, kscale, vscale}, 4))
        return fail(CLA_ERR_INVALID_ARG, "%s: a pointer is misaligned", fn);
    const size_t need = cla_window_attn_step8_workspace_size(B, H, Hkv, d, window, sinks);
    if (ws == nullptr || !aligned16(ws) || ws_bytes < need)
        return fail(CLA_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes, need);
    static const char *const names[] = {"q", "k", "v"};
    const int64_t heads[] = {H, Hkv, Hkv}, ds[] = {d, d, d};
    Triple r[3];
    int64_t full[9];
    if (strides != nullptr)
        for (int i = 0; i < 3; ++i) full[3 * i] = strides[2 * i], full[3 * i + 1] = strides[2 * i + 1], full[3 * i + 2] = d;
    if (int st = view_strides(fn, strides ? full : nullptr, names, heads, ds, 3, B, 1, 8, r)) return st;
    if (B * H == 0) {
        CLA_CUDA_TRY(cudaMemsetAsync(ws, 0, sizeof(WsHeader), (cudaStream_t)stream), fn);
        return CLA_OK;
    }
    const Step8Args g{pos,      scale * 1.4426950408889634f, window, sinks, sinks + window, (int)B, (int)H, (int)Hkv,
                      (int)((sinks + window + kC8Block - 1) / kC8Block), r[0], r[1], r[2]};
    cudaStream_t s = (cudaStream_t)stream;
    // heads of a group at once: 16, 8, or 4 with both parts of the weights in one product (64 x 32/8, in graphs: x 128, window
    // 4096 89 us, 91 with 8; x 64, window 8192 91 us, 95 with 8.  64 x 64/4 x 128, window 4096: 71 us with 16, 96 with 8,
    // which reads the cache twice)
    const bool bf = dtype == CLA_BF16;
    const int64_t heads_of = H / Hkv;
#define CLA_STEP8(E, D)                                                                                            \
    (heads_of > 8   ? c8_step<E, D, 16>(fn, q, k, v, kcache, vcache, kscale, vscale, o, g, ws, s) \
     : heads_of > 4 ? c8_step<E, D, 8>(fn, q, k, v, kcache, vcache, kscale, vscale, o, g, ws, s)  \
                    : c8_step<E, D, 4>(fn, q, k, v, kcache, vcache, kscale, vscale, o, g, ws, s))
    if (d == 128) return bf ? CLA_STEP8(__nv_bfloat16, 128) : CLA_STEP8(__half, 128);
    return bf ? CLA_STEP8(__nv_bfloat16, 64) : CLA_STEP8(__half, 64);
#undef CLA_STEP8
}
