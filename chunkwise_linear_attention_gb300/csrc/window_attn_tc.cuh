// window_attn_tc.cuh -- the training and prefill kernels of window_attn.cu on
// the fifth-generation tensor cores: TMA tile loads, tcgen05.mma with the
// accumulators in tensor memory, probabilities and their gradients rounded to
// the tensors' type and fed back as the A operand from tensor memory.
//
// Tiles are 128 tokens on both sides.  Every kernel is persistent (a block per
// SM, items taken in a fixed order) and has its roles in separate warps: 16
// math warps, one that issues the products, one that issues the loads, and one
// or two that form the rows' statistics and store what the math warps staged,
// so that loads, products and stores run beside the elementwise work.  A math
// warp reads the lane quarter of tensor memory that its rank in its group of
// four allows; the thread's lane is its row.
//
// Probabilities P and their gradients dS are rounded to the tensors' type for
// their products, with fp32 sums: the tensor cores take no fp32 operand, and
// two 16-bit parts would double the products that bound the kernels at d = 128.
// delta is the sum of dO o with the o that the backward is given, which is
// rounded too; a sum of P dP would need both formed once more.  Against a form
// that keeps all three in fp32 this adds about as much error to dq and dk as
// the rounding of the outputs does (bf16: 2.5e-3 against 1.7e-3 at a window of
// 512, of which dS is 1.7e-3 and delta 1.1e-3; delta's share grows as a query
// sees fewer keys, to twice the outputs' rounding at two).
//
// Measured on GB300 (B x H / Hkv x T x d, window, sinks; bf16):
//                                     4 x 16/16 x 8192 x 64   2 x 16/4 x 8192 x 128
//                                     512, 0                  2048, 16
//   forward                           117 us, 31% of the      198 us, 64%
//   dq                                141 us  40% tensor      252 us, 74%
//   dk, dv                            173 us, 41% pipe's      342 us, 74%
//   join                              6 us        cycles      8 us
// At d = 128 the products bound them (of the backward's seven, two are S and dP
// formed a second time, for rows of keys; all tiles are formed whole, also those
// that the window or the diagonal cuts: 17 where 16 would do at that window,
// 5 where 4 would at the other); at d = 64, where a pair of tiles has half the
// products and the same 16384 exponentials and roundings, the chain of a warp's
// elementwise work (load, 2^x, rounding, store, each behind the other; no unit
// above half of its rate), and the exchange and staging at the end of each item,
// a fifth of its time at five key tiles.  More overlap did not help there: next
// scores formed before the probabilities' product, in columns of their own, 452
// us for the pass against 446; nor cheaper polls of the barriers, 442, or sleep
// between them, 451.
//
// Waits are bounded: one that gives up marks the block, which then waits no
// more, and records the timeout in the block's entry of the workspace header.
// Most last a step; those for the end of a list or item, which may have any
// number of steps, give up only when the block's loads have stopped moving too.
#pragma once

#include "mma_sync.cuh"
#include "tc_ptx.cuh"

namespace cla {
namespace {

constexpr int kWT = 128;  // tokens of a tile
constexpr int kHalf = 64 * 128;  // bytes of 64 of its tokens in a block of 64 columns
// Every block takes all 512 columns of tensor memory, so its shared memory is kept above half of
// an SM's, which keeps a second block of these kernels off the SM.
constexpr int kMinSmem = 116 * 1024;

struct Str3 {
    long long b, h, t;
};

// Division of a number below 2^31 by one known on the host (the round-up method of Granlund and
// Montgomery): items are taken apart in every warp of a block, and a division is a hundred cycles.
struct Div {
    uint32_t d, mul, shift;
    __host__ Div(uint32_t n = 1) : d(n ? n : 1), mul(0), shift(0) {
        while ((1ull << shift) < d) ++shift;
        mul = (uint32_t)(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
    }
    __device__ __forceinline__ int operator()(int x) const {
        return (int)((__umulhi((uint32_t)x, mul) + (uint32_t)x) >> shift);
    }
};

// Token numbers, the window and the sinks (both at most T) fit 32 bits: T is at most 2^31 - 512.
struct WaArgs {
    const int32_t *lens;
    float scale;
    int T, window, sinks, B, H, Hkv;
    Div per, bh, hkv, heads, group;  // items of a group, B Hkv, Hkv, H, H / Hkv
};

// Of the inputs q, k, v, dO, and of the outputs: o, dq in `x`, dk in `x`, dv in `y`.
struct WaMaps {
    CUtensorMap q, k, v, g, x, y;
};

__device__ __forceinline__ int wa_len(const WaArgs &g, int b) {
    return g.lens == nullptr ? g.T : min(max(__ldg(g.lens + b), 0), g.T);
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_store_4d(const CUtensorMap *map, int x, int y, int z, int w, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(w), "r"(src)
                 : "memory");
}
// A value that is the same in all lanes, in a form that the compiler knows to be.  The warp that
// issues the products keeps its loops' bounds and operands so: descriptors that it takes for
// divergent are moved into uniform registers before each product, which took 75 cycles each.
__device__ __forceinline__ int uni(int v) { return __shfl_sync(~0u, v, 0); }
// The lane that issues them, chosen once.
__device__ __forceinline__ uint32_t elect() {
    uint32_t e;
    asm volatile("{\n .reg .pred p;\n .reg .b32 r;\n elect.sync r|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(e));
    return e;
}
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p, e;\n setp.ne.b32 e, %0, 0;\n setp.ne.b32 p, %5, 0;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%1], %2, %3, %4, p;\n}" ::"r"(lead),
        "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p, e;\n setp.ne.b32 e, %0, 0;\n setp.ne.b32 p, %5, 0;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%1], [%2], %3, %4, p;\n}" ::"r"(lead),
        "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t lead, uint32_t bar) {
    asm volatile(
        "{\n .reg .pred e;\n setp.ne.b32 e, %0, 0;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%1];\n}" ::"r"(lead),
        "r"(bar)
        : "memory");
}
// kind::f16 instruction descriptor, fp32 accumulate, A and B both bf16 or both fp16.
template <bool BF>
__host__ __device__ constexpr uint32_t idesc16(int N, int b_mn_major) {
    return (1u << 4) | (BF ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(kWT >> 4) << 24);
}
template <bool BF>
__device__ __forceinline__ uint32_t pack16(float2 v) {
    if constexpr (BF) {
        const __nv_bfloat162 h = __float22bfloat162_rn(v);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __float22half2_rn(v);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}
template <bool BF>
__device__ __forceinline__ float2 unpack16(uint32_t u) {
    if constexpr (BF) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    else return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}

// c += A B^T, A [16 x 16], B [8 x 16], by a warp.  The order of the 16 columns is free, so a lane
// (r = lane / 4, j = lane % 4) may hold any four of them of its rows r, r + 8 and r.
template <bool BF>
__device__ __forceinline__ void mma16x8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    if constexpr (BF)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The waits of a block: once one has given up none waits long any more.
struct Waits {
    volatile uint32_t *dead;  // 0, or the wait that gave up
    __device__ __forceinline__ static bool try_once(uint32_t bar, uint32_t parity) {
        uint32_t done;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
            : "=r"(done)
            : "r"(bar), "r"(parity)
            : "memory");
        return done != 0u;
    }
    __device__ __forceinline__ void operator()(uint32_t bar, uint32_t parity, unsigned int where) const {
        parity &= 1u;
        if (!try_once(bar, parity)) slow(bar, parity, where);
    }
    __device__ __noinline__ void slow(uint32_t bar, uint32_t parity, unsigned int where) const {
        for (uint32_t it = 0; it < (1u << 24); ++it) {
            if (try_once(bar, parity)) return;
            if ((it & 255u) == 255u && *dead != 0u) return;
        }
        *dead = where;
    }
    // For a list's or an item's end, which may be any number of steps away (2^24 polls are 24 s at the
    // 1.4 us that a poll lasts where nothing wakes the warp): the bound begins anew whenever the loads'
    // warp, which is a few steps ahead of the products at most, has moved.
    __device__ __forceinline__ void end(volatile uint32_t *loads, uint32_t bar, uint32_t parity, unsigned int where) const {
        if (!try_once(bar, parity & 1u)) slow_end(dead, loads, bar, parity & 1u, where);
    }
    // (its members as values: an object whose address is taken would lie in local memory)
    __device__ __noinline__ static void slow_end(volatile uint32_t *dead, volatile uint32_t *loads, uint32_t bar,
                                                 uint32_t parity, unsigned int where) {
        uint32_t seen = *loads;
        for (uint32_t it = 0; it < (1u << 24); ++it) {
            if (try_once(bar, parity)) return;
            if ((it & 255u) != 255u) continue;
            if (*dead != 0u) return;
            const uint32_t now = *loads;
            if (now != seen) seen = now, it = 0u;
        }
        *dead = where;
    }
};

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// After a timeout: the loads that were issued into a ring of S stages (n in all) land before the
// block leaves.
__device__ __forceinline__ void drain(uint32_t full, uint32_t n, uint32_t S) {
    for (uint32_t s = 0; s < S && s < n; ++s) (void)mbar_wait(full + 8 * s, ((n - 1 - s) / S) & 1u);
}

// A tile of [128 tokens][D] in blocks of 64 columns, each 128 rows of 128 swizzled bytes.
template <int D>
struct Tile {
    static constexpr int BYTES = kWT * D * 2;
    static constexpr int BLOCK = kWT * 128;
    static __device__ __forceinline__ void load(uint32_t dst, const CUtensorMap *m, int t, int h, int b, uint32_t bar) {
#pragma unroll
        for (int c = 0; c < D / 64; ++c) tma_load_4d(dst + c * BLOCK, m, c * 64, t, h, b, bar);
    }
    // operand over D (K-major), step kk of 16 columns
    static __device__ __forceinline__ uint64_t kmajor(uint32_t base) { return smem_desc(base, 16, 1024); }
    static __device__ __forceinline__ uint64_t kstep(int kk) { return (uint64_t)(((kk >> 2) * BLOCK + (kk & 3) * 32) >> 4); }
    // operand over the tokens (D along N), step kk of 16 tokens
    static __device__ __forceinline__ uint64_t nmajor(uint32_t base) { return smem_desc(base, BLOCK, 1024); }
    static __device__ __forceinline__ uint64_t nstep(int kk) { return (uint64_t)(kk * 2048 >> 4); }
    // Rows from `row` on become zero, by one warp: what lies behind a sequence's length must not
    // meet a zero probability in a product as a NaN.
    static __device__ __forceinline__ void zero_rows(uint32_t base, int row) {
        for (int i = row * 8 + (threadIdx.x & 31); i < kWT * 8; i += 32)
#pragma unroll
            for (int c = 0; c < D / 64; ++c) st_shared_v4(base + c * BLOCK + i * 16, 0.f, 0.f, 0.f, 0.f);
        fence_async_smem();
        __syncwarp();
    }
};

// acc = A B^T over D columns (both operands K-major): the scores of two tiles.  negate: 0, or
// kNegateA for -A B^T.
constexpr uint32_t kNegateA = 1u << 13;
template <int D, bool BF, int N = kWT>
__device__ __forceinline__ void mma_scores(uint32_t lead, uint32_t acc, uint32_t a, uint32_t b, uint32_t negate = 0u) {
    const uint64_t da = Tile<D>::kmajor(a), db = Tile<D>::kmajor(b);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
        mma_ss(lead, acc, da + Tile<D>::kstep(kk), db + Tile<D>::kstep(kk), idesc16<BF>(N, 0) | negate, kk ? 1u : 0u);
}
// acc (+)= P X: P [128 x K] in tensor memory, X a tile [128 tokens][D] from a token on.  P lies packed
// over the scores it came from in pieces of C columns, each at the start of its C score columns: a
// thread then writes only where it has read itself, and the threads of a row need not wait for another.
template <int D, bool BF, int C, int K = kWT>
__device__ __forceinline__ void mma_apply(uint32_t lead, uint32_t acc, uint32_t p, uint32_t x, bool add) {
    const uint64_t dx = Tile<D>::nmajor(x);
#pragma unroll
    for (int kk = 0; kk < K / 16; ++kk)
        mma_ts(lead, acc, p + (kk / (C / 16)) * C + (kk % (C / 16)) * 8, dx + Tile<D>::nstep(kk), idesc16<BF>(D, 1),
                 (add || kk) ? 1u : 0u);
}

__device__ __forceinline__ uint32_t tmem_alloc_all(uint32_t *slot) {
    if (threadIdx.x < 32) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(512u));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    return *slot;
}
__device__ __forceinline__ void tmem_free_all(uint32_t tmem) {
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x < 32)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
}
// Behind the tiles: the barriers, then the words below, then 512 floats.  The kernels have no
// static shared memory, so that the tiles start on the 1024 bytes that the swizzle needs; a base
// that did not is reported, not used.
constexpr int kSmall = 2560;
constexpr int kLast = 39;  // the barrier of products_done
struct Small {
    uint64_t bars[kLast + 1];
    uint32_t tmem, dead;
    uint32_t pad[45];
    uint32_t loads;  // issued of the tiles that a step takes, for the long waits
    float f[512];
};
static_assert(sizeof(Small) == kSmall, "layout behind the tiles");
__device__ __forceinline__ bool misplaced(uint32_t base, WsHeader *hdr) {
    if ((base & 1023u) == 0u) return false;
    if (threadIdx.x == 0) hdr->error = kErrTimeout, hdr->where = 1u;  // in every block
    return true;
}
// The call's status, by all threads at a kernel's end: each block's entry says which wait gave up (0:
// none).  The call's first kernel writes every entry, block 0 those that have no block, so that nothing
// has to be cleared before it; a later kernel adds to them.
template <bool FIRST>
__device__ __forceinline__ void leave_status(WsHeader *hdr, const Small &sm) {
    if (threadIdx.x == 0 && (FIRST || sm.dead != 0u)) hdr->block[blockIdx.x] = (unsigned char)sm.dead;
    if (!FIRST || blockIdx.x != 0) return;
    if (threadIdx.x == 0) hdr->error = kErrInBlocks, hdr->where = 0u;
    if (threadIdx.x >= gridDim.x && threadIdx.x < kStatusBlocks) hdr->block[threadIdx.x] = 0;
}
// By the warp that issues the products, in the end: none is in flight when tensor memory is given back.
// (The math warps have waited for the last of them, unless a wait was given up.)
__device__ __forceinline__ void products_done(uint32_t lead, uint32_t bars) {
    mma_commit(lead, bars + 8 * kLast);
    (void)mbar_wait(bars + 8 * kLast, 0u);
}
// Between the N warps that share a lane quarter, and so their rows.
template <int N>
__device__ __forceinline__ void quarter_sync(int id) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(32 * N) : "memory");
}
__device__ __forceinline__ void warp_arrive(uint32_t bar) {  // one arrival of a warp whose lanes are all done
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// The key tiles that a query tile sees: [lo, hi], and the sinks' below lo.
struct KeyTiles {
    int lo, hi, sinks;  // hi < lo: none
    __device__ __forceinline__ bool has(int tile) const { return tile <= hi && (tile >= lo || tile < sinks); }
};
__device__ __forceinline__ KeyTiles key_tiles(const WaArgs &g, int t0, int len) {
    if (t0 >= len) return KeyTiles{0, -1, 0};
    return KeyTiles{max(t0 - g.window + 1, 0) / kWT, min(t0 + kWT - 1, len - 1) / kWT, (g.sinks + kWT - 1) / kWT};
}
// Whether some pair of a query tile at t0 and a key tile at s0 is masked.
__device__ __forceinline__ bool tile_masked(const WaArgs &g, int t0, int s0) {
    return s0 + kWT - 1 > t0 || (t0 + kWT - 1 - s0 >= g.window && s0 + kWT > g.sinks);
}
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }
// Bit j: query t sees key s0 + j.
__device__ __forceinline__ uint32_t key_bits(const WaArgs &g, int t, int s0) {
    return bits_below(t - s0 + 1) & (~bits_below(t - s0 - g.window + 1) | bits_below(g.sinks - s0));
}
// Bit j: query t0 + j sees key s.
__device__ __forceinline__ uint32_t query_bits(const WaArgs &g, int t0, int s) {
    return ~bits_below(s - t0) & (s < g.sinks ? ~0u : bits_below(s - t0 + g.window));
}

// A query that sees one key: its weight is 1 whatever the score, and dS is 0.  It is made so, where
// dP - delta of two different sums would leave a rounding.
__device__ __forceinline__ bool sees_one(const WaArgs &g, int t) { return t == 0 || (g.window == 1 && g.sinks == 0); }

// Columns [col, col + N) of a row of an accumulator, times f, into a tile in shared memory, from
// where one store takes the tile out.  (Rows stored by their own threads are 32 lines an
// instruction; that took 4000 cycles a tile.)
template <int N, bool BF>
__device__ __forceinline__ void stage_row(uint32_t taddr, uint32_t tile, int row, int col, float f, bool zero) {
    constexpr int C = N < 32 ? N : 32;
#pragma unroll
    for (int c = 0; c < N; c += C) {
        uint32_t r[C];
        if constexpr (C == 32) tmem_ld32(taddr + c, r);
        else tmem_ld16(taddr + c, r);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < C / 8; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = zero ? 0u
                            : pack16<BF>(make_float2(__uint_as_float(r[k * 8 + 2 * j]) * f, __uint_as_float(r[k * 8 + 2 * j + 1]) * f));
            const int x = col + c + 8 * k;
            st_shared_v4(tile + (x >> 6) * (kWT * 128) + row * 128 + ((((x >> 3) ^ row) & 7) << 4), __uint_as_float(w[0]),
                         __uint_as_float(w[1]), __uint_as_float(w[2]), __uint_as_float(w[3]));
        }
    }
    fence_async_smem();
}
// By one thread, when the tile is staged.
template <int D>
__device__ __forceinline__ void store_tile(const CUtensorMap *m, uint32_t tile, int t, int h, int b) {
#pragma unroll
    for (int c = 0; c < D / 64; ++c) tma_store_4d(m, c * 64, t, h, b, tile + c * (kWT * 128));
    tma_store_commit();
}
template <int D>
__device__ __forceinline__ void zero_row(void *out, long long at) {
    uint4 *p = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + at);
#pragma unroll
    for (int k = 0; k < D / 8; ++k) p[k] = make_uint4(0u, 0u, 0u, 0u);
}

// ------------------------------------------------------------------ forward
// A block works on two query tiles at once that share their key tiles: two heads of a group, or
// two neighbouring tiles of one head where a group has an odd number of heads.  While one tile's
// eight warps form its probabilities, the tensor cores work for the other.  Two threads share a
// row, 64 columns each: with one warp a scheduler and tile the chain of loads, maxima and
// exponentials bounds the kernel by latency.  Tensor memory: two score tiles (a tile's
// probabilities lie over its scores) and two output accumulators.  The running maximum is moved
// only when a row's grows by more than 8 (in powers of two), so the accumulator is rescaled
// rarely and by the warps that own it; sums and outputs are fp32.
//
// 1 x 32/8 x 32768 x 128, window 1024, sinks 4: 495 us, of 284 us for the products of the visible
// pairs alone at the measured rate of a library's (10 tiles are formed where 8 would do).
// Tried and not kept: products of 16 columns for tiles that only sinks are seen of (no gain there,
// 3% slower without sinks), probabilities in two passes over half rows, a suspend-time hint on the
// waits (5% slower than spinning).
template <int D>
struct FwdCfg {
    static constexpr int STAGES = D == 128 ? 3 : 8;  // of keys and values, beside two pairs of query tiles
    static constexpr int SMEM = (4 + STAGES) * Tile<D>::BYTES + kSmall;
    static constexpr int THREADS = 608;  // 16 math warps, products, loads, stores
};

struct FwdItem {
    int b, hk, h, t0, step_h, step_t;  // the second tile: head h + step_h at t0 + step_t
};
// Items go from the last query tiles, which see the most, to the first: dealt out in turn they
// leave the blocks with almost equal shares.
__device__ __forceinline__ FwdItem fwd_item(const WaArgs &g, int item, int tiles) {
    FwdItem w;
    const int G = g.group.d, even = (G & 1) == 0, per = g.per.d, q = g.per(item), r = g.bh(q), bh = q - r * (int)g.bh.d;
    const int tt = (even ? tiles : (tiles + 1) / 2) - 1 - r;
    w.b = g.hkv(bh);
    w.hk = bh - w.b * g.Hkv;
    w.h = w.hk * G + (item - q * per) * (even ? 2 : 1);
    w.t0 = tt * (even ? kWT : 2 * kWT);
    w.step_h = even ? 1 : 0;
    w.step_t = even ? 0 : kWT;
    return w;
}
// The key tiles of both: the first's range begins no later than the second's, and is empty only
// if that is.
struct FwdTiles {
    KeyTiles a, b;
    int skip, count;  // the i-th tile is i below `skip` (sinks), then i - skip + a.lo
    __device__ __forceinline__ FwdTiles(const WaArgs &g, const FwdItem &w, int len)
        : a(key_tiles(g, w.t0, len)), b(key_tiles(g, w.t0 + w.step_t, len)) {
        skip = min(a.sinks, a.lo);
        count = a.hi < a.lo ? 0 : max(a.hi, b.hi) - a.lo + 1 + skip;
    }
    __device__ __forceinline__ int tile(int i) const { return i < skip ? i : a.lo + i - skip; }
};

template <int D, bool BF>
__global__ void __launch_bounds__(FwdCfg<D>::THREADS, 1)
wa_fwd_kernel(const __grid_constant__ WaMaps maps, void *__restrict__ o, float *__restrict__ lse, Str3 so, WaArgs g,
              int items, WsHeader *hdr) {
    constexpr int ST = FwdCfg<D>::STAGES, TB = Tile<D>::BYTES;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t sq = smem_u32(smem_raw), skv = sq + 4 * TB;
    Small &sm = *reinterpret_cast<Small *>(smem_raw + (4 + ST) * TB);
    static_assert(2 * ST + 14 <= kLast, "barriers");
    float(*s_row)[2][kWT] = reinterpret_cast<float(*)[2][kWT]>(sm.f);  // [tile][half][row]: maxima, in the end sums
    if (misplaced(sq, hdr)) return;
    const int warp = threadIdx.x >> 5, tiles = (g.T + kWT - 1) / kWT;
    const uint32_t b0 = smem_u32(sm.bars);
    const uint32_t q_full = b0, q_empty = b0 + 16, o_full = b0 + 32, s_full = b0 + 48, p_ready = b0 + 64, staged = b0 + 80;  // two each; of staged four, [tile][parity]
    const uint32_t kv_full = b0 + 112, kv_empty = kv_full + 8 * ST;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 8; ++i) mbar_init(b0 + 8 * i, 1);
        for (int i = 0; i < 6; ++i) mbar_init(p_ready + 8 * i, 8);  // and staged
        for (int i = 0; i < 2 * ST; ++i) mbar_init(kv_full + 8 * i, 1);
        mbar_init(b0 + 8 * kLast, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sm.dead = sm.loads = 0u;
    }
    const uint32_t tmem = tmem_alloc_all(&sm.tmem);
    const Waits wait{&sm.dead};
    volatile uint32_t *loads = &sm.loads;
    const uint32_t tS = tmem, tO = tmem + 256;

    if (warp == 17) {
        // ------------------------------------------------------------ loads
        if ((threadIdx.x & 31) == 0) {
            uint32_t n = 0, it = 0;
            for (int item = blockIdx.x; item < items; item += gridDim.x) {
                const FwdItem w = fwd_item(g, item, tiles);
                const FwdTiles kt(g, w, wa_len(g, w.b));
                if (kt.count == 0) continue;
                const uint32_t qb = it & 1;
                if (it > 1) wait(q_empty + 8 * qb, it / 2 - 1, 21);
                if (*wait.dead != 0u) break;
                const bool two = kt.b.hi >= kt.b.lo;
                mbar_expect_tx(q_full + 8 * qb, two ? 2 * TB : TB);
                Tile<D>::load(sq + 2 * qb * TB, &maps.q, w.t0, w.h, w.b, q_full + 8 * qb);
                if (two) Tile<D>::load(sq + (2 * qb + 1) * TB, &maps.q, w.t0 + w.step_t, w.h + w.step_h, w.b, q_full + 8 * qb);
                for (int i = 0; i < 2 * kt.count; ++i, ++n) {
                    const uint32_t s = n % ST;
                    if (n >= ST) wait(kv_empty + 8 * s, n / ST - 1, 22);
                    if (*wait.dead != 0u) break;
                    mbar_expect_tx(kv_full + 8 * s, TB);
                    Tile<D>::load(skv + s * TB, (i & 1) ? &maps.v : &maps.k, kt.tile(i >> 1) * kWT, w.hk, w.b, kv_full + 8 * s);
                    *loads = n + 1;
                }
                ++it;
            }
            if (*wait.dead != 0u) drain(q_full, it, 2), drain(kv_full, n, ST);
        }
        __syncwarp();
    } else if (warp == 16) {
        // ------------------------------------------------------------ products
        // One stream of steps over all items: for each of the two tiles the output of the step
        // before, then the scores of this one, so that a tile begins the next item while the other
        // still ends the last.
        const uint32_t lead = elect();
        uint32_t j = 0, it = 0, np[2] = {0, 0};  // steps, items, probabilities taken
        const uint32_t negate = g.scale < 0.f ? kNegateA : 0u;
        bool owed[2] = {false, false}, begun[2] = {false, false}, ends[2] = {false, false};
        int rows = kWT;  // of the values of the step before, that lie in the sequence
        auto settle = [&](int u, bool &got) {  // o += P v of the step before
            if (!owed[u]) return;
            const uint32_t s = (2 * j - 1) % ST;
            if (!got) {
                wait(kv_full + 8 * s, (2 * j - 1) / ST, 24);
                if (g.lens != nullptr && rows < kWT) Tile<D>::zero_rows(skv + s * TB, rows);
                got = true;
            }
            wait(p_ready + 8 * u, np[u]++, 25);
            tc_fence_after();
            mma_apply<D, BF, 64>(lead, tO + 128 * u, tS + 128 * u, skv + s * TB, begun[u]);
            begun[u] = !ends[u];
            if (ends[u]) mma_commit(lead, o_full + 8 * u);
            owed[u] = false;
        };
        for (int item = blockIdx.x; item < items; item += gridDim.x) {
            const FwdItem w = fwd_item(g, item, tiles);
            const int len = uni(wa_len(g, w.b));
            const FwdTiles kt(g, w, len);
            if (kt.count == 0) continue;
            const uint32_t qb = it & 1;
            for (int i = 0; i < kt.count; ++i, ++j) {
                const uint32_t s = 2 * j % ST;
                const int tile = kt.tile(i);
                bool got_v = false, got_k = false;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const KeyTiles &mine = u == 0 ? kt.a : kt.b;
                    settle(u, got_v);
                    if (!mine.has(tile)) continue;
                    if (i == 0) wait(q_full + 8 * qb, it / 2, 23);
                    if (!got_k) wait(kv_full + 8 * s, 2 * j / ST, 26);
                    got_k = true;
                    tc_fence_after();
                    mma_scores<D, BF>(lead, tS + 128 * u, sq + (2 * qb + u) * TB, skv + s * TB, negate);
                    mma_commit(lead, s_full + 8 * u);
                    owed[u] = true;
                    ends[u] = tile == mine.hi;
                }
                if (j > 0) mma_commit(lead, kv_empty + 8 * ((2 * j - 1) % ST));
                mma_commit(lead, kv_empty + 8 * s);
                rows = len - tile * kWT;
            }
            ++it;
        }
        bool got = false;
        settle(0, got);
        settle(1, got);
        products_done(lead, b0);
    } else if (warp == 18) {
        // ------------------------------------------------------------ stores, which give the query tiles back
        if ((threadIdx.x & 31) == 0) {
            uint32_t it = 0, n[2] = {0, 0};
            for (int item = blockIdx.x; item < items; item += gridDim.x) {
                const FwdItem w = fwd_item(g, item, tiles);
                const FwdTiles kt(g, w, wa_len(g, w.b));
                if (kt.count == 0) continue;
                for (int u = 0; u < 2; ++u)
                    if (u == 0 || kt.b.hi >= kt.b.lo) {
                        wait.end(loads, staged + 16 * u + 8 * (n[u] & 1), n[u] >> 1, 29);
                        ++n[u];
                        if (*wait.dead == 0u)
                            store_tile<D>(&maps.x, sq + (2 * (it & 1) + u) * TB, w.t0 + u * w.step_t, w.h + u * w.step_h, w.b);
                    }
                tma_store_wait_read();
                mbar_arrive(q_empty + 8 * (it & 1));
                ++it;
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ probabilities and output
        const int u = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3, row = quarter * 32 + (threadIdx.x & 31);
        const uint32_t lanes = (uint32_t)quarter << 21, ts = tS + 128 * u + lanes, to = tO + 128 * u + lanes + half * (D / 2);
        const int id = 1 + u * 4 + quarter;
        // the scores of a negative factor come negated, and a factor of 0 must leave masked scores at -inf
        const float c = fmaxf(fabsf(g.scale) * 1.4426950408889634f, 1e-30f);
        float *own = &s_row[u][half][row], *other = &s_row[u][half ^ 1][row];
        uint32_t ns = 0, no = 0, it = 0;
        for (int item = blockIdx.x; item < items; item += gridDim.x) {
            const FwdItem w = fwd_item(g, item, tiles);
            const int len = wa_len(g, w.b), t0 = w.t0 + u * w.step_t, t = t0 + row;
            const FwdTiles kt(g, w, len);
            const KeyTiles mine = u == 0 ? kt.a : kt.b;
            float m = -INFINITY, l = 0.f;  // maximum in use (times c) and this half's sum
            bool first = true;
            for (int i = 0; i < kt.count; ++i) {
                const int tile = kt.tile(i);
                if (!mine.has(tile)) continue;
                const int s0 = tile * kWT + 64 * half;
                wait(s_full + 8 * u, ns++, 27);
                tc_fence_after();
                uint32_t r[64];
                tmem_ld32(ts + 64 * half, *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
                tmem_ld32(ts + 64 * half + 32, *reinterpret_cast<uint32_t(*)[32]>(&r[32]));
                tmem_ld_wait();
                if (tile_masked(g, t0, tile * kWT)) {
                    const uint32_t b0 = key_bits(g, t, s0), b1 = key_bits(g, t, s0 + 32);
                    if (!__all_sync(~0u, (b0 & b1) == ~0u)) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            if (!(b0 & (1u << k))) r[k] = 0xff800000u;
                            if (!(b1 & (1u << k))) r[32 + k] = 0xff800000u;
                        }
                    }
                }
                float mx[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    mx[k] = fmaxf(__uint_as_float(r[16 * k]), __uint_as_float(r[16 * k + 1]));
#pragma unroll
                    for (int j = 2; j < 16; j += 2)
                        mx[k] = fmaxf(fmaxf(__uint_as_float(r[16 * k + j]), __uint_as_float(r[16 * k + j + 1])), mx[k]);
                }
                float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                *own = top;
                quarter_sync<2>(id);
                top = fmaxf(top, *other) * c;
                const bool move = top > m + 8.f;
                if (__any_sync(~0u, move)) {
                    const float f = move ? ex2(m - top) : 1.f;
                    if (move) m = top;
                    l *= f;
                    if (!first) {
#pragma unroll 1
                        for (int k = 0; k < D / 2; k += 16) {
                            uint32_t x[16];
                            tmem_ld16(to + k, x);
                            tmem_ld_wait();
#pragma unroll
                            for (int j = 0; j < 16; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * f);
                            tmem_st16(to + k, x);
                        }
                    }
                }
                first = false;
                const float mu = m == -INFINITY ? 0.f : m;
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t p[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float2 x = __ffma2_rn(make_float2(__uint_as_float(r[32 * k + 2 * j]), __uint_as_float(r[32 * k + 2 * j + 1])),
                                                    make_float2(c, c), make_float2(-mu, -mu));
                        const float2 e = make_float2(ex2(x.x), ex2(x.y));
                        sum[j & 1] = __fadd2_rn(sum[j & 1], e);
                        p[j] = pack16<BF>(e);
                    }
                    tmem_st16(ts + 64 * half + 16 * k, p);
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                tmem_st_wait();
                tc_fence_before();
                warp_arrive(p_ready + 8 * u);
            }
            if (!first) {
                wait(o_full + 8 * u, no++, 28);
                tc_fence_after();
            }
            if (t0 < g.T) {  // the same for the whole tile
                const int h = w.h + u * w.step_h;
                const bool dead = t >= len;
                if (first) {
                    if (t < g.T) zero_row<D / 2>(o, w.b * so.b + h * so.h + t * so.t + half * (D / 2));
                } else {
                    *own = l;
                    quarter_sync<2>(id);
                    l += *other;
                    // into the query tile, whose last product is done
                    stage_row<D / 2, BF>(to, sq + (2 * (it & 1) + u) * TB, row, half * (D / 2), __fdividef(1.f, l), dead);
                }
                if (half == 0 && t < g.T)
                    lse[((long long)w.b * g.H + h) * g.T + t] = dead ? -INFINITY : (m + __log2f(l)) * 0.6931471805599453f;
            }
            tc_fence_before();
            if (!first) {
                warp_arrive(staged + 16 * u + 8 * ((no - 1) & 1));
                quarter_sync<2>(id);  // *other has been read
                ++it;
            } else if (kt.count > 0) {
                ++it;
            }
        }
    }
    tmem_free_all(tmem);
    leave_status<true>(hdr, sm);
}

// ------------------------------------------------------------------ backward: dq (and delta)
// One query tile at a time; each row's 128 scores and their gradients are shared by four threads
// (32 columns each).  Tensor memory: two score tiles in turn (dS is written over the scores), one
// dP tile, the accumulator.  While the math warps work on key tile i, the tensor cores form the
// scores of i + 1, and when its dS is there, dP of i + 1 and then dq += dS k.  In two groups of 64
// key columns, as the dk/dv kernel has them, it was slower (64 columns: 454 us for the whole pass at
// d = 64 against 447; 299 us against 250 at d = 128, where products 64 wide read the row operand
// twice as often).
template <int D>
struct DqCfg {
    // pairs of q and dO tiles: two where they fit, so that an item begins while the last one ends
    static constexpr int QST = D == 128 ? 1 : 2, KST = D == 128 ? 3 : 5, VST = D == 128 ? 2 : 4;
    static constexpr int SMEM = (2 * QST + KST + VST) * Tile<D>::BYTES + kSmall;
    // 16 math warps, products, loads, two for the rows' statistics, of which one also stores: a warp
    // more would cost 16 registers a thread
    static constexpr int THREADS = 640;
};

template <int D, bool BF>
__global__ void __launch_bounds__(DqCfg<D>::THREADS, 1)
wa_dq_kernel(const __grid_constant__ WaMaps maps, const void *__restrict__ o, const void *__restrict__ dO,
             const float *__restrict__ lse, void *__restrict__ dq, float *__restrict__ delta, Str3 so, Str3 sg, Str3 sdq,
             WaArgs g, int items, WsHeader *hdr) {
    constexpr int QST = DqCfg<D>::QST, KST = DqCfg<D>::KST, VST = DqCfg<D>::VST, TB = Tile<D>::BYTES;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t sq = smem_u32(smem_raw), sk = sq + 2 * QST * TB, sv = sk + KST * TB;  // q, dO in turn
    Small &sm = *reinterpret_cast<Small *>(smem_raw + (2 * QST + KST + VST) * TB);
    static_assert(15 + 2 * (KST + VST) <= kLast, "barriers");
    float(*s_stat)[2][kWT] = reinterpret_cast<float(*)[2][kWT]>(sm.f);  // [item's parity][delta, lse log2 e][row]
    if (misplaced(sq, hdr)) return;
    const int warp = threadIdx.x >> 5, tiles = (g.T + kWT - 1) / kWT;
    const uint32_t b0 = smem_u32(sm.bars);
    const uint32_t q_full = b0, q_empty = b0 + 16, acc_full = b0 + 32, dp_full = b0 + 40, s_full = b0 + 48, ds_ready = b0 + 64;
    const uint32_t st_full = b0 + 72, st_empty = b0 + 88;  // two each, by the item's parity
    const uint32_t staged = b0 + 104, x_empty = b0 + 112, k_full = b0 + 120, k_empty = k_full + 8 * KST, v_full = k_empty + 8 * KST, v_empty = v_full + 8 * VST;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 8; ++i) mbar_init(b0 + 8 * i, 1);
        mbar_init(ds_ready, 16);
        for (int i = 0; i < 2; ++i) mbar_init(st_full + 8 * i, 2), mbar_init(st_empty + 8 * i, 16);
        mbar_init(staged, 16);
        mbar_init(x_empty, 1);
        for (int i = 0; i < 2 * (KST + VST); ++i) mbar_init(k_full + 8 * i, 1);
        mbar_init(b0 + 8 * kLast, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sm.dead = sm.loads = 0u;
    }
    const uint32_t tmem = tmem_alloc_all(&sm.tmem);
    const Waits wait{&sm.dead};
    volatile uint32_t *loads = &sm.loads;
    const uint32_t tS = tmem, tP = tmem + 256, tA = tmem + 384;
    // items: all heads of the last tile, then of the one before it (as in the forward)
    auto place = [&](int item, int &b, int &h, int &hk, int &t0) {
        const int r = g.bh(item), bh = item - r * (int)g.bh.d;  // here B H
        t0 = (tiles - 1 - r) * kWT;
        b = g.heads(bh);
        h = bh - b * g.H;
        hk = g.group(h);
    };

    if (warp == 17) {
        if ((threadIdx.x & 31) == 0) {
            uint32_t n = 0, it = 0;
            for (int item = blockIdx.x; item < items; item += gridDim.x) {
                int b, h, hk, t0;
                place(item, b, h, hk, t0);
                const KeyTiles kt = key_tiles(g, t0, wa_len(g, b));
                if (kt.hi < kt.lo) continue;
                const int ns = min(kt.sinks, kt.lo), count = kt.hi - kt.lo + 1 + ns;
                const uint32_t qb = it % QST;
                if (it >= QST) wait(q_empty + 8 * qb, it / QST - 1, 31);
                if (*wait.dead != 0u) break;
                mbar_expect_tx(q_full + 8 * qb, 2 * TB);
                Tile<D>::load(sq + 2 * qb * TB, &maps.q, t0, h, b, q_full + 8 * qb);
                Tile<D>::load(sq + (2 * qb + 1) * TB, &maps.g, t0, h, b, q_full + 8 * qb);
                for (int i = 0; i < count; ++i, ++n) {
                    const int s0 = (i < ns ? i : kt.lo + i - ns) * kWT;
                    const uint32_t a = n % KST, c = n % VST;
                    if (n >= KST) wait(k_empty + 8 * a, n / KST - 1, 32);
                    if (*wait.dead != 0u) break;
                    mbar_expect_tx(k_full + 8 * a, TB);
                    Tile<D>::load(sk + a * TB, &maps.k, s0, hk, b, k_full + 8 * a);
                    if (n >= VST) wait(v_empty + 8 * c, n / VST - 1, 33);
                    mbar_expect_tx(v_full + 8 * c, TB);
                    Tile<D>::load(sv + c * TB, &maps.v, s0, hk, b, v_full + 8 * c);
                    *loads = n + 1;
                }
                ++it;
            }
            if (*wait.dead != 0u) drain(q_full, it, QST), drain(k_full, n, KST), drain(v_full, n, VST);
        }
        __syncwarp();
    } else if (warp == 16) {
        const uint32_t lead = elect();
        uint32_t n = 0, it = 0;
        for (int item = blockIdx.x; item < items; item += gridDim.x) {
            int b, h, hk, t0;
            place(item, b, h, hk, t0);
            const int len = uni(wa_len(g, b));
            const KeyTiles kt = key_tiles(g, t0, len);
            if (kt.hi < kt.lo) continue;
            const int ns = min(kt.sinks, kt.lo), count = kt.hi - kt.lo + 1 + ns;
            const uint32_t qb = it % QST;
            auto scores = [&](uint32_t j, int i) {  // key tile i of the item, number j of the block
                wait(k_full + 8 * (j % KST), j / KST, 34);
                const int left = len - (i < ns ? i : kt.lo + i - ns) * kWT;
                if (g.lens != nullptr && left < kWT) Tile<D>::zero_rows(sk + (j % KST) * TB, left);
                tc_fence_after();
                mma_scores<D, BF>(lead, tS + 128 * (j & 1), sq + 2 * qb * TB, sk + (j % KST) * TB);
                mma_commit(lead, s_full + 8 * (j & 1));
            };
            auto grads = [&](uint32_t j) {
                wait(v_full + 8 * (j % VST), j / VST, 35);
                tc_fence_after();
                mma_scores<D, BF>(lead, tP, sq + (2 * qb + 1) * TB, sv + (j % VST) * TB);
                mma_commit(lead, dp_full);
                mma_commit(lead, v_empty + 8 * (j % VST));
            };
            wait(q_full + 8 * qb, it / QST, 36);
            scores(n, 0);
            grads(n);
            for (int i = 0; i < count; ++i, ++n) {
                if (i + 1 < count) scores(n + 1, i + 1);
                wait(ds_ready, n, 37);
                tc_fence_after();
                if (i + 1 < count) grads(n + 1);
                else mma_commit(lead, q_empty + 8 * qb);
                mma_apply<D, BF, 32>(lead, tA, tS + 128 * (n & 1), sk + (n % KST) * TB, i > 0);
                // an item's last key tile becomes the place of its output
                if (i + 1 < count) mma_commit(lead, k_empty + 8 * (n % KST));
            }
            mma_commit(lead, acc_full);
            ++it;
        }
        products_done(lead, b0);
    } else if (warp >= 18) {
        // ------------------------------------------------------------ delta = dO . o and lse of the next item's rows
        // A warp takes 64 rows; the second of them also stores dq, of the item before the one whose
        // statistics it has formed.  delta is the diagonal of dO o^T: 16 rows against 8 and 8, 16 bytes of
        // them a lane as they come from memory.  (Sums of unpacked products took 11000 cycles of one
        // warp, more than an item of five key tiles; so did the rows from DRAM, which are therefore
        // asked for into L2 an item before.)
        const int lane = threadIdx.x & 31, r = lane >> 2, col = (lane & 3) * 8;
        uint32_t all = 0, it = 0, last = 0;
        auto store = [&](int item) {
            int b, h, hk, t0;
            place(item, b, h, hk, t0);
            const KeyTiles kt = key_tiles(g, t0, wa_len(g, b));
            if (kt.hi < kt.lo) return;
            last += kt.hi - kt.lo + 1 + min(kt.sinks, kt.lo);
            const uint32_t s = (last - 1) % KST;
            if (lane == 0) {
                wait.end(loads, staged, it, 43);
                if (*wait.dead == 0u) store_tile<D>(&maps.x, sk + s * TB, t0, h, b);
                tma_store_wait_read();
                mbar_arrive(x_empty);
                mbar_arrive(k_empty + 8 * s);
            }
            __syncwarp();
            ++it;
        };
        for (int item = blockIdx.x; item < items; item += gridDim.x, ++all) {
            int b, h, hk, t0;
            place(item, b, h, hk, t0);
            const int len = wa_len(g, b);
            const uint16_t *x = static_cast<const uint16_t *>(o) + b * so.b + h * so.h + col;
            const uint16_t *y = static_cast<const uint16_t *>(dO) + b * sg.b + h * sg.h + col;
            const long long at = ((long long)b * g.H + h) * g.T;
            float ls[2];  // P, and with it dS, of a row without a gradient is 0
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int t = t0 + (warp - 18) * 64 + lane + 32 * k;
                ls[k] = t < len && !sees_one(g, t) ? __ldg(lse + at + t) * 1.4426950408889634f : INFINITY;
            }
            if (item < items - (int)gridDim.x) {
                int b, h, hk, t0;
                place(item + gridDim.x, b, h, hk, t0);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int t = t0 + (warp - 18) * 64 + lane + 32 * k;
                    if (t >= wa_len(g, b)) continue;
#pragma unroll
                    for (int c = 0; c < D; c += 64) {
                        prefetch_l2(static_cast<const uint16_t *>(o) + b * so.b + h * so.h + t * so.t + c);
                        prefetch_l2(static_cast<const uint16_t *>(dO) + b * sg.b + h * sg.h + t * sg.t + c);
                    }
                }
            }
            if (all > 1) wait.end(loads, st_empty + 8 * (all & 1), all / 2 - 1, 42);
            float *dst = s_stat[all & 1][0], *dst2 = s_stat[all & 1][1];
#pragma unroll
            for (int k = 0; k < 2; ++k) dst2[(warp - 18) * 64 + lane + 32 * k] = ls[k];
#pragma unroll 1
            for (int r0 = (warp - 18) * 64; r0 < (warp - 18) * 64 + 64; r0 += 32) {
                float acc[4][4];  // rows r0 + 8 k ..
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[k][0] = acc[k][1] = acc[k][2] = acc[k][3] = 0.f;
#pragma unroll 1
                for (int c = 0; c < D; c += 64) {
                    uint4 xv[4][2], yv[4][2];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int t = t0 + r0 + 8 * k + r;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            xv[k][e] = t < len ? __ldg(reinterpret_cast<const uint4 *>(x + t * so.t + c + 32 * e)) : make_uint4(0u, 0u, 0u, 0u);
                            yv[k][e] = t < len ? __ldg(reinterpret_cast<const uint4 *>(y + t * sg.t + c + 32 * e)) : make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint4 &a = yv[k & ~1][e], &b = yv[k | 1][e], &o = xv[k][e];
                            mma16x8<BF>(acc[k], a.x, b.x, a.y, b.y, o.x, o.y);
                            mma16x8<BF>(acc[k], a.z, b.z, a.w, b.w, o.z, o.w);
                        }
                }
                if ((lane & 3) == r >> 1) {  // the lanes that hold the diagonals
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float sum = (r & 1) ? acc[k][2 * (k & 1) + 1] : acc[k][2 * (k & 1)];
                        const int row = r0 + 8 * k + r, t = t0 + row;
                        dst[row] = sum;
                        if (t < g.T) delta[at + t] = sum;
                    }
                }
            }
            warp_arrive(st_full + 8 * (all & 1));
            if (warp == 19 && all > 0) store(item - gridDim.x);
        }
        if (warp == 19 && all > 0) store(blockIdx.x + (all - 1) * gridDim.x);
    } else {
        const int part = warp >> 2, quarter = warp & 3, row = quarter * 32 + (threadIdx.x & 31);  // columns 32 part ..
        const uint32_t lanes = (uint32_t)quarter << 21;
        const float c = g.scale * 1.4426950408889634f;
        uint32_t n = 0, it = 0, all = 0;
        for (int item = blockIdx.x; item < items; item += gridDim.x) {
            int b, h, hk, t0;
            place(item, b, h, hk, t0);
            const int len = wa_len(g, b), t = t0 + row;
            const KeyTiles kt = key_tiles(g, t0, len);
            const bool live = t < len;
            wait(st_full + 8 * (all & 1), all / 2, 41);
            const float dl = s_stat[all & 1][0][row], ls = s_stat[all & 1][1][row];
            warp_arrive(st_empty + 8 * (all & 1));
            ++all;
            const int ns = min(kt.sinks, kt.lo), count = kt.hi < kt.lo ? 0 : kt.hi - kt.lo + 1 + ns;
            for (int i = 0; i < count; ++i, ++n) {
                const int s0 = (i < ns ? i : kt.lo + i - ns) * kWT;
                const uint32_t ts = tS + 128 * (n & 1) + lanes;
                wait(s_full + 8 * (n & 1), n >> 1, 38);
                tc_fence_after();
                uint32_t r[32], e[32], ds[16];
                tmem_ld32(ts + 32 * part, r);
                tmem_ld_wait();
                float2 *x = reinterpret_cast<float2 *>(r);
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float2 y = __ffma2_rn(x[k], make_float2(c, c), make_float2(-ls, -ls));
                    x[k] = make_float2(ex2(y.x), ex2(y.y));
                }
                wait(dp_full, n, 39);
                tc_fence_after();
                tmem_ld32(tP + lanes + 32 * part, e);
                tmem_ld_wait();
                const float2 *y = reinterpret_cast<const float2 *>(e);
#pragma unroll
                for (int k = 0; k < 16; ++k) x[k] = __fmul2_rn(x[k], __fadd2_rn(y[k], make_float2(-dl, -dl)));
                if (tile_masked(g, t0, s0)) {
                    const uint32_t bits = key_bits(g, t, s0 + 32 * part);
                    if (!__all_sync(~0u, bits == ~0u)) {
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (!(bits & (1u << k))) r[k] = 0u;
                    }
                }
#pragma unroll
                for (int k = 0; k < 16; ++k) ds[k] = pack16<BF>(x[k]);
                tmem_st16(ts + 32 * part, ds);
                tmem_st_wait();
                tc_fence_before();
                warp_arrive(ds_ready);
            }
            if (count > 0) {
                if (it > 0) wait(x_empty, it - 1, 44);  // the item before this one's output has been read
                wait(acc_full, it, 40);
                tc_fence_after();
                stage_row<D / 4, BF>(tA + lanes + part * (D / 4), sk + (n - 1) % KST * TB, row, part * (D / 4), g.scale, !live);
                tc_fence_before();
                warp_arrive(staged);
                ++it;
            } else if (t < g.T) {
                zero_row<D / 4>(dq, b * sdq.b + h * sdq.h + t * sdq.t + part * (D / 4));
            }
        }
    }
    tmem_free_all(tmem);
    leave_status<true>(hdr, sm);
}

// ------------------------------------------------------------------ backward: dk, dv
// A key tile against the query tiles that see it, head by head of the group.  The scores are
// transposed (a row is a key), so that P^T and dS^T are A operands from tensor memory: S^T = K Q^T,
// dP^T = V dO^T, dv += P^T dO, dk += dS^T Q, with P^T over S^T and dS^T over dP^T.  The
// 128 queries of a step are two halves, each with its own eight warps, products and barriers and half
// a step behind the other, so that one forms P while the other forms dS (347 -> 343 us at d = 128,
// 176 -> 172 at d = 64 against all 16 warps in step).
//
// The lists of the key tiles, one behind the other (sequence, key head, tile), are cut into equal
// shares, one a block: few tiles with long lists (sinks are seen by every later query) and a
// number of tiles that the blocks do not divide cost nothing.  A list that is cut leaves fp32
// partial sums, which wa_join_kernel adds in their order; where the cuts are depends on the sizes, the
// lengths and the device's multiprocessors.
template <int D>
struct DkvCfg {
    // Stages of q and of dO, and pairs of k and v tiles: two where they fit, so that a list begins while
    // the last one ends.  The scores of step i + 2 are asked for before the last product with q of
    // step i is: q needs three stages.
    static constexpr int QST = D == 128 ? 3 : 4, GST = D == 128 ? 2 : 4, KVST = D == 128 ? 1 : 2;
    static constexpr int SMEM = (2 * KVST + QST + GST) * Tile<D>::BYTES + kSmall;
    static constexpr int THREADS = 640;  // 16 math warps, products, loads, statistics, stores
};

// The lists of a sequence of n tiles: tile k is seen by n - k query tiles if it has sinks (k < st),
// else by at most `span` of them.
struct Lists {
    int n, st, span;
    __host__ __device__ __forceinline__ Lists(int len, int window, int sinks)
        : n((int)(((long long)len + kWT - 1) / kWT)), st(0), span((int)(((long long)window + kWT - 2) / kWT) + 1) {
        st = (int)(((long long)sinks + kWT - 1) / kWT);
        if (st > n) st = n;
    }
    __host__ __device__ __forceinline__ int of(int k) const { return k < st || n - k < span ? n - k : span; }
    __host__ __device__ __forceinline__ long long all(long long x) const { return x * n - x * (x - 1) / 2; }
    __host__ __device__ __forceinline__ long long banded(long long x) const {
        const long long full = n - span + 1 > 0 ? n - span + 1 : 0;
        return x <= full ? x * span : full * span + all(x) - all(full);
    }
    __host__ __device__ __forceinline__ long long before(int k) const {  // query tiles in the lists of tiles below k
        return k <= st ? all(k) : all(st) + banded(k) - banded(st);
    }
};

// A place in the chain of lists: step i of `tile`'s (query tile tile + i % f of head i / f).
struct Place {
    int b, hk, tile, i;
};
// The whole chain's length, and the place of its step `pos`; by one warp, the result in all lanes.
__device__ __forceinline__ long long chain_length(const WaArgs &g) {
    if (g.lens == nullptr) {
        const Lists l(g.T, g.window, g.sinks);
        return (long long)g.B * g.H * l.before(l.n);
    }
    long long sum = 0;
    for (int b = threadIdx.x & 31; b < g.B; b += 32) {
        const Lists l(wa_len(g, b), g.window, g.sinks);
        sum += g.H * l.before(l.n);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    return sum;
}
__device__ __forceinline__ Place chain_place(const WaArgs &g, long long pos) {
    Place p{0, 0, 0, 0};
    if (g.lens == nullptr) {
        const Lists l(g.T, g.window, g.sinks);
        const long long u = g.H * l.before(l.n);
        p.b = (int)(pos / u);
        pos -= p.b * u;
    } else {
        for (int b = 0; b < g.B; b += 32) {
            const int mine = b + (threadIdx.x & 31);
            long long u = 0;
            if (mine < g.B) {
                const Lists l(wa_len(g, mine), g.window, g.sinks);
                u = g.H * l.before(l.n);
            }
            long long run = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long x = __shfl_up_sync(~0u, run, o);
                if ((int)(threadIdx.x & 31) >= o) run += x;
            }
            const unsigned int in = __ballot_sync(~0u, pos < run);
            if (in != 0u) {
                const int at = __ffs(in) - 1;
                p.b = b + at;
                pos -= __shfl_sync(~0u, run - u, at);
                break;
            }
            pos -= __shfl_sync(~0u, run, 31);
        }
    }
    const Lists l(wa_len(g, p.b), g.window, g.sinks);
    const int G = g.H / g.Hkv;
    const long long head = G * l.before(l.n);
    p.hk = (int)(pos / head);
    pos -= p.hk * head;
    int lo = 0, hi = l.n - 1;  // the last tile whose list begins at or before pos
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (G * l.before(mid) <= pos) lo = mid;
        else hi = mid - 1;
    }
    p.tile = lo;
    p.i = (int)(pos - G * l.before(lo));
    return p;
}
// Walks a block's share, a tile's part of it at a time: steps [i0, i1) of `list` of that tile.
struct Walk {
    const WaArgs &g;
    long long left;
    Place p;
    int len, f, i0, i1, list;
    __device__ __forceinline__ Walk(const WaArgs &a, const Place &start, long long steps) : g(a), left(steps), p(start), i1(start.i), list(0) {
        len = wa_len(g, p.b);
    }
    __device__ __forceinline__ bool next() {
        if (left <= 0) return false;
        if (list != 0) {  // not the first: the tile before was walked to its end
            i1 = 0;
            if (++p.tile * (long long)kWT >= len) {
                p.tile = 0;
                if (++p.hk == g.Hkv) {
                    p.hk = 0;
                    do len = wa_len(g, ++p.b);
                    while (len == 0);
                }
            }
        }
        const Lists l(len, g.window, g.sinks);
        f = l.of(p.tile);
        list = f * (g.H / g.Hkv);
        i0 = i1;
        i1 = left < list - i0 ? i0 + (int)left : list;
        left -= i1 - i0;
        return true;
    }
};

// What a block tells wa_join_kernel: the tile whose list it leaves before its end (tile < 0: none;
// its sums are part 1), and whether it joins a list after its start (part 0), and ends it.
struct CutList {
    int b, hk, tile;
    int joins;  // 0: no, 1: and leaves it before its end too, 2: to its end
};

template <int D, bool BF>
__global__ void __launch_bounds__(DkvCfg<D>::THREADS, 1)
wa_dkv_kernel(const __grid_constant__ WaMaps maps, const float *__restrict__ lse, const float *__restrict__ delta,
              void *__restrict__ dk, void *__restrict__ dv, float *__restrict__ parts, CutList *__restrict__ cuts, Str3 sdk,
              Str3 sdv, WaArgs g, WsHeader *hdr) {
    constexpr int QST = DkvCfg<D>::QST, GST = DkvCfg<D>::GST, KVST = DkvCfg<D>::KVST, TB = Tile<D>::BYTES;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t sk = smem_u32(smem_raw), sq = sk + 2 * KVST * TB, sg = sq + QST * TB;  // k, v in turn
    Small &sm = *reinterpret_cast<Small *>(smem_raw + (2 * KVST + QST + GST) * TB);
    static_assert(17 + 2 * (QST + GST) + 4 <= kLast, "barriers");
    static_assert(QST >= 3 && GST >= 2, "stages");
    float(*s_stat)[2][kWT] = reinterpret_cast<float(*)[2][kWT]>(sm.f);  // [slot][lse log2 e, delta][query]
    if (misplaced(sk, hdr)) {
        if (threadIdx.x == 0) cuts[blockIdx.x] = CutList{0, 0, -1, 0};  // nothing to join
        return;
    }
    const int warp = threadIdx.x >> 5, G = g.H / g.Hkv;
    const uint32_t b0 = smem_u32(sm.bars);
    const uint32_t kv_full = b0, kv_empty = b0 + 16, acc_full = b0 + 32;
    const uint32_t s_full = b0 + 40, dp_full = b0 + 56, p_ready = b0 + 72, ds_ready = b0 + 88;  // of each half
    const uint32_t staged = b0 + 104;  // [dk, dv][parity of the list]
    const uint32_t q_full = b0 + 136, q_empty = q_full + 8 * QST, g_full = q_empty + 8 * QST, g_empty = g_full + 8 * GST;
    const uint32_t st_full = g_empty + 8 * GST, st_empty = st_full + 16;
    if (warp == 1) {  // this block's share of the chain
        const long long total = chain_length(g), p0 = total * blockIdx.x / gridDim.x, p1 = total * (blockIdx.x + 1) / gridDim.x;
        Place p{0, 0, 0, 0};
        if (p1 > p0) p = chain_place(g, p0);
        if (threadIdx.x == 32) {
            *reinterpret_cast<Place *>(sm.pad) = p;
            *reinterpret_cast<long long *>(sm.pad + 4) = p1 - p0;
        }
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < 9; ++i) mbar_init(b0 + 8 * i, 1);
        for (int i = 0; i < 8; ++i) mbar_init(p_ready + 8 * i, 8);  // ds_ready and staged too
        for (int i = 0; i < 2 * (QST + GST); ++i) mbar_init(q_full + 8 * i, 1);
        for (int i = 0; i < 2; ++i) mbar_init(st_full + 8 * i, 1), mbar_init(st_empty + 8 * i, 16);
        mbar_init(b0 + 8 * kLast, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sm.dead = sm.loads = 0u;
    }
    const uint32_t tmem = tmem_alloc_all(&sm.tmem);
    const Waits wait{&sm.dead};
    volatile uint32_t *loads = &sm.loads;
    const uint32_t tS = tmem, tP = tmem + 128, tV = tmem + 256, tK = tmem + 384;
    Walk w(g, *reinterpret_cast<const Place *>(sm.pad), *reinterpret_cast<const long long *>(sm.pad + 4));
    // the head and the query tile of a step, without a division in the loops
    struct Step {
        int h, qt;
    };
    auto first_step = [&]() {
        if (w.i0 == 0) return Step{w.p.hk * G, w.p.tile};
        return Step{w.p.hk * G + w.i0 / w.f, w.p.tile + w.i0 % w.f};
    };
    auto advance = [&](Step &s) {
        if (++s.qt == w.p.tile + w.f) s.qt = w.p.tile, ++s.h;
    };

    if (warp == 17) {
        if ((threadIdx.x & 31) == 0) {
            uint32_t n = 0, it = 0;
            while (w.next()) {
                const uint32_t kb = it % KVST;
                if (it >= KVST) wait(kv_empty + 8 * kb, it / KVST - 1, 51);
                if (*wait.dead != 0u) break;
                mbar_expect_tx(kv_full + 8 * kb, 2 * TB);
                Tile<D>::load(sk + 2 * kb * TB, &maps.k, w.p.tile * kWT, w.p.hk, w.p.b, kv_full + 8 * kb);
                Tile<D>::load(sk + (2 * kb + 1) * TB, &maps.v, w.p.tile * kWT, w.p.hk, w.p.b, kv_full + 8 * kb);
                Step x = first_step();
                for (int i = w.i0; i < w.i1; ++i, ++n, advance(x)) {
                    const uint32_t s = n % QST, r = n % GST;
                    if (n >= QST) wait(q_empty + 8 * s, n / QST - 1, 42);
                    if (*wait.dead != 0u) break;
                    mbar_expect_tx(q_full + 8 * s, TB);
                    Tile<D>::load(sq + s * TB, &maps.q, x.qt * kWT, x.h, w.p.b, q_full + 8 * s);
                    if (n >= GST) wait(g_empty + 8 * r, n / GST - 1, 43);
                    mbar_expect_tx(g_full + 8 * r, TB);
                    Tile<D>::load(sg + r * TB, &maps.g, x.qt * kWT, x.h, w.p.b, g_full + 8 * r);
                    *loads = n + 1;
                }
                ++it;
            }
            if (*wait.dead != 0u) drain(kv_full, it, KVST), drain(q_full, n, QST), drain(g_full, n, GST);
        }
        __syncwarp();
    } else if (warp == 18) {
        // ------------------------------------------------------------ the rows' statistics, a tile ahead
        const int lane = threadIdx.x & 31;
        uint32_t n = 0;
        CutList cut{0, 0, -1, 0};
        while (w.next()) {
            if (w.i0 > 0) cut.joins = w.i1 < w.list ? 1 : 2;
            else if (w.i1 < w.list) cut.b = w.p.b, cut.hk = w.p.hk, cut.tile = w.p.tile;
            Step x = first_step();
            for (int i = w.i0; i < w.i1; ++i, ++n, advance(x)) {
                const uint32_t s = n & 1;
                const int t0 = x.qt * kWT;
                const long long at = ((long long)w.p.b * g.H + x.h) * g.T + t0;
                float a[4], d[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int j = lane + 32 * k;
                    const bool in = t0 + j < w.len;  // behind the length P is 0
                    a[k] = in ? __ldg(lse + at + j) * 1.4426950408889634f : INFINITY;
                    d[k] = in ? __ldg(delta + at + j) : 0.f;
                }
                if (n >= 2) wait(st_empty + 8 * s, n / 2 - 1, 44);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    s_stat[s][0][lane + 32 * k] = a[k];
                    s_stat[s][1][lane + 32 * k] = d[k];
                }
                warp_arrive(st_full + 8 * s);
            }
        }
        if (lane == 0) cuts[blockIdx.x] = cut;
    } else if (warp == 19) {
        // ------------------------------------------------------------ stores, which give the key tiles back
        if ((threadIdx.x & 31) == 0) {
            uint32_t it = 0;
            while (w.next()) {
                for (int which = 0; which < 2; ++which) {
                    wait.end(loads, staged + 16 * which + 8 * (it & 1), it >> 1, 54);
                    if (w.i0 == 0 && w.i1 == w.list && *wait.dead == 0u)
                        store_tile<D>(which == 0 ? &maps.x : &maps.y, sk + (2 * (it % KVST) + which) * TB, w.p.tile * kWT, w.p.hk, w.p.b);
                }
                tma_store_wait_read();
                mbar_arrive(kv_empty + 8 * (it % KVST));
                ++it;
            }
        }
        __syncwarp();
    } else if (warp == 16) {
        const uint32_t lead = elect();
        uint32_t n = 0, it = 0;
        while (w.next()) {
            const int i0 = uni(w.i0), i1 = uni(w.i1), len = uni(w.len), tile = uni(w.p.tile), f = uni(w.f);
            const uint32_t kb = it % KVST, kt = sk + 2 * kb * TB;
            auto scores = [&](uint32_t j, int qt, int u) {
                const uint32_t s = j % QST;
                if (u == 0) {
                    wait(q_full + 8 * s, j / QST, 45);
                    if (g.lens != nullptr && len - qt * kWT < kWT) Tile<D>::zero_rows(sq + s * TB, len - qt * kWT);
                }
                tc_fence_after();
                mma_scores<D, BF, 64>(lead, tS + 64 * u, kt, sq + s * TB + u * kHalf);
                mma_commit(lead, s_full + 8 * u);
            };
            auto grads = [&](uint32_t j, int qt, int u) {
                const uint32_t s = j % GST;
                if (u == 0) {
                    wait(g_full + 8 * s, j / GST, 46);
                    if (g.lens != nullptr && len - qt * kWT < kWT) Tile<D>::zero_rows(sg + s * TB, len - qt * kWT);
                }
                tc_fence_after();
                mma_scores<D, BF, 64>(lead, tP + 64 * u, kt + TB, sg + s * TB + u * kHalf);
                mma_commit(lead, dp_full + 8 * u);
            };
            // of step j: dv += P^T dO of a half, then the half's next scores; dk += dS^T Q, then its next dP
            auto values = [&](uint32_t j, int u, bool first, bool last, int next) {
                const uint32_t s = j % GST;
                wait(p_ready + 8 * u, j, 48);
                tc_fence_after();
                mma_apply<D, BF, 32, 64>(lead, tV, tS + 64 * u, sg + s * TB + u * kHalf, !first || u > 0);
                if (u == 1) mma_commit(lead, g_empty + 8 * s);
                if (!last) scores(j + 1, next, u);
            };
            auto keys = [&](uint32_t j, int u, bool first, bool last, int next) {
                const uint32_t s = j % QST;
                wait(ds_ready + 8 * u, j, 49);
                tc_fence_after();
                mma_apply<D, BF, 32, 64>(lead, tK, tP + 64 * u, sq + s * TB + u * kHalf, !first || u > 0);
                if (u == 1) mma_commit(lead, q_empty + 8 * s);
                if (!last) grads(j + 1, next, u);
            };
            int qt = tile + uni(i0 == 0 ? 0 : i0 % f);
            wait(kv_full + 8 * kb, it / KVST, 47);
#pragma unroll
            for (int u = 0; u < 2; ++u) scores(n, qt, u), grads(n, qt, u);
            for (int i = i0; i < i1; ++i, ++n) {
                const int now = qt;
                if (++qt == tile + f) qt = tile;  // of step i + 1
                const bool first = i == i0, last = i + 1 == i1;
                values(n, 0, first, last, qt);
                // the second half's gradients of the step before; in a list's first step its values, with
                // which its warps say that they have read the accumulators of the list before
                if (first) values(n, 1, first, last, qt);
                else keys(n - 1, 1, i - 1 == i0, false, now);
                keys(n, 0, first, last, qt);
                if (!first) values(n, 1, first, last, qt);
            }
            keys(n - 1, 1, i1 - 1 == i0, true, 0);
            mma_commit(lead, acc_full);
            ++it;
        }
        products_done(lead, b0);
    } else {
        const int part = warp >> 2, quarter = warp & 3, row = quarter * 32 + (threadIdx.x & 31);  // queries 32 part ..
        const uint32_t lanes = (uint32_t)quarter << 21;
        const float c = g.scale * 1.4426950408889634f;
        // dv by the first half's warps, dk by the second's: a list's first product for dv follows the
        // first half's probabilities, its first product for dk those of both
        const int u = part >> 1, which = u ^ 1, col = (part & 1) * (D / 2);
        uint32_t n = 0, it = 0;
        while (w.next()) {
            const int s0 = w.p.tile * kWT, key = s0 + row;
            Step st = first_step();
            for (int i = w.i0; i < w.i1; ++i, ++n, advance(st)) {
                const int t0 = st.qt * kWT;
                const uint32_t sl = n & 1;
                wait(st_full + 8 * sl, n >> 1, 50);
                wait(s_full + 8 * u, n, 51);
                tc_fence_after();
                uint32_t r[32], e[32], p[16];
                tmem_ld32(tS + lanes + 32 * part, r);
                tmem_ld_wait();
                float2 *x = reinterpret_cast<float2 *>(r);
                const float4 *ls = reinterpret_cast<const float4 *>(&s_stat[sl][0][32 * part]);
                const float4 *dl = reinterpret_cast<const float4 *>(&s_stat[sl][1][32 * part]);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float4 z = ls[k];
                    const float2 y0 = __ffma2_rn(x[2 * k], make_float2(c, c), make_float2(-z.x, -z.y));
                    const float2 y1 = __ffma2_rn(x[2 * k + 1], make_float2(c, c), make_float2(-z.z, -z.w));
                    x[2 * k] = make_float2(ex2(y0.x), ex2(y0.y));
                    x[2 * k + 1] = make_float2(ex2(y1.x), ex2(y1.y));
                }
                if (tile_masked(g, t0, s0)) {
                    const uint32_t bits = query_bits(g, t0 + 32 * part, key);
                    if (!__all_sync(~0u, bits == ~0u)) {
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (!(bits & (1u << k))) r[k] = 0u;
                    }
                }
#pragma unroll
                for (int k = 0; k < 16; ++k) p[k] = pack16<BF>(x[k]);
                tmem_st16(tS + lanes + 32 * part, p);
                tmem_st_wait();
                tc_fence_before();
                warp_arrive(p_ready + 8 * u);
                wait(dp_full + 8 * u, n, 52);
                tc_fence_after();
                tmem_ld32(tP + lanes + 32 * part, e);
                tmem_ld_wait();
                const float2 *y = reinterpret_cast<const float2 *>(e);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float4 z = dl[k];
                    p[2 * k] = pack16<BF>(__fmul2_rn(x[2 * k], __fadd2_rn(y[2 * k], make_float2(-z.x, -z.y))));
                    p[2 * k + 1] = pack16<BF>(__fmul2_rn(x[2 * k + 1], __fadd2_rn(y[2 * k + 1], make_float2(-z.z, -z.w))));
                }
                if (g.window == 1 && g.sinks == 0) {
#pragma unroll
                    for (int k = 0; k < 16; ++k) p[k] = 0u;
                } else if (t0 == 0 && part == 0) {
                    p[0] &= 0xffff0000u;  // query 0
                }
                tmem_st16(tP + lanes + 32 * part, p);
                tmem_st_wait();
                tc_fence_before();
                warp_arrive(ds_ready + 8 * u);
                warp_arrive(st_empty + 8 * sl);
            }
            const bool zero = key >= w.len, whole = w.i0 == 0 && w.i1 == w.list;
            wait(acc_full, it, 53);
            tc_fence_after();
            const uint32_t acc = (which == 0 ? tK : tV) + lanes + col;
            const uint32_t tile = sk + (2 * (it % KVST) + which) * TB;  // k's or v's, whose last product is done
            const float f = which == 0 ? g.scale : 1.f;
            if (whole) {
                stage_row<D / 2, BF>(acc, tile, row, col, f, zero);
            } else {
                // part 0 of a block: a list it joins after its start; part 1: one it leaves before its end.
                // Four columns of all rows next to each other.
                float4 *p = reinterpret_cast<float4 *>(parts + ((2ll * blockIdx.x + (w.i0 > 0 ? 0 : 1)) * 2 + which) * (kWT * D)) + row;
#pragma unroll
                for (int k = 0; k < D / 2; k += 16) {
                    uint32_t r[16];
                    tmem_ld16(acc + k, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        p[((col + k) / 4 + j) * kWT] = zero ? make_float4(0.f, 0.f, 0.f, 0.f)
                                                            : make_float4(__uint_as_float(r[4 * j]) * f, __uint_as_float(r[4 * j + 1]) * f,
                                                                          __uint_as_float(r[4 * j + 2]) * f, __uint_as_float(r[4 * j + 3]) * f);
                }
            }
            tc_fence_before();
            warp_arrive(staged + 16 * which + 8 * (it & 1));
            ++it;
        }
        // the tiles behind a sequence's length, which are in no list
        if (g.lens != nullptr) {
            const int tiles = (g.T + kWT - 1) / kWT;
            const long long units = (long long)g.B * g.Hkv * tiles;
            for (long long u = blockIdx.x; u < units; u += gridDim.x) {
                const int tile = (int)(u % tiles), hk = (int)(u / tiles % g.Hkv), b = (int)(u / tiles / g.Hkv);
                const int key = tile * kWT + row;
                if (tile * kWT < wa_len(g, b) || key >= g.T) continue;
                const Str3 st = which == 0 ? sdk : sdv;
                zero_row<D / 2>(which == 0 ? dk : dv, b * st.b + hk * st.h + key * st.t + col);
            }
        }
    }
    tmem_free_all(tmem);
    leave_status<false>(hdr, sm);
}

// Adds the parts of a list that was cut, in their order: block (x, y) those of the list that block x
// of wa_dkv_kernel left, y an eighth of the columns of dk and dv.  Parts come with the rows next to
// each other and go out with the columns so, through shared memory.  At 151 cuts of 128 x 128 it reads
// 40 MB in 10 us (4 TB/s).
constexpr int kJoinY = 8;
template <int D, bool BF>
__global__ void __launch_bounds__(256) wa_join_kernel(const float *__restrict__ parts, const CutList *__restrict__ cuts,
                                                      void *__restrict__ dk, void *__restrict__ dv, Str3 sdk, Str3 sdv, int T,
                                                      int blocks) {
    constexpr int C = D / 4, N = 2 * kWT * C, CY = C / kJoinY, PER = 2 * CY * kWT / 256;  // float4 columns: all, a block's
    __shared__ uint2 out[2 * kWT][CY + 1];
    const int x0 = blockIdx.x;
    const CutList c = cuts[x0];
    if (c.tile < 0) return;
    const float4 *src = reinterpret_cast<const float4 *>(parts);
    const int row = threadIdx.x % kWT, first = threadIdx.x / kWT;
    // the k-th of this thread: row `row` of column which * C + blockIdx.y * CY + j
    auto at = [&](int k) {
        const int u = first + 2 * k, which = u / CY, j = u % CY;
        return (which * C + blockIdx.y * CY + j) * kWT + row;
    };
    float4 s[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) s[k] = src[(2ll * x0 + 1) * N + at(k)];
    for (int x = x0 + 1; x < blocks; ++x) {
        const int joins = cuts[x].joins;
        if (joins == 0) continue;  // a block without a share
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const float4 y = src[2ll * x * N + at(k)];
            s[k].x += y.x;
            s[k].y += y.y;
            s[k].z += y.z;
            s[k].w += y.w;
        }
        if (joins == 2) break;
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int u = first + 2 * k;
        out[u / CY * kWT + row][u % CY] = make_uint2(pack16<BF>(make_float2(s[k].x, s[k].y)), pack16<BF>(make_float2(s[k].z, s[k].w)));
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int i = threadIdx.x + k * 256, r = i / CY, j = i % CY, which = r / kWT, key = c.tile * kWT + r % kWT;
        if (key >= T) continue;
        const Str3 st = which == 0 ? sdk : sdv;
        uint16_t *to = static_cast<uint16_t *>(which == 0 ? dk : dv) + c.b * st.b + c.hk * st.h + key * st.t;
        *reinterpret_cast<uint2 *>(to + 4 * (blockIdx.y * CY + j)) = out[r][j];
    }
}

// 4-D map over [B][heads][T][d] with the tensor's own strides, boxes of 64 columns x 128 tokens.
bool make_map_bht(CUtensorMap *m, const void *base, bool bf, int64_t d, int64_t T, int64_t heads, int64_t B, const Str3 &s) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)T, (cuuint64_t)heads, (cuuint64_t)B};
    // the stride of a dimension of one element is not used
    cuuint64_t strides[3] = {(cuuint64_t)(s.t ? s.t : d) * 2, (cuuint64_t)(s.h ? s.h : d) * 2, (cuuint64_t)(s.b ? s.b : d) * 2};
    cuuint32_t box[4] = {64u, (cuuint32_t)kWT, 1u, 1u}, estr[4] = {1u, 1u, 1u, 1u};
    return enc(m, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void *>(base), dims,
               strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace cla
