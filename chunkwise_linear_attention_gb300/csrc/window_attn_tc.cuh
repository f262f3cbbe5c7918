// window_attn_tc.cuh -- the training and prefill kernels of window_attn.cu on
// the fifth-generation tensor cores: TMA tile loads, tcgen05.mma with the
// accumulators in tensor memory, probabilities and their gradients rounded to
// the tensors' type and fed back as the A operand from tensor memory.
//
// Tiles are 128 tokens on both sides.  Every kernel is persistent (a block per
// SM, items taken in a fixed order) and has its roles in separate warps: 16
// math warps, one that issues the products, one that issues the loads (and in
// the dk/dv kernel one that stages the rows' statistics), so that loads and
// products run ahead of the elementwise work.  A math warp reads the lane
// quarter of tensor memory that its rank in its group of four allows; the
// thread's lane is its row.
//
// Waits are bounded: one that gives up marks the block, which then waits no
// more, and records the timeout in the workspace header.
#pragma once

#include "mma_sync.cuh"
#include "tc_ptx.cuh"

namespace cla {
namespace {

constexpr int kWT = 128;  // tokens of a tile
// Every block takes all 512 columns of tensor memory, so its shared memory is kept above half of
// an SM's, which keeps a second block of these kernels off the SM.
constexpr int kMinSmem = 116 * 1024;

struct Str3 {
    long long b, h, t;
};

// Token numbers, the window and the sinks (both at most T) fit 32 bits: T is at most 2^31 - 512.
struct WaArgs {
    const int32_t *lens;
    float scale;
    int T, window, sinks, B, H, Hkv;
};

struct WaMaps {
    CUtensorMap q, k, v, g;
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

// The waits of a block: once one has given up none waits long any more.
struct Waits {
    volatile uint32_t *dead;
    WsHeader *hdr;
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
        *dead = 1u;
        atomicOr(&hdr->error, kErrTimeout);
        atomicExch(&hdr->where, where);
    }
};

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
template <int D, bool BF>
__device__ __forceinline__ void mma_scores(uint32_t acc, uint32_t a, uint32_t b, uint32_t negate = 0u) {
    const uint64_t da = Tile<D>::kmajor(a), db = Tile<D>::kmajor(b);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
        mma_ss_w(acc, da + Tile<D>::kstep(kk), db + Tile<D>::kstep(kk), idesc16<BF>(kWT, 0) | negate, kk ? 1u : 0u);
}
// acc (+)= P X: P [128 x 128] packed in tensor memory, X a tile [128 tokens][D].
template <int D, bool BF>
__device__ __forceinline__ void mma_apply(uint32_t acc, uint32_t p, uint32_t x, bool add) {
    const uint64_t dx = Tile<D>::nmajor(x);
#pragma unroll
    for (int kk = 0; kk < kWT / 16; ++kk)
        mma_ts_w(acc, p + kk * 8, dx + Tile<D>::nstep(kk), idesc16<BF>(D, 1), (add || kk) ? 1u : 0u);
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
struct Small {
    uint64_t bars[32];
    uint32_t tmem, dead;
    uint32_t pad[62];
    float f[512];
};
static_assert(sizeof(Small) == kSmall, "layout behind the tiles");
__device__ __forceinline__ bool misplaced(uint32_t base, WsHeader *hdr) {
    if ((base & 1023u) == 0u) return false;
    if (threadIdx.x == 0) atomicOr(&hdr->error, kErrTimeout);
    return true;
}
// Between the N warps that share a lane quarter: what any has read of tensor memory is read.
template <int N>
__device__ __forceinline__ void quarter_sync(int id) {
    tc_fence_before();
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(32 * N) : "memory");
    tc_fence_after();
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

// One row of o, dq, dk or dv (D columns of an accumulator, times f) to memory.
template <int D, bool BF>
__device__ __forceinline__ void store_row(uint32_t taddr, void *out, long long at, float f, bool write, bool zero) {
#pragma unroll
    for (int c = 0; c < D; c += 16) {
        uint32_t r[16];
        tmem_ld16(taddr + c, r);
        tmem_ld_wait();
        if (write) {
            uint4 *p = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + at + c);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = zero ? 0u
                                : pack16<BF>(make_float2(__uint_as_float(r[k * 8 + 2 * j]) * f,
                                                         __uint_as_float(r[k * 8 + 2 * j + 1]) * f));
                p[k] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
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
template <int D>
struct FwdCfg {
    static constexpr int STAGES = D == 128 ? 5 : 8;
    static constexpr int SMEM = (2 + STAGES) * Tile<D>::BYTES + kSmall;
    static constexpr int THREADS = 576;  // 16 math warps, products, loads
};

struct FwdItem {
    int b, hk, h, t0, step_h, step_t;  // the second tile: head h + step_h at t0 + step_t
};
__device__ __forceinline__ FwdItem fwd_item(const WaArgs &g, int item, int tiles) {
    FwdItem w;
    const int G = g.H / g.Hkv;
    if ((G & 1) == 0) {
        const int pr = item % (G / 2), r = item / (G / 2), bh = r / tiles;
        w.b = bh / g.Hkv;
        w.hk = bh % g.Hkv;
        w.h = w.hk * G + 2 * pr;
        w.t0 = (r % tiles) * kWT;
        w.step_h = 1;
        w.step_t = 0;
    } else {
        const int pairs = (tiles + 1) / 2, r = item / G, bh = r / pairs;
        w.b = bh / g.Hkv;
        w.hk = bh % g.Hkv;
        w.h = w.hk * G + item % G;
        w.t0 = (r % pairs) * 2 * kWT;
        w.step_h = 0;
        w.step_t = kWT;
    }
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
    const uint32_t sq = smem_u32(smem_raw), skv = sq + 2 * TB;
    Small &sm = *reinterpret_cast<Small *>(smem_raw + (2 + ST) * TB);
    static_assert(2 * ST + 8 <= 32, "barriers");
    float(*s_row)[2][kWT] = reinterpret_cast<float(*)[2][kWT]>(sm.f);  // [tile][half][row]: maxima, in the end sums
    if (misplaced(sq, hdr)) return;
    const int warp = threadIdx.x >> 5, tiles = (g.T + kWT - 1) / kWT;
    const uint32_t b0 = smem_u32(sm.bars);
    const uint32_t q_full = b0, q_empty = b0 + 8, o_full = b0 + 16, s_full = b0 + 24, p_ready = b0 + 40;  // the last two x 2
    const uint32_t kv_full = b0 + 64, kv_empty = kv_full + 8 * ST;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 5; ++i) mbar_init(b0 + 8 * i, 1);
        mbar_init(p_ready, 8);
        mbar_init(p_ready + 8, 8);
        for (int i = 0; i < 2 * ST; ++i) mbar_init(kv_full + 8 * i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sm.dead = 0u;
        if (blockIdx.x == 0) hdr->error = 0u, hdr->where = 0u;
    }
    const uint32_t tmem = tmem_alloc_all(&sm.tmem);
    const Waits wait{&sm.dead, hdr};
    const uint32_t tS = tmem, tO = tmem + 256;

    if (warp == 17) {
        // ------------------------------------------------------------ loads
        if ((threadIdx.x & 31) == 0) {
            uint32_t n = 0, it = 0;
            for (int item = blockIdx.x; item < items; item += gridDim.x) {
                const FwdItem w = fwd_item(g, item, tiles);
                const FwdTiles kt(g, w, wa_len(g, w.b));
                if (kt.count == 0) continue;
                if (it > 0) wait(q_empty, it - 1, 21);
                if (*wait.dead != 0u) break;
                const bool two = kt.b.hi >= kt.b.lo;
                mbar_expect_tx(q_full, two ? 2 * TB : TB);
                Tile<D>::load(sq, &maps.q, w.t0, w.h, w.b, q_full);
                if (two) Tile<D>::load(sq + TB, &maps.q, w.t0 + w.step_t, w.h + w.step_h, w.b, q_full);
                for (int i = 0; i < 2 * kt.count; ++i, ++n) {
                    const uint32_t s = n % ST;
                    if (n >= ST) wait(kv_empty + 8 * s, n / ST - 1, 22);
                    if (*wait.dead != 0u) break;
                    mbar_expect_tx(kv_full + 8 * s, TB);
                    Tile<D>::load(skv + s * TB, (i & 1) ? &maps.v : &maps.k, kt.tile(i >> 1) * kWT, w.hk, w.b, kv_full + 8 * s);
                }
                ++it;
            }
            if (*wait.dead != 0u) drain(q_full, it, 1), drain(kv_full, n, ST);
        }
        __syncwarp();
    } else if (warp == 16) {
        // ------------------------------------------------------------ products
        uint32_t n = 0, it = 0, np[2] = {0, 0};
        const uint32_t negate = g.scale < 0.f ? kNegateA : 0u;
        for (int item = blockIdx.x; item < items; item += gridDim.x) {
            const FwdItem w = fwd_item(g, item, tiles);
            const int len = wa_len(g, w.b);
            const FwdTiles kt(g, w, len);
            const int count = kt.count;
            if (count == 0) continue;
            bool begun[2] = {false, false};
            wait(q_full, it, 23);
            // step i: for each of the two tiles the output of key tile i - 1, then the scores of i
            for (int i = 0; i <= count; ++i) {
                const uint32_t sk = (n + 2 * i) % ST, sv = (n + 2 * i - 1) % ST;
                const int ti = kt.tile(i), tp = kt.tile(i - 1);
                bool got_v = false, got_k = false;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const KeyTiles &mine = u == 0 ? kt.a : kt.b;
                    if (i > 0 && mine.has(tp)) {
                        if (!got_v) {
                            wait(kv_full + 8 * sv, (n + 2 * i - 1) / ST, 24);
                            if (g.lens != nullptr && len - tp * kWT < kWT) Tile<D>::zero_rows(skv + sv * TB, len - tp * kWT);
                            got_v = true;
                        }
                        wait(p_ready + 8 * u, np[u]++, 25);
                        tc_fence_after();
                        mma_apply<D, BF>(tO + 128 * u, tS + 128 * u, skv + sv * TB, begun[u]);
                        begun[u] = true;
                    }
                    if (i < count && mine.has(ti)) {
                        if (!got_k) wait(kv_full + 8 * sk, (n + 2 * i) / ST, 26);
                        got_k = true;
                        tc_fence_after();
                        mma_scores<D, BF>(tS + 128 * u, sq + u * TB, skv + sk * TB, negate);
                        mma_commit_w(s_full + 8 * u);
                    }
                }
                if (i > 0) mma_commit_w(kv_empty + 8 * sv);
                if (i < count) mma_commit_w(kv_empty + 8 * sk);
                if (i == count - 1) mma_commit_w(q_empty);
            }
            mma_commit_w(o_full);
            n += 2 * count;
            ++it;
        }
    } else {
        // ------------------------------------------------------------ probabilities and output
        const int u = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3, row = quarter * 32 + (threadIdx.x & 31);
        const uint32_t lanes = (uint32_t)quarter << 21, ts = tS + 128 * u + lanes, to = tO + 128 * u + lanes + half * (D / 2);
        const int id = 1 + u * 4 + quarter;
        // the scores of a negative factor come negated, and a factor of 0 must leave masked scores at -inf
        const float c = fmaxf(fabsf(g.scale) * 1.4426950408889634f, 1e-30f);
        float *own = &s_row[u][half][row], *other = &s_row[u][half ^ 1][row];
        uint32_t ns = 0, it = 0;
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
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        if (!(b0 & (1u << k))) r[k] = 0xff800000u;
                        if (!(b1 & (1u << k))) r[32 + k] = 0xff800000u;
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
                quarter_sync<2>(id);  // also: both halves hold their scores, P may be written over them
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
                    tmem_st16(ts + 32 * half + 16 * k, p);
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                tmem_st_wait();
                tc_fence_before();
                warp_arrive(p_ready + 8 * u);
            }
            if (kt.count > 0) {
                wait(o_full, it++, 28);
                tc_fence_after();
            }
            if (t0 < g.T) {  // the same for the whole tile
                const int h = w.h + u * w.step_h;
                const long long at = w.b * so.b + h * so.h + t * so.t + half * (D / 2);
                const bool dead = t >= len;
                if (first) {
                    if (t < g.T) zero_row<D / 2>(o, at);
                } else {
                    *own = l;
                    quarter_sync<2>(id);
                    l += *other;
                    store_row<D / 2, BF>(to, o, at, 1.f / l, t < g.T, dead);
                    quarter_sync<2>(id);  // *other has been read
                }
                if (half == 0 && t < g.T)
                    lse[((long long)w.b * g.H + h) * g.T + t] = dead ? -INFINITY : m * 0.6931471805599453f + logf(l);
            }
            tc_fence_before();
        }
    }
    tmem_free_all(tmem);
}

// ------------------------------------------------------------------ backward: dq (and delta)
// One query tile at a time; each row's 128 scores and their gradients are shared by four threads
// (32 columns each).  Tensor memory: two score tiles in turn (dS is written over the scores), one
// dP tile, the accumulator.  While the math warps work on key tile i, the tensor cores form the
// scores of i + 1, and when its dS is there, dP of i + 1 and then dq += dS k.
template <int D>
struct DqCfg {
    static constexpr int KST = D == 128 ? 3 : 5, VST = D == 128 ? 2 : 4;
    static constexpr int SMEM = (2 + KST + VST) * Tile<D>::BYTES + kSmall;
    static constexpr int THREADS = 576;  // 16 math warps, products, loads
};

template <int D, bool BF>
__global__ void __launch_bounds__(DqCfg<D>::THREADS, 1)
wa_dq_kernel(const __grid_constant__ WaMaps maps, const void *__restrict__ o, const void *__restrict__ dO,
             const float *__restrict__ lse, void *__restrict__ dq, float *__restrict__ delta, Str3 so, Str3 sg, Str3 sdq,
             WaArgs g, int items, WsHeader *hdr) {
    constexpr int KST = DqCfg<D>::KST, VST = DqCfg<D>::VST, TB = Tile<D>::BYTES;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t sq = smem_u32(smem_raw), sg_ = sq + TB, sk = sq + 2 * TB, sv = sk + KST * TB;
    Small &sm = *reinterpret_cast<Small *>(smem_raw + (2 + KST + VST) * TB);
    static_assert(8 + 2 * (KST + VST) <= 32, "barriers");
    float(*s_delta)[kWT] = reinterpret_cast<float(*)[kWT]>(sm.f);
    if (misplaced(sq, hdr)) return;
    const int warp = threadIdx.x >> 5, tiles = (g.T + kWT - 1) / kWT, G = g.H / g.Hkv;
    const uint32_t b0 = smem_u32(sm.bars);
    const uint32_t q_full = b0, q_empty = b0 + 8, acc_full = b0 + 16, dp_full = b0 + 24, s_full = b0 + 32, ds_ready = b0 + 48;
    const uint32_t k_full = b0 + 64, k_empty = k_full + 8 * KST, v_full = k_empty + 8 * KST, v_empty = v_full + 8 * VST;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 6; ++i) mbar_init(b0 + 8 * i, 1);
        mbar_init(ds_ready, 16);
        for (int i = 0; i < 2 * (KST + VST); ++i) mbar_init(k_full + 8 * i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sm.dead = 0u;
    }
    const uint32_t tmem = tmem_alloc_all(&sm.tmem);
    const Waits wait{&sm.dead, hdr};
    const uint32_t tS = tmem, tP = tmem + 256, tA = tmem + 384;
    // items: the heads of a group next to each other, then the tiles
    auto place = [&](int item, int &b, int &h, int &hk, int &t0) {
        const int gi = item % G, r = item / G, bh = r / tiles;
        t0 = r % tiles * kWT;
        hk = bh % g.Hkv;
        b = bh / g.Hkv;
        h = hk * G + gi;
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
                if (it > 0) wait(q_empty, it - 1, 31);
                if (*wait.dead != 0u) break;
                mbar_expect_tx(q_full, 2 * TB);
                Tile<D>::load(sq, &maps.q, t0, h, b, q_full);
                Tile<D>::load(sg_, &maps.g, t0, h, b, q_full);
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
                }
                ++it;
            }
            if (*wait.dead != 0u) drain(q_full, it, 1), drain(k_full, n, KST), drain(v_full, n, VST);
        }
        __syncwarp();
    } else if (warp == 16) {
        uint32_t n = 0, it = 0;
        for (int item = blockIdx.x; item < items; item += gridDim.x) {
            int b, h, hk, t0;
            place(item, b, h, hk, t0);
            const int len = wa_len(g, b);
            const KeyTiles kt = key_tiles(g, t0, len);
            if (kt.hi < kt.lo) continue;
            const int ns = min(kt.sinks, kt.lo), count = kt.hi - kt.lo + 1 + ns;
            auto scores = [&](uint32_t j, int i) {  // key tile i of the item, number j of the block
                wait(k_full + 8 * (j % KST), j / KST, 34);
                const int left = len - (i < ns ? i : kt.lo + i - ns) * kWT;
                if (g.lens != nullptr && left < kWT) Tile<D>::zero_rows(sk + (j % KST) * TB, left);
                tc_fence_after();
                mma_scores<D, BF>(tS + 128 * (j & 1), sq, sk + (j % KST) * TB);
                mma_commit_w(s_full + 8 * (j & 1));
            };
            auto grads = [&](uint32_t j) {
                wait(v_full + 8 * (j % VST), j / VST, 35);
                tc_fence_after();
                mma_scores<D, BF>(tP, sg_, sv + (j % VST) * TB);
                mma_commit_w(dp_full);
                mma_commit_w(v_empty + 8 * (j % VST));
            };
            wait(q_full, it, 36);
            scores(n, 0);
            grads(n);
            for (int i = 0; i < count; ++i, ++n) {
                if (i + 1 < count) scores(n + 1, i + 1);
                wait(ds_ready, n, 37);
                tc_fence_after();
                if (i + 1 < count) grads(n + 1);
                if (i + 1 == count) mma_commit_w(q_empty);
                mma_apply<D, BF>(tA, tS + 128 * (n & 1), sk + (n % KST) * TB, i > 0);
                mma_commit_w(k_empty + 8 * (n % KST));
            }
            mma_commit_w(acc_full);
            ++it;
        }
    } else {
        const int part = warp >> 2, quarter = warp & 3, row = quarter * 32 + (threadIdx.x & 31);  // columns 32 part ..
        const uint32_t lanes = (uint32_t)quarter << 21;
        const float c = g.scale * 1.4426950408889634f;
        uint32_t n = 0, it = 0;
        for (int item = blockIdx.x; item < items; item += gridDim.x) {
            int b, h, hk, t0;
            place(item, b, h, hk, t0);
            const int len = wa_len(g, b), t = t0 + row;
            const KeyTiles kt = key_tiles(g, t0, len);
            const bool live = t < len;
            const long long at = ((long long)b * g.H + h) * g.T + t;
            // delta = dO . o of the row, a quarter of the columns by each of its four threads
            float sum = 0.f;
            if (live) {
                const uint4 *x = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(o) + b * so.b + h * so.h + t * so.t) + part * (D / 32);
                const uint4 *y = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(dO) + b * sg.b + h * sg.h + t * sg.t) + part * (D / 32);
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                    const uint4 a = __ldg(x + k), e = __ldg(y + k);
                    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, ew[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 p = unpack16<BF>(aw[j]), q = unpack16<BF>(ew[j]);
                        sum = fmaf(p.x, q.x, fmaf(p.y, q.y, sum));
                    }
                }
            }
            s_delta[part][row] = sum;
            quarter_sync<4>(1 + quarter);
            const float dl = (s_delta[0][row] + s_delta[1][row]) + (s_delta[2][row] + s_delta[3][row]);
            const float ls = live ? lse[at] * 1.4426950408889634f : INFINITY;
            if (part == 0 && t < g.T) delta[at] = dl;
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
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (!(bits & (1u << k))) r[k] = 0u;
                }
#pragma unroll
                for (int k = 0; k < 16; ++k) ds[k] = pack16<BF>(x[k]);
                // the threads of a row write where others of them have read scores
                quarter_sync<4>(1 + quarter);
                tmem_st16(ts + 16 * part, ds);
                tmem_st_wait();
                tc_fence_before();
                warp_arrive(ds_ready);
            }
            const long long out = b * sdq.b + h * sdq.h + t * sdq.t + part * (D / 4);
            if (count > 0) {
                wait(acc_full, it++, 40);
                tc_fence_after();
                store_row<D / 4, BF>(tA + lanes + part * (D / 4), dq, out, g.scale, t < g.T, !live);
            } else if (t < g.T) {
                zero_row<D / 4>(dq, out);
            }
            tc_fence_before();
            quarter_sync<4>(1 + quarter);  // s_delta is free
        }
    }
    tmem_free_all(tmem);
}

// ------------------------------------------------------------------ backward: dk, dv
// One key tile at a time against the query tiles that see it, head by head of the group.  The
// scores are transposed (a row is a key), so that P^T and dS^T are A operands from tensor memory:
// S^T = K Q^T, dP^T = V dO^T, dv += P^T dO, dk += dS^T Q, with P^T over S^T and dS^T over dP^T.
// Each half of the elementwise work runs beside two products: forming P beside dk += and the next
// dP, forming dS beside dv += and the next S.  A tile with sinks is seen by every later query
// tile: its list is cut into pieces that leave fp32 partial sums, joined in their order.
template <int D>
struct DkvCfg {
    static constexpr int ST = D == 128 ? 2 : 4;
    static constexpr int SMEM = (2 + 2 * ST) * Tile<D>::BYTES + kSmall;
    static constexpr int THREADS = 608;  // 16 math warps, products, loads, statistics
};

struct DkvPlan {
    int sink_tiles, pieces, piece;  // tiles that are cut, pieces of each, query tiles of a piece
    float *part;                    // [b][hk][sink tile][piece][dk, dv][128][D]
};

template <int D, bool BF>
__global__ void __launch_bounds__(DkvCfg<D>::THREADS, 1)
wa_dkv_kernel(const __grid_constant__ WaMaps maps, const float *__restrict__ lse, const float *__restrict__ delta,
              void *__restrict__ dk, void *__restrict__ dv, Str3 sdk, Str3 sdv, WaArgs g, DkvPlan pl, int items,
              WsHeader *hdr) {
    constexpr int ST = DkvCfg<D>::ST, TB = Tile<D>::BYTES;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t sk = smem_u32(smem_raw), sv = sk + TB, sq = sk + 2 * TB, sg = sq + ST * TB;
    Small &sm = *reinterpret_cast<Small *>(smem_raw + (2 + 2 * ST) * TB);
    static_assert(8 + 4 * ST + 4 <= 32, "barriers");
    float(*s_stat)[2][kWT] = reinterpret_cast<float(*)[2][kWT]>(sm.f);  // [slot][lse log2 e, delta][query]
    if (misplaced(sk, hdr)) return;
    const int warp = threadIdx.x >> 5;
    const uint32_t b0 = smem_u32(sm.bars);
    const uint32_t kv_full = b0, kv_empty = b0 + 8, acc_full = b0 + 16, s_full = b0 + 24, dp_full = b0 + 32;
    const uint32_t p_ready = b0 + 40, ds_ready = b0 + 48;
    const uint32_t q_full = b0 + 64, q_empty = q_full + 8 * ST, g_full = q_empty + 8 * ST, g_empty = g_full + 8 * ST;
    const uint32_t st_full = g_empty + 8 * ST, st_empty = st_full + 16;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 5; ++i) mbar_init(b0 + 8 * i, 1);
        mbar_init(p_ready, 16);
        mbar_init(ds_ready, 16);
        for (int i = 0; i < 4 * ST; ++i) mbar_init(q_full + 8 * i, 1);
        for (int i = 0; i < 2; ++i) mbar_init(st_full + 8 * i, 1), mbar_init(st_empty + 8 * i, 16);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        sm.dead = 0u;
    }
    const uint32_t tmem = tmem_alloc_all(&sm.tmem);
    const Waits wait{&sm.dead, hdr};
    const uint32_t tS = tmem, tP = tmem + 128, tV = tmem + 256, tK = tmem + 384;
    const int tiles = (g.T + kWT - 1) / kWT, G = g.H / g.Hkv;
    const int per = pl.sink_tiles * pl.pieces + (tiles - pl.sink_tiles);  // items of a (batch, key head)
    struct Item {
        int b, hk, tile, piece, nq, i0, i1;  // piece < 0: whole; query tiles tile + i % nq of head i / nq, i in [i0, i1)
        int len;
    };
    auto place = [&](int item) {
        Item w;
        const int bh = item / per, r = item % per;
        w.b = bh / g.Hkv;
        w.hk = bh % g.Hkv;
        const bool cut = r < pl.sink_tiles * pl.pieces;
        w.tile = cut ? r / pl.pieces : r - pl.sink_tiles * (pl.pieces - 1);
        w.piece = cut ? r % pl.pieces : -1;
        w.len = wa_len(g, w.b);
        const int s0 = w.tile * kWT;
        if (s0 >= w.len) {
            w.nq = w.i0 = w.i1 = 0;
            return w;
        }
        // the last query that the tile's last key is in the window of, where the sequence reaches it
        const int room = w.len - 1 - s0, reach = kWT - 1 + g.window - 1;
        w.nq = (s0 + (s0 < g.sinks || reach < 0 || reach > room ? room : reach)) / kWT - w.tile + 1;
        w.i0 = cut ? min(w.piece * pl.piece, G * w.nq) : 0;
        w.i1 = cut ? min(w.i0 + pl.piece, G * w.nq) : G * w.nq;
        return w;
    };

    if (warp == 17) {
        if ((threadIdx.x & 31) == 0) {
            uint32_t n = 0, it = 0;
            for (int item = blockIdx.x; item < items; item += gridDim.x) {
                const Item w = place(item);
                if (w.i0 >= w.i1) continue;
                if (it > 0) wait(kv_empty, it - 1, 41);
                if (*wait.dead != 0u) break;
                mbar_expect_tx(kv_full, 2 * TB);
                Tile<D>::load(sk, &maps.k, w.tile * kWT, w.hk, w.b, kv_full);
                Tile<D>::load(sv, &maps.v, w.tile * kWT, w.hk, w.b, kv_full);
                for (int i = w.i0; i < w.i1; ++i, ++n) {
                    const uint32_t s = n % ST;
                    const int t0 = (w.tile + i % w.nq) * kWT;
                    const int h = w.hk * G + i / w.nq;
                    if (n >= ST) wait(q_empty + 8 * s, n / ST - 1, 42);
                    if (*wait.dead != 0u) break;
                    mbar_expect_tx(q_full + 8 * s, TB);
                    Tile<D>::load(sq + s * TB, &maps.q, t0, h, w.b, q_full + 8 * s);
                    if (n >= ST) wait(g_empty + 8 * s, n / ST - 1, 43);
                    mbar_expect_tx(g_full + 8 * s, TB);
                    Tile<D>::load(sg + s * TB, &maps.g, t0, h, w.b, g_full + 8 * s);
                }
                ++it;
            }
            if (*wait.dead != 0u) drain(kv_full, it, 1), drain(q_full, n, ST), drain(g_full, n, ST);
        }
        __syncwarp();
    } else if (warp == 18) {
        // ------------------------------------------------------------ the rows' statistics, a tile ahead
        const int lane = threadIdx.x & 31;
        uint32_t n = 0;
        for (int item = blockIdx.x; item < items; item += gridDim.x) {
            const Item w = place(item);
            for (int i = w.i0; i < w.i1; ++i, ++n) {
                const uint32_t s = n & 1;
                const int t0 = (w.tile + i % w.nq) * kWT;
                const long long at = ((long long)w.b * g.H + w.hk * G + i / w.nq) * g.T + t0;
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
    } else if (warp == 16) {
        uint32_t n = 0, it = 0;
        for (int item = blockIdx.x; item < items; item += gridDim.x) {
            const Item w = place(item);
            if (w.i0 >= w.i1) continue;
            auto scores = [&](uint32_t j, int i) {
                const uint32_t s = j % ST;
                wait(q_full + 8 * s, j / ST, 45);
                const int left = w.len - (w.tile + i % w.nq) * kWT;
                if (g.lens != nullptr && left < kWT) Tile<D>::zero_rows(sq + s * TB, left);
                tc_fence_after();
                mma_scores<D, BF>(tS, sk, sq + s * TB);
                mma_commit_w(s_full);
            };
            auto grads = [&](uint32_t j, int i) {
                const uint32_t s = j % ST;
                wait(g_full + 8 * s, j / ST, 46);
                const int left = w.len - (w.tile + i % w.nq) * kWT;
                if (g.lens != nullptr && left < kWT) Tile<D>::zero_rows(sg + s * TB, left);
                tc_fence_after();
                mma_scores<D, BF>(tP, sv, sg + s * TB);
                mma_commit_w(dp_full);
            };
            wait(kv_full, it, 47);
            scores(n, w.i0);
            grads(n, w.i0);
            for (int i = w.i0; i < w.i1; ++i, ++n) {
                const uint32_t s = n % ST;
                wait(p_ready, n, 48);
                tc_fence_after();
                mma_apply<D, BF>(tV, tS, sg + s * TB, i > w.i0);
                mma_commit_w(g_empty + 8 * s);
                if (i + 1 < w.i1) scores(n + 1, i + 1);
                wait(ds_ready, n, 49);
                tc_fence_after();
                mma_apply<D, BF>(tK, tP, sq + s * TB, i > w.i0);
                mma_commit_w(q_empty + 8 * s);
                if (i + 1 < w.i1) grads(n + 1, i + 1);
            }
            mma_commit_w(kv_empty);
            mma_commit_w(acc_full);
            ++it;
        }
    } else {
        const int part = warp >> 2, quarter = warp & 3, row = quarter * 32 + (threadIdx.x & 31);  // queries 32 part ..
        const uint32_t lanes = (uint32_t)quarter << 21;
        const float c = g.scale * 1.4426950408889634f;
        uint32_t n = 0, it = 0;
        for (int item = blockIdx.x; item < items; item += gridDim.x) {
            const Item w = place(item);
            const int s0 = w.tile * kWT, key = s0 + row;
            for (int i = w.i0; i < w.i1; ++i, ++n) {
                const int t0 = (w.tile + i % w.nq) * kWT;
                const uint32_t sl = n & 1;
                wait(st_full + 8 * sl, n >> 1, 50);
                wait(s_full, n, 51);
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
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (!(bits & (1u << k))) r[k] = 0u;
                }
#pragma unroll
                for (int k = 0; k < 16; ++k) p[k] = pack16<BF>(x[k]);
                quarter_sync<4>(1 + quarter);  // the threads of a row write where others of them have read
                tmem_st16(tS + lanes + 16 * part, p);
                tmem_st_wait();
                tc_fence_before();
                warp_arrive(p_ready);
                wait(dp_full, n, 52);
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
                quarter_sync<4>(1 + quarter);
                tmem_st16(tP + lanes + 16 * part, p);
                tmem_st_wait();
                tc_fence_before();
                warp_arrive(ds_ready);
                warp_arrive(st_empty + 8 * sl);
            }
            const bool any = w.i0 < w.i1, write = key < g.T, zero = key >= w.len;
            if (any) {
                wait(acc_full, it++, 53);
                tc_fence_after();
            }
            // dk by the first eight warps, dv by the others, half of the columns each
            const int which = part >> 1, col = (part & 1) * (D / 2);
            const uint32_t acc = (which == 0 ? tK : tV) + lanes + col;
            const float f = which == 0 ? g.scale : 1.f;
            if (w.piece < 0) {
                void *out = which == 0 ? dk : dv;
                const Str3 st = which == 0 ? sdk : sdv;
                const long long at = w.b * st.b + w.hk * st.h + key * st.t + col;
                if (any) store_row<D / 2, BF>(acc, out, at, f, write, zero);
                else if (write) zero_row<D / 2>(out, at);
            } else {
                float4 *p = reinterpret_cast<float4 *>(
                    pl.part + (((((long long)w.b * g.Hkv + w.hk) * pl.sink_tiles + w.tile) * pl.pieces + w.piece) * 2 + which) * (kWT * D) + row * D + col);
#pragma unroll
                for (int k = 0; k < D / 2; k += 32) {
                    uint32_t r[32];
                    if (any) {
                        tmem_ld32(acc + k, r);
                        tmem_ld_wait();
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        p[k / 4 + j] = any && !zero ? make_float4(__uint_as_float(r[4 * j]) * f, __uint_as_float(r[4 * j + 1]) * f,
                                                                  __uint_as_float(r[4 * j + 2]) * f, __uint_as_float(r[4 * j + 3]) * f)
                                                    : make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
            tc_fence_before();
        }
    }
    tmem_free_all(tmem);
}

// Adds the pieces of the cut tiles in their order: a thread for two columns of a row of dk or dv.
template <int D, bool BF>
__global__ void wa_join_kernel(void *__restrict__ dk, void *__restrict__ dv, Str3 sdk, Str3 sdv, WaArgs g, DkvPlan pl) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    constexpr int C = D / 2;
    const int col = (int)(i % C), row = (int)(i / C % kWT), which = (int)(i / C / kWT % 2);
    const long long u = i / C / kWT / 2;
    const int tile = (int)(u % pl.sink_tiles);
    const long long bh = u / pl.sink_tiles;
    if (bh >= (long long)g.B * g.Hkv) return;
    const long long key = (long long)tile * kWT + row;
    if (key >= g.T) return;
    const float2 *p = reinterpret_cast<const float2 *>(pl.part + ((u * pl.pieces * 2 + which) * kWT + row) * D) + col;
    float2 s = make_float2(0.f, 0.f);
    for (int k = 0; k < pl.pieces; ++k) {
        const float2 x = p[(long long)k * (kWT * D)];
        s.x += x.x;
        s.y += x.y;
    }
    const Str3 st = which == 0 ? sdk : sdv;
    uint16_t *out = static_cast<uint16_t *>(which == 0 ? dk : dv);
    *reinterpret_cast<uint32_t *>(out + (bh / g.Hkv) * st.b + (bh % g.Hkv) * st.h + key * st.t + 2 * col) = pack16<BF>(s);
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
