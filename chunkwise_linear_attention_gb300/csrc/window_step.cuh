// window_step.cuh -- one token against the rolling cache of window_attn.cu.
//
// What bounds it is reading the cache once.  A cluster of blocks shares the
// slots of one (sequence, key head); a warp takes 16 slots at a time, straight
// from memory into the operands of m16n8k16 products, with no staging: the
// slots are the rows and up to 8 (or two times 8) query heads the columns.
//   scores^T [16 slots x 8 heads] = K Q^T.  The order of the columns of d
//   within a product is free, so a lane loads 16 contiguous bytes of its slot
//   and of its head and uses them as they come.
//   o^T [16 columns of d x 8 heads] += V^T P^T.  A lane loads 8 columns of
//   four slots; a byte permutation pairs neighbouring slots.
// The probabilities keep their accuracy as two 16-bit parts.  The new token's
// key and value come from the arguments; the block that meets their slot
// writes them to the cache.  The warps' and the cluster's partial results meet
// in (distributed) shared memory, in a fixed order: no workspace, one launch.
//
// Measured on GB300: 64 x 32/8 x 128, window 4096, sinks 4: 180 us for 1.08 GB
// (6.0 TB/s, 88% of the measured copy rate) at 12 warps a multiprocessor; 4 x
// 16/4 x 128, window 1024: 13 us with its launch, of which the cold cache's
// latency and the cluster's two barriers are most; one sequence of 32772 slots
// and 8 key heads, in clusters of 16: 54 us (2.5 TB/s: 128 blocks of 4 warps).
#pragma once

#include "window_attn_tc.cuh"

namespace cla {
namespace {

constexpr int kStepWarps = 4;

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct StepArgs {
    float c;  // scale log2 e
    long long window, slots;
    int sinks, B, H, Hkv, splits, groups;  // groups: blocks of 8 NG query heads in a key head
};

template <int D, bool BF, int NG>
__global__ void __launch_bounds__(kStepWarps * 32)
wa_step_kernel(const uint16_t *__restrict__ q, const uint16_t *__restrict__ k, const uint16_t *__restrict__ v, uint16_t *kc,
               uint16_t *vc, const int32_t *__restrict__ pos, uint16_t *__restrict__ o, Str3 sq, Str3 sk, Str3 sv, StepArgs g) {
    constexpr int NH = 8 * NG, KC = D / 32, VG = D / 64;
    __shared__ float s_o[kStepWarps][NH][D], s_m[kStepWarps][NH], s_l[kStepWarps][NH];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3;
    const int split = blockIdx.x % g.splits;
    const long long unit = blockIdx.x / g.splits;
    const int z = (int)(unit % g.groups), hk = (int)(unit / g.groups % g.Hkv), b = (int)(unit / g.groups / g.Hkv);
    const int G = g.H / g.Hkv, h0 = hk * G + z * NH, nh = min(NH, G - z * NH);
    uint16_t *ob = o + ((long long)b * g.H + h0) * D;
    const long long p = pos[b];
    if (p < 0) {  // the whole cluster leaves
        if (split == 0)
            for (int i = threadIdx.x; i < nh * D / 2; i += blockDim.x) reinterpret_cast<uint32_t *>(ob)[i] = 0u;
        return;
    }
    const long long mine = p < g.sinks ? p : g.sinks + (p - g.sinks) % g.window, n = min(p + 1, g.slots);
    const uint16_t *kn = k + b * sk.b + hk * sk.h, *vn = v + b * sv.b + hk * sv.h;
    uint16_t *kb = kc + ((long long)b * g.Hkv + hk) * g.slots * D, *vb = vc + ((long long)b * g.Hkv + hk) * g.slots * D;

    uint4 qf[NG][KC];
#pragma unroll
    for (int a = 0; a < NG; ++a)
#pragma unroll
        for (int c = 0; c < KC; ++c)
            qf[a][c] = 8 * a + r < nh ? *reinterpret_cast<const uint4 *>(q + b * sq.b + (h0 + 8 * a + r) * sq.h + 32 * c + 8 * j)
                                      : make_uint4(0u, 0u, 0u, 0u);
    const long long tiles = (n + 15) / 16, share = (tiles + g.splits - 1) / g.splits;
    const long long first = split * share + warp, end = min(tiles, (split + 1) * share);

    uint4 kx[2][KC], vx[4][VG];
    auto load_k = [&](long long t) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const long long s = t * 16 + r + 8 * i;
            const uint16_t *row = (s == mine ? kn : kb + s * D) + 8 * j;
#pragma unroll
            for (int c = 0; c < KC; ++c)
                kx[i][c] = s < n ? __ldcs(reinterpret_cast<const uint4 *>(row + 32 * c)) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    auto load_v = [&](long long t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const long long s = t * 16 + 2 * j + (i & 1) + 8 * (i >> 1);
            const uint16_t *row = (s == mine ? vn : vb + s * D) + 8 * r;
#pragma unroll
            for (int a = 0; a < VG; ++a)
                vx[i][a] = s < n ? __ldcs(reinterpret_cast<const uint4 *>(row + 64 * a)) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    float acc[NG][VG][4][4];  // [heads][64 columns][16 of them][row pair x head pair]
    float m[NG][2], l[NG][2];
#pragma unroll
    for (int a = 0; a < NG; ++a) {
        m[a][0] = m[a][1] = -INFINITY;
        l[a][0] = l[a][1] = 0.f;
#pragma unroll
        for (int x = 0; x < VG; ++x)
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[a][x][t][0] = acc[a][x][t][1] = acc[a][x][t][2] = acc[a][x][t][3] = 0.f;
    }
    if (first < end) {
        load_k(first);
        load_v(first);
    }
    for (long long t = first; t < end; t += kStepWarps) {
        if (z == 0) {  // the new token goes into its slot
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (t * 16 + r + 8 * i == mine) {
#pragma unroll
                    for (int c = 0; c < KC; ++c) *reinterpret_cast<uint4 *>(kb + mine * D + 32 * c + 8 * j) = kx[i][c];
                }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (t * 16 + 2 * j + (i & 1) + 8 * (i >> 1) == mine) {
#pragma unroll
                    for (int a = 0; a < VG; ++a) *reinterpret_cast<uint4 *>(vb + mine * D + 64 * a + 8 * r) = vx[i][a];
                }
        }
        float s[NG][4];
#pragma unroll
        for (int a = 0; a < NG; ++a) {
            s[a][0] = s[a][1] = s[a][2] = s[a][3] = 0.f;
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                mma16x8<BF>(s[a], kx[0][c].x, kx[1][c].x, kx[0][c].y, kx[1][c].y, qf[a][c].x, qf[a][c].y);
                mma16x8<BF>(s[a], kx[0][c].z, kx[1][c].z, kx[0][c].w, kx[1][c].w, qf[a][c].z, qf[a][c].w);
            }
        }
        if (t + kStepWarps < end) load_k(t + kStepWarps);
        const bool in0 = t * 16 + r < n, in1 = t * 16 + r + 8 < n;
        uint32_t hi[NG][2], lo[NG][2];
#pragma unroll
        for (int a = 0; a < NG; ++a) {
            // s: (slot r, heads 2j, 2j + 1), (slot r + 8, the same heads)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[a][i] = (i < 2 ? in0 : in1) ? s[a][i] * g.c : -INFINITY;
            float top[2] = {fmaxf(s[a][0], s[a][2]), fmaxf(s[a][1], s[a][3])};
            if (__any_sync(~0u, top[0] > m[a][0] + 8.f || top[1] > m[a][1] + 8.f)) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) top[e] = fmaxf(top[e], __shfl_xor_sync(~0u, top[e], x));
                    const float mn = fmaxf(m[a][e], top[e]), f = mn == -INFINITY ? 1.f : ex2(m[a][e] - mn);
                    m[a][e] = mn;
                    l[a][e] *= f;
#pragma unroll
                    for (int x = 0; x < VG; ++x)
#pragma unroll
                        for (int y = 0; y < 4; ++y) acc[a][x][y][e] *= f, acc[a][x][y][2 + e] *= f;
                }
            }
            const float mu[2] = {m[a][0] == -INFINITY ? 0.f : m[a][0], m[a][1] == -INFINITY ? 0.f : m[a][1]};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 e = make_float2(ex2(s[a][2 * i] - mu[0]), ex2(s[a][2 * i + 1] - mu[1]));
                l[a][0] += e.x;
                l[a][1] += e.y;
                const uint32_t h = pack16<BF>(e);
                const float2 eh = unpack16<BF>(h);
                hi[a][i] = transpose8x8(h);
                lo[a][i] = transpose8x8(pack16<BF>(make_float2(e.x - eh.x, e.y - eh.y)));
            }
        }
#pragma unroll
        for (int x = 0; x < VG; ++x) {
            const uint32_t w[4][4] = {{vx[0][x].x, vx[0][x].y, vx[0][x].z, vx[0][x].w},
                                      {vx[1][x].x, vx[1][x].y, vx[1][x].z, vx[1][x].w},
                                      {vx[2][x].x, vx[2][x].y, vx[2][x].z, vx[2][x].w},
                                      {vx[3][x].x, vx[3][x].y, vx[3][x].z, vx[3][x].w}};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                // row r: column 64 x + 8 r + 2 y, row r + 8: the next column
                const uint32_t a0 = __byte_perm(w[0][y], w[1][y], 0x5410), a1 = __byte_perm(w[0][y], w[1][y], 0x7632);
                const uint32_t a2 = __byte_perm(w[2][y], w[3][y], 0x5410), a3 = __byte_perm(w[2][y], w[3][y], 0x7632);
#pragma unroll
                for (int a = 0; a < NG; ++a) {
                    mma16x8<BF>(acc[a][x][y], a0, a1, a2, a3, hi[a][0], hi[a][1]);
                    mma16x8<BF>(acc[a][x][y], a0, a1, a2, a3, lo[a][0], lo[a][1]);
                }
            }
        }
        if (t + kStepWarps < end) load_v(t + kStepWarps);
    }
#pragma unroll
    for (int a = 0; a < NG; ++a)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) l[a][e] += __shfl_xor_sync(~0u, l[a][e], x);
            const int h = 8 * a + 2 * j + e;
            if (r == 0) s_m[warp][h] = m[a][e], s_l[warp][h] = l[a][e];
#pragma unroll
            for (int x = 0; x < VG; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    *reinterpret_cast<float2 *>(&s_o[warp][h][64 * x + 8 * r + 2 * y]) = make_float2(acc[a][x][y][e], acc[a][x][y][2 + e]);
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
        reinterpret_cast<uint32_t *>(ob)[i] = pack16<BF>(make_float2(x / lt, y / lt));
    }
    if (g.splits > 1) cluster_sync();  // no block leaves while its part is being read
}

}  // namespace
}  // namespace cla
