// Matrix product of 16-bit operands on the tensor cores (tcgen05), fed by tiled copies.
//
// out(i,j) = epilogue(sum_k B(i,k) A(j,k)): the product is computed with the output's contiguous
// index j on the accumulator's lanes.  A CTA pair owns a tile of 256 j (128 in each CTA's tensor
// memory) x NT i; each CTA stages its 128 rows of A and half of B's rows, and the pair's matrix
// instruction reads both halves of B, so each B element is staged once for 256 lanes.  At
// NT = 256 a 64-deep step moves 32 KB into a CTA's shared memory and 32 KB out of it in the 512
// clocks of its four instructions: 128 bytes a clock, the port's rate.
//
// Roles in a CTA (10 warps): 8 warps of epilogue, one thread of tiled copies, one thread of
// matrix instructions (the pair's first CTA).  Operand stages form a ring (full/empty barriers);
// the accumulator is double buffered in tensor memory, so a tile's epilogue runs under the next
// tile's products.  The epilogue turns 32-column pieces through shared memory so that a warp
// reads and writes 128 contiguous elements of an output row.
//
// With few tiles the cluster is 2*S CTAs: S pairs take a share of k each and add their
// accumulators, in order, through each other's shared memory (no workspace, no atomics, equal
// bits every time).
//
// Every wait is bounded: one that runs out sets the device status and ends the launch early.
#pragma once

#include <type_traits>

#include "linear.cuh"
#include "tensor.cuh"

namespace symar {

constexpr int kTcThreads = 320, kTcEpiWarps = 8;
constexpr int kTcBK = 64;                          // k elements per stage: one 128-byte swizzle row
constexpr uint32_t kTcStageA = 128 * kTcBK * 2;    // bytes of A per stage and CTA
constexpr uint32_t kTcRing = 192 * 1024;           // bytes of all stages
constexpr uint32_t kTcStaging = 32 * 128 * 4;      // one epilogue group's piece

__host__ __device__ constexpr uint32_t tc_stage_bytes(int NT) { return kTcStageA + (uint32_t)NT / 2 * kTcBK * 2; }
__host__ __device__ constexpr int tc_stages(int NT) {
    return (int)(kTcRing / tc_stage_bytes(NT)) > 12 ? 12 : (int)(kTcRing / tc_stage_bytes(NT));
}
constexpr size_t kTcSmem = 1024 + kTcRing + 2 * kTcStaging + 512;

struct TcArgs {
    CUtensorMap a, b;
    MatmulArgs m;              // m.m rows i, m.n columns j, m.kk terms; the epilogue
    uint32_t tiles_i, tiles_j, group;
    uint32_t kblocks;
    uint32_t splits;           // S: pairs per cluster
    uint32_t* status;
    uint64_t timeout_ns;
};

struct TcShared {              // after the ring and the staging
    uint64_t full[12], empty[12], acc_full[2], acc_empty[2];
    uint32_t tmem;
    volatile uint32_t abort;
};

// Waits for a barrier's phase, at most timeout_ns or until another wait of the CTA gave up.
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, const TcArgs& a, TcShared* s, uint32_t what) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1; it < (1u << 30); ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 0u && (s->abort || globaltimer_ns() - t0 > a.timeout_ns)) break;
    }
    if (!s->abort) {
        s->abort = 1;
        report_timeout(a.status, nullptr, 0, kSiteLinearStage, what, blockIdx.x);
    }
    return false;
}

// Tile t of the launch: groups of `group` row tiles, column tiles outer within a group, so the
// tiles in flight share rows and columns in L2.
__device__ __forceinline__ void tc_tile(const TcArgs& a, uint32_t t, uint32_t& ti, uint32_t& tj) {
    const uint32_t per = a.group * a.tiles_j, g = t / per, r = t - g * per;
    const uint32_t gi = min(a.group, a.tiles_i - g * a.group);
    tj = r / gi;
    ti = g * a.group + (r - tj * gi);
}

// Four neighbouring elements of 16 or 32 bits.
template <class T>
struct Quad;
template <>
struct Quad<float> {
    using V = float4;
    static __device__ __forceinline__ void get(const V& v, float (&f)[4]) {
        f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    }
    static __device__ __forceinline__ V put(const float (&f)[4]) { return make_float4(f[0], f[1], f[2], f[3]); }
};
template <>
struct Quad<__nv_bfloat16> {
    using V = uint2;
    static __device__ __forceinline__ void get(const V& v, float (&f)[4]) {
        f[0] = __uint_as_float(v.x << 16), f[1] = __uint_as_float(v.x & 0xFFFF0000u);
        f[2] = __uint_as_float(v.y << 16), f[3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
    static __device__ __forceinline__ V put(const float (&f)[4]) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
        return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
};
template <>
struct Quad<__half> {
    using V = uint2;
    static __device__ __forceinline__ void get(const V& v, float (&f)[4]) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
        f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
    }
    static __device__ __forceinline__ V put(const float (&f)[4]) {
        const __half2 a = __floats2half2_rn(f[0], f[1]), b = __floats2half2_rn(f[2], f[3]);
        return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
};

// The epilogue of one lane: R rows of a tile, four columns of each.  VEC: four neighbouring ones, by
// accesses of four elements (every row of the output and of what is read with it starts at such a
// boundary and the columns come in fours); else columns 32 apart, so that a warp's accesses of single
// elements are still contiguous.
template <class X, class O, bool VEC>
struct TcColumns {
    static constexpr int STEP = VEC ? 1 : 32;
    size_t j;
    int live;                 // of columns j, j + STEP, ... those that exist
    float bias[4];

    __device__ __forceinline__ void set(const MatmulArgs& m, size_t j0, int lane) {
        j = j0 + (VEC ? lane * 4 : lane);
        live = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            bias[e] = 0.f;
            if (j + e * STEP < m.n) {
                live = e + 1;
                if (m.bias) bias[e] = load_f<X>(m.bias, j + e * STEP);
            }
        }
    }

    // Where the lane's four sums of a 128-column row are in shared memory.
    static __device__ __forceinline__ float4 sums(const float* row, int lane) {
        if (VEC) return *reinterpret_cast<const float4*>(row + lane * 4);
        return make_float4(row[lane], row[lane + 32], row[lane + 64], row[lane + 96]);
    }

    template <class T, int R>
    struct Rows {
        typename Quad<T>::V v[VEC ? R : 1];
        T e[VEC ? 1 : R][4];

        __device__ __forceinline__ void load(const TcColumns& c, const void* p, size_t ld, size_t i0, size_t m) {
            const T* q = static_cast<const T*>(p) + i0 * ld + c.j;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (i0 + r >= m || !c.live) continue;
                if (VEC) {
                    v[r] = *reinterpret_cast<const typename Quad<T>::V*>(q + r * ld);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < c.live) e[r][k] = q[r * ld + k * 32];
                }
            }
        }
        __device__ __forceinline__ void add(int r, int live, float (&z)[4]) const {
            float f[4];
            if (VEC) {
                Quad<T>::get(v[r], f);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) f[k] = k < live ? to_f(e[r][k]) : 0.f;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) z[k] += f[k];
        }
    };

    template <class T>
    __device__ __forceinline__ void store(void* p, size_t at, const float (&z)[4]) const {
        T* q = static_cast<T*>(p) + at + j;
        if (VEC) {
            *reinterpret_cast<typename Quad<T>::V*>(q) = Quad<T>::put(z);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < live) q[k * 32] = from_f<T>(z[k]);
        }
    }

    __device__ __forceinline__ void activate(const MatmulArgs& m, size_t i, float4 sum, float (&z)[4]) const {
        z[0] = sum.x + bias[0], z[1] = sum.y + bias[1], z[2] = sum.z + bias[2], z[3] = sum.w + bias[3];
        if (m.pre) store<X>(m.pre, i * m.ldp, z);
        if (m.act != SYM_ACT_NONE) {
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = act_value(z[e], m.act);
        }
    }
};

// A_MN / B_MN: the operand's contiguous index is j / i (else k).
template <class X, class O, bool A_MN, bool B_MN, int NT, bool VEC>
__global__ void __launch_bounds__(kTcThreads, 1) k_matmul_tc(const __grid_constant__ TcArgs a) {
    constexpr int STAGES = tc_stages(NT), CW = NT < 32 ? NT : 32, CHUNKS = NT / CW;
    constexpr int GROUPS = CHUNKS > 1 ? 2 : 1;                       // epilogue groups of 4 warps at work
    constexpr uint32_t STAGE = tc_stage_bytes(NT), COLUMNS = 2 * NT < 32 ? 32 : 2 * NT;
    static_assert(!B_MN || NT >= 128, "a 128-byte swizzle row holds 64 contiguous elements");
    extern __shared__ uint8_t raw[];
    uint8_t* ring = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    float* staging = reinterpret_cast<float*>(ring + kTcRing);
    TcShared* s = reinterpret_cast<TcShared*>(ring + kTcRing + 2 * kTcStaging);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_rank(), half = rank & 1, split = rank >> 1, lead = rank & ~1u;
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&s->full[i], 1);
            mbar_init(&s->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s->acc_full[i], 1);
            mbar_init(&s->acc_empty[i], 2 * 4 * GROUPS);             // one lane of each epilogue warp of the pair
        }
        s->abort = 0;
        fence_mbar_init();
    }
    if (warp == 9) tmem_alloc(&s->tmem, COLUMNS);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = s->tmem;

    const uint32_t S = a.splits, tiles = a.tiles_i * a.tiles_j;
    const uint32_t first = blockIdx.x / (2 * S), step = gridDim.x / (2 * S);
    const uint32_t k0 = (uint32_t)((uint64_t)a.kblocks * split / S), k1 = (uint32_t)((uint64_t)a.kblocks * (split + 1) / S);

    if (warp == 8) {
        // ---- tiled copies: this CTA's 128 rows of A and NT/2 rows of B, counted at the first CTA's barrier
        if (lane == 0) {
            prefetch_map(&a.a);
            prefetch_map(&a.b);
            uint32_t st = 0, ph = 1;                                 // a fresh barrier's previous phase is complete
            bool ok = true;
            for (uint32_t t = first; ok && t < tiles; t += step) {
                uint32_t ti, tj;
                tc_tile(a, t, ti, tj);
                const int j = (int)(tj * 256 + half * 128), i = (int)(ti * NT + half * (NT / 2));
                for (uint32_t k = k0; k < k1; ++k) {
                    if (!(ok = tc_wait(&s->empty[st], ph, a, s, 1))) break;
                    const uint32_t bar = map_rank(smem_u32(&s->full[st]), lead);
                    if (half == 0) mbar_expect_tx(&s->full[st], 2 * STAGE);
                    const uint32_t sa = smem_u32(ring + st * STAGE), sb = sa + kTcStageA;
                    const int kk = (int)(k * kTcBK);
                    if (A_MN) {
                        tma_load_2d(sa, &a.a, j, kk, bar);
                        tma_load_2d(sa + kTcStageA / 2, &a.a, j + 64, kk, bar);
                    } else {
                        tma_load_2d(sa, &a.a, kk, j, bar);
                    }
                    if (B_MN) {
#pragma unroll
                        for (int c = 0; c < NT / 128; ++c) tma_load_2d(sb + c * 8192, &a.b, i + c * 64, kk, bar);
                    } else {
                        tma_load_2d(sb, &a.b, kk, i, bar);
                    }
                    if (++st == STAGES) st = 0, ph ^= 1;
                }
            }
        }
    } else if (warp == 9) {
        // ---- matrix instructions
        if (lane == 0 && half == 0) {
            constexpr bool BF = std::is_same<X, __nv_bfloat16>::value;
            constexpr uint32_t idesc = 1u << 4 | (BF ? 1u << 7 | 1u << 10 : 0u) | (A_MN ? 1u << 15 : 0u) |
                                       (B_MN ? 1u << 16 : 0u) | (uint32_t)(NT / 8) << 17 | (256u / 16) << 24;
            const uint16_t mask = (uint16_t)(3u << lead);
            uint32_t st = 0, ph = 0, n = 0;
            bool ok = true;
            for (uint32_t t = first; ok && t < tiles; t += step, ++n) {
                const uint32_t buf = n & 1, aph = (n >> 1 & 1) ^ 1;
                if (!(ok = tc_wait(&s->acc_empty[buf], aph, a, s, 2))) break;
                tc_fence_after();
                for (uint32_t k = k0; k < k1; ++k) {
                    if (!(ok = tc_wait(&s->full[st], ph, a, s, 3))) break;
                    tc_fence_after();
                    const uint32_t sa = smem_u32(ring + st * STAGE), sb = sa + kTcStageA;
                    const uint64_t da = smem_desc(sa, A_MN ? kTcStageA / 2 : 16, 1024);
                    const uint64_t db = smem_desc(sb, B_MN ? 8192 : 16, 1024);
#pragma unroll
                    for (int q = 0; q < kTcBK / 16; ++q)             // 16 k: 32 bytes of a row, or two atoms of 8 rows
                        mma_f16_pair(tmem + buf * NT, da + q * (A_MN ? 128 : 2), db + q * (B_MN ? 128 : 2), idesc,
                                     k != k0 || q != 0);
                    mma_commit_pair(&s->empty[st], mask);
                    if (++st == STAGES) st = 0, ph ^= 1;
                }
                if (ok) mma_commit_pair(&s->acc_full[buf], mask);
            }
        }
    } else if (S == 1) {
        // ---- epilogue: pieces of CW rows i x 128 columns j
        const int g = warp / 4, q = warp % 4;
        float* stage = staging + g * (kTcStaging / 4);
        uint32_t n = 0;
        for (uint32_t t = first; g < GROUPS && t < tiles; t += step, ++n) {
            uint32_t ti, tj;
            tc_tile(a, t, ti, tj);
            const uint32_t buf = n & 1;
            const bool late = !tc_wait(&s->acc_full[buf], n >> 1 & 1, a, s, 4);
            if (named_any(1 + g, 128, late)) break;                  // the group's threads agree: no barrier is left open
            tc_fence_after();
            TcColumns<X, O, VEC> col;
            col.set(a.m, (size_t)tj * 256 + half * 128, lane);
#pragma unroll 1
            for (int c = g; c < CHUNKS; c += GROUPS) {
                constexpr int R = CW / 4;                            // rows of the piece that this warp finishes
                const size_t i0 = (size_t)ti * NT + c * CW + q * R;
                typename TcColumns<X, O, VEC>::template Rows<X, R> res;
                typename TcColumns<X, O, VEC>::template Rows<O, R> old;
                if (a.m.residual) res.load(col, a.m.residual, a.m.ldr, i0, a.m.m);
                if (a.m.accumulate) old.load(col, a.m.out, a.m.ldo, i0, a.m.m);
                float v[CW];
                tmem_load(tmem + buf * NT + c * CW + ((uint32_t)(q * 32) << 16), v);
                if (c + GROUPS >= CHUNKS) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(map_rank(smem_u32(&s->acc_empty[buf]), lead));
                }
#pragma unroll
                for (int r = 0; r < CW; ++r) stage[r * 128 + q * 32 + lane] = v[r];
                named_sync(1 + g, 128);
                if (col.live) {
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        if (i0 + r >= a.m.m) break;
                        float z[4];
                        col.activate(a.m, i0 + r, col.sums(stage + (q * R + r) * 128, lane), z);
                        if (a.m.residual) res.add(r, col.live, z);
                        if (a.m.accumulate) old.add(r, col.live, z);
                        col.template store<O>(a.m.out, (i0 + r) * a.m.ldo, z);
                    }
                }
                named_sync(1 + g, 128);
            }
        }
    }
    if (S > 1) {
        // ---- one tile per cluster: each pair's sums into shared memory, then every CTA adds its share of rows
        float* sums = reinterpret_cast<float*>(ring);                // [NT][128]; the ring is idle by now
        bool ok = true;
        if (warp < kTcEpiWarps) {
            ok = __all_sync(~0u, tc_wait(&s->acc_full[0], 0, a, s, 4));
            tc_fence_after();
            const int g = warp / 4, q = warp % 4;
            if (ok && g < GROUPS)
#pragma unroll 1
                for (int c = g; c < CHUNKS; c += GROUPS) {
                    float v[CW];
                    tmem_load(tmem + c * CW + ((uint32_t)(q * 32) << 16), v);
#pragma unroll
                    for (int r = 0; r < CW; ++r) sums[(c * CW + r) * 128 + q * 32 + lane] = v[r];
                }
        }
        __syncwarp();
        cluster_sync();
        if (warp < kTcEpiWarps && !s->abort) {
            uint32_t ti, tj;
            tc_tile(a, first, ti, tj);
            TcColumns<X, O, VEC> col;
            col.set(a.m, (size_t)tj * 256 + half * 128, lane);
            for (uint32_t r = split + S * warp; r < NT; r += S * kTcEpiWarps) {
                const size_t i = (size_t)ti * NT + r;
                if (i >= a.m.m || !col.live) break;
                typename TcColumns<X, O, VEC>::template Rows<X, 1> res;
                typename TcColumns<X, O, VEC>::template Rows<O, 1> old;
                if (a.m.residual) res.load(col, a.m.residual, a.m.ldr, i, a.m.m);
                if (a.m.accumulate) old.load(col, a.m.out, a.m.ldo, i, a.m.m);
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
                const uint32_t at = smem_u32(sums + r * 128);
                for (uint32_t p = 0; p < S; ++p) {
                    const uint32_t from = map_rank(at, 2 * p + half);
                    const float4 w = VEC ? ld_cluster_f4(from + lane * 16)
                                         : make_float4(ld_cluster_f(from + lane * 4), ld_cluster_f(from + lane * 4 + 128),
                                                       ld_cluster_f(from + lane * 4 + 256),
                                                       ld_cluster_f(from + lane * 4 + 384));
                    sum.x += w.x, sum.y += w.y, sum.z += w.z, sum.w += w.w;
                }
                float z[4];
                col.activate(a.m, i, sum, z);
                if (a.m.residual) res.add(0, col.live, z);
                if (a.m.accumulate) old.add(0, col.live, z);
                col.template store<O>(a.m.out, i * a.m.ldo, z);
            }
        }
    }
    __syncwarp();
    if (s->abort && lane == 0 && warp >= 8) {
        // copies and products may still be under way: let them land before the memory is given up
        const uint64_t t0 = globaltimer_ns();
        for (int it = 0; it < 100000 && globaltimer_ns() - t0 < 5000000; ++it) __nanosleep(200);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    if (warp == 9) tmem_free(tmem, COLUMNS);
    cluster_sync();
}

}  // namespace symar
