// Clipped policy loss with a KL term, from logits, and its gradient.
//
// For row t with weight w_t != 0, z = logits_t / temperature, y = target:
//   lse  = log sum_j exp(z_j)             logp = z_y - lse
//   d    = clamp(logp - old, -20, 20)     rho  = exp(d)
//   k    = clamp(ref - logp, -20, 20)     kl   = exp(k) - k - 1
//   L_t  = -min(rho A, clip(rho, 1-lo, 1+hi) A) + beta kl
//   dL_t/dlogp = -A rho (0 where the clipped product is the smaller one, or
//                d is clamped) + beta (1 - exp(k)) (0 where k is clamped)
//   dlogits_j  = grad w_t dL_t/dlogp (1[j=y] - exp(z_j - lse)) / temperature
// The sums over a row are held in binary32.  A row of weight 0 is not read:
// its outputs are 0 whatever stands there.
#include <cmath>
#include <type_traits>

#include "tensor.cuh"
#include "training.cuh"

namespace symar {

constexpr float kClampLog = 20.f;

struct PolicyArgs {
    const void* logits;
    size_t ld;
    size_t T, V;
    const int64_t* targets;
    const float* old_logp;
    const float* ref_logp;     // null: no KL term
    const float* adv;
    const float* weights;      // null: 1
    const float* grad_out;     // device scalar; null: 1
    float lo, hi, beta, inv_t;
    float* stats;
    float* logp;
    float* lse;
    void* dlogits;             // null: no gradient
    size_t ldd;
    uint32_t* status;
};

struct RowTerms {
    float policy, kl, slope;
    bool clipped;
};

// A row's inputs but its logits.
struct RowInputs {
    float A, old, ref, go;
    __device__ __forceinline__ RowInputs(const PolicyArgs& a, size_t t) {
        A = a.adv[t];
        old = a.old_logp[t];
        ref = a.ref_logp ? a.ref_logp[t] : 0.f;
        go = a.grad_out ? *a.grad_out : 1.f;
    }
};

__device__ __forceinline__ RowTerms row_terms(const PolicyArgs& a, const RowInputs& in, float logp) {
    RowTerms o;
    const float A = in.A;
    const float d0 = logp - in.old, d = fminf(fmaxf(d0, -kClampLog), kClampLog);
    const float rho = expf(d), bounded = fminf(fmaxf(rho, a.lo), a.hi);
    o.clipped = bounded * A < rho * A;
    o.policy = d0 != d0 ? d0 : -fminf(rho * A, bounded * A);
    o.slope = o.clipped || fabsf(d0) > kClampLog ? 0.f : -A * rho;
    o.kl = 0.f;
    if (a.ref_logp) {
        const float k0 = in.ref - logp, k = fminf(fmaxf(k0, -kClampLog), kClampLog);
        const float kr = expf(k);
        o.kl = k0 != k0 ? k0 : kr - k - 1.f;
        if (!(fabsf(k0) > kClampLog)) o.slope += a.beta * (1.f - kr);
    }
    if (d0 != d0) o.slope = d0;
    return o;
}

// The row's weight, 0 (with the status word set) where its target is no column.
__device__ __forceinline__ float row_weight(const PolicyArgs& a, size_t t, bool report) {
    const float w = a.weights ? a.weights[t] : 1.f;
    if (w == 0.f) return 0.f;
    const int64_t y = a.targets[t];
    if (y >= 0 && (uint64_t)y < a.V) return w;
    if (report && threadIdx.x == 0 && (atomicOr(a.status, kStatusBadArg) & kStatusBadArg) == 0) {
        a.status[1] = kSitePolicyTarget;
        a.status[2] = (uint32_t)t;
        a.status[3] = (uint32_t)y;
    }
    return 0.f;
}

// One element of a row, as 16-byte vectors of E elements counted from the 16-byte boundary at or
// before the row's start: vector v holds elements v*E - phase and on.
template <class X>
struct Row {
    static constexpr int E = 16 / sizeof(X);
    X* p;
    int phase;
    __device__ __forceinline__ Row(const void* base, size_t at) {
        p = const_cast<X*>(static_cast<const X*>(base)) + at;
        phase = (int)((uintptr_t)p / sizeof(X) % E);
    }
};

template <class X>
__device__ __forceinline__ uint32_t minus_inf_bits();
template <>
__device__ __forceinline__ uint32_t minus_inf_bits<float>() { return 0xFF800000u; }
template <>
__device__ __forceinline__ uint32_t minus_inf_bits<__nv_bfloat16>() { return 0xFF80FF80u; }
template <>
__device__ __forceinline__ uint32_t minus_inf_bits<__half>() { return 0xFC00FC00u; }

// Element pair k of a vector.
template <class X>
__device__ __forceinline__ void unpack2(const uint4& v, int k, float& x, float& y) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (sizeof(X) == 4) {
        x = __uint_as_float(w[2 * k]), y = __uint_as_float(w[2 * k + 1]);
    } else if (std::is_same<X, __nv_bfloat16>::value) {
        x = __uint_as_float(w[k] << 16), y = __uint_as_float(w[k] & 0xFFFF0000u);
    } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
        x = f.x, y = f.y;
    }
}

template <class X>
__device__ __forceinline__ void pack2(uint4& v, int k, float x, float y) {
    uint32_t* w = &v.x;
    if (sizeof(X) == 4) {
        w[2 * k] = __float_as_uint(x), w[2 * k + 1] = __float_as_uint(y);
    } else if (std::is_same<X, __nv_bfloat16>::value) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
        w[k] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
        const __half2 h = __floats2half2_rn(x, y);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
}

// Largest of a vector's elements and m; NaN elements are passed over (their exponentials are NaN).
template <class X>
__device__ __forceinline__ float max_vector(const uint4& v, float m) {
    if (sizeof(X) == 4) {
        m = fmaxf(m, fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)));
        return fmaxf(m, fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    }
    float x, y;
    uint4 t;
    if (std::is_same<X, __nv_bfloat16>::value) {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
        const __nv_bfloat162 b = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        t.x = *reinterpret_cast<const uint32_t*>(&b);
    } else {
        const __half2* h = reinterpret_cast<const __half2*>(&v);
        const __half2 b = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        t.x = *reinterpret_cast<const uint32_t*>(&b);
    }
    t.y = t.z = t.w = 0;
    unpack2<X>(t, 0, x, y);
    return fmaxf(m, fmaxf(x, y));
}

// Vector v of a row; what lies outside the row's V elements reads as -infinity (weight 0).
template <class X>
__device__ __forceinline__ uint4 load_vector(const Row<X>& r, int64_t v, int64_t V) {
    constexpr int E = Row<X>::E;
    const int64_t j = v * E - r.phase;
    if (j >= 0 && j + E <= V) return __ldcs(reinterpret_cast<const uint4*>(r.p + j));
    const uint32_t inf = minus_inf_bits<X>();
    uint4 x = make_uint4(inf, inf, inf, inf);
    X* h = reinterpret_cast<X*>(&x);
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (j + e >= 0 && j + e < V) h[e] = r.p[j + e];
    return x;
}

// Writes the elements of vector v (counted in a row with `phase`) that are inside.
template <class X>
__device__ __forceinline__ void store_vector(const Row<X>& r, int phase, int64_t v, int64_t V, const uint4& x) {
    constexpr int E = Row<X>::E;
    const int64_t j = v * E - phase;
    if (phase == r.phase && j >= 0 && j + E <= V) {
        __stcs(reinterpret_cast<uint4*>(r.p + j), x);
        return;
    }
    const X* h = reinterpret_cast<const X*>(&x);
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (j + e >= 0 && j + e < V) r.p[j + e] = h[e];
}

__device__ __forceinline__ float exp2_approx(float x) {      // 2 ulp; below 2^-126: 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Adds exp2(c x - b) of a vector's elements to two sums.
template <class X>
__device__ __forceinline__ void add_vector(const uint4& v, F2 c, F2 b, F2& s) {
#pragma unroll
    for (int k = 0; k < Row<X>::E / 2; ++k) {
        float x, y;
        unpack2<X>(v, k, x, y);
        split(fma2(f2(x, y), c, b), x, y);
        s = add2(s, f2(exp2_approx(x), exp2_approx(y)));
    }
}

// Joins two (maximum, sum) pairs.
__device__ __forceinline__ void join(float c, float& m, float& s, float m2, float s2) {
    const float M = fmaxf(m, m2), b = M == -INFINITY ? 0.f : M * c;
    s = s * exp2_approx(fmaf(m, c, -b)) + s2 * exp2_approx(fmaf(m2, c, -b));
    m = M;
}

// The gradient's common factors of a row: dlogits_j = -coef exp2(c x_j - lse2) (+ coef at the target).
struct RowGrad {
    float shift;               // log2|coef| - lse2
    uint32_t flip;             // sign bits of -coef, for one 32-bit word of X
    float coef, lse2;
};

template <class X>
__device__ __forceinline__ RowGrad row_grad(float coef, float lse) {
    RowGrad g;
    g.coef = coef;
    g.lse2 = lse * 1.44269504f;
    g.shift = log2f(fabsf(coef)) - g.lse2;
    g.flip = coef > 0.f ? (sizeof(X) == 4 ? 0x80000000u : 0x80008000u) : 0u;
    return g;
}

// Its magnitudes are 2^(c x + shift): one product, one exponential, one rounding an element; the sign
// is set on the rounded word.
template <class X>
__device__ __forceinline__ uint4 grad_vector(const uint4& v, F2 c, F2 shift, uint32_t flip) {
    uint4 o;
#pragma unroll
    for (int k = 0; k < Row<X>::E / 2; ++k) {
        float x, y;
        unpack2<X>(v, k, x, y);
        split(fma2(f2(x, y), c, shift), x, y);
        pack2<X>(o, k, exp2_approx(x), exp2_approx(y));
    }
    o.x ^= flip, o.y ^= flip, o.z ^= flip, o.w ^= flip;
    return o;
}

// The target's element, by the thread that wrote its vector, after it.
template <class X>
__device__ __forceinline__ void fix_target(const Row<X>& d, int phase, int64_t v, int64_t y, float c, float xy,
                                           const RowGrad& g) {
    const int64_t j = v * Row<X>::E - phase;
    if (y >= j && y < j + Row<X>::E) d.p[y] = from_f<X>(g.coef - g.coef * exp2_approx(fmaf(xy, c, -g.lse2)));
}

// A cluster of CTAs per row (1, 2, 4 or 8), each with a run of its vectors, VPT a thread at a time,
// neighbouring threads on neighbouring vectors.  KEEP: the run fits the threads' registers, so the
// logits are read once and the gradient comes from registers; else they are read again for it.
template <class X, int THREADS, int VPT, bool KEEP>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) k_policy_loss(PolicyArgs a, int64_t run) {
    __shared__ float s_m[THREADS / 32], s_s[THREADS / 32], s_cm[8], s_cs[8];
    __shared__ RowGrad s_g;
    uint32_t rank = 0, C = 1;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(C));
    const size_t t = blockIdx.x / C;
    const int64_t V = (int64_t)a.V;
    const Row<X> x(a.logits, t * a.ld), d(a.dlogits, a.dlogits ? t * a.ldd : 0);
    const int64_t vectors = (V + x.phase + Row<X>::E - 1) / Row<X>::E;
    const int64_t v0 = (int64_t)rank * run + threadIdx.x, v1 = min((int64_t)(rank + 1) * run, vectors);
    uint4 r[VPT];
    const float w = row_weight(a, t, rank == 0);
    if (w == 0.f) {                                          // the same in every CTA of the cluster
        if (rank == 0 && threadIdx.x == 0) a.logp[t] = a.lse[t] = 0.f;
        if (a.dlogits)
            for (int64_t v = v0; v < v1; v += THREADS) store_vector<X>(d, x.phase, v, V, make_uint4(0, 0, 0, 0));
        return;
    }
    const RowInputs in(a, t);
    const int64_t y = a.targets[t];
    const float xy = to_f(x.p[y]);                           // before a gradient in place can replace it
    if (C > 1) cluster_arrive();                             // waited for before the first remote store
    const float c = a.inv_t * 1.44269504f;
    float m = -INFINITY, s = 0.f;
    for (int64_t v = v0; v < v1; v += (int64_t)THREADS * VPT) {
        const uint32_t inf = minus_inf_bits<X>();
#pragma unroll
        for (int k = 0; k < VPT; ++k)
            r[k] = v + k * THREADS < v1 ? load_vector<X>(x, v + k * THREADS, V) : make_uint4(inf, inf, inf, inf);
        float M = m;
#pragma unroll
        for (int k = 0; k < VPT; ++k) M = max_vector<X>(r[k], M);
        const float b = M == -INFINITY ? 0.f : -M * c;       // all -inf so far: every term is 0
        F2 sum = f2(KEEP ? 0.f : s * exp2_approx(fmaf(m, c, b)), 0.f);
#pragma unroll
        for (int k = 0; k < VPT; ++k) add_vector<X>(r[k], f2(c, c), f2(b, b), sum);
        float s1;
        split(sum, s, s1);
        s += s1;
        m = M;
        if (KEEP) break;
    }
    const float wm = warp_max(m);
    s = warp_sum(s * exp2_approx(fmaf(m, c, wm == -INFINITY ? 0.f : -wm * c)));
    if (threadIdx.x % 32 == 0) {
        s_m[threadIdx.x / 32] = wm;
        s_s[threadIdx.x / 32] = s;
    }
    __syncthreads();
    if (C > 1) cluster_wait();
    if (threadIdx.x < 32) {
        constexpr int W = THREADS / 32;
        m = threadIdx.x < W ? s_m[threadIdx.x] : -INFINITY;
        s = threadIdx.x < W ? s_s[threadIdx.x] : 0.f;
#pragma unroll
        for (int o = 1; o < W; o <<= 1) join(c, m, s, __shfl_xor_sync(~0u, m, o), __shfl_xor_sync(~0u, s, o));
        if (C > 1 && threadIdx.x < C) {                      // to every CTA of the cluster
            st_cluster_f32(map_rank(smem_u32(&s_cm[rank]), threadIdx.x), m);
            st_cluster_f32(map_rank(smem_u32(&s_cs[rank]), threadIdx.x), s);
        }
    }
    if (C > 1) {
        __syncwarp();
        cluster_sync();
    }
    if (threadIdx.x == 0) {
        if (C > 1) {
            m = s_cm[0], s = s_cs[0];
            for (uint32_t q = 1; q < C; ++q) join(c, m, s, s_cm[q], s_cs[q]);
        }
        const float lse = m * a.inv_t + logf(s), logp = xy * a.inv_t - lse;
        if (rank == 0) {
            a.logp[t] = logp;
            a.lse[t] = lse;
        }
        if (a.dlogits) s_g = row_grad<X>(in.go * w * row_terms(a, in, logp).slope * a.inv_t, lse);
    }
    if (!a.dlogits) return;
    __syncthreads();
    const RowGrad g = s_g;
    for (int64_t v = v0; v < v1; v += (int64_t)THREADS * VPT) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int64_t u = v + k * THREADS;
            if (u >= v1) break;
            if (!KEEP) r[k] = load_vector<X>(x, u, V);
            store_vector<X>(d, x.phase, u, V, grad_vector<X>(r[k], f2(c, c), f2(g.shift, g.shift), g.flip));
            fix_target<X>(d, x.phase, u, y, c, xy, g);
        }
        if (KEEP) break;
    }
}

// The gradient alone: a block takes kBackThreads * kBackVectors vectors of a row.
constexpr int kBackThreads = 256, kBackVectors = 4;

template <class X>
__global__ void __launch_bounds__(kBackThreads) k_policy_backward(PolicyArgs a, uint32_t blocks_per_row) {
    __shared__ RowGrad s_g;
    const size_t t = blockIdx.x / blocks_per_row;
    const int64_t V = (int64_t)a.V;
    const Row<X> x(a.logits, t * a.ld), d(a.dlogits, t * a.ldd);
    const int64_t v0 = (int64_t)(blockIdx.x % blocks_per_row) * (kBackThreads * kBackVectors) + threadIdx.x;
    const int64_t vectors = (V + x.phase + Row<X>::E - 1) / Row<X>::E;
    const float w = row_weight(a, t, blockIdx.x % blocks_per_row == 0);
    if (w == 0.f) {
#pragma unroll
        for (int k = 0; k < kBackVectors; ++k)
            if (v0 + k * kBackThreads < vectors)
                store_vector<X>(d, x.phase, v0 + k * kBackThreads, V, make_uint4(0, 0, 0, 0));
        return;
    }
    uint4 r[kBackVectors];
#pragma unroll
    for (int k = 0; k < kBackVectors; ++k)
        if (v0 + k * kBackThreads < vectors) r[k] = load_vector<X>(x, v0 + k * kBackThreads, V);
    const int64_t y = a.targets[t];
    const float c = a.inv_t * 1.44269504f;
    if (threadIdx.x == 0) {
        const RowInputs in(a, t);
        s_g = row_grad<X>(in.go * w * row_terms(a, in, a.logp[t]).slope * a.inv_t, a.lse[t]);
    }
    __syncthreads();
    const RowGrad g = s_g;
#pragma unroll
    for (int k = 0; k < kBackVectors; ++k) {
        const int64_t v = v0 + k * kBackThreads, j = v * Row<X>::E - x.phase;
        if (v >= vectors) break;
        const bool target = y >= j && y < j + Row<X>::E;
        const float xy = target ? to_f(x.p[y]) : 0.f;        // this thread's own vector: not yet replaced
        store_vector<X>(d, x.phase, v, V, grad_vector<X>(r[k], f2(c, c), f2(g.shift, g.shift), g.flip));
        if (target) fix_target<X>(d, x.phase, v, y, c, xy, g);
    }
}

// stats = {loss, policy part, kl, weight of clipped rows}, summed in a fixed order by one
// block of a launch of its own: a counter that finds the last block of the first launch would
// have to live somewhere, and two calls in flight (or a replayed graph) would share it.
constexpr int kStatsThreads = 512;

template <int THREADS>
__global__ void __launch_bounds__(THREADS) k_policy_stats(PolicyArgs a) {
    __shared__ float red[THREADS / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");       // launched while the rows' kernel still runs
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    for (size_t t = threadIdx.x; t < a.T; t += THREADS) {
        float w = a.weights ? a.weights[t] : 1.f;
        const int64_t y = a.targets[t];
        if (w == 0.f || y < 0 || (uint64_t)y >= a.V) continue;
        const RowTerms r = row_terms(a, RowInputs(a, t), a.logp[t]);
        s[0] += w * (r.policy + a.beta * r.kl);
        s[1] += w * r.policy;
        s[2] += w * r.kl;
        s[3] += r.clipped ? w : 0.f;
    }
    for (int i = 0; i < 4; ++i) {
        const float v = block_sum<THREADS>(s[i], red);
        if (threadIdx.x == 0) a.stats[i] = v;
    }
}

// CTAs per row, threads and vectors per thread: the smallest block that holds the row in registers, the
// row shared out further while there are fewer CTAs than SMs.
struct LossShape {
    int threads, vpt;
    uint32_t cluster;
    bool keep;
};

static LossShape loss_shape(size_t T, size_t vectors, int num_sms) {
    LossShape s{128, 2, 1, true};
    while (s.vpt < 8 && (size_t)s.threads * s.vpt < vectors) s.vpt *= 2;
    if ((size_t)s.threads * s.vpt < vectors) s = {512, 4, 1, true};
    if ((size_t)s.threads * s.vpt < vectors) s.vpt = 8;
    while (s.cluster < 8 && (size_t)s.threads * s.vpt * s.cluster < vectors) s.cluster *= 2;
    while (s.cluster < 8 && s.vpt > 2 && T * s.cluster < (size_t)num_sms) s.cluster *= 2, s.vpt /= 2;
    s.keep = (size_t)s.threads * s.vpt * s.cluster >= vectors;
    return s;
}

// 16-byte vectors that a row can touch: one more where rows start between their boundaries.
static size_t row_vectors(const void* logits, size_t ld, size_t rows, size_t vocab, size_t es) {
    const size_t per = 16 / es;
    const bool aligned = (uintptr_t)logits % 16 == 0 && (rows == 1 || ld % per == 0);
    return ceil_div(vocab + (aligned ? 0 : per - 1), per);
}

template <class X>
static const void* loss_kernel(const LossShape& s) {
    if (!s.keep) return (const void*)k_policy_loss<X, 512, 8, false>;
    if (s.threads == 128)
        return s.vpt == 2   ? (const void*)k_policy_loss<X, 128, 2, true>
               : s.vpt == 4 ? (const void*)k_policy_loss<X, 128, 4, true>
                            : (const void*)k_policy_loss<X, 128, 8, true>;
    return s.vpt == 2   ? (const void*)k_policy_loss<X, 512, 2, true>
           : s.vpt == 4 ? (const void*)k_policy_loss<X, 512, 4, true>
                        : (const void*)k_policy_loss<X, 512, 8, true>;
}

}  // namespace symar

using namespace symar;

// A launch with one attribute: a cluster size, or leave to start before the kernel before it has ended.
static cudaError_t launch_with(const void* kernel, unsigned grid, int threads, void** args, cudaStream_t st,
                               cudaLaunchAttributeID id, uint32_t value) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = id;
    if (id == cudaLaunchAttributeClusterDimension) attr.val.clusterDim.x = value, attr.val.clusterDim.y = 1, attr.val.clusterDim.z = 1;
    else attr.val.programmaticStreamSerializationAllowed = (int)value;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, kernel, args);
}

static sym_status_t check_policy(const PolicyArgs& a, sym_dtype_t dtype, double clip_low, double clip_high,
                                 double kl_coef, double temperature) {
    const size_t es = dtype_size(dtype);
    if (!es) return SYM_ERR_INVALID_ARG;
    if (!(temperature > 0) || !std::isfinite(temperature) || !(clip_low >= 0) || !(clip_high >= 0) ||
        !std::isfinite(kl_coef))
        return SYM_ERR_INVALID_ARG;
    if (a.T >= (1ull << 31) || a.V >= (1ull << 31)) return SYM_ERR_UNSUPPORTED;
    if (a.T == 0) return SYM_OK;
    if (a.V == 0 || a.ld < a.V || (a.dlogits && a.ldd < a.V)) return SYM_ERR_INVALID_ARG;
    if (!a.logits || !a.targets || !a.old_logp || !a.adv || !a.logp || !a.lse) return SYM_ERR_INVALID_ARG;
    if ((uintptr_t)a.logits % es || (uintptr_t)a.dlogits % es || (uintptr_t)a.targets % 8) return SYM_ERR_INVALID_ARG;
    for (const void* p : {(const void*)a.old_logp, (const void*)a.ref_logp, (const void*)a.adv,
                          (const void*)a.weights, (const void*)a.grad_out, (const void*)a.logp, (const void*)a.lse,
                          (const void*)a.stats})
        if ((uintptr_t)p % 4) return SYM_ERR_INVALID_ARG;
    if (a.dlogits) {
        // in place (the same rows) or apart; anything between would overwrite logits not yet read
        const uintptr_t x0 = (uintptr_t)a.logits, x1 = x0 + ((a.T - 1) * a.ld + a.V) * es;
        const uintptr_t g0 = (uintptr_t)a.dlogits, g1 = g0 + ((a.T - 1) * a.ldd + a.V) * es;
        if (x0 < g1 && g0 < x1 && !(x0 == g0 && (a.ld == a.ldd || a.T == 1))) {
            set_last_error("sym_policy_loss: dlogits overlaps logits without being the same rows");
            return SYM_ERR_INVALID_ARG;
        }
    }
    return SYM_OK;
}

extern "C" {

sym_status_t sym_policy_loss(const void* logits, size_t ld, size_t rows, size_t vocab, sym_dtype_t dtype,
                             const int64_t* targets, const float* old_logp, const float* ref_logp,
                             const float* advantages, const float* weights, double clip_low, double clip_high,
                             double kl_coef, double temperature, float* stats, float* logp, float* lse, void* dlogits,
                             size_t ldd, const float* grad_out, sym_stream_t stream) {
    PolicyArgs a{logits, ld, rows, vocab, targets, old_logp, ref_logp, advantages, weights, grad_out,
                 (float)(1.0 - clip_low), (float)(1.0 + clip_high), (float)kl_coef, (float)(1.0 / temperature),
                 stats, logp, lse, dlogits, ldd, nullptr};
    if (!stats) return SYM_ERR_INVALID_ARG;
    sym_status_t s = check_policy(a, dtype, clip_low, clip_high, kl_coef, temperature);
    if (s != SYM_OK) return s;
    int dev = 0;
    SYM_CUDA(cudaGetDevice(&dev));
    DevCtx* ctx = dev_ctx(dev);
    if (!ctx) return SYM_ERR_CUDA;
    cudaStream_t st = (cudaStream_t)stream;
    a.status = ctx->status;
    if (rows) {
        const size_t vectors = row_vectors(logits, ld, rows, vocab, dtype_size(dtype));
        const LossShape sh = loss_shape(rows, vectors, ctx->num_sms);
        if (rows * sh.cluster >= (1ull << 31)) return SYM_ERR_UNSUPPORTED;
        int64_t run = (int64_t)ceil_div(vectors, (size_t)sh.cluster);
        const void* k = dtype == SYM_F32    ? loss_kernel<float>(sh)
                        : dtype == SYM_BF16 ? loss_kernel<__nv_bfloat16>(sh)
                                            : loss_kernel<__half>(sh);
        void* args[] = {&a, &run};
        SYM_CUDA(launch_with(k, (unsigned)(rows * sh.cluster), sh.threads, args, st,
                             cudaLaunchAttributeClusterDimension, sh.cluster));
    }
    {
        void* args[] = {&a};
        SYM_CUDA(launch_with((const void*)k_policy_stats<kStatsThreads>, 1, kStatsThreads, args, st,
                             cudaLaunchAttributeProgrammaticStreamSerialization, 1));
    }
    count_launch(rows ? 2 : 1);
    SYM_CUDA(cudaGetLastError());
    return SYM_OK;
}

sym_status_t sym_policy_loss_backward(const void* logits, size_t ld, size_t rows, size_t vocab, sym_dtype_t dtype,
                                      const int64_t* targets, const float* old_logp, const float* ref_logp,
                                      const float* advantages, const float* weights, double clip_low,
                                      double clip_high, double kl_coef, double temperature, const float* logp,
                                      const float* lse, void* dlogits, size_t ldd, const float* grad_out,
                                      sym_stream_t stream) {
    PolicyArgs a{logits, ld, rows, vocab, targets, old_logp, ref_logp, advantages, weights, grad_out,
                 (float)(1.0 - clip_low), (float)(1.0 + clip_high), (float)kl_coef, (float)(1.0 / temperature),
                 nullptr, const_cast<float*>(logp), const_cast<float*>(lse), dlogits, ldd, nullptr};
    sym_status_t s = check_policy(a, dtype, clip_low, clip_high, kl_coef, temperature);
    if (s != SYM_OK) return s;
    if (rows == 0) return SYM_OK;
    if (!dlogits) return SYM_ERR_INVALID_ARG;
    int dev = 0;
    SYM_CUDA(cudaGetDevice(&dev));
    DevCtx* ctx = dev_ctx(dev);
    if (!ctx) return SYM_ERR_CUDA;
    a.status = ctx->status;
    cudaStream_t st = (cudaStream_t)stream;
    const size_t bpr = ceil_div(row_vectors(logits, ld, rows, vocab, dtype_size(dtype)),
                                (size_t)(kBackThreads * kBackVectors));
    if (rows * bpr >= (1ull << 31)) return SYM_ERR_UNSUPPORTED;
    const unsigned grid = (unsigned)(rows * bpr);
    switch (dtype) {
        case SYM_F32: k_policy_backward<float><<<grid, kBackThreads, 0, st>>>(a, (uint32_t)bpr); break;
        case SYM_BF16: k_policy_backward<__nv_bfloat16><<<grid, kBackThreads, 0, st>>>(a, (uint32_t)bpr); break;
        case SYM_F16: k_policy_backward<__half><<<grid, kBackThreads, 0, st>>>(a, (uint32_t)bpr); break;
    }
    count_launch();
    SYM_CUDA(cudaGetLastError());
    return SYM_OK;
}

}  // extern "C"
