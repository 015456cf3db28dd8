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

__device__ __forceinline__ RowTerms row_terms(const PolicyArgs& a, size_t t, float logp) {
    RowTerms o;
    const float A = a.adv[t];
    const float d0 = logp - a.old_logp[t], d = fminf(fmaxf(d0, -kClampLog), kClampLog);
    const float rho = expf(d), bounded = fminf(fmaxf(rho, a.lo), a.hi);
    o.clipped = bounded * A < rho * A;
    o.policy = d0 != d0 ? d0 : -fminf(rho * A, bounded * A);
    o.slope = o.clipped || fabsf(d0) > kClampLog ? 0.f : -A * rho;
    o.kl = 0.f;
    if (a.ref_logp) {
        const float k0 = a.ref_logp[t] - logp, k = fminf(fmaxf(k0, -kClampLog), kClampLog);
        const float kr = expf(k);
        o.kl = k0 != k0 ? k0 : kr - k - 1.f;
        if (!(fabsf(k0) > kClampLog)) o.slope += a.beta * (1.f - kr);
    }
    if (d0 != d0) o.slope = d0;
    return o;
}

// The row's weight, 0 (with the status word set) where its target is no column.
__device__ __forceinline__ float row_weight(const PolicyArgs& a, size_t t) {
    const float w = a.weights ? a.weights[t] : 1.f;
    if (w == 0.f) return 0.f;
    const int64_t y = a.targets[t];
    if (y >= 0 && (uint64_t)y < a.V) return w;
    if (threadIdx.x == 0 && (atomicOr(a.status, kStatusBadArg) & kStatusBadArg) == 0) {
        a.status[1] = kSitePolicyTarget;
        a.status[2] = (uint32_t)t;
        a.status[3] = (uint32_t)y;
    }
    return 0.f;
}

// stats = {loss, policy part, kl, weight of clipped rows}, summed in a fixed order by one
// block of a launch of its own: a counter that finds the last block of the first launch would
// have to live somewhere, and two calls in flight (or a replayed graph) would share it.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) k_policy_stats(PolicyArgs a) {
    __shared__ double red[THREADS / 32];
    double s[4] = {0., 0., 0., 0.};
    for (size_t t = threadIdx.x; t < a.T; t += THREADS) {
        float w = a.weights ? a.weights[t] : 1.f;
        const int64_t y = a.targets[t];
        if (w == 0.f || y < 0 || (uint64_t)y >= a.V) continue;
        const RowTerms r = row_terms(a, t, a.logp[t]);
        s[0] += (double)(w * (r.policy + a.beta * r.kl));
        s[1] += (double)(w * r.policy);
        s[2] += (double)(w * r.kl);
        s[3] += r.clipped ? (double)w : 0.;
    }
    for (int i = 0; i < 4; ++i) {
        const double v = block_sum<THREADS>(s[i], red);
        if (threadIdx.x == 0) a.stats[i] = (float)v;
    }
}

constexpr int kLossThreads = 512;
constexpr int kStatsThreads = 512;

template <class X>
__device__ __forceinline__ void write_gradient(const PolicyArgs& a, size_t t, float c, float lse) {
    const X* x = static_cast<const X*>(a.logits) + t * a.ld;
    X* g = static_cast<X*>(a.dlogits) + t * a.ldd;
    const size_t y = (size_t)a.targets[t];
    for (size_t j = threadIdx.x; j < a.V; j += kLossThreads) {
        float v = -c * expf(to_f(x[j]) * a.inv_t - lse);
        if (j == y) v += c;
        g[j] = from_f<X>(v);
    }
}

template <class X>
__device__ __forceinline__ void write_zeros(const PolicyArgs& a, size_t t) {
    X* g = static_cast<X*>(a.dlogits) + t * a.ldd;
    for (size_t j = threadIdx.x; j < a.V; j += kLossThreads) g[j] = from_f<X>(0.f);
}

template <class X>
__global__ void __launch_bounds__(kLossThreads) k_policy_loss(PolicyArgs a) {
    __shared__ float s_m[kLossThreads / 32], s_s[kLossThreads / 32];
    const size_t t = blockIdx.x;
    const float w = row_weight(a, t);
    if (w == 0.f) {
        if (threadIdx.x == 0) a.logp[t] = a.lse[t] = 0.f;
        if (a.dlogits) write_zeros<X>(a, t);
    } else {
        const X* x = static_cast<const X*>(a.logits) + t * a.ld;
        float m = -INFINITY, s = 0.f;
        for (size_t j = threadIdx.x; j < a.V; j += kLossThreads) {
            const float z = to_f(x[j]) * a.inv_t;
            const float M = fmaxf(m, z);
            if (M != -INFINITY) s = s * expf(m - M) + expf(z - M);
            else if (z != z) s = z;
            m = M;
        }
        const float wm = warp_max(m);
        s = warp_sum(wm == -INFINITY ? s : s * expf(m - wm));
        if ((threadIdx.x & 31) == 0) {
            s_m[threadIdx.x >> 5] = wm;
            s_s[threadIdx.x >> 5] = s;
        }
        __syncthreads();
        m = -INFINITY;
        for (int i = 0; i < kLossThreads / 32; ++i) m = fmaxf(m, s_m[i]);
        s = 0.f;
        for (int i = 0; i < kLossThreads / 32; ++i) s += m == -INFINITY ? s_s[i] : s_s[i] * expf(s_m[i] - m);
        const float lse = m + logf(s);
        const float logp = to_f(x[(size_t)a.targets[t]]) * a.inv_t - lse;
        if (threadIdx.x == 0) {
            a.logp[t] = logp;
            a.lse[t] = lse;
        }
        if (a.dlogits) {
            const float go = a.grad_out ? *a.grad_out : 1.f;
            __syncthreads();                       // the target's logit is read before in-place gradients replace it
            write_gradient<X>(a, t, go * w * row_terms(a, t, logp).slope * a.inv_t, lse);
        }
    }
}

template <class X>
__global__ void __launch_bounds__(kLossThreads) k_policy_backward(PolicyArgs a) {
    const size_t t = blockIdx.x;
    const float w = row_weight(a, t);
    if (w == 0.f) {
        write_zeros<X>(a, t);
        return;
    }
    const float go = a.grad_out ? *a.grad_out : 1.f;
    write_gradient<X>(a, t, go * w * row_terms(a, t, a.logp[t]).slope * a.inv_t, a.lse[t]);
}

}  // namespace symar

using namespace symar;

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
    if (rows) switch (dtype) {
        case SYM_F32: k_policy_loss<float><<<(unsigned)rows, kLossThreads, 0, st>>>(a); break;
        case SYM_BF16: k_policy_loss<__nv_bfloat16><<<(unsigned)rows, kLossThreads, 0, st>>>(a); break;
        case SYM_F16: k_policy_loss<__half><<<(unsigned)rows, kLossThreads, 0, st>>>(a); break;
    }
    k_policy_stats<kStatsThreads><<<1, kStatsThreads, 0, st>>>(a);
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
    switch (dtype) {
        case SYM_F32: k_policy_backward<float><<<(unsigned)rows, kLossThreads, 0, st>>>(a); break;
        case SYM_BF16: k_policy_backward<__nv_bfloat16><<<(unsigned)rows, kLossThreads, 0, st>>>(a); break;
        case SYM_F16: k_policy_backward<__half><<<(unsigned)rows, kLossThreads, 0, st>>>(a); break;
    }
    count_launch();
    SYM_CUDA(cudaGetLastError());
    return SYM_OK;
}

}  // extern "C"
