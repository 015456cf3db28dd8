// What the linear operators' kernels share: one matrix product's description and its epilogue.
#pragma once

#include "training.cuh"

namespace symar {

// C(i,j) = sum_k A(i,k) B(j,k), then the epilogue.  A's element (i,k) is at i*ai + k*ak, one of
// ai, ak being 1; B likewise.  Rows i < m, columns j < n, terms k < kk.
struct MatmulArgs {
    const void* a;
    const void* b;
    size_t ai, ak, bj, bk;
    size_t m, n, kk;
    // z = C + bias[j]; pre(i,j) = z; out(i,j) = act(z) + residual(i,j).  bias and pre are of the operands'
    // type, residual of out's: an accumulating product passes `out` itself.
    const void* bias;
    const void* residual;
    size_t ldr;
    void* pre;
    size_t ldp;
    void* out;
    size_t ldo;
    int act;
};

// exp(-z^2/2).  PRECISE carries the roundings of z^2 and of its product with log2(e) along, which an
// exponent of tens would turn into several units of the last place.
template <bool PRECISE>
__device__ __forceinline__ float gauss(float z) {
    constexpr float c = -0.72134752f;                       // -log2(e)/2
    const float zz = z * z, y = zz * c;
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y));
    if (PRECISE && y > -150.f) e = fmaf(e, 0.69314718f * fmaf(fmaf(z, z, -zz), c, fmaf(zz, c, -y)), e);
    return e;
}

// Phi(-|z|) = erfc(|z|/sqrt 2)/2 = e Q(t), e = exp(-z^2/2), t = 1/(1 + 0.3 |z|), for two z.  Q is the
// polynomial of degree 8 without a constant term that is nearest to Phi(-|z|)/e in relative distance for
// |z| <= 14.5 (fitted on 4000 Chebyshev nodes by reweighted least squares: 1.7e-7 off at most); beyond, e
// is 0.  One exponential and one reciprocal: 3 times as fast as erfcf, and, unlike 1 + erf, exact digits at
// both ends.
__device__ __forceinline__ void lower_tail2(float z0, float z1, float e0, float e1, float& h0, float& h1) {
    const F2 t = f2(__fdividef(1.f, fmaf(fabsf(z0), 0.3f, 1.f)), __fdividef(1.f, fmaf(fabsf(z1), 0.3f, 1.f)));
    auto both = [](float c) { return f2(c, c); };
    F2 q = fma2(both(0.0354238595f), t, both(-0.156158936f));
    q = fma2(q, t, both(0.20455757f));
    q = fma2(q, t, both(-0.0520346846f));
    q = fma2(q, t, both(0.127692095f));
    q = fma2(q, t, both(0.100175859f));
    q = fma2(q, t, both(0.120712149f));
    q = fma2(q, t, both(0.119632006f));
    float q0, q1, t0, t1;
    split(q, q0, q1);
    split(t, t0, t1);
    h0 = q0 * t0 * e0;
    h1 = q1 * t1 * e1;
}

// Activations of two elements.  X: the type that they are rounded to; 32-bit ones get the slower, closer
// forms.
template <class X, int ACT>
__device__ __forceinline__ void act_value2(float& z0, float& z1) {
    constexpr bool PRECISE = sizeof(X) == 4;
    if (ACT == SYM_ACT_RELU) {
        z0 = z0 < 0.f ? 0.f : z0;
        z1 = z1 < 0.f ? 0.f : z1;
    } else if (ACT == SYM_ACT_GELU) {
        float h0, h1;
        lower_tail2(z0, z1, gauss<PRECISE>(z0), gauss<PRECISE>(z1), h0, h1);
        z0 *= z0 < 0.f ? h0 : 1.f - h0;
        z1 *= z1 < 0.f ? h1 : 1.f - h1;
    } else if (ACT == SYM_ACT_SILU) {
        z0 = PRECISE ? z0 / (1.f + expf(-z0)) : __fdividef(z0, 1.f + __expf(-z0));
        z1 = PRECISE ? z1 / (1.f + expf(-z1)) : __fdividef(z1, 1.f + __expf(-z1));
    }
}

template <class X>
__device__ __forceinline__ float act_value(float z, int act) {
    float other = 0.f;
    if (act == SYM_ACT_RELU) act_value2<X, SYM_ACT_RELU>(z, other);
    else if (act == SYM_ACT_GELU) act_value2<X, SYM_ACT_GELU>(z, other);
    else if (act == SYM_ACT_SILU) act_value2<X, SYM_ACT_SILU>(z, other);
    return z;
}

template <class X, int ACT>
__device__ __forceinline__ void act_slope2(float z0, float z1, float& a0, float& a1) {
    constexpr bool PRECISE = sizeof(X) == 4;
    if (ACT == SYM_ACT_RELU) {
        a0 = z0 > 0.f ? 1.f : 0.f;
        a1 = z1 > 0.f ? 1.f : 0.f;
    } else if (ACT == SYM_ACT_GELU) {
        const float e0 = gauss<PRECISE>(z0), e1 = gauss<PRECISE>(z1);
        float h0, h1;
        lower_tail2(z0, z1, e0, e1, h0, h1);
        a0 = fmaf(z0 * 0.39894228f, e0, z0 < 0.f ? h0 : 1.f - h0);
        a1 = fmaf(z1 * 0.39894228f, e1, z1 < 0.f ? h1 : 1.f - h1);
    } else if (ACT == SYM_ACT_SILU) {
        const float p0 = PRECISE ? 1.f / (1.f + expf(-z0)) : __fdividef(1.f, 1.f + __expf(-z0));
        const float p1 = PRECISE ? 1.f / (1.f + expf(-z1)) : __fdividef(1.f, 1.f + __expf(-z1));
        a0 = p0 * fmaf(z0, 1.f - p0, 1.f);
        a1 = p1 * fmaf(z1, 1.f - p1, 1.f);
    }
}

// linear_bf16.cu, linear_f16.cu: 16-bit operands on the tensor cores, rows of both operands 16-byte
// aligned.  a_mn: b is contiguous along j; b_mn: a is contiguous along i.  nt rows of the output per tile
// (16, 32, 64, 128, 256; b_mn: 128, 256), k shared out to `splits` (1, 2, 4) CTA pairs.
sym_status_t matmul_tc_bf16(const MatmulArgs& m, sym_dtype_t out, bool a_mn, bool b_mn, int nt, uint32_t splits,
                            cudaStream_t st);
sym_status_t matmul_tc_f16(const MatmulArgs& m, sym_dtype_t out, bool a_mn, bool b_mn, int nt, uint32_t splits,
                           cudaStream_t st);

// linear_f32.cu: 32-bit operands on the tensor cores, any strides; nt 16, 32, 64 or 128 (b_mn: 128).
sym_status_t matmul_f32(const MatmulArgs& m, bool a_mn, bool b_mn, int nt, uint32_t splits, cudaStream_t st);

// The three products and their layouts: forward (both operands contiguous along k), dX (m.b contiguous
// along j), dW (m.b along j, m.a along i).
enum class Product { kForward, kDx, kDw };

// linear_skinny.cu: few rows (m.m; kDw: few terms, m.kk), any strides.
bool matmul_is_skinny(size_t rows, sym_dtype_t in, Product product);
sym_status_t matmul_skinny(const MatmulArgs& m, sym_dtype_t in, sym_dtype_t out, Product product, int num_sms,
                           cudaStream_t st);

// How many clusters of 2, 4 and 8 CTAs of these kernels a device holds at once: held[1], held[2], held[4].
sym_status_t matmul_tc_held(int device, int num_sms, uint32_t* held);

}  // namespace symar
