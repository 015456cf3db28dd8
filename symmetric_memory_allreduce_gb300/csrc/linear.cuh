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
    // z = C + bias[j]; pre(i,j) = z; out(i,j) = act(z) + residual(i,j), or out += it
    const void* bias;
    const void* residual;
    size_t ldr;
    void* pre;
    size_t ldp;
    void* out;
    size_t ldo;
    int act;
    bool accumulate;
};

// gelu through erfc, not 1 + erf: the latter loses all digits where z is well below zero.
__device__ __forceinline__ float act_value(float z, int act) {
    switch (act) {
        case SYM_ACT_RELU: return z < 0.f ? 0.f : z;
        case SYM_ACT_GELU: return 0.5f * z * erfcf(z * -0.70710678f);
        case SYM_ACT_SILU: return __fdividef(z, 1.f + __expf(-z));
    }
    return z;
}

__device__ __forceinline__ float act_slope(float z, int act) {
    switch (act) {
        case SYM_ACT_RELU: return z > 0.f ? 1.f : 0.f;
        case SYM_ACT_GELU:
            return fmaf(z * 0.39894228f, __expf(-0.5f * z * z), 0.5f * erfcf(z * -0.70710678f));
        case SYM_ACT_SILU: {
            const float p = __fdividef(1.f, 1.f + __expf(-z));
            return p * fmaf(z, 1.f - p, 1.f);
        }
    }
    return 1.f;
}

// One element's epilogue, from the 32-bit sum.
template <class X, class O>
__device__ __forceinline__ void epilogue_one(const MatmulArgs& a, size_t i, size_t j, float z) {
    if (a.bias) z += load_f<X>(a.bias, j);
    if (a.pre) store_f<X>(a.pre, i * a.ldp + j, z);
    z = act_value(z, a.act);
    if (a.residual) z += load_f<X>(a.residual, i * a.ldr + j);
    if (a.accumulate) z += load_f<O>(a.out, i * a.ldo + j);
    store_f<O>(a.out, i * a.ldo + j, z);
}

// linear_bf16.cu, linear_f16.cu: 16-bit operands on the tensor cores, rows of both operands 16-byte
// aligned.  a_mn: b is contiguous along j; b_mn: a is contiguous along i.  nt rows of the output per tile
// (16, 32, 64, 128, 256; b_mn: 128, 256), k shared out to `splits` (1, 2, 4) CTA pairs.
sym_status_t matmul_tc_bf16(const MatmulArgs& m, sym_dtype_t out, bool a_mn, bool b_mn, int nt, uint32_t splits,
                            cudaStream_t st);
sym_status_t matmul_tc_f16(const MatmulArgs& m, sym_dtype_t out, bool a_mn, bool b_mn, int nt, uint32_t splits,
                           cudaStream_t st);

// linear_simt.cu: products in 32 bits on the FMA units, any strides
sym_status_t matmul_simt(const MatmulArgs& a, sym_dtype_t in, sym_dtype_t out, cudaStream_t st);

}  // namespace symar
