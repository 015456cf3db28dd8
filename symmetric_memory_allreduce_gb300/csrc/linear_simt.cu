// Matrix product on the FMA units, for any sizes and strides: 32-bit operands
// (whose products the tensor cores would round).
#include "linear.cuh"

namespace symar {

constexpr int kSimtTile = 64, kSimtK = 16, kSimtThreads = 256;

// One 64 x 64 tile per block, 4 x 4 sums per thread; the operands' tiles go through shared memory.
template <class X, class O>
__global__ void __launch_bounds__(kSimtThreads) k_matmul_simt(MatmulArgs a) {
    __shared__ float sa[kSimtK][kSimtTile + 4], sb[kSimtK][kSimtTile + 4];
    const size_t i0 = (size_t)blockIdx.x * kSimtTile, j0 = (size_t)blockIdx.y * kSimtTile;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float c[4][4] = {};
    for (size_t k0 = 0; k0 < a.kk; k0 += kSimtK) {
        for (int e = threadIdx.x; e < kSimtTile * kSimtK; e += kSimtThreads) {
            // neighbouring threads follow the operand's contiguous index
            const int ia = a.ak == 1 ? e / kSimtK : e % kSimtTile, ka = a.ak == 1 ? e % kSimtK : e / kSimtTile;
            const int jb = a.bk == 1 ? e / kSimtK : e % kSimtTile, kb = a.bk == 1 ? e % kSimtK : e / kSimtTile;
            const size_t i = i0 + ia, j = j0 + jb;
            sa[ka][ia] = i < a.m && k0 + ka < a.kk ? load_f<X>(a.a, i * a.ai + (k0 + ka) * a.ak) : 0.f;
            sb[kb][jb] = j < a.n && k0 + kb < a.kk ? load_f<X>(a.b, j * a.bj + (k0 + kb) * a.bk) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kSimtK; ++k) {
            const float4 x = *reinterpret_cast<const float4*>(&sa[k][ty * 4]);
            const float4 y = *reinterpret_cast<const float4*>(&sb[k][tx * 4]);
            const float u[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int p = 0; p < 4; ++p)
#pragma unroll
                for (int q = 0; q < 4; ++q) c[p][q] = fmaf(u[p], v[q], c[p][q]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const size_t i = i0 + ty * 4 + p, j = j0 + tx * 4 + q;
            if (i < a.m && j < a.n) epilogue_one<X, O>(a, i, j, c[p][q]);
        }
}

template <class X>
static const void* simt_kernel(sym_dtype_t out) {
    if (out == SYM_F32) return (const void*)k_matmul_simt<X, float>;
    return (const void*)k_matmul_simt<X, X>;
}

sym_status_t matmul_simt(const MatmulArgs& a, sym_dtype_t in, sym_dtype_t out, cudaStream_t st) {
    const void* k = in == SYM_F32    ? simt_kernel<float>(out)
                    : in == SYM_BF16 ? simt_kernel<__nv_bfloat16>(out)
                                     : simt_kernel<__half>(out);
    const size_t gx = ceil_div(a.m, (size_t)kSimtTile), gy = ceil_div(a.n, (size_t)kSimtTile);
    if (gx >= (1u << 31) || gy > 65535) return SYM_ERR_UNSUPPORTED;
    void* args[] = {const_cast<MatmulArgs*>(&a)};
    SYM_CUDA(cudaLaunchKernel(k, dim3((unsigned)gx, (unsigned)gy), dim3(kSimtThreads), args, 0, st));
    count_launch();
    return SYM_OK;
}

}  // namespace symar
