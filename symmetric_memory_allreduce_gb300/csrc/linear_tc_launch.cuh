// Host side of the tensor-core matrix product: operand maps, tile shape, launch.
#pragma once

#include <cudaTypedefs.h>

#include "linear_tc.cuh"

namespace symar {

// cuTensorMapEncodeTiled, looked up through the runtime (the library does not link the driver's).
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encode() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return (PFN_cuTensorMapEncodeTiled_v12000)p;
    }();
    return fn;
}

// `rows` rows of `cols` contiguous 16-bit elements, `ld` apart, copied in boxes of 64 x `box` rows.
inline bool encode_map(CUtensorMap* map, sym_dtype_t t, const void* p, size_t rows, size_t cols, size_t ld, int box) {
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {(rows > 1 ? ld : ceil_div(cols, (size_t)8) * 8) * 2};   // one row has no stride
    const cuuint32_t boxes[2] = {kTcBK, (cuuint32_t)box};
    const cuuint32_t es[2] = {1, 1};
    return tensor_map_encode()(map, t == SYM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                               2, const_cast<void*>(p), dims, strides, boxes, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class X, class O, bool A_MN, bool B_MN, int NT>
sym_status_t launch_tc(const MatmulArgs& m, sym_dtype_t t, uint32_t splits, cudaStream_t st) {
    const bool vec = columns_in_eights(m);
    const void* kernel = vec ? (const void*)k_matmul_tc<X, O, A_MN, B_MN, NT, true>
                             : (const void*)k_matmul_tc<X, O, A_MN, B_MN, NT, false>;
    int dev = 0;
    SYM_CUDA(cudaGetDevice(&dev));
    DevCtx* ctx = dev_ctx(dev);
    if (!ctx) return SYM_ERR_CUDA;
    TcArgs a{};
    // the product's A is the operand along the output's contiguous index: m.b
    const size_t lda = A_MN ? m.bk : m.bj, ldb = B_MN ? m.ak : m.ai;
    if (!tensor_map_encode() ||
        !(A_MN ? encode_map(&a.a, t, m.b, m.kk, m.n, lda, kTcBK) : encode_map(&a.a, t, m.b, m.n, m.kk, lda, 128)) ||
        !(B_MN ? encode_map(&a.b, t, m.a, m.kk, m.m, ldb, kTcBK) : encode_map(&a.b, t, m.a, m.m, m.kk, ldb, NT / 2))) {
        set_last_error("linear: cuTensorMapEncodeTiled failed");
        return SYM_ERR_CUDA;
    }
    a.m = m;
    a.tiles_i = (uint32_t)ceil_div(m.m, (size_t)NT);
    a.tiles_j = (uint32_t)ceil_div(m.n, (size_t)256);
    a.group = 8;
    a.kblocks = (uint32_t)ceil_div(m.kk, (size_t)kTcBK);
    while (splits > a.kblocks) splits /= 2;               // a pair without terms would have nothing to commit
    a.splits = splits;
    a.status = ctx->status;
    a.timeout_ns = default_timeout_ns();
    if ((uint64_t)a.tiles_i * a.tiles_j >= (1ull << 26)) return SYM_ERR_UNSUPPORTED;
    const uint32_t tiles = a.tiles_i * a.tiles_j;
    static std::atomic<uint64_t> ready[2];                // devices whose limit is set
    if (dev >= 64 || !(ready[vec].load(std::memory_order_acquire) >> dev & 1)) {
        SYM_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTcSmem));
        if (dev < 64) ready[vec].fetch_or(1ull << dev, std::memory_order_release);
    }
    const uint32_t pairs = (uint32_t)ctx->num_sms / 2;
    const TcConfig c(splits > 1 ? tiles * 2 * splits : 2 * std::min(tiles, pairs), kTcThreads, kTcSmem, 2 * splits, st);
    void* args[] = {&a};
    SYM_CUDA(cudaLaunchKernelExC(&c.cfg, kernel, args));
    count_launch();
    return SYM_OK;
}

struct TcShape {
    int nt;
    uint32_t splits;
};

template <class X, class O, bool A_MN>
sym_status_t launch_tc_rows(const MatmulArgs& m, sym_dtype_t t, TcShape s, cudaStream_t st) {
    switch (s.nt) {
        case 16: return launch_tc<X, O, A_MN, false, 16>(m, t, s.splits, st);
        case 32: return launch_tc<X, O, A_MN, false, 32>(m, t, s.splits, st);
        case 64: return launch_tc<X, O, A_MN, false, 64>(m, t, s.splits, st);
        case 128: return launch_tc<X, O, A_MN, false, 128>(m, t, s.splits, st);
    }
    return launch_tc<X, O, A_MN, false, 256>(m, t, s.splits, st);
}

template <class X, class O>
sym_status_t launch_tc_cols(const MatmulArgs& m, sym_dtype_t t, TcShape s, cudaStream_t st) {
    if (s.nt == 128 || sizeof(O) == 4) return launch_tc<X, O, true, true, 128>(m, t, s.splits, st);
    return launch_tc<X, O, true, true, sizeof(O) == 4 ? 128 : 256>(m, t, s.splits, st);
}

// The layouts of the three products: forward (both operands contiguous along k), dX (m.b contiguous
// along j) and dW (m.b along j, m.a along i).
template <class X>
sym_status_t launch_tc_type(const MatmulArgs& m, sym_dtype_t t, sym_dtype_t out, bool a_mn, bool b_mn, TcShape s,
                            cudaStream_t st) {
    if (b_mn) return out == SYM_F32 ? launch_tc_cols<X, float>(m, t, s, st) : launch_tc_cols<X, X>(m, t, s, st);
    return a_mn ? launch_tc_rows<X, X, true>(m, t, s, st) : launch_tc_rows<X, X, false>(m, t, s, st);
}

}  // namespace symar
