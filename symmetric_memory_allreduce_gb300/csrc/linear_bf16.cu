// Tensor-core matrix products of bf16 operands.
#include "linear_tc_launch.cuh"

namespace symar {

sym_status_t matmul_tc_bf16(const MatmulArgs& m, sym_dtype_t out, bool a_mn, bool b_mn, int nt, uint32_t splits,
                            cudaStream_t st) {
    return launch_tc_type<__nv_bfloat16>(m, SYM_BF16, out, a_mn, b_mn, {nt, splits}, st);
}

}  // namespace symar
