// Tensor-core matrix products of f16 operands.
#include "linear_tc_launch.cuh"

namespace symar {

sym_status_t matmul_tc_f16(const MatmulArgs& m, sym_dtype_t out, bool a_mn, bool b_mn, int nt, uint32_t splits,
                           cudaStream_t st) {
    return launch_tc_type<__half>(m, SYM_F16, out, a_mn, b_mn, {nt, splits}, st);
}

}  // namespace symar
