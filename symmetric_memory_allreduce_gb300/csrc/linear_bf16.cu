// Tensor-core matrix products of bf16 operands.
#include <array>
#include <cstdio>
#include <map>
#include <mutex>

#include "linear_tc_launch.cuh"

namespace symar {

sym_status_t matmul_tc_bf16(const MatmulArgs& m, sym_dtype_t out, bool a_mn, bool b_mn, int nt, uint32_t splits,
                            cudaStream_t st) {
    return launch_tc_type<__nv_bfloat16>(m, SYM_BF16, out, a_mn, b_mn, {nt, splits}, st);
}

sym_status_t matmul_tc_held(int device, int num_sms, uint32_t* held_out) {
    static std::mutex mu;
    static std::map<int, std::array<uint32_t, 5>> known;
    std::lock_guard<std::mutex> lk(mu);
    auto it = known.find(device);
    if (it == known.end()) {
        const void* k = (const void*)k_matmul_tc<__nv_bfloat16, __nv_bfloat16, false, false, 128, true>;
        SYM_CUDA(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTcSmem));
        std::array<uint32_t, 5> n{};
        n[1] = (uint32_t)num_sms / 2;
        for (uint32_t s = 2; s <= 4; s *= 2) {
            const TcConfig c(2 * s * 64, kTcThreads, kTcSmem, 2 * s, nullptr);
            int held = 0;
            SYM_CUDA(cudaOccupancyMaxActiveClusters(&held, k, &c.cfg));
            n[s] = (uint32_t)std::max(held, 0);
        }
        it = known.emplace(device, n).first;
        if (trace_on()) fprintf(stderr, "[symar] linear: %u, %u, %u clusters of 2, 4, 8 CTAs at once\n", n[1], n[2], n[4]);
    }
    std::copy(it->second.begin(), it->second.end(), held_out);
    return SYM_OK;
}

}  // namespace symar
