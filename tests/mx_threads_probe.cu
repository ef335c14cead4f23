// Several threads make their first microscaled and routing launches at the same time, on a host stand-in for the CUDA
// runtime; built with the thread sanitizer, which reports unsynchronised accesses to what the launchers keep.
#include <cstdlib>
#include <thread>
#include <vector>

#include "../gemm_uq_gb300/csrc/uq_kernels.h"

int main() {
    std::vector<std::thread> all;
    static uint8_t at[4096] __attribute__((aligned(256)));
    for (int i = 0; i < 4; ++i)
        all.emplace_back([] {
            for (int rows : {1, 40, 4096}) {
                uq::MxGemmArgs a = {};
                a.xscales = a.wscales = a.wscales_up = at;
                a.y = at;
                a.rows = rows;
                a.experts = 1;
                a.N = 1024;
                a.K = 8192;
                a.alpha = 1.f;
                for (int fmt : {UQ_MXFP4, UQ_NVFP4})
                    for (const uint8_t* up : {(const uint8_t*)nullptr, (const uint8_t*)at})
                        if (uq::launch_mx_gemm(fmt, at, at, up, a, 152, nullptr) != cudaSuccess) _Exit(2);
            }
            if (uq::launch_moe_sort((const int32_t*)at, 100000, 64, (int32_t*)at, (int32_t*)at, (int32_t*)at, nullptr) != cudaSuccess)
                _Exit(3);
        });
    for (auto& t : all) t.join();
    return 0;
}
