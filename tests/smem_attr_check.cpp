// The table of shared memory limits against a stand-in of the CUDA runtime: how
// often the attribute call is made.  Prints the counts, one a line.
#include <cstdint>
#include <cstdio>

#include "hs_smem_attr.h"

static int calls = 0, device = 0, limit[200][2] = {};
extern "C" cudaError_t cudaGetDevice(int* d) { return *d = device, cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void* fn, cudaFuncAttribute, int bytes) {
    ++calls;
    limit[(uintptr_t)fn][device] = bytes;
    return cudaSuccess;
}

static const void* kernel(int i) { return (const void*)(uintptr_t)i; }

int main() {
    auto count = [&](auto&& f) { return calls = 0, f(), printf("%d\n", calls), 0; };
    // one kernel at 100 growing sizes, each twice: each size once
    count([] { for (int b = 1; b <= 200; ++b) hs_host::set_smem_attr(kernel(1), 50000 + b / 2 * 16); });
    // 40 others, three times: once each, the first kernel's sizes have left them room
    count([] { for (int r = 0; r < 3; ++r) for (int k = 2; k < 42; ++k) hs_host::set_smem_attr(kernel(k), 60000); });
    // smaller sizes: none, and the limit stays
    count([] { for (int b = 0; b < 50; ++b) hs_host::set_smem_attr(kernel(1), 50000 + b); });
    printf("%d\n", limit[1][0]);
    // another device has limits of its own
    device = 1;
    count([] { for (int r = 0; r < 3; ++r) hs_host::set_smem_attr(kernel(1), 50000); });
    // more kernels than the table holds: still set, on every call
    device = 0;
    count([] { for (int r = 0; r < 2; ++r) for (int k = 50; k < 150; ++k) hs_host::set_smem_attr(kernel(k), 70000); });
    printf("%d\n", limit[149][0]);
}
