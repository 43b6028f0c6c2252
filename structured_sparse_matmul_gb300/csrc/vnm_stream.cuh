// Loads of the kernels that stream a weight matrix from global memory into registers.
#pragma once

#include <stdint.h>

namespace vnm {

// 16 bytes of W: read once, not kept in L1.
__device__ __forceinline__ uint4 load_once(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// The same of memory that the grid before, beside which this one was started, may have written.
__device__ __forceinline__ uint4 load_once_coherent(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// 16 bytes of a row from column k on, 0 from column K on (the last, shorter block).
// Rows are 16-byte aligned, so the 16 bytes lie within the row's pitch; the last
// row's pitch may not be all there, and its last bytes are read one by one.
static __device__ __noinline__ uint4 load_edge(const uint8_t* row, int64_t k, int64_t K, bool last_row) {
    const int n = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(16), K - k)));  // bytes that exist
    uint32_t u[4] = {0u, 0u, 0u, 0u};
    if (n == 16 || (n > 0 && !last_row)) {
        const uint4 v = load_once(row + k);
        u[0] = v.x;
        u[1] = v.y;
        u[2] = v.z;
        u[3] = v.w;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int left = n - 4 * j;
            u[j] = left >= 4 ? u[j] : left <= 0 ? 0u : u[j] & (0xFFFFFFFFu >> (8 * (4 - left)));
        }
    } else {
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            const uint32_t byte = row[k + i];
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] |= j == i / 4 ? byte << (8 * (i & 3)) : 0u;
        }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

}  // namespace vnm
