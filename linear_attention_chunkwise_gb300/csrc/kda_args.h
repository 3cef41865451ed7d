// kda_args.h -- argument checks shared by the C-ABI front ends, and what kda_api.cu does for the others.
#pragma once

#include <cstddef>
#include <cstdint>

#include "kda_internal.h"

namespace kda {

// SMs of the current device (0 when the runtime cannot say).
int device_sm_count();

// Tensor map over a bf16 [T][H][128] tensor with boxes of box_rows tokens of one head and box_inner
// channels; false when the driver refuses it.
bool make_tensor_map(CUtensorMap* m, const void* base, uint64_t H, uint64_t T, uint32_t box_inner, uint32_t box_rows,
                     CUtensorMapSwizzle sw);

constexpr size_t kAlign = 256;  // workspaces and the regions inside them

inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};
inline Range range_of(const void* p, size_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Range{a, a + bytes};
}
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo; }

// Whether the product fits comfortably in int64.
inline bool sizes_ok(int64_t a, int64_t b, int64_t c, int64_t d) {
    const double prod = static_cast<double>(a) * static_cast<double>(b) * static_cast<double>(c) *
                        static_cast<double>(d);
    return prod < 4.0e18;
}

inline size_t esize_of(kda_dtype t) { return t == KDA_DTYPE_F32 ? 4 : 2; }

// Lets a kernel have `bytes` of dynamic shared memory (48 KB need no leave), on first use per device.
template <typename K>
inline cudaError_t set_smem(K kernel, uint32_t bytes, int* configured) {
    if (bytes <= 48 * 1024) return cudaSuccess;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess || (dev >= 0 && dev < 64 && configured[dev])) return err;
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (err == cudaSuccess && dev >= 0 && dev < 64) configured[dev] = 1;
    return err;
}

}  // namespace kda
