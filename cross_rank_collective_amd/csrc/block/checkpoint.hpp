// checkpoint.hpp -- activations to 8 bits and back.
//
// Bound by memory: 2 or 4 bytes an element on one side, 33/32 on the other.
// Slots are numbered straight through the rows, one per lane, so that a block
// of 32 elements lies in 4 (or 8) neighbouring lanes: a row takes a whole
// number of those.
#pragma once

#include "block_device.hpp"

namespace ptored {
namespace block {

constexpr int kPackThreads = 256;

template <int DT, bool TAIL>
__global__ __launch_bounds__(kPackThreads) void pack_kernel(const PackArgs a, uint32_t row_slots,
                                                            int64_t slots) {
    constexpr int V = Elem<DT>::V;
    // whole waves walk together: pack_slot needs every lane
    const int64_t end = (slots + 63) / 64 * 64;
    for (int64_t n = (int64_t)blockIdx.x * kPackThreads + threadIdx.x; n < end;
         n += (int64_t)gridDim.x * kPackThreads) {
        const int64_t row = n / row_slots;
        const int col = (int)(n - row * row_slots) * V;
        float v[V];
        const bool in = n < slots;
        load_slot<DT, TAIL>(a.x.p + row * a.x.ld, in ? col : a.cols, a.cols, v);
        pack_slot<V, TAIL>(a.k, row, in ? col : a.cols, a.cols, v);
    }
}

template <int DT, bool TAIL>
__global__ __launch_bounds__(kPackThreads) void unpack_kernel(const PackArgs a,
                                                              uint32_t row_slots, int64_t slots) {
    constexpr int V = Elem<DT>::V;
    for (int64_t n = (int64_t)blockIdx.x * kPackThreads + threadIdx.x; n < slots;
         n += (int64_t)gridDim.x * kPackThreads) {
        const int64_t row = n / row_slots;
        const int col = (int)(n - row * row_slots) * V;
        float v[V];
        unpack_slot<V, TAIL>(a.k, row, col, a.cols, v);
        store_slot<DT, TAIL>(a.x.p + row * a.x.ld, col, a.cols, v);
    }
}

template <int DT, bool PACK>
int pack_launch(const PackArgs& a, hipStream_t stream) {
    constexpr int V = Elem<DT>::V;
    const bool tail = a.cols % V != 0;
    uint32_t row_slots = (uint32_t)((a.cols + 31) / 32 * 32 / V);
    int64_t slots = a.rows * (int64_t)row_slots;
    const void* k =
        PACK ? (tail ? reinterpret_cast<const void*>(pack_kernel<DT, true>)
                     : reinterpret_cast<const void*>(pack_kernel<DT, false>))
             : (tail ? reinterpret_cast<const void*>(unpack_kernel<DT, true>)
                     : reinterpret_cast<const void*>(unpack_kernel<DT, false>));
    int64_t grid = (slots + kPackThreads - 1) / kPackThreads;
    if (grid > (1 << 20)) grid = 1 << 20;
    void* args[] = {const_cast<PackArgs*>(&a), &row_slots, &slots};
    return hipLaunchKernel(k, dim3((uint32_t)grid), dim3(kPackThreads), args, 0, stream) ==
                   hipSuccess
               ? kOk
               : kFailed;
}

}  // namespace block
}  // namespace ptored
