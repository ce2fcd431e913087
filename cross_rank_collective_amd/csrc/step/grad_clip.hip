// grad_clip.hip -- the norm over many gradients, and their scaling.
//
//     n = sqrt(sum g^2),   out = g c,   c = min(1, max / n)
//
// Bound by memory: one pass that reads, one that reads and writes.  The table
// of gradients travels in the kernels' arguments (4 KB hold kGradEntries), so
// that a call allocates and copies nothing and can be captured; more gradients
// take more launches.  A workgroup takes one chunk of one gradient.  Squares
// are exact in binary64 and summed there: no sum of 32-bit gradients passes
// its range or drops below it, and it costs two instructions an element, which
// memory hides.  Partial sums are added in a fixed order.
#include <hip/hip_runtime.h>

#include "block/block_device.hpp"
#include "step_plan.h"

namespace ptored {
namespace step {

using namespace block;

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // slots of a thread in flight

// This workgroup's entry and chunk in it.  Entries' first workgroups ascend.
struct Place {
    int entry, chunk;
};
__device__ __forceinline__ Place find(const GradList& a) {
    const int id = (int)blockIdx.x, lane = (int)threadIdx.x & 63;
    int found = 0;
#pragma unroll
    for (int at = 0; at < kGradEntries; at += 64) {
        const int i = at + lane;
        const bool starts = i < a.count && a.e[i < kGradEntries ? i : 0].first <= id;
        found += __builtin_popcountll(__ballot(starts));
    }
    const int entry = __builtin_amdgcn_readfirstlane(found - 1);
    return {entry, id - a.e[entry].first};
}

// Calls f(data, out, elements) for the chunk's runs of consecutive elements.
template <typename F>
__device__ __forceinline__ void walk(const GradList& a, const GradEntry& e, int chunk, int es, int oes,
                                     F f) {
    if (e.chunks > 0) {
        const int64_t row = e.chunks == 1 ? chunk : chunk / e.chunks;
        const int64_t at = (chunk - row * e.chunks) * a.chunk;
        const int64_t n = e.cols - at < a.chunk ? e.cols - at : a.chunk;
        f(e.data + (row * e.ld + at) * es, e.out + (row * e.out_ld + at) * oes, (int)n);
        return;
    }
    const int group = (int)(a.chunk / e.cols);
    const int64_t first = (int64_t)chunk * group;
    const int rows = (int)(e.rows - first < group ? e.rows - first : group);
    for (int r = 0; r < rows; ++r)
        f(e.data + (first + r) * e.ld * es, e.out + (first + r) * e.out_ld * oes, (int)e.cols);
}

template <int DT>
__device__ __forceinline__ void add_squares(const char* p, int n, double* sum) {
    using E = Elem<DT>;
    constexpr int V = E::V;
    auto slot = [&](u32x4 w, double& to) {
        float v[V];
        E::widen(w, v);
#pragma unroll
        for (int i = 0; i < V; ++i) to = __builtin_fma((double)v[i], (double)v[i], to);
    };
    const int slots = n / V;
    int s = (int)threadIdx.x;
    for (; s + (kAhead - 1) * kThreads < slots; s += kAhead * kThreads) {
        u32x4 w[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            w[k] = *reinterpret_cast<const u32x4_any*>(p + (int64_t)(s + k * kThreads) * 16);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) slot(w[k], sum[k]);
    }
    for (; s < slots; s += kThreads)
        slot(*reinterpret_cast<const u32x4_any*>(p + (int64_t)s * 16), sum[0]);
    const int i = slots * V + (int)threadIdx.x;
    if (i < n) {
        const double v = E::load1(p + (int64_t)i * E::kBytes);
        sum[0] = __builtin_fma(v, v, sum[0]);
    }
}

// The workgroup's sum, in thread 0.
__device__ __forceinline__ double block_total(double v) {
    __shared__ double part[kThreads / 64];
#pragma unroll
    for (int by = 32; by >= 1; by /= 2) v += __shfl_xor(v, by);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    return (part[0] + part[1]) + (part[2] + part[3]);
}

__global__ __launch_bounds__(kThreads) void sums_kernel(const GradList a) {
    const Place at = find(a);
    const GradEntry& e = a.e[at.entry];
    double sum[kAhead] = {};
    switch (e.type & 0xFF) {
        case PTORED_F32:
            walk(a, e, at.chunk, 4, 0, [&](const char* p, char*, int n) { add_squares<PTORED_F32>(p, n, sum); });
            break;
        case PTORED_BF16:
            walk(a, e, at.chunk, 2, 0, [&](const char* p, char*, int n) { add_squares<PTORED_BF16>(p, n, sum); });
            break;
        default:
            walk(a, e, at.chunk, 2, 0, [&](const char* p, char*, int n) { add_squares<PTORED_F16>(p, n, sum); });
    }
    const double total = block_total((sum[0] + sum[1]) + (sum[2] + sum[3]));
    if (threadIdx.x == 0) a.sums[blockIdx.x] = total;
}

// The norm from every partial sum, the same in all threads of every workgroup.
__device__ __forceinline__ double joined(const GradList& a) {
    double sum = 0.0;
#pragma unroll 4
    for (int i = (int)threadIdx.x; i < a.all_count; i += kThreads) sum += a.all[i];
    return sqrt(block_total(sum));
}

__global__ __launch_bounds__(kThreads) void join_kernel(const GradList a) {
    const double n = joined(a);
    if (threadIdx.x == 0) a.norm[0] = (float)n;
}

template <int DT, int OT>
__device__ __forceinline__ void scale_run(const char* p, char* q, int n, float by) {
    using E = Elem<DT>;
    using O = Elem<OT>;
    constexpr int V = E::V;
    auto slot = [&](u32x4 w, int s) {
        float v[V];
        E::widen(w, v);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= by;
        char* to = q + (int64_t)s * (V * O::kBytes);
        *reinterpret_cast<u32x4_any*>(to) = O::narrow(v);
        if constexpr (O::V < V) *reinterpret_cast<u32x4_any*>(to + 16) = O::narrow(v + 4);
    };
    const int slots = n / V;
    int s = (int)threadIdx.x;
    for (; s + (kAhead - 1) * kThreads < slots; s += kAhead * kThreads) {
        u32x4 w[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            w[k] = *reinterpret_cast<const u32x4_any*>(p + (int64_t)(s + k * kThreads) * 16);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) slot(w[k], s + k * kThreads);
    }
    for (; s < slots; s += kThreads) slot(*reinterpret_cast<const u32x4_any*>(p + (int64_t)s * 16), s);
    const int i = slots * V + (int)threadIdx.x;
    if (i < n) O::store1(q + (int64_t)i * O::kBytes, E::load1(p + (int64_t)i * E::kBytes) * by);
}

__global__ __launch_bounds__(kThreads) void scale_kernel(const GradList a) {
    const Place at = find(a);
    const GradEntry& e = a.e[at.entry];
    double n;
    if (a.all != nullptr) {
        n = joined(a);
        if (a.norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) a.norm[0] = (float)n;
        // as a norm that was handed over: the same factor either way
        n = (double)(float)n;
    } else {
        n = (double)a.norm[0];
    }
    const float by = n > (double)a.max_norm ? (float)((double)a.max_norm / n) : n == n ? 1.0f : (float)n;
    if (by == 1.0f && e.data == e.out) return;  // in place, nothing changes
#define PTORED_SCALE(DT, OT)                                                          \
    walk(a, e, at.chunk, Elem<DT>::kBytes, Elem<OT>::kBytes,                          \
         [&](const char* p, char* q, int m) { scale_run<DT, OT>(p, q, m, by); })
    switch (e.type) {
        case PTORED_F32: PTORED_SCALE(PTORED_F32, PTORED_F32); break;
        case PTORED_BF16 | PTORED_BF16 << 8: PTORED_SCALE(PTORED_BF16, PTORED_BF16); break;
        case PTORED_F16 | PTORED_F16 << 8: PTORED_SCALE(PTORED_F16, PTORED_F16); break;
        case PTORED_BF16: PTORED_SCALE(PTORED_BF16, PTORED_F32); break;
        default: PTORED_SCALE(PTORED_F16, PTORED_F32);
    }
#undef PTORED_SCALE
}

int launch(const void* k, const GradList& a, int groups, hipStream_t stream) {
    void* args[] = {const_cast<GradList*>(&a)};
    return hipLaunchKernel(k, dim3((uint32_t)groups), dim3(kThreads), args, 0, stream) == hipSuccess
               ? kOk
               : kFailed;
}

}  // namespace

int grad_sums(const GradList& a, hipStream_t stream) {
    return launch(reinterpret_cast<const void*>(sums_kernel), a, a.groups, stream);
}
int grad_join(const GradList& a, hipStream_t stream) {
    return launch(reinterpret_cast<const void*>(join_kernel), a, 1, stream);
}
int grad_scale(const GradList& a, hipStream_t stream) {
    return launch(reinterpret_cast<const void*>(scale_kernel), a, a.groups, stream);
}

}  // namespace step
}  // namespace ptored
