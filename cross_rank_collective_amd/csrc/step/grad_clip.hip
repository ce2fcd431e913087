// grad_clip.hip -- the norm over many gradients, and their scaling.
//
//     n = sqrt(sum g^2),   out = g c,   c = min(1, max / n)
//
// Bound by memory: one pass that reads, one that reads and writes.  The table
// of gradients travels in the kernels' arguments (4 KB hold kGradEntries), so
// that a call allocates nothing, copies nothing from the host and can be
// captured.  Of more gradients the table is first put together in the
// workspace, and both passes stay one launch each: in launches of their own,
// each waits for the last one's slowest workgroup.  Its launches (two for 300
// tensors) take 4.7 us each, most of it the way of the arguments from host memory,
// so that the table is packed on that way (unpacked 8).
//
// All gradients are cut into chunks of kGradChunk elements, and each workgroup
// takes an equal run of consecutive chunks, over the ends of gradients: as many
// workgroups as the chip holds at once, all with the same work.  A slot's
// squares are added in binary32 and the slots' sums in binary64; a slot whose
// sum leaves binary32's safe range is taken again in binary64, so that no norm
// passes the range on the way or drops below it.  Partial sums are added in a
// fixed order, by every workgroup of the scaling itself.
//
// Measured: 85 M elements in 300 tensors, 174 MB of bf16 and some F32, 96% of them
// into outputs that do not begin at multiples of 16 bytes, 44% in rows with gaps: 130
// us; as profiled, sums 36 (4.8 TB/s), scaling 89 (3.9 TB/s, a read and a write where a
// copy reaches 6.2), tables 4.8 each.  101 M bf16 elements in few matrices without
// gaps: sums 37, scaling 79 (5.1 TB/s).  8 tensors of 100000 elements in all 9.2 us,
// two launches.
#include <hip/hip_runtime.h>

#include "block/block_device.hpp"
#include "step_plan.h"

namespace ptored {
namespace step {

using namespace block;

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // slots of a thread in flight

template <bool TABLE>
__device__ __forceinline__ const GradEntry& entry_of(const GradList& a, int i) {
    if constexpr (TABLE)
        return a.table[i];
    else
        return a.e[i];
}

// The entry that chunk `id` lies in.  Entries' first chunks ascend.
template <bool TABLE>
__device__ __forceinline__ int find(const GradList& a, int id) {
    const int lane = (int)threadIdx.x & 63;
    int found = 0;
    for (int at = 0; at < a.count; at += 64) {
        const int i = at + lane;
        const bool starts = i < a.count && entry_of<TABLE>(a, i < a.count ? i : 0).first <= id;
        found += __builtin_popcountll(__ballot(starts));
    }
    return __builtin_amdgcn_readfirstlane(found - 1);
}

// Calls f(entry, its chunk, how many chunks) over this workgroup's run.
template <bool TABLE, typename F>
__device__ __forceinline__ void each_run(const GradList& a, F f) {
    int id = (int)((int64_t)a.chunks * blockIdx.x / a.groups);
    const int end = (int)((int64_t)a.chunks * (blockIdx.x + 1) / a.groups);
    for (int i = find<TABLE>(a, id); id < end; ++i) {
        const int next = i + 1 < a.count ? entry_of<TABLE>(a, i + 1).first : a.chunks;
        const GradEntry e = entry_of<TABLE>(a, i);
        const int stop = min(next, end);
        f(e, id - e.first, stop - id);
        id = stop;
    }
}

// A launch's entries to their place in the workspace's table.
__global__ __launch_bounds__(kThreads) void table_kernel(const GradPack a) {
    static_assert(kGradSlots <= kThreads, "a thread for each slot");
    __shared__ int sums[2][kThreads];
    const int i = (int)threadIdx.x;
    int rank = 0;  // heads before this slot
#pragma unroll
    for (int w = 0; w < kGradSlots / 32; ++w) {
        const int below = min(max(i - 32 * w, 0), 32);
        rank += __builtin_popcount(below == 32 ? a.heads[w] : a.heads[w] & ((1u << below) - 1));
    }
    const bool head = i < a.slots && (a.heads[i / 32 % (kGradSlots / 32)] >> (i % 32) & 1);
    GradEntry e{};
    int chunks = 0;
    if (head) {
        const uint64_t d = a.data[i];
        e.data = reinterpret_cast<const char*>(d & 0xFFFFFFFFFFFFull);
        e.out = reinterpret_cast<char*>(a.out[i]);
        e.cols = (int64_t)((d >> 48 & 0xFF) << 32 | a.cols[i]);
        e.rows = 1;
        const int type = (int)(d >> 56 & 7);
        e.type = type > PTORED_F16 ? type - 3 : type | type << 8;
        if (d >> 59 & 1) {
            e.rows = (int32_t)(uint32_t)a.data[i + 1];
            e.ld = (int32_t)(a.data[i + 1] >> 32);
            e.out_ld = (int32_t)a.out[i + 1];
        }
        chunks = (int)grad_chunks(e.rows, e.cols, e.type & 0xFF);
    }
    // the entries' first chunks: sums over the slots before
    int turn = 0;
    sums[0][i] = chunks;
    __syncthreads();
#pragma unroll
    for (int by = 1; by < kThreads; by *= 2) {
        sums[1 - turn][i] = sums[turn][i] + (i >= by ? sums[turn][i - by] : 0);
        turn = 1 - turn;
        __syncthreads();
    }
    e.first = a.first + sums[turn][i] - chunks;
    if (head) a.table[rank] = e;
}

// Elements of `ES` bytes through buffer resources: what lies past the end reads
// as zeros and is not stored, so that loads need no branch.
constexpr int kMostBytes = 1 << 30;  // of a resource
constexpr uint32_t kNowhere = 0x80000000u;
__device__ __forceinline__ u32x4 load_slot(rsrc_t r, uint32_t off) {
    return __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, kPolicyStream);
}
template <int ES>
__device__ __forceinline__ uint32_t load_one(rsrc_t r, uint32_t off) {
    if constexpr (ES == 4)
        return __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0);
    else
        return __builtin_amdgcn_raw_buffer_load_b16(r, (int)off, 0, 0);
}

// The chunks' slots: f(words, elements, out, offset in it, k), kAhead of a thread
// in flight.  A slot of fewer than V elements has zeros behind them.
template <int ES, int OES, typename F>
__device__ __forceinline__ void walk(const GradEntry& e, int chunk, int count, F f) {
    constexpr int V = 16 / ES, kSlots = kGradChunk / V;
    if (e.rows == 1) {
        while (count > 0) {
            const int take = min(count, kMostBytes / (kGradChunk * 4));  // a resource's
            const int64_t at = (int64_t)chunk * kGradChunk;
            const int n = (int)min(e.cols - at, (int64_t)take * kGradChunk);
            const char* p = e.data + at * ES;
            char* q = e.out + at * OES;
            // slots begin where the output is aligned
            const int head = min(n, OES == 0 ? 0 : (int)(-reinterpret_cast<uintptr_t>(q) & 15) / max(OES, 1));
            const int slots = (n - head) / V, behind = head + slots * V;
            const rsrc_t r = row_rsrc(p + head * ES, slots * 16);
            const rsrc_t to = row_rsrc(q + head * OES, slots * V * OES);
            for (int s = (int)threadIdx.x; s < slots; s += kAhead * kThreads) {
                u32x4 w[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) w[k] = load_slot(r, (uint32_t)(s + k * kThreads) * 16);
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    f(w[k], V, to, (uint32_t)(s + k * kThreads) * (V * OES), k);
            }
            const int i = (int)threadIdx.x < head ? (int)threadIdx.x : behind + (int)threadIdx.x - head;
            if (i < n)
                f((u32x4){load_one<ES>(row_rsrc(p, n * ES), (uint32_t)i * ES), 0u, 0u, 0u}, 1,
                  row_rsrc(q, n * OES), (uint32_t)i * OES, 0);
            chunk += take;
            count -= take;
        }
        return;
    }
    // slots numbered through the rows: rows shorter than a workgroup are not
    // waited for one by one, and long ones do not make chunks longer
    const int cols = (int)e.cols;
    const uint32_t per_row = (uint32_t)(cols + V - 1) / V;
    const int64_t pitch = (int64_t)e.ld * ES, out_pitch = (int64_t)e.out_ld * OES;
    int64_t first = (int64_t)chunk * kSlots;
    const int64_t end = min((int64_t)e.rows * per_row, first + (int64_t)count * kSlots);
    // rows of a resource, of which the first may be begun
    const int64_t most = (kMostBytes / max(pitch, out_pitch) - 1) * per_row;
    while (first < end) {
        const int64_t row0 = first / per_row;
        const uint32_t begun = (uint32_t)(first - row0 * per_row);
        const uint32_t slots = (uint32_t)min(end - first, most);
        const uint32_t rows = (begun + slots + per_row - 1) / per_row;
        const rsrc_t r = row_rsrc(e.data + row0 * pitch, (int)((rows - 1) * pitch + cols * ES));
        const rsrc_t to = row_rsrc(e.out + row0 * out_pitch, (int)((rows - 1) * out_pitch + cols * OES));
        for (uint32_t s0 = threadIdx.x; s0 < slots; s0 += kAhead * kThreads) {
            u32x4 w[kAhead];
            uint32_t row[kAhead];
            int col[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const uint32_t s = begun + s0 + k * kThreads;
                row[k] = s / per_row;
                col[k] = s0 + k * kThreads < slots ? (int)(s - row[k] * per_row) * V : cols;
                const uint32_t at = row[k] * (uint32_t)pitch;
                if (cols >= V) {
                    // what is left of a row is loaded so that it ends with it
                    w[k] = load_slot(r, col[k] < cols ? at + min(col[k], cols - V) * ES : kNowhere);
                } else {
                    uint32_t u[4] = {};
#pragma unroll
                    for (int i = 0; i < V - 1; ++i)
                        u[i * ES / 4] |= load_one<ES>(r, col[k] + i < cols ? at + i * ES : kNowhere)
                                         << (i * ES % 4 * 8);
                    w[k] = (u32x4){u[0], u[1], u[2], u[3]};
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int n = min(cols - col[k], V);
                if (cols % V != 0 && cols >= V) w[k] = shift_down(w[k], (n > 0 ? V - n : 0) * ES);
                f(w[k], n, to, n > 0 ? row[k] * (uint32_t)out_pitch + col[k] * OES : kNowhere, k);
            }
        }
        first += slots;
    }
}

__device__ __forceinline__ bool all_zero(u32x4 w) { return (w[0] | w[1] | w[2] | w[3]) == 0; }

template <int DT>
__device__ __forceinline__ void add_squares(const GradEntry& e, int chunk, int count, double* sum) {
    using E = Elem<DT>;
    constexpr int V = E::V;
    walk<E::kBytes, 0>(
        e, chunk, count,
        [&](u32x4 w, int, rsrc_t, uint32_t, int k) {
            float v[V];
            E::widen(w, v);
            float t = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) t = __builtin_fmaf(v[i], v[i], t);
            // squares below 2^-126 may have lost bits, unless they are beside
            // far larger ones; a NaN goes on as it is
            if (__builtin_expect((t >= 0x1p-90f && t < 0x1p127f) || (t == 0.0f && all_zero(w)), 1)) {
                sum[k] += (double)t;
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) sum[k] = __builtin_fma((double)v[i], (double)v[i], sum[k]);
            }
        });
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

template <bool TABLE>
__global__ __launch_bounds__(kThreads, kGradPerUnit) void sums_kernel(const GradList a) {
    double sum[kAhead] = {};
    each_run<TABLE>(a, [&](const GradEntry& e, int chunk, int count) {
        switch (e.type & 0xFF) {
            case PTORED_F32: add_squares<PTORED_F32>(e, chunk, count, sum); break;
            case PTORED_BF16: add_squares<PTORED_BF16>(e, chunk, count, sum); break;
            default: add_squares<PTORED_F16>(e, chunk, count, sum);
        }
    });
    const double total = block_total((sum[0] + sum[1]) + (sum[2] + sum[3]));
    if (threadIdx.x == 0) a.sums[blockIdx.x] = total;
}

// The norm from every partial sum, the same in all threads of every workgroup.
__device__ __forceinline__ double joined(const GradList& a) {
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kGradGroups / kThreads; ++i) {
        const int at = i * kThreads + (int)threadIdx.x;
        sum += at < a.all_count ? a.all[at] : 0.0;
    }
    return sqrt(block_total(sum));
}

__global__ __launch_bounds__(kThreads) void join_kernel(const GradList a) {
    const double n = joined(a);
    if (threadIdx.x == 0) a.norm[0] = (float)n;
}

template <int DT, int OT>
__device__ __forceinline__ void scale_run(const GradEntry& e, int chunk, int count, float by) {
    using E = Elem<DT>;
    using O = Elem<OT>;
    constexpr int V = E::V;
    walk<E::kBytes, O::kBytes>(
        e, chunk, count,
        [&](u32x4 w, int n, rsrc_t to, uint32_t off, int) {
            float v[V];
            E::widen(w, v);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] *= by;
            const u32x4 lo = O::narrow(v), hi = O::V < V ? O::narrow(v + O::V % V) : lo;
            if (__builtin_expect(n >= V, 1)) {
                __builtin_amdgcn_raw_buffer_store_b128(lo, to, (int)off, 0, kPolicyStream);
                if constexpr (O::V < V)
                    __builtin_amdgcn_raw_buffer_store_b128(hi, to, (int)(off + 16), 0, kPolicyStream);
                return;
            }
#pragma unroll
            for (int i = 0; i < V - 1; ++i) {
                const uint32_t at = i < n ? off + i * O::kBytes : kNowhere;
                const uint32_t word = (i / O::V ? hi : lo)[i % O::V * O::kBytes / 4];
                if constexpr (O::kBytes == 4)
                    __builtin_amdgcn_raw_buffer_store_b32(word, to, (int)at, 0, 0);
                else
                    __builtin_amdgcn_raw_buffer_store_b16((unsigned short)(word >> (16 * (i % 2))), to,
                                                          (int)at, 0, 0);
            }
        });
}

template <bool TABLE>
__global__ __launch_bounds__(kThreads, kGradPerUnit) void scale_kernel(const GradList a) {
    double n;
    if (a.all != nullptr) {
        n = joined(a);
        if (blockIdx.x == 0 && threadIdx.x == 0) a.norm[0] = (float)n;
        // as a norm that was handed over: the same factor either way
        n = (double)(float)n;
    } else {
        n = (double)a.norm[0];
    }
    const float by = n > (double)a.max_norm ? (float)((double)a.max_norm / n) : n == n ? 1.0f : (float)n;
    each_run<TABLE>(a, [&](const GradEntry& e, int chunk, int count) {
        if (by == 1.0f && e.data == e.out) return;  // in place, nothing changes
        switch (e.type) {
            case PTORED_F32: scale_run<PTORED_F32, PTORED_F32>(e, chunk, count, by); break;
            case PTORED_BF16 | PTORED_BF16 << 8: scale_run<PTORED_BF16, PTORED_BF16>(e, chunk, count, by); break;
            case PTORED_F16 | PTORED_F16 << 8: scale_run<PTORED_F16, PTORED_F16>(e, chunk, count, by); break;
            case PTORED_BF16: scale_run<PTORED_BF16, PTORED_F32>(e, chunk, count, by); break;
            default: scale_run<PTORED_F16, PTORED_F32>(e, chunk, count, by);
        }
    });
}

template <typename A>
int launch(const void* k, const A& a, int groups, hipStream_t stream) {
    void* args[] = {const_cast<A*>(&a)};
    return hipLaunchKernel(k, dim3((uint32_t)groups), dim3(kThreads), args, 0, stream) == hipSuccess
               ? kOk
               : kFailed;
}

}  // namespace

#define PTORED_PICK(kernel, a)                                             \
    ((a).table != nullptr ? reinterpret_cast<const void*>(kernel<true>)    \
                          : reinterpret_cast<const void*>(kernel<false>))
int grad_table(const GradPack& a, hipStream_t stream) {
    return launch(reinterpret_cast<const void*>(table_kernel), a, 1, stream);
}
int grad_sums(const GradList& a, hipStream_t stream) {
    return launch(PTORED_PICK(sums_kernel, a), a, a.groups, stream);
}
int grad_join(const GradList& a, hipStream_t stream) {
    return launch(reinterpret_cast<const void*>(join_kernel), a, 1, stream);
}
int grad_scale(const GradList& a, hipStream_t stream) {
    return launch(PTORED_PICK(scale_kernel, a), a, a.groups, stream);
}
#undef PTORED_PICK

}  // namespace step
}  // namespace ptored
