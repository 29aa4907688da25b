// clip.hip -- the norm that all gradients have together, and their scaling to a
// largest norm.
//
//   norm = (sum over tensors and their values of x^2)^(1/2)
//   factor = max_norm / norm where norm is finite and above max_norm, else 1
//   out = factor x
//
// A tensor is groups of rows; of a group's rows the first take part, as many as
// its count in device memory says (a table's row gradients), or all of them.
// Squares are summed in 64 bits: fp32 would lose 1e-20 and overflow at 1e20,
// and the adds are far below the rate of memory.  One launch sums (a
// partial sum a workgroup, joined in a fixed order: no atomics), a second joins
// the partial sums in each of its workgroups and scales.  Up to kEntries
// tensors go in a launch's arguments; more take more launches.
//
// Bound by memory: the values are read twice and written once, and the norm has
// to be whole before the first is scaled.  The second launch takes the chunks
// from the last to the first, so that what the last-level cache (256 MB) still
// holds is not read from memory again.  480 million fp32 values in 25 tensors: 345 us for the
// norm (5.6 TB/s) and 738 us for the scaling (5.2 TB/s).  A small layer's seven
// tensors (0.7 million values) take 9 us, two launches.
#include <algorithm>

#include "engram_internal.h"
#include "vec8.h"

namespace engram {
namespace {

constexpr int kEntries = 48;           // tensors of a launch (2.7 KB of arguments)
constexpr int kThreads = 256;
constexpr int kUnits = 4;              // 8-value units of a thread and chunk
constexpr int kChunk = kThreads * kUnits * 8;
constexpr int kMostBlocks = 1024;      // four a CU: 128 KB of loads in flight

struct ClipEntry {
    const void *x;
    void *out;                         // null: only the norm is wanted
    const int32_t *counts;             // rows of each group that take part, or null
    int64_t group;                     // values of a group
    int64_t rows, row_len;             // group = rows * row_len
    int32_t group_chunks;              // chunks of a group
    int32_t bf16;
};
struct ClipList {
    ClipEntry e[kEntries];
    int32_t first[kEntries + 1];       // first chunk of each tensor; first[n]: how many
    int32_t n;
};

// Where a chunk lies: its values [at, at + n) of tensor e.
struct ClipPlace {
    int e;
    int64_t at;
    int32_t n;
};
__device__ __forceinline__ ClipPlace place_of(const ClipList &l, int32_t chunk) {
    int lo = 0, hi = l.n - 1;  // the last tensor whose first chunk is not above (empty ones hold none)
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (l.first[mid] <= chunk)
            lo = mid;
        else
            hi = mid - 1;
    }
    const ClipEntry &e = l.e[lo];
    const uint32_t in = (uint32_t)(chunk - l.first[lo]), g = in / (uint32_t)e.group_chunks;
    const int64_t o = (int64_t)(in - g * (uint32_t)e.group_chunks) * kChunk;
    int64_t len = e.group;
    if (e.counts) len = min(max((int64_t)e.counts[g], (int64_t)0), e.rows) * e.row_len;
    return ClipPlace{lo, g * e.group + o, (int32_t)min(max(len - o, (int64_t)0), (int64_t)kChunk)};
}

template <typename T>
__device__ __forceinline__ F8 load_upto8(const T *p, int32_t left) {
    F8 v = {};
    if (left >= 8) return load_any8(p).get();
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < left) {
            if constexpr (sizeof(T) == 2)
                v.v[i] = bf16_to_f32(p[i]);
            else
                v.v[i] = p[i];
        }
    return v;
}

template <typename T>
__device__ __forceinline__ void store_upto8(T *p, int32_t left, const F8 &v) {
    if (left >= 8) {
        store_any8(p, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < left) {
            if constexpr (sizeof(T) == 2)
                p[i] = (uint16_t)pack_bf16x2(v.v[i], 0.f);
            else
                p[i] = v.v[i];
        }
}

template <typename T>
__device__ __forceinline__ double squares(const T *x, int32_t n, double sum) {
    F8 v[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const int32_t i = (u * kThreads + (int)threadIdx.x) * 8;
        v[u] = load_upto8(x + i, n - i);
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += (double)v[u].v[i] * (double)v[u].v[i];
    return sum;
}

// Sum over a workgroup, in a fixed order.
__device__ __forceinline__ double block_sum(double x, double (&red)[kThreads / 64]) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
    __syncthreads();
    double t = red[0];
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w) t += red[w];
    return t;
}

__global__ __launch_bounds__(kThreads) void clip_norm_kernel(ClipList l, double *part) {
    __shared__ double red[kThreads / 64];
    double sum = 0.;
    for (int32_t c = blockIdx.x; c < l.first[l.n]; c += gridDim.x) {
        const ClipPlace p = place_of(l, c);
        if (p.n == 0) continue;
        if (l.e[p.e].bf16)
            sum = squares(static_cast<const uint16_t *>(l.e[p.e].x) + p.at, p.n, sum);
        else
            sum = squares(static_cast<const float *>(l.e[p.e].x) + p.at, p.n, sum);
    }
    sum = block_sum(sum, red);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

template <typename T>
__device__ __forceinline__ void scale_chunk(const T *x, T *out, int32_t n, float factor) {
    F8 v[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const int32_t i = (u * kThreads + (int)threadIdx.x) * 8;
        v[u] = load_upto8(x + i, n - i);
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const int32_t i = (u * kThreads + (int)threadIdx.x) * 8;
#pragma unroll
        for (int k = 0; k < 8; ++k) v[u].v[k] *= factor;
        store_upto8(out + i, n - i, v[u]);
    }
}

__global__ __launch_bounds__(kThreads) void clip_scale_kernel(ClipList l, const double *part, int32_t parts,
                                                              float max_norm, float *norm, bool first) {
    __shared__ double red[kThreads / 64];
    double sum = 0.;
    for (int32_t i = threadIdx.x; i < parts; i += kThreads) sum += part[i];
    const double total = sqrt(block_sum(sum, red));
    float factor = 1.f;
    if (total > (double)max_norm && total < (double)INFINITY) factor = (float)((double)max_norm / total);
    if (first && blockIdx.x == 0 && threadIdx.x == 0) {
        norm[0] = (float)total;
        norm[1] = factor;
    }
    for (int32_t c = l.first[l.n] - 1 - (int32_t)blockIdx.x; c >= 0; c -= gridDim.x) {
        const ClipPlace p = place_of(l, c);
        const ClipEntry &e = l.e[p.e];
        if (p.n == 0 || !e.out || (e.out == e.x && factor == 1.f)) continue;
        if (e.bf16)
            scale_chunk(static_cast<const uint16_t *>(e.x) + p.at, static_cast<uint16_t *>(e.out) + p.at, p.n, factor);
        else
            scale_chunk(static_cast<const float *>(e.x) + p.at, static_cast<float *>(e.out) + p.at, p.n, factor);
    }
}

int64_t group_chunks(const engram_grad &g) { return (g.rows * g.row_len + kChunk - 1) / kChunk; }

}  // namespace

int64_t clip_chunks(const engram_grad &g) { return g.n_groups * group_chunks(g); }

size_t clip_workspace(int64_t n_grads) { return (size_t)((n_grads + kEntries - 1) / kEntries) * kMostBlocks * sizeof(double); }

void launch_clip(const engram_grad *grads, int32_t n_grads, float max_norm, float *norm, double *part, hipStream_t s) {
    auto list_of = [&](int32_t from, ClipList &l) {
        l.n = std::min(kEntries, n_grads - from);
        l.first[0] = 0;
        for (int32_t i = 0; i < l.n; ++i) {
            const engram_grad &g = grads[from + i];
            const bool some = g.n_groups * g.rows * g.row_len > 0;
            l.e[i] = ClipEntry{g.data, g.out, g.row_counts, g.rows * g.row_len, g.rows, g.row_len,
                               some ? (int32_t)group_chunks(g) : 1, g.dtype == ENGRAM_BF16};
            l.first[i + 1] = l.first[i] + (some ? (int32_t)clip_chunks(g) : 0);
        }
    };
    ClipList l;
    int32_t parts = 0;
    for (int32_t from = 0; from < n_grads; from += kEntries) {
        list_of(from, l);
        const int32_t blocks = std::min(kMostBlocks, std::max(1, l.first[l.n]));
        launch_kernel(clip_norm_kernel, dim3((unsigned)blocks), dim3(kThreads), s, l, part + parts);
        parts += blocks;
    }
    for (int32_t from = 0; from < n_grads; from += kEntries) {
        list_of(from, l);
        bool any = false;
        for (int32_t i = 0; i < l.n; ++i) any |= l.e[i].out != nullptr;
        if (!any && from > 0) continue;
        const int32_t blocks = any ? std::min(2 * kMostBlocks, std::max(1, l.first[l.n])) : 1;
        if (!any) l.n = 0, l.first[0] = 0;
        launch_kernel(clip_scale_kernel, dim3((unsigned)blocks), dim3(kThreads), s, l, part, parts, max_norm, norm,
                      from == 0);
    }
}

}  // namespace engram
