// rope3d_paged.h -- host helpers of the operators around a paged cache
// (rope3d_axes.cu, rope3d_paged.cu, rope3d_paged_tc.cu, rope3d_pages.cu): the
// memory that strided views cover, whether two of them can meet, device checks
// and launches.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <utility>

#include "../../include/rope3d.h"

namespace rope3d_paged {

// A strided view of `elem` bytes an element: up to three strided dimensions
// over rows of `row` contiguous elements.
struct View {
    const void *p;
    int64_t row;
    int64_t count[3], stride[3];
    int elem;
};

inline View view(const void *p, int elem, int64_t row, int64_t n0, int64_t s0, int64_t n1 = 1, int64_t s1 = 0,
                 int64_t n2 = 1, int64_t s2 = 0) {
    return View{p, row, {n0, n1, n2}, {s0, s1, s2}, elem};
}

// Elements from the first to behind the last one.
inline int64_t extent(const View &v) {
    int64_t e = v.row;
    for (int i = 0; i < 3; ++i) e += (v.count[i] - 1) * v.stride[i];
    return e;
}

// Strides that a written view may have: sorted by size, each steps over all that
// lies below it, so that no element is written twice.
inline bool rows_apart(const View &v) {
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int a, int b) { return v.stride[a] < v.stride[b]; });
    int64_t below = v.row;
    for (int i : order) {
        if (v.count[i] <= 1) continue;
        if (v.stride[i] < below) return false;
        below += (v.count[i] - 1) * v.stride[i];
    }
    return true;
}

// Whether a (written) and b can share memory. Address ranges that do not meet
// cannot; nor can views of one buffer that repeat at a common stride with
// their rows beside one another there (the thirds of a projection, the K and V
// halves of a cache's pages).
inline bool may_meet(const View &a, const View &b) {
    if (!a.p || !b.p) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    if (x >= y + uint64_t(extent(b)) * b.elem || y >= x + uint64_t(extent(a)) * a.elem) return false;
    if (a.elem != b.elem || (y - x) % uintptr_t(a.elem) != 0) return true;
    const int64_t d = (int64_t(y) - int64_t(x)) / a.elem;
    for (int i = 0; i < 3; ++i) {
        const int64_t s = a.stride[i];
        if (s <= 0) continue;
        bool fits = true;
        int64_t below[2];
        for (int v = 0; v < 2; ++v) {   // every larger stride a multiple of s; what is smaller, below it
            const View &w = v ? b : a;
            below[v] = w.row;
            for (int j = 0; j < 3; ++j) {
                if (w.count[j] <= 1) continue;
                if (w.stride[j] < s) below[v] += (w.count[j] - 1) * w.stride[j];
                else fits = fits && w.stride[j] % s == 0;
            }
        }
        if (!fits) continue;
        const int64_t r = ((d % s) + s) % s;
        if (r >= below[0] && r + below[1] <= s) return false;
    }
    return true;
}

inline bool same_view(const View &a, const View &b) {
    if (a.p != b.p) return false;
    for (int i = 0; i < 3; ++i)
        if (a.count[i] > 1 && a.stride[i] != b.stride[i]) return false;
    return true;
}

inline bool aligned(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % uintptr_t(bytes) == 0; }

// Rows that can be read and written as 16-byte vectors.
inline bool vectors(const View &v) {
    if (!v.p) return true;
    if (!aligned(v.p, 16) || v.row * v.elem % 16 != 0) return false;
    for (int i = 0; i < 3; ++i)
        if (v.count[i] > 1 && v.stride[i] * v.elem % 16 != 0) return false;
    return true;
}

constexpr int64_t kMaxStride = int64_t(1) << 40;

inline bool bad_strides(const View &v) {
    for (int i = 0; i < 3; ++i)
        if (v.stride[i] < 0 || v.stride[i] > kMaxStride) return true;
    return false;
}

inline int on_current_device(const void *const *p, int n) {
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) {
        cudaGetLastError();
        return ROPE3D_ERR_CUDA;
    }
    for (int i = 0; i < n; ++i) {
        if (!p[i]) continue;
        cudaPointerAttributes attr{};
        if (cudaPointerGetAttributes(&attr, p[i]) != cudaSuccess) {
            cudaGetLastError();
            return ROPE3D_ERR_DEVICE;
        }
        if (attr.type != cudaMemoryTypeManaged && (attr.type != cudaMemoryTypeDevice || attr.device != device))
            return ROPE3D_ERR_DEVICE;
    }
    return ROPE3D_OK;
}

// The SMs of the current device (asked once a device); 0 on an error.
inline int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return 0;
    }
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        known[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

// A launch whose blocks may become resident while the stream's previous kernel
// ends (each waits for it before it touches memory).
template <typename... P, typename... A>
int launch(void (*fn)(P...), dim3 grid, int block, size_t smem, cudaStream_t st, A &&...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(block));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, fn, std::forward<A>(args)...) != cudaSuccess) {
        cudaGetLastError();
        return ROPE3D_ERR_CUDA;
    }
    return ROPE3D_OK;
}

constexpr int64_t kMaxTokens = int64_t(1) << 28, kMaxSeqs = int64_t(1) << 20, kMaxHeads = int64_t(1) << 12;
constexpr int64_t kMaxPlaces = int64_t(1) << 30;   // tokens that one row of a page table can name

// The description of a batch that the cache's operators share.
inline int check_batch(const rope3d_paged_batch &b, int64_t tokens) {
    if (!b.page_table || !b.seq_lens) return ROPE3D_ERR_NULL;
    if (b.seqs <= 0 || b.seqs > kMaxSeqs || b.table_width <= 0 || b.table_stride < b.table_width ||
        b.table_stride > kMaxStride || b.pages <= 0 || b.pages > 0x7fffffff || b.page_size <= 0 ||
        b.page_size > kMaxPlaces || b.table_width > kMaxPlaces / b.page_size)
        return ROPE3D_ERR_SHAPE;
    if (!b.q_starts && tokens % b.seqs != 0) return ROPE3D_ERR_SHAPE;
    if (!aligned(b.page_table, 4) || !aligned(b.seq_lens, 4) || !aligned(b.q_starts, 4)) return ROPE3D_ERR_ALIGN;
    return ROPE3D_OK;
}

// The batch as the kernels have it.
struct Batch {
    const int *table, *lens, *starts;
    int64_t table_stride;
    int seqs, width, pages, page_size, tokens;
};

inline Batch device_batch(const rope3d_paged_batch &b, int64_t tokens) {
    return Batch{b.page_table, b.seq_lens, b.q_starts, b.table_stride, int(b.seqs), int(b.table_width), int(b.pages),
                 int(b.page_size), int(tokens)};
}

#ifdef __CUDACC__
// The new tokens [lo, hi) of sequence s, and its length with them; whatever the
// arrays hold, they stay within the call's tokens and the table's row.
__host__ __device__ __forceinline__ void sequence(const Batch &b, int s, int &lo, int &hi, int &len) {
    if (b.starts) {
        lo = min(max(b.starts[s], 0), b.tokens);
        hi = min(max(b.starts[s + 1], lo), b.tokens);
    } else {
        const int n = b.tokens / b.seqs;
        lo = s * n;
        hi = lo + n;
    }
    len = min(max(b.lens[s], 0), b.width * b.page_size);
}
#endif

}  // namespace rope3d_paged
