// rope3d_pages.cu -- whole pages of a paged cache, for all layers at once:
// rope3d_cache_fork (children that share their parents' full pages and copy the
// last one) and rope3d_cache_compact (the pages in use move to the front).
//
// Both are copies, bounded by memory: a page is cut into pieces of 32 KB, one to
// a block at a time, eight 16-byte vectors in flight a thread and up to eight blocks
// queued for an SM. (3,016 pages of 8 planes of 16 KB: 133 us with the tables, 5,940 GB/s; 136 with
// four vectors.) What is copied where is read from device memory by the blocks themselves, so
// nothing waits for the host.
//
// Compaction numbers the pages with a bitmap of the pages in use. One block, or a cluster of
// eight for large tables, makes it (each marks its share of the tables' rows in its own shared
// memory, and merges its share of the words), counts it, and writes the list of
// moves: with U pages in use, the k-th page in use at U or above goes to the k-th
// free page below U. A second kernel rewrites the tables and copies the pages.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/rope3d.h"
#include "rope3d_internal.h"
#include "rope3d_paged.h"
#include "rope3d_tc.cuh"

namespace {

using namespace rope3d_paged;

constexpr int kThreads = 256;
constexpr int kVectors = 8;
constexpr int kPiece = kThreads * kVectors * 16;   // bytes a block copies at a time
constexpr int kMarkBlocks = 8, kMarkThreads = 1024;
// Entries of a table that one block reads; both kernels of a compaction that moves nothing, one block / a cluster,
// us: 32 sequences of 256 entries 4.3 / 7.5, 96 of 152 6.4 / 7.2, 32 of 1000 7.8 / 12.2, 128 of 256 8.0 / 7.9, 2 of
// 16,384 40 / 65; above, 256 of 256 12.4 / 8.1, but 16 of 4096 13.7 / 21.9 (a warp marks a row).
constexpr int64_t kSmallTable = 32768;
constexpr int64_t kMaxPages = int64_t(1) << 20;   // their bitmap is 128 KB of shared memory

struct Planes {
    char *p;
    int64_t plane, page, bytes;   // strides and a page's size in bytes
    int planes, pages, pieces;
};

// Piece `piece` of page src into page dst.
__device__ __forceinline__ void copy_piece(const Planes &c, int plane, int src, int dst, int piece) {
    const int64_t at = int64_t(piece) * kPiece + threadIdx.x * 16;
    const char *from = c.p + plane * c.plane + src * c.page + at;
    char *to = c.p + plane * c.plane + dst * c.page + at;
    uint4 v[kVectors];
#pragma unroll
    for (int i = 0; i < kVectors; ++i)
        if (at + i * kThreads * 16 < c.bytes) v[i] = __ldcs(reinterpret_cast<const uint4 *>(from + i * kThreads * 16));
#pragma unroll
    for (int i = 0; i < kVectors; ++i)
        if (at + i * kThreads * 16 < c.bytes) __stcs(reinterpret_cast<uint4 *>(to + i * kThreads * 16), v[i]);
}

// ---- forks -------------------------------------------------------------------------

struct ForkParams {
    Planes cache;
    int *table, *lens;
    const int *parents, *children, *new_pages;
    int *invalid;
    int64_t table_stride;
    int seqs, width, page_size, forks;
};

// Units 0 .. forks - 1 write a child's row of the table, the others copy pieces.
__global__ void __launch_bounds__(kThreads) cache_fork_kernel(const __grid_constant__ ForkParams p) {
    rope3d_tc::grid_release();
    rope3d_tc::grid_wait();
    const int64_t each = int64_t(p.cache.planes) * p.cache.pieces, units = p.forks + p.forks * each;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int i = u < p.forks ? int(u) : int((u - p.forks) / each);
        const int parent = p.parents[i], child = p.children[i], fresh = p.new_pages[i];
        int n = -1, whole = 0, last = -1;
        if (parent >= 0 && parent < p.seqs && child >= 0 && child < p.seqs && child != parent && fresh >= 0 && fresh < p.cache.pages) {
            n = p.lens[parent];
            whole = n / p.page_size;
            if (n < 0 || whole >= p.width) n = -1;
            else if (n % p.page_size) {
                last = p.table[parent * p.table_stride + whole];
                if (last < 0 || last >= p.cache.pages) n = -1;
            }
        }
        if (u < p.forks) {
            if (n < 0) {
                if (threadIdx.x == 0 && p.invalid) atomicAdd(p.invalid, 1);
                continue;
            }
            const int *from = p.table + parent * p.table_stride;
            int *to = p.table + child * p.table_stride;
            for (int j = threadIdx.x; j < whole; j += kThreads) to[j] = from[j];
            if (threadIdx.x == 0) {
                to[whole] = fresh;
                p.lens[child] = n;
            }
        } else if (n >= 0 && last >= 0 && last != fresh) {
            const int64_t r = (u - p.forks) % each;
            copy_piece(p.cache, int(r / p.cache.pieces), last, fresh, int(r % p.cache.pieces));
        }
    }
}

// ---- compaction ----------------------------------------------------------------------

struct CompactParams {
    Planes cache;
    const int *table, *lens;
    int *table_out, *used;
    int64_t table_stride, out_stride, reserve;
    int seqs, width, page_size;
    int *moves;            // workspace: how many pages move
    int *src, *dst;        // workspace: [pages / 2 + 1] their old and new numbers
    int *rank;             // workspace: [pages] a moving page's place in the lists
};

// Entries that row s of the table holds.
__device__ __forceinline__ int held(const CompactParams &p, int s) {
    const int64_t n = p.lens[s];
    if (n <= 0) return 0;
    return int(min((n + p.reserve + p.page_size - 1) / p.page_size, int64_t(p.width)));
}

__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// The sum of v over the threads before this one, and over all.
__device__ int block_scan(int v, int *s_warp, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        int w = s_warp[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, w, d);
            if (lane >= d) w += o;
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    const int before = inc - v + (warp ? s_warp[warp - 1] : 0);
    *total = s_warp[31];
    __syncthreads();
    return before;
}

template <int kBlocks>
__global__ void __cluster_dims__(kBlocks, 1, 1) __launch_bounds__(kMarkThreads)
    cache_mark_kernel(const __grid_constant__ CompactParams p) {
    constexpr int kWords = kBlocks == 1 ? 1 : 4;   // of a thread
    extern __shared__ uint32_t s_map[];   // a bit for every page
    __shared__ int s_warp[32], s_share[2];
    const int tid = threadIdx.x, rank = kBlocks == 1 ? 0 : int(rope3d_tc::cluster_rank());
    auto meet = [] {
        if constexpr (kBlocks == 1) __syncthreads();
        else rope3d_tc::cluster_sync();
    };
    auto of_block = [](const void *at, int r) {   // a word of block r's shared memory
        if constexpr (kBlocks == 1) return *static_cast<const uint32_t *>(at);
        else return ld_cluster(rope3d_tc::map_rank(rope3d_tc::smem_u32(at), uint32_t(r)));
    };
    const int words = (p.cache.pages + 31) / 32;
    for (int w = tid; w < words; w += kMarkThreads) s_map[w] = 0;
    rope3d_tc::grid_release();
    rope3d_tc::grid_wait();
    __syncthreads();
    for (int s = rank * (kMarkThreads / 32) + (tid >> 5); s < p.seqs; s += kBlocks * (kMarkThreads / 32)) {
        const int n = held(p, s);
        for (int j = tid & 31; j < n; j += 32) {
            const int e = p.table[s * p.table_stride + j];
            if (e >= 0 && e < p.cache.pages) atomicOr(&s_map[e >> 5], 1u << (e & 31));
        }
    }
    __syncthreads();
    meet();

    // this block's words, of all eight maps: words in a row to a thread, so that a scan orders them
    const int mine = (words + kBlocks - 1) / kBlocks, first = min(rank * mine, words), end = min(first + mine, words);
    const int each = (mine + kMarkThreads - 1) / kMarkThreads;   // up to kWords
    uint32_t map[kWords];
    int ones = 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        const int w = first + tid * each + i;
        map[i] = 0;
        if (i < each && w < end) {
            for (int r = 0; r < kBlocks; ++r)
                map[i] |= of_block(&s_map[w], r);
            ones += __popc(map[i]);
        }
    }
    int sum;
    int before = block_scan(ones, s_warp, &sum);
    if (tid == 0) s_share[0] = sum;
    __syncthreads();
    meet();
    int total = 0, earlier = 0;
    for (int r = 0; r < kBlocks; ++r) {
        const int n = int(of_block(&s_share[0], r));
        total += n;
        if (r < rank) earlier += n;
    }
    before += earlier;   // pages in use below this thread's first word

    // pages in use below `total`: of which word holds it, or all where no word does
    if (tid == 0) s_share[1] = 0;
    __syncthreads();
    {
        int b = before;
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const int w = first + tid * each + i;
            if (i < each && w < end) {
                if (total >> 5 == w) s_share[1] = b + __popc(map[i] & ((1u << (total & 31)) - 1u));
                b += __popc(map[i]);
            }
        }
    }
    __syncthreads();
    meet();
    int low = 0;
    for (int r = 0; r < kBlocks; ++r)
        low += int(of_block(&s_share[1], r));
    if (total >> 5 >= words) low = total;   // every page is in use

    int b = before;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        const int w = first + tid * each + i;
        if (i >= each || w >= end) continue;
        // pages in use at `total` or above, then free ones below it
        const int from = total - w * 32;
        const uint32_t below = from <= 0 ? 0u : from >= 32 ? 0xffffffffu : (1u << from) - 1u;
        for (uint32_t high = map[i] & ~below; high; high &= high - 1) {
            const int bit = __ffs(int(high)) - 1, place = b + __popc(map[i] & ((1u << bit) - 1u)) - low;
            p.src[place] = w * 32 + bit;
            p.rank[w * 32 + bit] = place;
        }
        for (uint32_t hole = ~map[i] & below; hole; hole &= hole - 1) {
            const int bit = __ffs(int(hole)) - 1;
            p.dst[w * 32 + bit - b - __popc(map[i] & ((1u << bit) - 1u))] = w * 32 + bit;
        }
        b += __popc(map[i]);
    }
    if (rank == 0 && tid == 0) {
        *p.moves = total - low;
        *p.used = total;
    }
    if constexpr (kBlocks > 1) meet();   // no block leaves while another still reads its shared memory
}

__global__ void __launch_bounds__(kThreads) cache_move_kernel(const __grid_constant__ CompactParams p) {
    rope3d_tc::grid_release();
    rope3d_tc::grid_wait();
    const int total = *p.used, moves = *p.moves;
    const int64_t entries = int64_t(p.seqs) * p.width;
    for (int64_t i = blockIdx.x * kThreads + threadIdx.x; i < entries; i += int64_t(gridDim.x) * kThreads) {
        const int s = int(i / p.width), j = int(i - int64_t(s) * p.width);
        int e = -1;
        if (j < held(p, s)) {
            e = p.table[s * p.table_stride + j];
            if (e < 0 || e >= p.cache.pages) e = -1;
            else if (e >= total) e = p.dst[p.rank[e]];
        }
        p.table_out[s * p.out_stride + j] = e;
    }
    const int64_t each = int64_t(p.cache.planes) * p.cache.pieces, units = moves * each;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int m = int(u / each), r = int(u - m * each);
        copy_piece(p.cache, r / p.cache.pieces, p.src[m], p.dst[m], r % p.cache.pieces);
    }
}

// ---- host ------------------------------------------------------------------------------

int check_cache(const void *cache, int64_t planes, int64_t pages, int64_t page_bytes, int64_t plane_stride, int64_t page_stride,
                int64_t seqs, int64_t width, int64_t table_stride, int64_t page_size, Planes *c, View *v) {
    if (planes <= 0 || planes > (1 << 20) || pages <= 0 || pages > kMaxPages || page_bytes <= 0 || page_bytes > (int64_t(1) << 30) ||
        seqs <= 0 || seqs > kMaxSeqs || width <= 0 || table_stride < width || table_stride > kMaxStride || page_size <= 0 ||
        page_size > kMaxPlaces || width > kMaxPlaces / page_size)
        return ROPE3D_ERR_SHAPE;
    *v = view(cache, 1, page_bytes, planes, plane_stride, pages, page_stride);
    if (bad_strides(*v) || !rows_apart(*v)) return ROPE3D_ERR_SHAPE;
    if (!aligned(cache, 16) || page_bytes % 16 || (planes > 1 && plane_stride % 16) || (pages > 1 && page_stride % 16))
        return ROPE3D_ERR_ALIGN;
    const int64_t pieces = (page_bytes + kPiece - 1) / kPiece;
    *c = Planes{const_cast<char *>(static_cast<const char *>(cache)), plane_stride, page_stride, page_bytes, int(planes), int(pages),
                int(pieces)};
    if (planes * pieces > 0x7fffffff) return ROPE3D_ERR_SHAPE;
    return ROPE3D_OK;
}

// Outputs meet neither one another nor an input. (Bytes and 32-bit words: by address.)
int check_views(const View *out, int nout, const View *in, int nin) {
    for (int i = 0; i < nout; ++i)
        if (!aligned(out[i].p, out[i].elem)) return ROPE3D_ERR_ALIGN;
    for (int i = 0; i < nin; ++i)
        if (!aligned(in[i].p, in[i].elem)) return ROPE3D_ERR_ALIGN;
    for (int i = 0; i < nout; ++i) {
        for (int j = 0; j < nin; ++j)
            if (may_meet(out[i], in[j])) return ROPE3D_ERR_ALIAS;
        for (int j = i + 1; j < nout; ++j)
            if (may_meet(out[i], out[j])) return ROPE3D_ERR_ALIAS;
    }
    return ROPE3D_OK;
}

int fork(const rope3d_cache_fork_args *a, bool go, bool check_device, cudaStream_t st) {
    if (!a || !a->cache || !a->page_table || !a->seq_lens || !a->parents || !a->children || !a->new_pages) return ROPE3D_ERR_NULL;
    ForkParams p{};
    View cache;
    int rc = check_cache(a->cache, a->planes, a->pages, a->page_bytes, a->plane_stride, a->page_stride, a->seqs, a->table_width,
                         a->table_stride, a->page_size, &p.cache, &cache);
    if (rc != ROPE3D_OK) return rc;
    if (a->forks <= 0 || a->forks > kMaxSeqs) return ROPE3D_ERR_SHAPE;
    const View out[] = {cache, view(a->page_table, 4, a->table_width, a->seqs, a->table_stride), view(a->seq_lens, 4, a->seqs, 1, 0),
                        view(a->invalid_count, 4, 1, 1, 0)};
    const View in[] = {view(a->parents, 4, a->forks, 1, 0), view(a->children, 4, a->forks, 1, 0), view(a->new_pages, 4, a->forks, 1, 0)};
    if ((rc = check_views(out, 4, in, 3)) != ROPE3D_OK) return rc;
    if (check_device) {
        const void *const all[] = {a->cache, a->page_table, a->seq_lens, a->parents, a->children, a->new_pages, a->invalid_count};
        if ((rc = on_current_device(all, 7)) != ROPE3D_OK) return rc;
    }
    if (!go) return ROPE3D_OK;
    const int sms = sm_count();
    if (sms <= 0) return ROPE3D_ERR_CUDA;
    p.table = a->page_table;
    p.lens = a->seq_lens;
    p.parents = a->parents;
    p.children = a->children;
    p.new_pages = a->new_pages;
    p.invalid = a->invalid_count;
    p.table_stride = a->table_stride;
    p.seqs = int(a->seqs);
    p.width = int(a->table_width);
    p.page_size = int(a->page_size);
    p.forks = int(a->forks);
    const int64_t units = a->forks * (1 + int64_t(p.cache.planes) * p.cache.pieces);
    return launch(cache_fork_kernel, dim3(unsigned(std::min<int64_t>(units, sms * 8))), kThreads, 0, st, p);
}

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

// The workspace: the count of moves, the lists, the ranks.
int64_t compact_bytes(int64_t pages) { return 256 + 2 * up256((pages / 2 + 1) * 4) + up256(pages * 4); }

int compact(const rope3d_cache_compact_args *a, bool go, bool check_device, int64_t *need, cudaStream_t st) {
    if (!a || !a->cache || !a->page_table || !a->seq_lens || !a->table_out || !a->used) return ROPE3D_ERR_NULL;
    CompactParams p{};
    View cache;
    int rc = check_cache(a->cache, a->planes, a->pages, a->page_bytes, a->plane_stride, a->page_stride, a->seqs, a->table_width,
                         a->table_stride, a->page_size, &p.cache, &cache);
    if (rc != ROPE3D_OK) return rc;
    if (a->table_out_stride < a->table_width || a->table_out_stride > kMaxStride || a->reserve < 0 || a->reserve > kMaxPlaces)
        return ROPE3D_ERR_SHAPE;
    const int64_t bytes = compact_bytes(a->pages);
    if (need) *need = bytes;
    else if (!a->workspace) return ROPE3D_ERR_NULL;
    else if (a->workspace_bytes < bytes) return ROPE3D_ERR_SCRATCH;
    const bool in_place = a->table_out == a->page_table && a->table_out_stride == a->table_stride;
    const View table = view(a->page_table, 4, a->table_width, a->seqs, a->table_stride);
    const View out[] = {cache, view(a->table_out, 4, a->table_width, a->seqs, a->table_out_stride), view(a->used, 4, 1, 1, 0),
                        View{need ? nullptr : a->workspace, bytes, {1, 1, 1}, {0, 0, 0}, 1}};
    const View in[] = {view(a->seq_lens, 4, a->seqs, 1, 0), in_place ? View{nullptr, 1, {1, 1, 1}, {0, 0, 0}, 4} : table};
    if (!need && !aligned(a->workspace, 256)) return ROPE3D_ERR_ALIGN;
    if ((rc = check_views(out, 4, in, 2)) != ROPE3D_OK) return rc;
    if (check_device) {
        const void *const all[] = {a->cache, a->page_table, a->seq_lens, a->table_out, a->used, a->workspace};
        if ((rc = on_current_device(all, 6)) != ROPE3D_OK) return rc;
    }
    if (need || !go) return ROPE3D_OK;
    const int sms = sm_count();
    if (sms <= 0) return ROPE3D_ERR_CUDA;
    p.table = a->page_table;
    p.lens = a->seq_lens;
    p.table_out = a->table_out;
    p.used = a->used;
    p.table_stride = a->table_stride;
    p.out_stride = a->table_out_stride;
    p.reserve = a->reserve;
    p.seqs = int(a->seqs);
    p.width = int(a->table_width);
    p.page_size = int(a->page_size);
    char *ws = static_cast<char *>(a->workspace);
    const int64_t list = up256((a->pages / 2 + 1) * 4);
    p.moves = reinterpret_cast<int *>(ws);
    p.src = reinterpret_cast<int *>(ws + 256);
    p.dst = reinterpret_cast<int *>(ws + 256 + list);
    p.rank = reinterpret_cast<int *>(ws + 256 + 2 * list);
    const size_t smem = size_t((a->pages + 31) / 32) * 4;
    static std::atomic<bool> ready[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return ROPE3D_ERR_CUDA;
    if (!ready[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(cache_mark_kernel<kMarkBlocks>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMaxPages / 8)) !=
            cudaSuccess) {
            cudaGetLastError();
            return ROPE3D_ERR_CUDA;
        }
        ready[dev].store(true, std::memory_order_release);
    }
    const int64_t entries = a->seqs * a->table_width;
    if (entries <= kSmallTable && a->pages <= kMarkThreads * 32) rc = launch(cache_mark_kernel<1>, dim3(1), kMarkThreads, smem, st, p);
    else rc = launch(cache_mark_kernel<kMarkBlocks>, dim3(kMarkBlocks), kMarkThreads, smem, st, p);
    if (rc != ROPE3D_OK) return rc;
    const int64_t most = std::max((entries + kThreads - 1) / kThreads, a->pages / 2 * p.cache.planes * p.cache.pieces);
    return launch(cache_move_kernel, dim3(unsigned(std::min<int64_t>(std::max<int64_t>(most, 1), sms * 8))), kThreads, 0, st, p);
}

}  // namespace

extern "C" int rope3d_cache_fork(const rope3d_cache_fork_args *args, void *stream) {
    return fork(args, true, true, static_cast<cudaStream_t>(stream));
}

extern "C" int rope3d_cache_fork_check(const rope3d_cache_fork_args *args, int32_t check_device) {
    return fork(args, false, check_device != 0, nullptr);
}

extern "C" int rope3d_cache_compact(const rope3d_cache_compact_args *args, void *stream) {
    return compact(args, true, true, nullptr, static_cast<cudaStream_t>(stream));
}

extern "C" int rope3d_cache_compact_check(const rope3d_cache_compact_args *args, int32_t check_device) {
    return compact(args, false, check_device != 0, nullptr, nullptr);
}

extern "C" int rope3d_cache_compact_workspace(const rope3d_cache_compact_args *args, int64_t *bytes) {
    if (!bytes) return ROPE3D_ERR_NULL;
    return compact(args, false, false, bytes, nullptr);
}
