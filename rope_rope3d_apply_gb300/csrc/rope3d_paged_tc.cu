// rope3d_paged_tc.cu -- the attention over pages for many query rows, on the tensor
// cores (tcgen05). An item is 128 query rows of a sequence and key/value head (M =
// 128; the query heads of a group side by side, so that its keys are loaded
// once), its keys come in blocks of 128 places. One persistent block an SM walks its
// part of the line of blocks (rope3d_paged.cuh); its 16 warps have one job each and
// hand over through mbarriers, so that copies, products and softmax overlap, also
// across items:
//   warp 0: K by TMA, a copy for every run of places on a page and 64 channels (lanes
//     issue side by side), into a ring of pieces; warp 3: V likewise. Rows of V
//     that no row sees (behind a length, on an absent page) are zeroed: a weight of
//     zero times what lies there may be NaN.
//   warp 2 (one thread): S = Q K^T into one of kSBufs buffers of tensor memory
//   warp 1 (one thread): O += P V, with P read from tensor memory
//   warps 4-7: the next item's Q rows into shared memory; each item's result
//   warps 8-15: the softmax, a thread a row, in two groups of four warps that take
//     blocks in turn: one's exponentials run while the other waits for S, finds its maximum
//     or hands over. The maximum that weights refer to goes from group to group through
//     shared memory (before the exponentials); it moves only when it is exceeded by more
//     than 2^kLazy, and O is rescaled in tensor memory then (a published way to rescale seldom; the
//     weights, up to 2^8, and their sums have the room; they are rounded as in rope3d_paged.cu). A row's 128 scores stay in
//     registers (the other warps give some of theirs up) from one read of tensor memory to
//     the weights, which are written over S as pairs of 16 bits.
// head_dim is padded to 64, 128 or 256 channels by TMA's zero fill. At 256 a block's K
// comes as two pieces of 128 channels and its V as two of 64 places, so that five
// pieces of 32 KB fit beside Q.
//
// Pairs (kPair): two blocks of a cluster share an item of 256 rows, 128 each, and its keys:
// the products are those of cta_group::2, issued by the first block, for which each
// block holds half of the places of K and half of the channels of V. That halves what
// each SM loads and keeps of K and V, and reads of them for a product. A block's softmax,
// Q and results stay its own; what the issuing threads wait for is signalled to the first
// block's barriers, and what their products free or finish to both blocks'. An item is cut
// between blocks of 256 places (each two of 128 here).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/rope3d.h"
#include "rope3d_internal.h"
#include "rope3d_paged.cuh"
#include "rope3d_paged.h"
#include "rope3d_tc.cuh"

namespace {

using namespace rope3d_paged;
using namespace rope3d_tc;

constexpr int kKeys = 128;       // places of a block of keys
constexpr int kLanes = 128;      // rows of a block of threads: tensor memory's lanes
constexpr int kThreads = 512, kSoftWarp = 8;
constexpr float kLazy = 8.0f;
constexpr int64_t kMostTilePlaces = int64_t(1) << 23;   // see tiles_fit
// Registers of a thread: 512 threads have 128 each at launch; the softmax's 256 have
// kSoftRegs and the others kOtherRegs, no more together. (The compiler spills 8 to 10 of them, with 440 to 488
// bytes of stores and 332 to 412 of loads in the text; of a copy without the softmax's part 2.
// Other splits between the copying, the output's and the softmax's warps, 48 to 104 / 56 to 80 /
// 168 to 192: the same times, or up to 5 % longer where the copying and issuing warps have fewer than 72.)
constexpr int kSoftRegs = 184, kOtherRegs = 72;
static_assert(256 * (kSoftRegs + kOtherRegs) <= kThreads * 128, "no more registers than the block has");
constexpr uint32_t kColBlock = kLanes * 128;   // bytes of 64 channels of 128 rows

__device__ unsigned int g_paged_wait_timeouts;

// Shared memory and tensor memory at kD channels.
template <int kD, bool kPair>
struct Lay {
    static constexpr int kPieces = kD == 256 && !kPair ? 2 : 1;   // pieces of a block's K, and of its V
    static constexpr int kKRows = kPair ? 64 : 128;               // places and channels / 64 of a K piece
    static constexpr int kKCols = kPair ? kD / 64 : (kD < 128 ? kD : 128) / 64;
    static constexpr int kVRows = kKeys / kPieces;                // places and channels / 64 of a V piece
    static constexpr int kVCols = kPair ? kD / 128 : kD / 64;
    static constexpr uint32_t kKPiece = kKRows * kKCols * 128, kVPiece = kVRows * kVCols * 128;
    static constexpr int kKSlots = kPair ? (kD == 256 ? 3 : 5) : kD == 256 ? 3 : kD == 128 ? 2 : 4;
    static constexpr int kVSlots = kPair ? (kD == 256 ? 2 : 5) : kD == 64 ? 4 : 2;
    static constexpr int kQBufs = kD == 256 ? 1 : 2;
    static constexpr uint32_t kQBytes = kLanes * kD * 2;
    static constexpr int kSBufs = kD == 256 ? 2 : 3;
    static constexpr uint32_t kColO = kSBufs * 128;
    static constexpr uint32_t kOffK = kQBufs * kQBytes, kOffV = kOffK + kKSlots * kKPiece;
    static constexpr uint32_t kOffMax = kOffV + kVSlots * kVPiece;   // float [2][128]: a row's maximum, from each group
    static constexpr uint32_t kOffSum = kOffMax + 2 * 128 * 4;      // float [2][128] sums, [128] maxima
    static constexpr uint32_t kOffBar = kOffSum + 3 * 128 * 4;
    static constexpr int kBars = 2 * kQBufs + 2 * kKSlots + 2 * kVSlots + 3 * kSBufs + 5;
    static constexpr uint32_t kBytes = kOffBar + kBars * 8 + 16;
    static_assert(kColO + kD <= 512, "S and O fit tensor memory");
    static_assert(kOffMax % 1024 == 0 && kOffV % 1024 == 0 && kKPiece % 1024 == 0, "the swizzle's period");
    static_assert(kBytes <= 232448, "one block an SM");
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

template <bool kF16>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    uint32_t w;
    if constexpr (kF16) {
        const __half2 h = __floats2half2_rn(x, y);
        memcpy(&w, &h, 4);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        memcpy(&w, &h, 4);
    }
    return w;
}

// A box of 64 channels by some places of one head and page. kPair: `bar` may be the
// other block's.
template <bool kPair>
__device__ __forceinline__ void tma_load4(uint32_t dst, const CUtensorMap *map, int c, int slot, int head, int page, uint32_t bar) {
    if constexpr (kPair)
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
            "[%0], [%1, {%2, %3, %4, %5}], [%6];"
            ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c), "r"(slot), "r"(head), "r"(page), "r"(bar) : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
            ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c), "r"(slot), "r"(head), "r"(page), "r"(bar) : "memory");
}

__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// An arrival on the first block's barrier (this block's, without pairs): with this
// thread's writes to shared memory, for the cluster; or light, where what it hands over lies in
// tensor memory (complete and fenced before) or is still to be copied. (A release to the
// cluster waits for all of the thread's writes: 1,000 clocks of each block's hand-over, measured.)
template <bool kPair>
__device__ __forceinline__ void arrive_first(uint32_t bar) {
    if constexpr (kPair) mbar_arrive_cluster(map_rank(bar, 0));
    else arrive(bar);
}
template <bool kPair>
__device__ __forceinline__ void arrive_first_light(uint32_t bar) {
    if constexpr (kPair)
        asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(map_rank(bar, 0)) : "memory");
    else
        arrive(bar);
}
// ... and with the bytes that copies of this block will report there.
template <bool kPair>
__device__ __forceinline__ void expect_first(uint32_t bar, uint32_t bytes) {
    if constexpr (kPair)
        asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;"
                     ::"r"(map_rank(bar, 0)), "r"(bytes) : "memory");
    else
        mbar_expect_tx(bar, bytes);
}

// An arrival once this thread's products so far are done, in both blocks.
template <bool kPair>
__device__ __forceinline__ void commit_all(uint32_t bar) {
    if constexpr (kPair) commit_pair(bar);
    else commit(bar);
}

// D += A B with A (16 columns, pairs of 16 bits to one of tensor memory) read from there.
template <bool kPair>
__device__ __forceinline__ void mma_ta(uint32_t tmem, uint32_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
            ::"r"(tmem), "r"(a), "l"(b), "r"(id), "r"(accumulate) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
            ::"r"(tmem), "r"(a), "l"(b), "r"(id), "r"(accumulate) : "memory");
}

__device__ __forceinline__ void tmem_ld32(float *v, uint32_t addr) {
    uint32_t r[32];
    __syncwarp();
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr) : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// The loads so far are complete; uses of v stay behind this.
template <int kN>
__device__ __forceinline__ void tmem_hold(float *v) {
    tmem_wait();
#pragma unroll
    for (int i = 0; i < kN; ++i) asm volatile("" : "+f"(v[i]));
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *w) {
    __syncwarp();
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "r"(w[8]),
          "r"(w[9]), "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]), "r"(w[15]) : "memory");
}

__device__ __forceinline__ void tmem_stored() {
    __syncwarp();
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// The blocks of 128 places that a part of an item has.
template <int kLine>
struct Blocks {
    int begin, end;
    __device__ Blocks(const Item &it)
        : begin(max(it.begin * (kLine / kKeys), it.tile.k0 / kKeys)),
          end(min(it.end * (kLine / kKeys), (it.tile.k1 + kKeys - 1) / kKeys)) {}
};

// box_places: places of a copy, the greatest power of two that divides the page, 64 at most
template <bool kF16, int kD, bool kPair>
__global__ void __cluster_dims__(kPair ? 2 : 1, 1, 1) __launch_bounds__(kThreads, 1)
    paged_tile_kernel(const __grid_constant__ AttnParams p, const int box_places, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v) {
    using L = Lay<kD, kPair>;
    constexpr int kRows = kPair ? kPairRows : kTileRows, kLine = kPair ? 256 : 128;   // of an item; places of the line's blocks
    const int rank = kPair ? int(cluster_rank()) : 0, part = int(blockIdx.x) / (kPair ? 2 : 1);
    extern __shared__ __align__(1024) char sm[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = smem_u32(sm), bars = base + L::kOffBar;
    // barriers: of Q, K, V, S buffers, then single ones
    constexpr int kB1 = 2 * L::kQBufs, kB2 = kB1 + 2 * L::kKSlots, kB3 = kB2 + 2 * L::kVSlots, kB4 = kB3 + 3 * L::kSBufs;
    auto q_full = [&](int i) { return bars + 8u * uint32_t(2 * i); };
    auto q_empty = [&](int i) { return bars + 8u * uint32_t(2 * i + 1); };
    auto k_full = [&](int i) { return bars + 8u * uint32_t(kB1 + 2 * i); };
    auto k_empty = [&](int i) { return bars + 8u * uint32_t(kB1 + 2 * i + 1); };
    auto v_full = [&](int i) { return bars + 8u * uint32_t(kB2 + 2 * i); };
    auto v_empty = [&](int i) { return bars + 8u * uint32_t(kB2 + 2 * i + 1); };
    auto s_full = [&](int i) { return bars + 8u * uint32_t(kB3 + 3 * i); };
    auto s_empty = [&](int i) { return bars + 8u * uint32_t(kB3 + 3 * i + 1); };
    auto p_full = [&](int i) { return bars + 8u * uint32_t(kB3 + 3 * i + 2); };
    const uint32_t o_full = bars + 8u * kB4, o_empty = o_full + 8, sum_full = o_full + 16, sum_empty = o_full + 24,
                   v_land = o_full + 32;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::kOffBar + L::kBars * 8);
    unsigned int *late = &g_paged_wait_timeouts;

    // what needs nothing of earlier kernels comes before the wait for them
    if (tid == 0) {
        for (int i = 0; i < L::kQBufs; ++i) {
            mbar_init(q_full(i), kPair ? 8 : 4);
            mbar_init(q_empty(i), 1);
        }
        for (int i = 0; i < L::kKSlots; ++i) {
            mbar_init(k_full(i), kPair ? 2 : 1);
            mbar_init(k_empty(i), 1);
        }
        for (int i = 0; i < L::kVSlots; ++i) {
            mbar_init(v_full(i), kPair ? 2 : 1);
            mbar_init(v_empty(i), 1);
        }
        for (int i = 0; i < L::kSBufs; ++i) {
            mbar_init(s_full(i), 1);
            mbar_init(s_empty(i), 1);
            mbar_init(p_full(i), kPair ? 8 : 4);
        }
        mbar_init(o_full, 1);
        mbar_init(o_empty, kPair ? 8 : 4);
        mbar_init(sum_full, 8);
        mbar_init(sum_empty, 4);
        mbar_init(v_land, 1);
        mbar_fence_init();
        prefetch_map(&map_k);
        prefetch_map(&map_v);
    }
    grid_wait();
    grid_release();
    if (warp == 1) tmem_alloc<kPair>(smem_u32(tmem_slot), 512);
    // where this part begins, by way of the (yet unused) Q buffer
    find_start<kRows, kLine, kThreads>(p, part, reinterpret_cast<Start *>(sm), reinterpret_cast<long long *>(sm + 256));
    const Start st = *reinterpret_cast<Start *>(sm);
    if (tid == 0 && rank == 0) write_note(p, part, st);
    tc_fence_before();
    __syncthreads();   // (also: everyone has read `st`)
    if constexpr (kPair) cluster_sync();   // both blocks' barriers are there
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    bool dead = false;
    __syncwarp();
    Walker<kRows, kLine> walk(p, st);
    Item it;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 0 || warp == 3) {
            // ---- copies of K (warp 0) or V (warp 3)
            const bool is_v = warp == 3;
            const CUtensorMap *map = is_v ? &map_v : &map_k;
            const int slots = is_v ? L::kVSlots : L::kKSlots;
            const uint32_t ring = base + (is_v ? L::kOffV : L::kOffK);
            int n = 0, landings = 0;   // pieces so far; of them, those that were waited for here
            while (walk.next(it)) {
                const int *table = p.batch.table + it.s * p.batch.table_stride;
                const Blocks<kLine> bl(it);
                for (int b = bl.begin; b < bl.end; ++b) {
                    const int k0 = max(it.tile.k0 - b * kKeys, 0), k1 = min(it.tile.k1 - b * kKeys, kKeys);   // what rows see
    #pragma unroll
                    for (int piece = 0; piece < L::kPieces; ++piece, ++n) {
                        const int slot = n % slots;
                        const uint32_t full = is_v ? v_full(slot) : k_full(slot), empty = is_v ? v_empty(slot) : k_empty(slot);
                        // this piece: places row0 .. row0 + rows - 1 of the block, 64 cols channels from `channel0` on
                        const int row0 = is_v ? piece * L::kVRows : rank * L::kKRows, rows = is_v ? L::kVRows : L::kKRows;
                        const int cols = is_v ? L::kVCols : L::kKCols;
                        const int channel0 = is_v ? rank * L::kVCols * 64 : piece * L::kKCols * 64;
                        // boxes [from, to) of the block hold places of the piece that rows see
                        const int from = max(k0, row0) / box_places, to = (min(k1, row0 + rows) + box_places - 1) / box_places;
                        const int count = max(to - from, 0);
                        if (n >= slots) mbar_wait(empty, uint32_t(n / slots - 1) & 1u, dead, late);
                        dead = __any_sync(0xffffffffu, dead);
                        const bool clean = !is_v || (k0 <= row0 && k1 >= row0 + rows);   // nothing to be zeroed
                        const uint32_t dst = ring + uint32_t(slot) * (is_v ? L::kVPiece : L::kKPiece);
                        if (count && !dead) {
                            const uint32_t bytes = uint32_t(count * cols * box_places) * 128u;
                            if (lane == 0) {
                                if (clean) expect_first<kPair>(full, bytes);
                                else mbar_expect_tx(v_land, bytes);
                            }
                            __syncwarp();
                            const uint32_t bar = !clean ? v_land : kPair ? map_rank(full, 0) : full;
                            for (int i = lane; i < count * cols; i += 32) {
                                const int box = from + i / cols, col = i % cols;
                                const int place = b * kKeys + box * box_places, index = int(udiv(uint32_t(place), p.page));
                                int page = index < p.batch.width ? table[index] : -1;
                                if (page < 0 || page >= p.batch.pages) page = p.batch.pages;   // outside: filled with zeros
                                tma_load4<kPair>(dst + uint32_t(col * rows + box * box_places - row0) * 128u, map, channel0 + col * 64,
                                                 place - index * p.batch.page_size, it.h, page, bar);
                            }
                            __syncwarp();
                        }
                        if (!clean) {
                            if (count && !dead) {
                                mbar_wait(v_land, uint32_t(landings) & 1u, dead, late);
                                dead = __any_sync(0xffffffffu, dead);
                                ++landings;
                            }
                            const int a = min(max(k0 - row0, 0), rows), z = max(min(k1 - row0, rows), a);   // rows [a, z) are seen
                            for (int i = lane; i < (rows - (z - a)) * 8 * cols; i += 32) {
                                const int chunk = i % 8, col = i / 8 % cols, r = i / (8 * cols);
                                const int row = r < a ? r : r + (z - a);
                                *reinterpret_cast<uint4 *>(sm + (dst - base) + uint32_t(col * rows + row) * 128u + chunk * 16) =
                                    make_uint4(0, 0, 0, 0);
                            }
                            fence_async_smem();
                            __syncwarp();
                            if (lane == 0) arrive_first<kPair>(full);
                        } else if (!count && lane == 0) {
                            arrive_first_light<kPair>(full);
                        }
                    }
                }
            }
            if (dead && lane == 0 && rank == 0) {   // (the other block of a pair waits below)
                const int first = max(n - slots, 0);
                for (int i = first; i < n; ++i) {
                    bool gone = false;
                    mbar_wait(is_v ? v_full(i % slots) : k_full(i % slots), uint32_t(i / slots) & 1u, gone, late);
                }
            }
            if (dead && lane == 0 && is_v && landings) {
                bool gone = false;
                mbar_wait(v_land, uint32_t(landings - 1) & 1u, gone, late);
            }
        } else if (warp == 1) {
            // ---- O += P V
            if (lane == 0 && rank == 0) {
                constexpr uint32_t id = idesc(kRows, kD, !kF16, false, true);
                int g = 0, n = 0, items = 0;
                while (walk.next(it)) {
                    if (it.begin >= it.end) continue;
                    if (items) mbar_wait(o_empty, uint32_t(items - 1) & 1u, dead, late);
                    ++items;
                    const Blocks<kLine> bl(it);
                    for (int b = bl.begin; b < bl.end; ++b, ++g) {
                        const int sb = g % L::kSBufs;
                        mbar_wait(p_full(sb), uint32_t(g / L::kSBufs) & 1u, dead, late);
    #pragma unroll
                        for (int piece = 0; piece < L::kPieces; ++piece, ++n) {
                            const int slot = n % L::kVSlots;
                            mbar_wait(v_full(slot), uint32_t(n / L::kVSlots) & 1u, dead, late);
                            tc_fence_after();
                            const uint32_t v = base + L::kOffV + uint32_t(slot) * L::kVPiece;
                            const uint32_t pa = tmem + uint32_t(sb * 128 + piece * (L::kVRows / 2));
    #pragma unroll
                            for (int j = 0; j < L::kVRows / 16; ++j)
                                mma_ta<kPair>(tmem + L::kColO, pa + uint32_t(8 * j), sdesc(v + uint32_t(j) * 2048u, L::kVRows * 128, 1024),
                                              id, b > bl.begin || piece > 0 || j > 0 ? 1u : 0u);
                            commit_all<kPair>(v_empty(slot));
                        }
                        commit_all<kPair>(s_empty(sb));
                        if (b == bl.end - 1) commit_all<kPair>(o_full);
                    }
                }
            }
        } else if (warp == 2) {
            // ---- S = Q K^T
            if (lane == 0 && rank == 0) {
                constexpr uint32_t id = idesc(kRows, kKeys, !kF16, false, false);
                int g = 0, n = 0, items = 0;
                while (walk.next(it)) {
                    if (it.begin >= it.end) continue;
                    const int qb = items % L::kQBufs;
                    mbar_wait(q_full(qb), uint32_t(items / L::kQBufs) & 1u, dead, late);
                    ++items;
                    const uint32_t q = base + uint32_t(qb) * L::kQBytes;
                    const Blocks<kLine> bl(it);
                    for (int b = bl.begin; b < bl.end; ++b, ++g) {
                        const int sb = g % L::kSBufs;
                        if (g >= L::kSBufs) mbar_wait(s_empty(sb), uint32_t(g / L::kSBufs - 1) & 1u, dead, late);
    #pragma unroll
                        for (int piece = 0; piece < L::kPieces; ++piece, ++n) {
                            const int slot = n % L::kKSlots;
                            mbar_wait(k_full(slot), uint32_t(n / L::kKSlots) & 1u, dead, late);
                            tc_fence_after();
                            const uint32_t k = base + L::kOffK + uint32_t(slot) * L::kKPiece;
                            const uint32_t qp = q + uint32_t(piece * L::kKCols) * kColBlock;
    #pragma unroll
                            for (int j = 0; j < 4 * L::kKCols; ++j) {
                                const uint32_t off = uint32_t(j & 3) * 32u;
                                mma<kPair>(tmem + uint32_t(sb * 128), sdesc(qp + uint32_t(j >> 2) * kColBlock + off, 16, 1024),
                                           sdesc(k + uint32_t(j >> 2) * (L::kKRows * 128) + off, 16, 1024), id, piece > 0 || j > 0 ? 1u : 0u);
                            }
                            commit_all<kPair>(k_empty(slot));
                        }
                        commit_all<kPair>(s_full(sb));
                        if (b == bl.end - 1) commit_all<kPair>(q_empty(qb));
                    }
                }
            }
        }
    } else if (warp < kSoftWarp) {
        // ---- Q in, results out
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        const int row = rank * kLanes + tid - 128;   // this thread's row of results
        const uint32_t lanes = uint32_t(warp & 3) << 21;
        constexpr int kChunks = kD / 8;
        const int chunks = p.head_dim / 8;
        int loads = 0, items = 0;
        auto load_q = [&](const Item &of) {
            if (of.begin >= of.end) return;
            const int qb = loads % L::kQBufs;
            if (loads >= L::kQBufs) mbar_wait(q_empty(qb), uint32_t(loads / L::kQBufs - 1) & 1u, dead, late);
            ++loads;
            // A warp copies kPer rows at once, rows kPer (4 e + warp % 4) + sub for e = 0, 1, ...;
            // lane kPer e + sub finds where row (e, sub) lies.
            constexpr int kPer = 32 / kChunks, kSteps = kLanes / (4 * kPer);
            static_assert(kSteps * kPer == 32, "a row to a lane");
            const int mine = kPer * (4 * (lane / kPer) + (warp & 3)) + lane % kPer;
            const RowOf o = row_of<kRows>(p, of, rank * kLanes + mine);
            const long long at = rank * kLanes + mine < of.rows ? o.token * p.q_token + o.head * p.q_head : -1;
            const int c = lane % kChunks;
            const uint32_t to = base + uint32_t(qb) * L::kQBytes + uint32_t(c >> 3) * kColBlock;
#pragma unroll 4
            for (int e = 0; e < kSteps; ++e) {
                const int r = kPer * (4 * e + (warp & 3)) + lane / kChunks;
                const long long from = __shfl_sync(0xffffffffu, at, kPer * e + lane / kChunks);
                const bool live = from >= 0 && c < chunks;   // zeros elsewhere
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                             ::"r"(to + uint32_t(r) * 128u + uint32_t(((c & 7) ^ (r & 7)) << 4)), "l"(p.q + (live ? from + c * 16 : 0)),
                             "r"(live ? 16 : 0) : "memory");
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_async_smem();
            __syncwarp();
            if (lane == 0) arrive_first<kPair>(q_full(qb));
        };
        const float *sums = reinterpret_cast<const float *>(sm + L::kOffSum);
        auto finish = [&](const Item &of) {
            const RowOf o = row_of<kRows>(p, of, row);
            const bool on = row < of.rows;
            char *out = p.out + o.token * p.out_token + o.head * p.out_head;
            if (of.begin >= of.end) {   // no row sees a key
                if (on) {
                    for (int c = 0; c < chunks; ++c) *reinterpret_cast<uint4 *>(out + c * 16) = make_uint4(0, 0, 0, 0);
                    if (p.lse) p.lse[o.token * p.lse_token + o.head] = -INFINITY;
                }
                return;
            }
            mbar_wait(sum_full, uint32_t(items) & 1u, dead, late);
            const int in = tid - 128;
            const float sum = sums[in] + sums[128 + in], top = sums[256 + in];
            mbar_wait(o_full, uint32_t(items) & 1u, dead, late);
            ++items;
            __syncwarp();
            tc_fence_after();
            if (lane == 0) arrive(sum_empty);
            float *slot = slot_of<kRows>(p, part, of.head);
            const float inv = sum > 0.f ? 1.f / sum : sum;
            for (int c0 = 0; c0 < p.head_dim; c0 += 32) {
                float v[32];
                tmem_ld32(v, tmem + L::kColO + lanes + uint32_t(c0));
                tmem_hold<32>(v);
                if (!on) continue;
                if (of.whole) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
                        if (c0 + i < p.head_dim)
                            *reinterpret_cast<uint4 *>(out + (c0 + i) * 2) =
                                make_uint4(pack2<kF16>(v[i] * inv, v[i + 1] * inv), pack2<kF16>(v[i + 2] * inv, v[i + 3] * inv),
                                           pack2<kF16>(v[i + 4] * inv, v[i + 5] * inv), pack2<kF16>(v[i + 6] * inv, v[i + 7] * inv));
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        if (c0 + i < p.head_dim)
                            *reinterpret_cast<float4 *>(slot + int64_t((c0 + i) / 4 * kRows + row) * 4) =
                                make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                }
            }
            __syncwarp();
            tc_fence_before();
            if (lane == 0) arrive_first_light<kPair>(o_empty);
            if (!on) return;
            if (of.whole) {
                if (p.lse) p.lse[o.token * p.lse_token + o.head] = sum > 0.f ? (top + log2f(sum)) * 0.69314718f : sum == 0.f ? -INFINITY : sum;
            } else {
                slot[int64_t(p.head_dim) * kRows + row] = top;
                slot[int64_t(p.head_dim) * kRows + kRows + row] = sum;
            }
        };
        bool more = walk.next(it);
        if (more) load_q(it);
        while (more) {
            const Item now = it;
            more = walk.next(it);
            if (more) load_q(it);
            finish(now);
        }
    } else {
        // ---- softmax: row `row`, every second block
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        const int group = (warp - kSoftWarp) >> 2, row = (warp & 3) * 32 + lane;   // (of this block's)
        const uint32_t lanes = uint32_t(warp & 3) << 21;
        float *passed = reinterpret_cast<float *>(sm + L::kOffMax), *sums = reinterpret_cast<float *>(sm + L::kOffSum);
        // named barriers of the four pairs of warps, one for each direction
        const int to_other = 1 + group * 4 + (warp & 3), from_other = 1 + (group ^ 1) * 4 + (warp & 3);
        int g = 0, items = 0;
        while (walk.next(it)) {
            if (it.begin >= it.end) continue;
            const RowOf ro = row_of<kRows>(p, it, rank * kLanes + row);
            const bool any_row = rank * kLanes + (warp & 3) * 32 < it.rows;   // the same for the pair of warps
            const Blocks<kLine> bl(it);
            const int *table = p.batch.table + it.s * p.batch.table_stride;
            auto page_at = [&](int b) {   // of eight places, by lane
                const uint32_t index = udiv(uint32_t(b * kKeys + (lane & 15) * 8), p.page);
                return b < bl.end && index < uint32_t(p.batch.width) ? table[index] : -1;
            };
            float m = -INFINITY, l = 0.f;
            auto receive = [&] {   // the maximum that the other group's last block refers to
                asm volatile("bar.sync %0, 64;" ::"r"(from_other) : "memory");
                const float now = passed[(group ^ 1) * 128 + row];
                if (now > m) {
                    l *= m == -INFINITY ? 0.f : ex2(m - now);
                    m = now;
                }
            };
            const int mine = bl.begin + ((g ^ group) & 1);   // this group's first block
            int page = page_at(mine);
            for (int b = bl.begin; b < bl.end; ++b, ++g) {
                if ((g & 1) != group) continue;
                const int sb = g % L::kSBufs, place = b * kKeys;
                const uint32_t s = tmem + uint32_t(sb * 128) + lanes;
                const uint32_t there = __ballot_sync(0xffffffffu, page >= 0 && page < p.batch.pages) & 0xffffu;
                page = page_at(b + 2);
                mbar_wait(s_full(sb), uint32_t(g / L::kSBufs) & 1u, dead, late);
                __syncwarp();
                tc_fence_after();
                if (any_row) {
                    const int a = max(ro.lo - place, 0), z = min(ro.hi - place, kKeys);
                    const bool masked = __any_sync(0xffffffffu, a > 0 || z < kKeys || there != 0xffffu);
                    auto sees = [&](int c) {   // of columns 32 c .. 32 c + 31
                        const int from = max(a - 32 * c, 0), to = min(z - 32 * c, 32);
                        uint32_t bits = from < to ? (0xffffffffu >> (32 - (to - from))) << from : 0u;
                        const uint32_t four = there >> (4 * c) & 15u;
                        if (four != 15u)
                            for (int e = 0; e < 4; ++e)
                                if (!(four >> e & 1u)) bits &= ~(0xffu << (8 * e));
                        return bits;
                    };
                    float x[128];
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32(x + 32 * c, s + uint32_t(32 * c));
                    tmem_hold<128>(x);
                    if (masked) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint32_t bits = sees(c);
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[32 * c + e] = bits >> e & 1u ? x[32 * c + e] : -INFINITY;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 128; e += 8)
#pragma unroll
                        for (int j = 0; j < 4; ++j) top[j] = max3(top[j], x[e + 2 * j], x[e + 2 * j + 1]);
                    const float best = max3(top[0], top[1], fmaxf(top[2], top[3])) * p.scale_log2;
                    if (b > bl.begin) receive();
                    const bool move = best > m + kLazy || m == -INFINITY;
                    const bool rescale = move && m != -INFINITY;
                    float f = 1.f;
                    if (move) {
                        const float to = fmaxf(m, best);
                        f = rescale ? ex2(m - to) : 0.f;
                        m = to;
                        l *= f;
                    }
                    passed[group * 128 + row] = m;
                    asm volatile("bar.arrive %0, 64;" ::"r"(to_other) : "memory");
                    const float neg = m == -INFINITY ? 0.f : -m;
                    const float2 c2 = make_float2(p.scale_log2, p.scale_log2), n2 = make_float2(neg, neg);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const float2 y = __ffma2_rn(make_float2(x[32 * c + e], x[32 * c + e + 1]), c2, n2);
                            const float u = ex2(y.x), t = ex2(y.y);
                            sum[(e >> 1) & 1] = __fadd2_rn(sum[(e >> 1) & 1], make_float2(u, t));
                            w[e / 2] = pack2<kF16>(u, t);
                        }
                        tmem_st16(s + uint32_t(16 * c), w);
                    }
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    if (__any_sync(0xffffffffu, rescale)) {   // O holds the blocks before
                        mbar_wait(s_empty((g - 1) % L::kSBufs), uint32_t((g - 1) / L::kSBufs) & 1u, dead, late);
                        __syncwarp();
                        tc_fence_after();
#pragma unroll 1
                        for (int c0 = 0; c0 < kD; c0 += 16) {
                            float o[16];
                            const uint32_t at = tmem + L::kColO + lanes + uint32_t(c0);
                            tmem_ld16(o, at);
                            tmem_wait();
                            tmem_tie16(o);
                            uint32_t u[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e] * f);
                            tmem_st16(at, u);
                        }
                    }
                    tmem_stored();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_first_light<kPair>(p_full(sb));
            }
            const bool last = ((g - 1) & 1) == group;   // the item's last block was this group's
            if (any_row && !last) receive();
            if (items) mbar_wait(sum_empty, uint32_t(items - 1) & 1u, dead, late);
            ++items;
            sums[group * 128 + row] = l;
            if (last) sums[256 + row] = m;
            __syncwarp();
            if (lane == 0) arrive(sum_full);
        }
    }
    // neither block of a pair leaves while the other may name its memory or barriers
    tc_fence_before();
    __syncthreads();
    if constexpr (kPair) cluster_sync();
    tc_fence_after();
    if (warp == 1) tmem_free<kPair>(tmem, 512);
}

// ---- host --------------------------------------------------------------------------

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                   const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
    static const EncodeTiledFn fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return EncodeTiledFn(nullptr);
        }
        return reinterpret_cast<EncodeTiledFn>(ptr);
    }();
    return fn;
}

// A cache as (channels, places of a page, heads, pages).
bool make_map(CUtensorMap *map, const void *p, const rope3d_paged_attention_args &a, int64_t page, int64_t slot, int64_t head, int box) {
    const EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    const rope3d_paged_batch &b = a.batch;
    const cuuint64_t dims[4] = {cuuint64_t(a.head_dim), cuuint64_t(b.page_size), cuuint64_t(a.kv_heads), cuuint64_t(b.pages)};
    // (of a dimension of one, any stride)
    const cuuint64_t row = cuuint64_t(a.head_dim) * 2;
    const cuuint64_t strides[3] = {b.page_size > 1 ? cuuint64_t(slot) * 2 : row, a.kv_heads > 1 ? cuuint64_t(head) * 2 : row,
                                   b.pages > 1 ? cuuint64_t(page) * 2 : row};
    const cuuint32_t boxes[4] = {64, cuuint32_t(box), 1, 1}, one[4] = {1, 1, 1, 1};
    return fn(map, a.dtype == ROPE3D_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(p),
              dims, strides, boxes, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kF16, int kD, bool kPair>
int launch_tile(const AttnParams &p, int box, const CUtensorMap &k, const CUtensorMap &v, cudaStream_t st) {
    static std::atomic<bool> ready[64];
    auto *fn = paged_tile_kernel<kF16, kD, kPair>;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return ROPE3D_ERR_CUDA;
    if (!ready[dev].load(std::memory_order_acquire)) {
        cudaFuncAttributes attr{};   // (a block launched with fewer registers would wait for more without an end)
        if (cudaFuncGetAttributes(&attr, fn) != cudaSuccess || attr.numRegs * kThreads < 256 * (kSoftRegs + kOtherRegs) ||
            cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Lay<kD, kPair>::kBytes)) != cudaSuccess) {
            cudaGetLastError();
            return ROPE3D_ERR_CUDA;
        }
        ready[dev].store(true, std::memory_order_release);
    }
    return launch(fn, dim3(unsigned(p.parts) * (kPair ? 2u : 1u)), kThreads, Lay<kD, kPair>::kBytes, st, p, box, k, v);
}

template <bool kF16>
int launch_tile(const AttnParams &p, bool pair, int box, const CUtensorMap &k, const CUtensorMap &v, cudaStream_t st) {
    if (p.head_dim <= 64) return launch_tile<kF16, 64, false>(p, box, k, v, st);
    if (p.head_dim <= 128) return pair ? launch_tile<kF16, 128, true>(p, box, k, v, st) : launch_tile<kF16, 128, false>(p, box, k, v, st);
    return pair ? launch_tile<kF16, 256, true>(p, box, k, v, st) : launch_tile<kF16, 256, false>(p, box, k, v, st);
}

}  // namespace

// What the tensor maps can describe: pages of whole groups of eight places (the
// swizzle's period in shared memory), strides above zero. And items that end within a
// bounded wait: an item's result is waited for from its beginning on, for 10^9 clocks at most,
// and a block of 128 places takes up to 5,600 (256 channels, every SM reading 128 KB of its own at
// the memory's rate). 2^23 places are 3.7 * 10^8 clocks; longer rows go to the kernel for few rows,
// which waits for nothing.
bool rope3d_paged::tiles_fit(const rope3d_paged_attention_args &a) {
    const rope3d_paged_batch &b = a.batch;
    if (b.page_size % 8 != 0 || b.table_width * b.page_size > kMostTilePlaces) return false;
    for (const int64_t s : {a.k_slot_stride, a.v_slot_stride})
        if (b.page_size > 1 && (s <= 0 || s * 2 >= kMaxStride)) return false;
    for (const int64_t s : {a.k_cache_head_stride, a.v_cache_head_stride})
        if (a.kv_heads > 1 && (s <= 0 || s * 2 >= kMaxStride)) return false;
    for (const int64_t s : {a.k_page_stride, a.v_page_stride})
        if (b.pages > 1 && (s <= 0 || s * 2 >= kMaxStride)) return false;
    return true;
}

// A pair's blocks each hold half of the channels of V, in whole 64s.
bool rope3d_paged::pairs_fit(const rope3d_paged_attention_args &a) { return a.head_dim > 64; }

int rope3d_paged::launch_tiles(const AttnParams &p, const rope3d_paged_attention_args &a, bool pair, cudaStream_t st) {
    int box = 8;
    while (box < 64 && a.batch.page_size % (2 * box) == 0) box *= 2;
    CUtensorMap k, v;
    if (!make_map(&k, a.k_cache, a, a.k_page_stride, a.k_slot_stride, a.k_cache_head_stride, box) ||
        !make_map(&v, a.v_cache, a, a.v_page_stride, a.v_slot_stride, a.v_cache_head_stride, box))
        return ROPE3D_ERR_CUDA;
    return a.dtype == ROPE3D_F16 ? launch_tile<true>(p, pair, box, k, v, st) : launch_tile<false>(p, pair, box, k, v, st);
}

int rope3d_paged::tiles_wait_timeouts(unsigned int *count, bool reset) {
    const unsigned int zero = 0;
    if (cudaMemcpyFromSymbol(count, g_paged_wait_timeouts, sizeof(zero)) != cudaSuccess ||
        (reset && cudaMemcpyToSymbol(g_paged_wait_timeouts, &zero, sizeof(zero)) != cudaSuccess)) {
        cudaGetLastError();
        return ROPE3D_ERR_CUDA;
    }
    return ROPE3D_OK;
}
