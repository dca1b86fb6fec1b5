// rope3d_paged.cu -- attention of new tokens over the pages of a cache:
// rope3d_paged_attention, its kernel for few query rows and the kernel that adds
// partial results. (rope3d_paged_tc.cu has the kernel for many rows, rope3d_paged.cuh
// the division of the work.)
//
//     out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j - m_i)
// in one pass over the keys, with the maximum m_i so far: where it moves, the sums so
// far are multiplied by exp(old - new).
//
// Few rows (one new token of a sequence and the query heads that share its keys): reading
// the cache is all there is, 1 to 16 rows to 2 bytes an element. Every warp streams
// places of its own through its own ring of shared memory (16 of every 64, by
// 16-byte cp.async copies, rows outside the mask filled with zeros and not read) and
// keeps a maximum, a sum and sums of V of its own, so that warps meet only at an
// item's end. Products are warp MMAs (m16n8k16): at 16 rows the tensor cores have
// next to nothing to do, and fragments come straight from the swizzled ring. The weights are rounded to the
// cache's type for the second product, as its operand has to be (their sum is of the unrounded ones): the
// result's relative error (2-norm, against 64 bits) is 0.0020 to 0.0021 in bf16 and 0.00027 to 0.00028 in fp16
// where that of weights kept in 32 bits is 0.0016 to 0.0017 and 0.00021, the rounding of the result itself.
// Measured: 64 sequences of 100 to 16,000 places of 8 heads of 128, fp16, pages of 16: 317 us,
// 6,620 GB/s, 97.5 % of a copy; of 8192 places of 4 heads of 256, bf16: 327 us, 6,570 GB/s; of 64:
// 97 us, 5,530 GB/s (the softmax's instructions are the same for half the bytes). One sequence
// of 8191 places of 4 heads of 256: 15.2 us for 33.6 MB, half of it the chain of loads before the
// first keys and behind the last.
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

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kWarpKeys = 16;                    // places of a block that one warp takes
constexpr int kKeys = kWarpKeys * kWarps;        // places of a block
constexpr int kRows = kFewRows;
constexpr int kMostParts = 3 * kTileParts;       // see kPerSm

// Stages of a warp's ring, and blocks that fit an SM beside one another with them.
template <int kD> constexpr int kStagesOf = kD == 64 ? 4 : 3;
template <int kD> constexpr int kPerSm = kD == 256 ? 1 : kD == 128 ? 2 : 3;
template <int kD> constexpr int kStageBytes = 2 * kWarpKeys * kD * 2;   // K, then V
template <int kD> constexpr int kSmemBytes = kRows * kD * 2 + kWarps * kStagesOf<kD> * kStageBytes<kD>;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

template <bool kF16>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (kF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// Byte offset of 16-byte chunk c of row r in a tile of rows of kD elements: chunks
// permuted within 128 bytes by the row, so that eight rows' chunks lie in
// eight different bank groups.
template <int kD>
__device__ __forceinline__ uint32_t at(int r, int c) { return uint32_t(r * kD * 2 + ((c ^ (r & 7)) << 4)); }

// log sum exp in base e of a row with maximum m (base 2) and sum l.
__device__ __forceinline__ float lse_of(float m, float l) {
    return l > 0.f ? (m + log2f(l)) * 0.69314718f : l == 0.f ? -INFINITY : l;
}

// Four results of a row, rounded.
template <bool kF16>
__device__ __forceinline__ void store4(char *to, float4 v, float inv) {
    *reinterpret_cast<uint2 *>(to) = make_uint2(pack2<kF16>(v.x * inv, v.y * inv), pack2<kF16>(v.z * inv, v.w * inv));
}

template <bool kF16, int kD>
__global__ void __launch_bounds__(kThreads) paged_rows_kernel(const __grid_constant__ AttnParams p) {
    constexpr int kStages = kStagesOf<kD>, kChunks = kD / 8, kPass = 32 / kChunks;   // rows that the warp copies at once
    constexpr int kHalf = kWarpKeys * kD * 2;   // bytes of a stage's K
    extern __shared__ __align__(128) char sm[];
    __shared__ Start s_start;
    __shared__ long long s_sums[kWarps];
    __shared__ uint32_t s_live[kWarps][kStages];
    __shared__ float s_max[kWarps][kRows], s_sum[kWarps][kRows];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane >> 2, col = lane & 3;
    const uint32_t sq = rope3d_tc::smem_u32(sm);
    char *ring = sm + kRows * kD * 2 + warp * kStages * kStageBytes<kD>;
    const uint32_t sring = rope3d_tc::smem_u32(ring);

    rope3d_tc::grid_release();
    rope3d_tc::grid_wait();
    find_start<kRows, kKeys, kThreads>(p, blockIdx.x, &s_start, s_sums);
    const Start st = s_start;
    if (tid == 0) write_note(p, blockIdx.x, st);
    const int chunks = p.head_dim / 8;

    Walker<kRows, kKeys> walk(p, st);
    Item it;
    while (walk.next(it)) {
        const int steps = it.end - it.begin;
        const char *kbase = p.k + it.h * p.k_head, *vbase = p.v + it.h * p.v_head;
        const int *table = p.batch.table + it.s * p.batch.table_stride;
        const int place0 = it.begin * kKeys + warp * kWarpKeys;

        // the page of this lane's place of a step (lanes 0-15); -1 where no row sees it
        auto page_of = [&](int step) {
            const int place = place0 + step * kKeys + (lane & 15);
            int page = -1;
            if (step < steps && place >= it.tile.k0 && place < it.tile.k1) page = table[udiv(uint32_t(place), p.page)];
            return page;
        };
        auto issue = [&](int step, int page) {
            const uint32_t place = uint32_t(place0 + step * kKeys + (lane & 15));
            const int slot_of = int(place - udiv(place, p.page) * p.page.d);
            const bool live = page >= 0 && page < p.batch.pages;
            const uint32_t all = __ballot_sync(0xffffffffu, live) & 0xffffu;
            const int slot = step % kStages;
            if (lane == 0) s_live[warp][slot] = all;
            if (step < steps) {
                const int64_t ko = live ? page * p.k_page + slot_of * p.k_slot : 0;
                const int64_t vo = live ? page * p.v_page + slot_of * p.v_slot : 0;
                const uint32_t dst = sring + slot * kStageBytes<kD>;
                const int c = lane % kChunks;
#pragma unroll
                for (int i = 0; i < kWarpKeys / kPass; ++i) {
                    const int r = i * kPass + lane / kChunks;
                    const bool on = (all >> r & 1u) && c < chunks;
                    const int64_t off = __shfl_sync(0xffffffffu, ko, r);
                    copy16(dst + at<kD>(r, c), kbase + (on ? off + c * 16 : 0), on);
                }
#pragma unroll
                for (int i = 0; i < kWarpKeys / kPass; ++i) {
                    const int r = i * kPass + lane / kChunks;
                    const bool on = (all >> r & 1u) && c < chunks;
                    const int64_t off = __shfl_sync(0xffffffffu, vo, r);
                    copy16(dst + kHalf + at<kD>(r, c), vbase + (on ? off + c * 16 : 0), on);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };

        // the rows of q, behind one another, zeros past head_dim and past the item (with step 0's copies)
        __syncthreads();   // the item before is done with shared memory
        for (int i = tid; i < kRows * kChunks; i += kThreads) {
            const int r = i / kChunks, c = i % kChunks;
            const bool on = r < it.rows && c < chunks;
            const RowOf o = row_of<kRows>(p, it, r);
            copy16(sq + at<kD>(r, c), p.q + (on ? o.token * p.q_token + o.head * p.q_head + c * 16 : 0), on);
        }
        constexpr bool kKeepQ = kD <= 128;   // q's fragments in registers
        uint32_t qf[kKeepQ ? kD / 16 : 1][4];
        const int qr = (lane & 7) + (lane & 8), qc = lane >> 4;
        const RowOf r0 = row_of<kRows>(p, it, quad), r1 = row_of<kRows>(p, it, quad + 8);

        float o[kD / 8][4];
#pragma unroll
        for (int i = 0; i < kD / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

        // A step issues the copies of kStages - 1 steps on; first those of steps 0 .. kStages - 2.
        int page = page_of(0);
#pragma unroll 1   // (a call of a few microseconds waits for its instructions too)
        for (int step = 0; step < kStages - 1; ++step) {
            const int after = page_of(step + 1);
            issue(step, page);
            page = after;
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        __syncthreads();   // every warp's part of q is there
        if constexpr (kKeepQ) {
#pragma unroll
            for (int k = 0; k < kD / 16; ++k) ldm4(qf[k], sq + at<kD>(qr, 2 * k + qc));
        }

#pragma unroll 1
        for (int step = 0; step < steps; ++step) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
            __syncwarp();
            const int slot = step % kStages;
            const uint32_t sk = sring + slot * kStageBytes<kD>, sv = sk + kHalf;
            const uint32_t live = s_live[warp][slot];
            if (live) {
                float sa[2][4] = {}, sb[2][4] = {};   // even and odd k: chains half as long
#pragma unroll
                for (int k = 0; k < kD / 16; ++k) {
                    uint32_t b[4], a[4];
                    ldm4(b, sk + at<kD>((lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
                    if constexpr (kKeepQ) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) a[e] = qf[k][e];
                    } else {
                        ldm4(a, sq + at<kD>(qr, 2 * k + qc));
                    }
                    mma16<kF16>(k & 1 ? sb[0] : sa[0], a, b[0], b[1]);
                    mma16<kF16>(k & 1 ? sb[1] : sa[1], a, b[2], b[3]);
                }
                float s[2][4], x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = n * 8 + col * 2 + (e & 1), place = place0 + step * kKeys + key;
                        const RowOf &r = e < 2 ? r0 : r1;
                        const bool sees = (live >> key & 1u) && place >= r.lo && place < r.hi;
                        s[n][e] = sees ? (sa[n][e] + sb[n][e]) * p.scale_log2 : -INFINITY;
                        if (e < 2) x0 = fmaxf(x0, s[n][e]);
                        else x1 = fmaxf(x1, s[n][e]);
                    }
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
                x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
                x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
                const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
                const float z0 = n0 == -INFINITY ? 0.f : n0, z1 = n1 == -INFINITY ? 0.f : n1;
                if (__any_sync(0xffffffffu, n0 > m0 || n1 > m1)) {
                    const float f0 = ex2(m0 - z0), f1 = ex2(m1 - z1);
                    l0 *= f0;
                    l1 *= f1;
#pragma unroll
                    for (int i = 0; i < kD / 8; ++i) {
                        o[i][0] *= f0;
                        o[i][1] *= f0;
                        o[i][2] *= f1;
                        o[i][3] *= f1;
                    }
                    m0 = n0;
                    m1 = n1;
                }
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[n][e] = ex2(s[n][e] - (e < 2 ? z0 : z1));
                        if (e < 2) l0 += s[n][e];
                        else l1 += s[n][e];
                    }
                const uint32_t pa[4] = {pack2<kF16>(s[0][0], s[0][1]), pack2<kF16>(s[0][2], s[0][3]),
                                        pack2<kF16>(s[1][0], s[1][1]), pack2<kF16>(s[1][2], s[1][3])};
#pragma unroll
                for (int i = 0; i < kD / 16; ++i) {
                    uint32_t b[4];
                    ldm4t(b, sv + at<kD>((lane & 7) + (lane & 8), 2 * i + (lane >> 4)));
                    mma16<kF16>(o[2 * i], pa, b[0], b[1]);
                    mma16<kF16>(o[2 * i + 1], pa, b[2], b[3]);
                }
            }
            __syncwarp();
            const int after = page_of(step + kStages);
            issue(step + kStages - 1, page);
            page = after;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");

        // the warps' results joined: by each row's greatest maximum, in the warps' order
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
        if (col == 0) {
            s_max[warp][quad] = m0;
            s_max[warp][quad + 8] = m1;
            s_sum[warp][quad] = l0;
            s_sum[warp][quad + 8] = l1;
        }
        __syncthreads();
        float g0 = s_max[0][quad], g1 = s_max[0][quad + 8];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            g0 = fmaxf(g0, s_max[w][quad]);
            g1 = fmaxf(g1, s_max[w][quad + 8]);
        }
        const float f0 = m0 == -INFINITY ? 0.f : ex2(m0 - g0), f1 = m1 == -INFINITY ? 0.f : ex2(m1 - g1);
        float *mine = reinterpret_cast<float *>(ring);
        constexpr int kLd = kD + 8;   // floats between rows: quads of rows in different banks
        static_assert(kRows * kLd * 4 <= kStagesOf<kD> * kStageBytes<kD>, "a warp's sums fit its ring");
#pragma unroll
        for (int i = 0; i < kD / 8; ++i) {
            *reinterpret_cast<float2 *>(mine + quad * kLd + i * 8 + col * 2) = make_float2(o[i][0] * f0, o[i][1] * f0);
            *reinterpret_cast<float2 *>(mine + (quad + 8) * kLd + i * 8 + col * 2) = make_float2(o[i][2] * f1, o[i][3] * f1);
        }
        __syncthreads();
        float *slot = slot_of<kRows>(p, blockIdx.x, it.head);
        const int vecs = p.head_dim / 4;
        for (int i = tid; i < it.rows * vecs; i += kThreads) {
            const int r = i / vecs, c = i % vecs;
            float big = -INFINITY, sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) big = fmaxf(big, s_max[w][r]);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 x = *reinterpret_cast<const float4 *>(
                    reinterpret_cast<const float *>(sm + kRows * kD * 2 + w * kStages * kStageBytes<kD>) + r * kLd + c * 4);
                v.x += x.x;
                v.y += x.y;
                v.z += x.z;
                v.w += x.w;
                sum += s_max[w][r] == big ? s_sum[w][r] : s_sum[w][r] * ex2(s_max[w][r] - big);
            }
            if (it.whole) {
                const RowOf row = row_of<kRows>(p, it, r);
                store4<kF16>(p.out + row.token * p.out_token + row.head * p.out_head + c * 8, v, sum > 0.f ? 1.f / sum : sum);
                if (c == 0 && p.lse) p.lse[row.token * p.lse_token + row.head] = lse_of(big, sum);
            } else {
                *reinterpret_cast<float4 *>(slot + (c * kRows + r) * 4) = v;
                if (c == 0) {
                    slot[vecs * kRows * 4 + r] = big;
                    slot[vecs * kRows * 4 + kRows + r] = sum;
                }
            }
        }
    }
}

// ---- partial results ---------------------------------------------------------------

// Few rows: as many parts as 456, and little in each: blocks of many threads. Tiles: two or
// three parts, and much: more blocks beside one another (512 threads of 88 registers left one
// on an SM, 42 us of 224 at 8192 x 8192 x 256).
template <int kTile> constexpr int kJoinThreadsOf = kTile == kFewRows ? 512 : 256;
template <int kTile> constexpr int kJoinAtOnce = kTile == kFewRows ? 8 : 4;   // a thread's loads
template <int kTile> constexpr int kJoinRowsOf = kTile == kFewRows ? 16 : 32;   // of a block

// The sum of weights by the greater of two maxima. (A row that saw nothing has a maximum of
// -infinity and a sum of 0; one whose scores are all NaN, a sum of NaN.)
__device__ __forceinline__ float joined(float m, float l, float n, float k) {
    const float top = fmaxf(m, n);
    return (m == top ? l : l * ex2(m - top)) + (n == top ? k : k * ex2(n - top));
}

// Block (c, y): if the cut at the beginning of part c falls into an item (behind its first
// block), rows kJoinRows y and on of that item from all parts that computed some of it, in
// order; the blocks of all cuts in an item share its vectors, and where a block has fewer
// vectors than threads, threads share a vector's parts. What bounds it is the chain of
// loads from L2 (notes, then maxima, sums and vectors), a microsecond each: each is
// made for all parts at once.
template <bool kF16, int kTile>
__global__ void __launch_bounds__(kJoinThreadsOf<kTile>, kTile == kFewRows ? 2 : 4) paged_join_kernel(const __grid_constant__ AttnParams p) {
    constexpr int kJoinThreads = kJoinThreadsOf<kTile>, kJoinRows = kJoinRowsOf<kTile>, kMost = kTile == kFewRows ? kMostParts : kTileParts;
    __shared__ float s_w[kJoinRows][kMost + 1];   // a row's maxima, then weights
    __shared__ int s_part[kMost + 1];             // the item's parts: the part, negative (~part) in its first slot
    __shared__ int s_count[kJoinThreads / 32], s_from[kJoinThreads / 32], s_mine;
    rope3d_tc::grid_release();
    rope3d_tc::grid_wait();
    const int c = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    static_assert(kMost <= kJoinThreads, "a part to a thread");
    const PartNote n = p.notes[c];
    const long long begin = tid < p.parts ? p.notes[tid].begin : 0, end = tid < p.parts ? p.notes[tid].end : 0;
    const long long first = n.item + p.item_cost;   // the item's first block on the line
    if (n.begin == n.end || n.begin <= first) return;
    // The item's parts: the last that begins at or before its first block, and those that begin
    // behind that and in it (parts without blocks among them have none of it)
    const bool its = begin > first && begin < n.item + n.cost && begin < end;
    const uint32_t bits = __ballot_sync(0xffffffffu, its), at_first = __ballot_sync(0xffffffffu, begin <= first && begin < end);
    if (lane == 0) {
        s_count[warp] = __popc(bits);
        s_from[warp] = at_first ? warp * 32 + 31 - __clz(int(at_first)) : -1;
    }
    Item it;
    it.s = n.s;
    it.h = n.h;
    it.t = n.t;
    it.q = seq_of<kTile>(p, n.s);
    it.rows = int(min(uint32_t(kTile), uint32_t(it.q.n) * p.group.d - uint32_t(n.t) * kTile));
    __syncthreads();
    int before = 1 + __popc(bits & ((1u << lane) - 1u)), cuts = 0, from = 0;
    for (int w = 0; w < kJoinThreads / 32; ++w) {
        if (w < warp) before += s_count[w];
        cuts += s_count[w];
        from = max(from, s_from[w]);
    }
    if (its) s_part[before] = ~tid;
    if (tid == 0) s_part[0] = from;
    if (tid == c) s_mine = before - 1;   // which of the item's cuts this block's is
    __syncthreads();
    const int parts = cuts + 1, mine = s_mine;
    const int row0 = blockIdx.y * kJoinRows, rows = min(kJoinRows, it.rows - row0);
    if (rows <= 0) return;
    const int vecs = p.head_dim / 4, all = rows * vecs, i_begin = all * mine / cuts, i_end = all * (mine + 1) / cuts;
    const int count = i_end - i_begin;
    if (count == 0 && !(p.lse && mine == 0)) return;
    auto slot_at = [&](int k) {
        const int of = s_part[k];
        return slot_of<kTile>(p, of < 0 ? ~of : of, of < 0);
    };

    // each thread's first vectors are on their way while the weights are found
    int shares = 1;     // threads to a vector
    while (shares < 32 && 2 * shares * count <= kJoinThreads && 2 * shares <= parts) shares *= 2;
    const int share = tid % shares;
    constexpr int kAtOnce = kJoinAtOnce<kTile>;
    float4 x[kAtOnce];
    auto fetch = [&](int i, int k0) {
        const int r = i % rows, v4 = i / rows;
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k0 + j * shares < parts)
                x[j] = *reinterpret_cast<const float4 *>(slot_at(k0 + j * shares) + (v4 * kTile + row0 + r) * 4);
        }
    };
    const int i_first = i_begin + tid / shares;
    if (i_first < i_end) fetch(i_first, share);

    // a warp a row: the greatest maximum, the parts' weights by it, their sum
    for (int r = warp; r < rows; r += kJoinThreads / 32) {
        float top = -INFINITY, sum = 0.f;
        constexpr int kLoads = 4;
        for (int k0 = lane; k0 < parts; k0 += 32 * kLoads) {
            float m[kLoads], l[kLoads];
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const float *of = slot_at(min(k0 + 32 * j, parts - 1)) + vecs * kTile * 4 + row0 + r;
                m[j] = of[0];
                l[j] = of[kTile];
            }
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                if (k0 + 32 * j >= parts) break;
                s_w[r][k0 + 32 * j] = m[j];
                sum = joined(top, sum, m[j], l[j]);
                top = fmaxf(top, m[j]);
            }
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const float m = __shfl_xor_sync(0xffffffffu, top, d), l = __shfl_xor_sync(0xffffffffu, sum, d);
            sum = joined(top, sum, m, l);
            top = fmaxf(top, m);
        }
        const float inv = sum > 0.f ? 1.f / sum : sum, ref = top == -INFINITY ? 0.f : top;
        for (int k = lane; k < parts; k += 32) s_w[r][k] = ex2(s_w[r][k] - ref) * inv;
        if (lane == 0 && p.lse && mine == 0) {
            const RowOf row = row_of<kTile>(p, it, row0 + r);
            p.lse[row.token * p.lse_token + row.head] = lse_of(top, sum);
        }
    }
    __syncthreads();
    for (int i0 = i_begin; i0 < i_end; i0 += kJoinThreads / shares) {
        const int i = i0 + tid / shares, r = i % rows;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < i_end) {
            for (int k0 = share; k0 < parts; k0 += kAtOnce * shares) {   // (a part in which the row saw nothing has zeros)
                if (i0 > i_begin || k0 > share) fetch(i, k0);
#pragma unroll
                for (int j = 0; j < kAtOnce; ++j) {
                    if (k0 + j * shares >= parts) break;
                    const float w = s_w[r][k0 + j * shares];
                    v.x += x[j].x * w;
                    v.y += x[j].y * w;
                    v.z += x[j].z * w;
                    v.w += x[j].w * w;
                }
            }
        }
        for (int d = shares / 2; d; d >>= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, d);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, d);
            v.z += __shfl_xor_sync(0xffffffffu, v.z, d);
            v.w += __shfl_xor_sync(0xffffffffu, v.w, d);
        }
        if (i < i_end && share == 0) {
            const RowOf row = row_of<kTile>(p, it, row0 + r);
            store4<kF16>(p.out + row.token * p.out_token + row.head * p.out_head + i / rows * 8, v, 1.f);
        }
    }
}

// ---- host --------------------------------------------------------------------------

thread_local int t_paged_kernel = 0;   // 1 few rows, 2 tiles, 3 tiles of pairs

template <bool kF16, int kD>
int launch_rows(const AttnParams &p, cudaStream_t st) {
    static std::atomic<bool> ready[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return ROPE3D_ERR_CUDA;
    if (!ready[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(paged_rows_kernel<kF16, kD>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes<kD>) !=
            cudaSuccess) {
            cudaGetLastError();
            return ROPE3D_ERR_CUDA;
        }
        ready[dev].store(true, std::memory_order_release);
    }
    return launch(paged_rows_kernel<kF16, kD>, dim3(unsigned(p.parts)), kThreads, kSmemBytes<kD>, st, p);
}

template <bool kF16>
int launch_rows(const AttnParams &p, cudaStream_t st) {
    if (p.head_dim <= 64) return launch_rows<kF16, 64>(p, st);
    return p.head_dim <= 128 ? launch_rows<kF16, 128>(p, st) : launch_rows<kF16, 256>(p, st);
}

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

// How a call is computed: the kernel (0 few rows, 1 tiles, 2 tiles of pairs), its parts and
// its workspace.
struct Choice {
    int kind, rows, keys, parts;
    int64_t notes, bytes;
};

Choice choose(const rope3d_paged_attention_args &a) {
    const rope3d_paged_batch &b = a.batch;
    const int64_t group = a.q_heads / a.kv_heads;
    int64_t most = b.q_starts ? a.tokens : a.tokens / b.seqs;
    if (a.max_new) most = std::min(most, a.max_new);
    Choice c{};
    // By the rows that share keys, at the borders (us). Few rows / tiles: 32 sequences of 8192 places of 4 heads of
    // 128, 16 rows 94 / 137 (pairs), 24 rows 172 / 106; of 4 heads of 256, 177 / 201 and 333 / 198; of 8 heads of
    // 64, 109 / 147 and 166 / 149; 8 sequences of 2000 places of 4 heads of 256, 23 / 28 and 34 / 31. Tiles / pairs:
    // the first of these, 128 rows 112 / 140, 160 rows 195 / 141; the second, 211 / 214 and 371 / 219; the last,
    // 35 / 39 and 47 / 41. (Where all is short, few rows stay ahead for longer, by up to a third: 32 rows of one
    // sequence of 2000 places of 4 heads of 128 14 and 18, of 8192 17 and 24, 8 sequences of 2000 21 and 23; the
    // lengths are not known here. Tiles and pairs are then within 1 us of one another.)
    if (most * group > kFewRows && tiles_fit(a)) c.kind = most * group > kTileRows && pairs_fit(a) ? 2 : 1;
    c.rows = c.kind == 2 ? kPairRows : c.kind ? kTileRows : kFewRows;
    c.keys = c.kind == 2 ? 256 : c.kind ? 128 : kKeys;
    const int limit = c.kind == 2 ? kPairParts : c.kind ? kTileParts
                      : kTileParts * (a.head_dim <= 64 ? kPerSm<64> : a.head_dim <= 128 ? kPerSm<128> : kPerSm<256>);
    // no more parts than blocks there can be
    const int64_t items = (a.tokens * group + c.rows - 1) / c.rows + std::min(b.seqs, a.tokens);
    const int64_t blocks = (b.table_width * b.page_size + c.keys - 1) / c.keys;
    const int64_t most_blocks = items > limit || blocks > limit ? limit : items * blocks * a.kv_heads;
    c.parts = int(std::min<int64_t>(limit, most_blocks));
    c.notes = up256(int64_t(c.parts) * int64_t(sizeof(PartNote)));
    const int d = int(a.head_dim);
    const int64_t floats = c.kind == 2 ? slot_floats<kPairRows>(d) : c.kind ? slot_floats<kTileRows>(d) : slot_floats<kFewRows>(d);
    c.bytes = c.notes + up256(2 * c.parts * floats * 4);
    return c;
}

template <bool kF16>
int launch_join(const AttnParams &p, const Choice &c, cudaStream_t st) {
    auto *join = c.kind == 2 ? paged_join_kernel<kF16, kPairRows> : c.kind ? paged_join_kernel<kF16, kTileRows>
                                                                           : paged_join_kernel<kF16, kFewRows>;
    const int rows = c.kind ? kJoinRowsOf<kTileRows> : kJoinRowsOf<kFewRows>;
    const int threads = c.kind ? kJoinThreadsOf<kTileRows> : kJoinThreadsOf<kFewRows>;
    return launch(join, dim3(unsigned(c.parts), unsigned(c.rows / rows)), threads, 0, st, p);
}

int attention(const rope3d_paged_attention_args *a, bool go, bool check_device, int64_t *need, cudaStream_t st) {
    if (!a || !a->q || !a->k_cache || !a->v_cache || !a->out) return ROPE3D_ERR_NULL;
    const rope3d_paged_batch &b = a->batch;
    const int64_t T = a->tokens, H = a->q_heads, K = a->kv_heads, D = a->head_dim;
    if (T <= 0 || T > kMaxTokens || H <= 0 || H > kMaxHeads || K <= 0 || K > H || H % K != 0 || D <= 0 || D > 256 || D % 8 != 0 ||
        T * H > 0x7fffffff)
        return ROPE3D_ERR_SHAPE;
    int rc = check_batch(b, T);
    if (rc != ROPE3D_OK) return rc;
    if (a->dtype != ROPE3D_BF16 && a->dtype != ROPE3D_F16) return ROPE3D_ERR_DTYPE;
    const float scale = float(a->scale * 1.4426950408889634);
    if (!(scale > 0.f) || !std::isfinite(scale) || (a->causal != 0 && a->causal != 1) || a->window < 0 || a->max_new < 0)
        return ROPE3D_ERR_ARG;
    const View q = view(a->q, 2, D, T, a->q_token_stride, H, a->q_head_stride);
    const View out = view(a->out, 2, D, T, a->out_token_stride, H, a->out_head_stride);
    const View k = view(a->k_cache, 2, D, b.pages, a->k_page_stride, b.page_size, a->k_slot_stride, K, a->k_cache_head_stride);
    const View v = view(a->v_cache, 2, D, b.pages, a->v_page_stride, b.page_size, a->v_slot_stride, K, a->v_cache_head_stride);
    const View lse = view(a->lse, 4, H, T, a->lse_stride);
    const View table = view(b.page_table, 4, b.table_width, b.seqs, b.table_stride), lens = view(b.seq_lens, 4, b.seqs, 1, 0),
               starts = view(b.q_starts, 4, b.seqs + 1, 1, 0);
    if (bad_strides(q) || bad_strides(out) || bad_strides(k) || bad_strides(v) || !rows_apart(out) ||
        (a->lse && (bad_strides(lse) || !rows_apart(lse))))
        return ROPE3D_ERR_SHAPE;
    if (!vectors(q) || !vectors(out) || !vectors(k) || !vectors(v) || !aligned(a->lse, 4)) return ROPE3D_ERR_ALIGN;
    const Choice c = choose(*a);
    if (need) *need = c.bytes;
    else if (!a->workspace) return ROPE3D_ERR_NULL;
    else if (a->workspace_bytes < c.bytes) return ROPE3D_ERR_SCRATCH;
    if (!need && !aligned(a->workspace, 256)) return ROPE3D_ERR_ALIGN;
    const View ws{need ? nullptr : a->workspace, c.bytes, {1, 1, 1}, {0, 0, 0}, 1};
    for (const View *o : {&out, &lse, &ws})
        for (const View *in : {&q, &k, &v, &table, &lens, &starts})
            if (may_meet(*o, *in)) return ROPE3D_ERR_ALIAS;
    if (may_meet(out, lse) || may_meet(out, ws) || may_meet(lse, ws)) return ROPE3D_ERR_ALIAS;
    if (check_device) {
        const void *const all[] = {a->q, a->k_cache, a->v_cache, a->out, a->lse, b.page_table, b.seq_lens, b.q_starts, a->workspace};
        if ((rc = on_current_device(all, 9)) != ROPE3D_OK) return rc;
    }
    if (need || !go) return ROPE3D_OK;

    AttnParams p{};
    p.q = static_cast<const char *>(a->q);
    p.k = static_cast<const char *>(a->k_cache);
    p.v = static_cast<const char *>(a->v_cache);
    p.out = static_cast<char *>(a->out);
    p.lse = a->lse;
    p.batch = device_batch(b, T);
    p.group = rope3d::make_fastdiv(uint32_t(H / K));
    p.page = rope3d::make_fastdiv(uint32_t(b.page_size));
    p.span = rope3d::make_fastdiv(uint32_t(H / K) * uint32_t(c.keys / c.rows));
    p.cuts = rope3d::make_fastdiv(uint32_t(c.parts));
    // An item's beginning and end, in blocks of the line. Measured, us at 0 / 1 / 2 / 3: pairs, 8192 x 8192
    // causal of 8 / 4 heads of 256 222 / 200 / 207 / 213, 13 ragged chunks of 16 / 2 heads of 128 920 / 776 /
    // 744 / 743; tiles, 8192 x 8192 of 16 / 4 heads of 64 229 / 203 / 194 / 197; few rows, 64 sequences
    // of 32 / 8 heads of 128 329 / 323 / 319 / 318.
    p.item_cost = c.kind == 0 ? 3 : c.kind == 2 && D > 128 ? 1 : 2;
    p.kv_heads = int(K);
    p.head_dim = int(D);
    p.causal = a->causal;
    p.window = int(std::min<int64_t>(a->window, kMaxPlaces));   // a longer one leaves nothing out
    if (a->window > kMaxPlaces) p.window = 0;
    p.q_token = a->q_token_stride * 2;
    p.q_head = a->q_head_stride * 2;
    p.out_token = a->out_token_stride * 2;
    p.out_head = a->out_head_stride * 2;
    p.lse_token = a->lse_stride;
    p.k_page = a->k_page_stride * 2;
    p.k_slot = a->k_slot_stride * 2;
    p.k_head = a->k_cache_head_stride * 2;
    p.v_page = a->v_page_stride * 2;
    p.v_slot = a->v_slot_stride * 2;
    p.v_head = a->v_cache_head_stride * 2;
    p.scale_log2 = scale;
    p.parts = c.parts;
    p.notes = static_cast<PartNote *>(a->workspace);
    p.partial = reinterpret_cast<float *>(static_cast<char *>(a->workspace) + c.notes);
    const bool f16 = a->dtype == ROPE3D_F16;
    if (c.kind) rc = launch_tiles(p, *a, c.kind == 2, st);
    else rc = f16 ? launch_rows<true>(p, st) : launch_rows<false>(p, st);
    if (rc != ROPE3D_OK) return rc;
    t_paged_kernel = c.kind + 1;
    return f16 ? launch_join<true>(p, c, st) : launch_join<false>(p, c, st);
}

}  // namespace

extern "C" int rope3d_paged_attention(const rope3d_paged_attention_args *args, void *stream) {
    return attention(args, true, true, nullptr, static_cast<cudaStream_t>(stream));
}

extern "C" int rope3d_paged_attention_check(const rope3d_paged_attention_args *args, int32_t check_device) {
    return attention(args, false, check_device != 0, nullptr, nullptr);
}

extern "C" int rope3d_paged_attention_workspace(const rope3d_paged_attention_args *args, int64_t *bytes) {
    if (!bytes) return ROPE3D_ERR_NULL;
    return attention(args, false, false, bytes, nullptr);
}

extern "C" int rope3d_paged_attention_last_kernel(void) { return t_paged_kernel; }

extern "C" int rope3d_testing_paged_wait_timeouts(int64_t *count, int32_t reset) {
    if (!count) return ROPE3D_ERR_NULL;
    unsigned int n = 0;
    if (tiles_wait_timeouts(&n, reset != 0) != 0) return ROPE3D_ERR_CUDA;
    *count = n;
    return ROPE3D_OK;
}
