// rope3d_norm.cuh -- what the forward (rope3d_norm.cu) and backward
// (rope3d_norm_back.cu) kernels of the norms around a transformer block share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <type_traits>

#include "../../include/rope3d.h"
#include "rope3d_internal.h"
#include "rope3d_tc.cuh"

namespace rope3d_norm {

using rope3d_tc::drain;
using rope3d_tc::grid_release;
using rope3d_tc::grid_wait;
using rope3d_tc::mbar_expect_tx;
using rope3d_tc::mbar_fence_init;
using rope3d_tc::mbar_init;
using rope3d_tc::mbar_wait;
using rope3d_tc::smem_u32;

// Bounded waits that ran out, counted in each of the two files
// (rope3d_testing_norm_wait_timeouts).
static __device__ unsigned int g_norm_wait_timeouts;

struct NormParams {
    const void *x, *y, *post_weight, *gate, *pre_weight, *scale, *shift;
    void *r, *n;
    const void *dr, *dn;
    void *dx, *dy;
    void *d_post_weight, *d_gate, *d_pre_weight, *d_scale, *d_shift;
    long long ldx, ldy, ldr, ldn, ldg, ldsc, ldsh, lddr, lddn, lddx, lddy, ldgrad;
    int rows, channels, rows_per_group, groups;
    float eps, res, offset;
    int post, pre;        // ROPE3D_NORM_*
    int dtype, param_f32;
    // backward: chunks of rows and their partial column sums
    float *part;          // [chunks][3][channels]: sums of a part of a group, or the weights' sums of whole groups
    float *group_sums;    // [groups][2][channels]: the groups' parts of the weights' gradients
    float *stats;         // general kernels: [rows][6], then [rows][2] (mean f, mean f yh)
    int chunk_rows, chunks_per_group, groups_per_chunk, chunks;
    int sums;             // column sums are wanted
    int stages;           // ring kernels: rows in shared memory
};

// ---- elements -------------------------------------------------------------------

// One bf16 value. (Not as bits << 16: right behind a 16-bit load that shift makes
// the loads wait for one another; 8000 x 2049, backward: 375 us instead of 159.)
__device__ __forceinline__ float from_bf16(uint16_t v) { return __bfloat162float(__ushort_as_bfloat16(v)); }

__device__ __forceinline__ float load1(const void *p, long long i, int dtype) {
    if (dtype == ROPE3D_F32) return static_cast<const float *>(p)[i];
    const uint16_t v = static_cast<const uint16_t *>(p)[i];
    return dtype == ROPE3D_F16 ? __half2float(__ushort_as_half(v)) : from_bf16(v);
}

__device__ __forceinline__ void store1(void *p, long long i, float v, int dtype) {
    if (dtype == ROPE3D_F32) static_cast<float *>(p)[i] = v;
    else
        static_cast<uint16_t *>(p)[i] = dtype == ROPE3D_F16 ? __half_as_ushort(__float2half_rn(v))
                                                             : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

template <int kT>
constexpr int kPer = kT == ROPE3D_F32 ? 4 : 8;   // elements of a 16-byte vector

template <int kT>
__device__ __forceinline__ void unpack(const uint4 &v, float *f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kT == ROPE3D_F32) {
            f[i] = __uint_as_float(w[i]);
        } else if constexpr (kT == ROPE3D_BF16) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
            __half2 h;
            memcpy(&h, &w[i], 4);
            const float2 t = __half22float2(h);
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        }
    }
}

template <int kT>
__device__ __forceinline__ uint4 pack(const float *f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kT == ROPE3D_F32) {
            w[i] = __float_as_uint(f[i]);
        } else if constexpr (kT == ROPE3D_BF16) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            memcpy(&w[i], &b, 4);
        } else {
            const __half2 b = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            memcpy(&w[i], &b, 4);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Row data: read once, not kept in L1 beside the parameters.
__device__ __forceinline__ uint4 ld_row(const void *base, long long elem, int elem_bytes) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(static_cast<const char *>(base) + elem * elem_bytes)
                 : "memory");
    return r;
}

__device__ __forceinline__ void st_row(void *base, long long elem, int elem_bytes, const uint4 &v) {
    asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(static_cast<char *>(base) + elem * elem_bytes),
                 "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

// kPer<kT> parameters from element i, fp32 or of the rows' type; `fill` where
// the parameter is absent.
template <int kT>
__device__ __forceinline__ void ld_param(const void *base, long long i, bool f32, float fill, float *f) {
    constexpr int V = kPer<kT>;
    if (!base) {
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = fill;
    } else if (f32 || kT == ROPE3D_F32) {
        const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + i);
#pragma unroll
        for (int j = 0; j < V / 4; ++j) {
            const float4 t = s[j];
            f[4 * j] = t.x; f[4 * j + 1] = t.y; f[4 * j + 2] = t.z; f[4 * j + 3] = t.w;
        }
    } else {
        unpack<kT>(*reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + i), f);
    }
}

// The weights of a norm plus their offset; ones where there is no weight.
template <int kT>
__device__ __forceinline__ void ld_weight(const void *base, long long i, bool f32, float offset, float *f) {
    ld_param<kT>(base, i, f32, 1.0f, f);
    if (base)
#pragma unroll
        for (int j = 0; j < kPer<kT>; ++j) f[j] += offset;
}

template <int kT>
__device__ __forceinline__ void st_param(void *base, long long i, bool f32, const float *f) {
    constexpr int V = kPer<kT>;
    if (f32 || kT == ROPE3D_F32) {
#pragma unroll
        for (int j = 0; j < V; j += 4)
            *reinterpret_cast<float4 *>(static_cast<float *>(base) + i + j) =
                make_float4(f[j], f[j + 1], f[j + 2], f[j + 3]);
    } else {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + i) = pack<kT>(f);
    }
}

// ---- teams ---------------------------------------------------------------------------

// A team is kTeam threads: 8 or 32 neighbouring lanes, a block of a fixed size
// above 32, or (0) a block of any size.
__host__ __device__ constexpr bool is_block(int team) { return team == 0 || team > 32; }

// Sums of kN values over the threads of a team: by shuffles, and for a block
// through shared memory (two alternating slots: one barrier a sum). Every thread
// gets the result; warps are added in order.
template <int kTeam>
struct Sums {
    float *red;   // [2][2][32]
    int slot;
    template <int kN>
    __device__ __forceinline__ void operator()(float (&v)[kN]) {
        constexpr int kFirst = is_block(kTeam) ? 16 : kTeam / 2;
        // (a team's lanes only: another team of the warp may have fewer rows)
        const uint32_t mask =
            kTeam == 8 ? 0xffu << (threadIdx.x & 24) : 0xffffffffu;
#pragma unroll
        for (int o = kFirst; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < kN; ++i) v[i] += __shfl_xor_sync(mask, v[i], o);
        if constexpr (is_block(kTeam)) {
            float *s = red + slot * 2 * 32;
            slot ^= 1;
            const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = (blockDim.x + 31) >> 5;
            if (lane == 0)
#pragma unroll
                for (int i = 0; i < kN; ++i) s[i * 32 + warp] = v[i];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                v[i] = lane < warps ? s[i * 32 + lane] : 0.0f;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
            }
        }
    }
};

// The threads of a row: `size` of them, and this one's place; teams of the block.
template <int kTeam>
struct TeamOf {
    int size, lane, team, teams;
    __device__ __forceinline__ TeamOf()
        : size(kTeam ? kTeam : int(blockDim.x)),
          lane(is_block(kTeam) ? int(threadIdx.x) : int(threadIdx.x) & (kTeam - 1)),
          team(is_block(kTeam) ? 0 : int(threadIdx.x) / (kTeam ? kTeam : 1)),
          teams(is_block(kTeam) ? 1 : int(blockDim.x) / (kTeam ? kTeam : 1)) {}
};

// kE elements of a row that one thread holds: vectors of 16 bytes (kVec), or
// single elements where rows are not whole aligned vectors; piece j is W elements
// from channel (lane + j * size) * W on. Work goes by batches of 8 elements.
// Single elements want a team of a fixed size, so that their addresses are one
// address and constants.
template <int kT, bool kVec, int kE>
struct RowPart {
    static constexpr int W = kVec ? kPer<kT> : 1, N = kE / W, PB = 8 / W, kBytes = kT == ROPE3D_F32 ? 4 : 2;
    using Raw = std::conditional_t<kVec, uint4, std::conditional_t<kT == ROPE3D_F32, uint32_t, uint16_t>>;
    Raw raw[N];

    static __device__ __forceinline__ int chan(int lane, int size, int j) { return (lane + j * size) * W; }
    // the row at `at` of base; zeros without one
    __device__ __forceinline__ void load(const void *base, long long at, int lane, int size, int channels) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int c = chan(lane, size, j);
            if constexpr (kVec) {
                raw[j] = base && c < channels ? ld_row(base, at + c, kBytes) : make_uint4(0, 0, 0, 0);
            } else {
                raw[j] = base && c < channels ? (static_cast<const Raw *>(base) + at + lane)[j * size] : Raw(0);
            }
        }
    }
    // batch b
    __device__ __forceinline__ void get(int b, float *f) const {
#pragma unroll
        for (int j = 0; j < PB; ++j) {
            if constexpr (kVec) unpack<kT>(raw[b * PB + j], f + j * W);
            else if constexpr (kT == ROPE3D_F32) f[j] = __uint_as_float(raw[b * PB + j]);
            else if constexpr (kT == ROPE3D_BF16) f[j] = from_bf16(raw[b * PB + j]);
            else f[j] = __half2float(__ushort_as_half(raw[b * PB + j]));
        }
    }
    static __device__ __forceinline__ void put(void *base, long long at, int lane, int size, int channels, int b,
                                               const float *f) {
#pragma unroll
        for (int j = 0; j < PB; ++j) {
            const int c = chan(lane, size, b * PB + j);
            if (c >= channels) continue;
            if constexpr (kVec) st_row(base, at + c, kBytes, pack<kT>(f + j * W));
            else if constexpr (kT == ROPE3D_F32) (static_cast<float *>(base) + at + lane)[(b * 8 + j) * size] = f[j];
            else
                (static_cast<uint16_t *>(base) + at + lane)[(b * 8 + j) * size] =
                    kT == ROPE3D_F16 ? __half_as_ushort(__float2half_rn(f[j])) : __bfloat16_as_ushort(__float2bfloat16_rn(f[j]));
        }
    }
    // 8 parameters from a row of them (fp32 or of the rows' type); `fill` where
    // there are none, anything at absent channels
    static __device__ __forceinline__ void param(const void *base, long long at, bool f32, float fill, int lane, int size,
                                                 int channels, int b, float *f) {
        if (!base) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = fill;
        } else if constexpr (kVec) {
#pragma unroll
            for (int j = 0; j < PB; ++j) {
                const int c = chan(lane, size, b * PB + j);
                ld_param<kT>(base, at + (c < channels ? c : 0), f32, fill, f + j * W);
            }
        } else if (f32 || kT == ROPE3D_F32) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f[j] = chan(lane, size, b * 8 + j) < channels
                           ? (static_cast<const float *>(base) + at + lane)[(b * 8 + j) * size] : 0.0f;
        } else {
            uint16_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[j] = chan(lane, size, b * 8 + j) < channels
                           ? (static_cast<const uint16_t *>(base) + at + lane)[(b * 8 + j) * size] : uint16_t(0);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f[j] = kT == ROPE3D_BF16 ? from_bf16(w[j]) : __half2float(__ushort_as_half(w[j]));
        }
    }
    static __device__ __forceinline__ void weight(const void *base, bool f32, float offset, int lane, int size, int channels,
                                                  int b, float *f) {
        param(base, 0, f32, 1.0f, lane, size, channels, b, f);
        if (base)
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] += offset;
    }
    static __device__ __forceinline__ void put_param(void *base, long long at, bool f32, int lane, int size, int channels,
                                                     int b, const float *f) {
#pragma unroll
        for (int j = 0; j < PB; ++j) {
            const int c = chan(lane, size, b * PB + j);
            if (c >= channels) continue;
            if constexpr (kVec) st_param<kT>(base, at + c, f32, f + j * W);
            else store1(base, at + c, f[j], f32 ? ROPE3D_F32 : kT);
        }
    }
};

// Mean and 1 / std of the row v (kE elements a thread); real(i): element i exists.
template <int kE, int kTeam, typename Real>
__device__ __forceinline__ void row_stats(const float *v, int kind, Real real, float inv_c, float eps,
                                          Sums<kTeam> &sum, float *mean, float *k) {
    *mean = 0.0f;
    *k = 1.0f;
    if (kind == ROPE3D_NORM_NONE) return;
    float s[1] = {0.0f};
    if (kind == ROPE3D_NORM_LAYER) {
#pragma unroll
        for (int i = 0; i < kE; ++i) s[0] += v[i];   // absent elements are zero
        sum(s);
        *mean = s[0] * inv_c;
        s[0] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kE; ++i) {
        const float d = real(i) ? v[i] - *mean : 0.0f;
        s[0] += d * d;
    }
    sum(s);
    *k = rsqrtf(s[0] * inv_c + eps);
}

// ---- any row ---------------------------------------------------------------------------

// One element of a row, from its statistics.
struct RowOps {
    const NormParams &p;
    long long row;
    int g;
    float my, ky, mr, kr;   // mean and 1 / std of y and r
    __device__ __forceinline__ float param(const void *b, long long i, float fill) const {
        return b ? load1(b, i, p.param_f32 ? ROPE3D_F32 : p.dtype) : fill;
    }
    __device__ __forceinline__ float wp(int c) const {
        return p.post_weight ? param(p.post_weight, c, 0.0f) + p.offset : 1.0f;
    }
    __device__ __forceinline__ float wq(int c) const {
        return p.pre_weight ? param(p.pre_weight, c, 0.0f) + p.offset : 1.0f;
    }
    __device__ __forceinline__ float gate(int c) const { return param(p.gate, g * p.ldg + c, 1.0f); }
    __device__ __forceinline__ float scale1(int c) const { return 1.0f + param(p.scale, g * p.ldsc + c, 0.0f); }
    __device__ __forceinline__ float yh(int c) const {
        return (load1(p.y, row * p.ldy + c, p.dtype) - my) * ky;
    }
    __device__ __forceinline__ float r(int c) const {
        float v = p.res * load1(p.x, row * p.ldx + c, p.dtype);
        if (p.y) v += gate(c) * (yh(c) * wp(c));
        return v;
    }
    __device__ __forceinline__ float z(int c) const { return (r(c) - mr) * kr; }
    __device__ __forceinline__ float dn(int c) const { return p.dn ? load1(p.dn, row * p.lddn + c, p.dtype) : 0.0f; }
    __device__ __forceinline__ float e(int c) const { return dn(c) * wq(c) * scale1(c); }
};

// Statistics of a row read element by element: get(c) for each of its channels.
template <typename Get, typename Sum>
__device__ __forceinline__ void scan_stats(Get get, const NormParams &p, int kind, Sum &sum, float *mean, float *k) {
    *mean = 0.0f;
    *k = 1.0f;
    if (kind == ROPE3D_NORM_NONE) return;
    const float inv_c = 1.0f / float(p.channels);
    if (kind == ROPE3D_NORM_LAYER) {
        float s[2] = {0.0f, 0.0f};
        for (int c = threadIdx.x; c < p.channels; c += blockDim.x) s[0] += get(c);
        sum(s);
        *mean = s[0] * inv_c;
    }
    float s[2] = {0.0f, 0.0f};
    for (int c = threadIdx.x; c < p.channels; c += blockDim.x) {
        const float d = get(c) - *mean;
        s[0] += d * d;
    }
    sum(s);
    *k = rsqrtf(s[0] * inv_c + p.eps);
}

constexpr int kGeneralThreads = 256;

// ---- many rows: rows through a ring in shared memory -------------------------------------------
//
// A row's bytes have to arrive before its statistics, and its statistics before
// its results, so a team that loads a row when it gets to it waits for memory in
// every row. Here one thread keeps a ring of whole rows on the way into shared
// memory (bulk copies that complete on an mbarrier), a few rows ahead of the
// team, and several teams share an SM. Forward, a block takes a contiguous range
// of rows; backward, one chunk. Of the parameters a row needs only
//   m = gate * wp,  q = wq * (1 + scale)  (and shift, forward),
// which stay in shared memory until the group changes. A thread owns 16 channels
// and works on pairs of them with packed fp32 arithmetic: the kernels would
// otherwise be bound by instruction issue, not by memory.
constexpr int kRingE = 16;
constexpr int kRingBars = 8;   // most stages

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long x, y, z, d;
    memcpy(&x, &a, 8);
    memcpy(&y, &b, 8);
    memcpy(&z, &c, 8);
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
    memcpy(&a, &d, 8);
    return a;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long x, y, d;
    memcpy(&x, &a, 8);
    memcpy(&y, &b, 8);
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
    memcpy(&a, &d, 8);
    return a;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long x, y, d;
    memcpy(&x, &a, 8);
    memcpy(&y, &b, 8);
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
    memcpy(&a, &d, 8);
    return a;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

template <int kT>
__device__ __forceinline__ void unpack2(const uint4 &v, float2 *f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (kT == ROPE3D_F32) {
        f[0] = make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
        f[1] = make_float2(__uint_as_float(w[2]), __uint_as_float(w[3]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kT == ROPE3D_BF16) {
                f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
            } else {
                __half2 h;
                memcpy(&h, &w[i], 4);
                f[i] = __half22float2(h);
            }
        }
    }
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void bulk_row(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// This thread's 16 values of one fp32 array in shared memory: 16-byte pieces,
// each piece contiguous over the threads.
struct Kept {
    uint32_t base;   // + this thread's 16 bytes
    uint32_t step;   // bytes of one piece of all threads
    // kPairs pairs from pair kPairs * j on
    template <int kPairs>
    __device__ __forceinline__ void load_part(int j, float2 *f) const {
#pragma unroll
        for (int i = 0; i < kPairs / 2; ++i) {
            const uint4 v = lds128(base + uint32_t(j * kPairs / 2 + i) * step);
            f[2 * i] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
            f[2 * i + 1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
        }
    }
    __device__ __forceinline__ void load(float2 *f) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 v = lds128(base + uint32_t(i) * step);
            f[2 * i] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
            f[2 * i + 1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
        }
    }
    __device__ __forceinline__ void store(const float *f) const {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(base + uint32_t(i) * step), "f"(f[4 * i]),
                         "f"(f[4 * i + 1]), "f"(f[4 * i + 2]), "f"(f[4 * i + 3]) : "memory");
    }
};

// Sums over a block of two values a thread: the warp's by shuffles that fold
// both values into one (the halves of a warp take one value each), then the
// warps' pairs in order, read as vectors. Two alternating slots: one barrier a
// sum. `warps` rounded up to an even number; a slot past the last warp is zero.
struct BlockSums {
    float2 *red;   // [2][16]
    int slot, warps;
    __device__ __forceinline__ float2 operator()(float a, float b) {
        const bool upper = threadIdx.x & 16;
        const float other = __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
        float v = (upper ? b : a) + other;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        float2 *s = red + slot * 16;
        slot ^= 1;
        if ((threadIdx.x & 15) == 0) reinterpret_cast<float *>(s + (threadIdx.x >> 5))[upper ? 1 : 0] = v;
        __syncthreads();
        float2 t = make_float2(0.0f, 0.0f);
        for (int w = 0; w < warps; w += 2) {
            const float4 q = *reinterpret_cast<const float4 *>(s + w);
            t = add2(t, add2(make_float2(q.x, q.y), make_float2(q.z, q.w)));
        }
        return t;
    }
    __device__ __forceinline__ float one(float a) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
        float *s = reinterpret_cast<float *>(red + slot * 16);
        slot ^= 1;
        if ((threadIdx.x & 31) == 0) s[2 * (threadIdx.x >> 5)] = a;
        __syncthreads();
        float t = 0.0f;
        for (int w = 0; w < warps; w += 2) {
            const float4 q = *reinterpret_cast<const float4 *>(s + 2 * w);
            t += q.x + q.z;
        }
        return t;
    }
};

__device__ __forceinline__ float fold(float2 v) { return v.x + v.y; }

struct Ring {
    uint32_t base, bars, row_bytes, stage_bytes;
    int stages;
};

// What the two ring kernels share: the ring, the group's parameters in shared
// memory, this thread's channels. kFull: every thread owns 16 channels (else
// some own fewer, and `real` says which vectors exist).
template <int kT, bool kFull>
struct RingTeam {
    static constexpr int V = kPer<kT>, kVecs = kRingE / V, P = V / 2, H = kRingE / 2, kBytes = 16 / V;
    const NormParams &p;
    int size, tid;
    bool real_[kVecs];
    float inv_c;
    uint32_t base;

    __device__ __forceinline__ RingTeam(const NormParams &params, const uint8_t *raw)
        : p(params), size(int(blockDim.x)), tid(int(threadIdx.x)), inv_c(1.0f / float(params.channels)),
          base((smem_u32(raw) + 127u) & ~127u) {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) real_[j] = tid + j * size < params.channels / V;
    }
    __device__ __forceinline__ bool real(int j) const { return kFull || real_[j]; }
    __device__ __forceinline__ int channel(int j) const { return (tid + j * size) * V; }
    __device__ __forceinline__ Kept kept(int i) const {
        return Kept{base + uint32_t(i) * 64u * uint32_t(size) + 16u * uint32_t(tid), 16u * uint32_t(size)};
    }
    // vector j of this thread in a row in shared memory; zeros where absent
    __device__ __forceinline__ uint4 read(uint32_t row, int j) const {
        return real(j) ? lds128(row + 16u * uint32_t(tid + j * size)) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void unpack_row(uint32_t row, float2 *f) const {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) unpack2<kT>(read(row, j), f + j * P);
    }
    __device__ __forceinline__ void write(void *out, long long at, const float2 *f) const {
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
            if (real(j)) st_row(out, at + channel(j), kBytes, pack<kT>(reinterpret_cast<const float *>(f + j * P)));
    }
    // m = gate * wp and q = wq * (1 + scale) of group g; zero for absent channels
    __device__ __forceinline__ void group(int g, float *m, float *q) const {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            const int c = real(j) ? channel(j) : 0;
            float a[V];
            ld_weight<kT>(p.post_weight, c, p.param_f32, p.offset, m + j * V);
            ld_param<kT>(p.gate, g * p.ldg + c, p.param_f32, 1.0f, a);
#pragma unroll
            for (int i = 0; i < V; ++i) m[j * V + i] = real(j) ? m[j * V + i] * a[i] : 0.0f;
            ld_weight<kT>(p.pre_weight, c, p.param_f32, p.offset, q + j * V);
            ld_param<kT>(p.scale, g * p.ldsc + c, p.param_f32, 0.0f, a);
#pragma unroll
            for (int i = 0; i < V; ++i) q[j * V + i] = real(j) ? q[j * V + i] * (1.0f + a[i]) : 0.0f;
        }
    }
    // v minus its mean (layer norm): absent channels stay zero
    __device__ __forceinline__ void center(float2 *v, float mean) const {
        const float2 m = both(-mean);
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
            if (real(j))
#pragma unroll
                for (int i = 0; i < P; ++i) v[j * P + i] = add2(v[j * P + i], m);
    }
    static __device__ __forceinline__ float total(const float2 *v) {
        float2 t = v[0];
#pragma unroll
        for (int i = 1; i < H; ++i) t = add2(t, v[i]);
        return fold(t);
    }
    static __device__ __forceinline__ float dot(const float2 *v, const float2 *w) {
        float2 t = mul2(v[0], w[0]);
#pragma unroll
        for (int i = 1; i < H; ++i) t = fma2(v[i], w[i], t);
        return fold(t);
    }
    // v normalised in place; returns 1 / std
    template <bool kLayer>
    __device__ __forceinline__ float normalise(float2 *v, int kind, BlockSums &sum) const {
        if (kLayer && kind == ROPE3D_NORM_LAYER) center(v, sum.one(total(v)) * inv_c);
        const float k = rsqrtf(sum.one(dot(v, v)) * inv_c + p.eps);
        const float2 k2 = both(k);
#pragma unroll
        for (int i = 0; i < H; ++i) v[i] = mul2(v[i], k2);
        return k;
    }
};

// ---- kernels of the two files -----------------------------------------------------------

using NormFn = void (*)(NormParams);

// The backward kernels: rows in registers (vec: whole aligned vectors; elements of
// a thread; team), rows through the ring, and the general ones.
NormFn back_team_fn(int dtype, bool vec, int elems, int team);
NormFn back_ring_fn(int dtype, bool layer, bool full, bool shift);
NormFn back_any_fn();
NormFn back_cols_fn();
NormFn finish_fn(int rows);   // 8, 16 or 32 rows of 32 threads
NormFn groups_fn();

// The backward file's count of waits that ran out; a CUDA error code.
int back_wait_timeouts(unsigned int *count, bool reset);

}  // namespace rope3d_norm
