// rope3d_norm.cu -- the norms around a transformer block: rope3d_block_norm and
// its backward pass.
//
//   r = res * x + gate_g * post(y) * wp,   n = pre(r) * wq * (1 + scale_g) + shift_g
// (wp, wq: the weights plus their offset; g: the row's group). Backward, with
// yh = (y - mean) k_y and z = (r - mean) k_r the normalised rows, k = 1 / std:
//   e  = dn * wq * (1 + scale_g)
//   dR = dr + k_r (e - mean(e) - z mean(e z))          the whole gradient of r
//   f  = dR * gate_g * wp
//   dx = res * dR,  dy = k_y (f - mean(f) - yh mean(f yh))
// (the plain means of e and f only in a layer norm; identity norms pass e and f
// through) and, per channel,
//   S_g = sum dn z, T_g = sum dn, U_g = sum dR yh   over the rows of group g:
//   d_scale_g = wq S_g, d_shift_g = T_g, d_gate_g = wp U_g,
//   d_pre_weight = sum_g (1 + scale_g) S_g, d_post_weight = sum_g gate_g U_g,
// so that three sums give all five parameter gradients.
//
// Every operation is element-wise or a sum along one row, 2-4 streams of bytes
// forward and up to 6 backward for some 12-30 flops an element: bound by memory.
// A team of threads (a warp, or a block) keeps a row in registers from its one
// read to its one write, statistics included; the backward pass computes the
// statistics again instead of reading saved ones, and keeps its threads on the
// same channels for a whole chunk of rows, so that the three column sums stay
// in registers too. Chunks leave partial sums in a workspace, added in chunk
// order by a second small kernel: no atomics, the same bits every time.
// Rows that are no multiple of 16 bytes, unaligned or too long for registers
// take general kernels that read a row once for each of its sums.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/rope3d.h"
#include "rope3d_internal.h"
#include "rope3d_tc.cuh"

namespace {

using rope3d_tc::grid_release;
using rope3d_tc::grid_wait;
using rope3d_tc::mbar_expect_tx;
using rope3d_tc::mbar_fence_init;
using rope3d_tc::mbar_init;
using rope3d_tc::mbar_wait;
using rope3d_tc::smem_u32;

// Bounded waits that ran out (rope3d_testing_norm_wait_timeouts).
__device__ unsigned int g_norm_wait_timeouts;

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
    float *stats;         // general kernels: [rows][6]
    int chunk_rows, chunks_per_group, groups_per_chunk, chunks;
    int sums;             // column sums are wanted
    int stages;           // ring kernels: rows in shared memory
};

// ---- elements -------------------------------------------------------------------

__device__ __forceinline__ float load1(const void *p, long long i, int dtype) {
    if (dtype == ROPE3D_F32) return static_cast<const float *>(p)[i];
    const uint16_t v = static_cast<const uint16_t *>(p)[i];
    return dtype == ROPE3D_F16 ? __half2float(__ushort_as_half(v)) : __uint_as_float(uint32_t(v) << 16);
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

// ---- sums over a team --------------------------------------------------------------

// kN sums over the threads of a team: a warp, or a whole block through shared
// memory (two alternating slots: one barrier a sum). Every thread gets the
// result; warps are added in order.
template <int kN, bool kWarp>
struct Sums {
    float *red;   // [2][kN][32]
    int slot;
    __device__ __forceinline__ void operator()(float *v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < kN; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        if constexpr (!kWarp) {
            float *s = red + slot * kN * 32;
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

// ---- forward, rows in registers -------------------------------------------------------

// Mean and 1 / std of the row v (kE elements a thread, `mine` of them real).
template <int kE, int kN, bool kWarp>
__device__ __forceinline__ void row_stats(const float *v, int kind, bool const *real, int per, float inv_c,
                                          float eps, Sums<kN, kWarp> &sum, float *mean, float *k) {
    *mean = 0.0f;
    *k = 1.0f;
    if (kind == ROPE3D_NORM_NONE) return;
    float s[kN] = {};
    if (kind == ROPE3D_NORM_LAYER) {
#pragma unroll
        for (int i = 0; i < kE; ++i) s[0] += v[i];   // absent elements are zero
        sum(s);
        *mean = s[0] * inv_c;
#pragma unroll
        for (int i = 0; i < kN; ++i) s[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kE; ++i) {
        const float d = real[i / per] ? v[i] - *mean : 0.0f;
        s[0] += d * d;
    }
    sum(s);
    *k = rsqrtf(s[0] * inv_c + eps);
}

template <int kT, int kVecs, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 128 : 512)
block_norm_vec_kernel(const __grid_constant__ NormParams p) {
    constexpr int V = kPer<kT>, E = V * kVecs, kBytes = 16 / V;
    __shared__ float red[2 * 32];
    Sums<1, kWarp> sum{red, 0};
    const int size = kWarp ? 32 : int(blockDim.x), lane = kWarp ? int(threadIdx.x & 31) : int(threadIdx.x);
    const int teams = kWarp ? int(blockDim.x >> 5) : 1;
    const int n_vec = p.channels / V;
    const float inv_c = 1.0f / float(p.channels);
    bool real[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) real[j] = lane + j * size < n_vec;
    grid_wait();
    grid_release();
    for (long long row = (long long)blockIdx.x * teams + (kWarp ? threadIdx.x >> 5 : 0); row < p.rows;
         row += (long long)gridDim.x * teams) {
        uint4 xv[kVecs], yv[kVecs];
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            xv[j] = yv[j] = make_uint4(0, 0, 0, 0);
            const int c = (lane + j * size) * V;
            if (real[j]) {
                xv[j] = ld_row(p.x, row * p.ldx + c, kBytes);
                if (p.y) yv[j] = ld_row(p.y, row * p.ldy + c, kBytes);
            }
        }
        const int g = int(uint32_t(row) / uint32_t(p.rows_per_group));
        float v[E];
#pragma unroll
        for (int j = 0; j < kVecs; ++j) unpack<kT>(xv[j], v + j * V);
        if (p.y) {
            float y[E], mean, k;
#pragma unroll
            for (int j = 0; j < kVecs; ++j) unpack<kT>(yv[j], y + j * V);
            row_stats<E>(y, p.post, real, V, inv_c, p.eps, sum, &mean, &k);
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                if (!real[j]) continue;
                const int c = (lane + j * size) * V;
                float w[V], gt[V];
                ld_weight<kT>(p.post_weight, c, p.param_f32, p.offset, w);
                ld_param<kT>(p.gate, g * p.ldg + c, p.param_f32, 1.0f, gt);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    v[j * V + i] = p.res * v[j * V + i] + gt[i] * ((y[j * V + i] - mean) * k * w[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) v[i] *= p.res;
        }
        if (p.r) {
#pragma unroll
            for (int j = 0; j < kVecs; ++j)
                if (real[j]) st_row(p.r, row * p.ldr + (lane + j * size) * V, kBytes, pack<kT>(v + j * V));
        }
        if (p.n) {
            float mean, k;
            row_stats<E>(v, p.pre, real, V, inv_c, p.eps, sum, &mean, &k);
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                if (!real[j]) continue;
                const int c = (lane + j * size) * V;
                float w[V], sc[V], sh[V];
                ld_weight<kT>(p.pre_weight, c, p.param_f32, p.offset, w);
                ld_param<kT>(p.scale, g * p.ldsc + c, p.param_f32, 0.0f, sc);
                ld_param<kT>(p.shift, g * p.ldsh + c, p.param_f32, 0.0f, sh);
                float o[V];
#pragma unroll
                for (int i = 0; i < V; ++i)
                    o[i] = (v[j * V + i] - mean) * k * w[i] * (1.0f + sc[i]) + sh[i];
                st_row(p.n, row * p.ldn + c, kBytes, pack<kT>(o));
            }
        }
    }
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

__global__ void __launch_bounds__(kGeneralThreads) block_norm_any_kernel(const __grid_constant__ NormParams p) {
    __shared__ float red[2 * 2 * 32];
    Sums<2, false> sum{red, 0};
    grid_wait();
    grid_release();
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        RowOps o{p, row, int(uint32_t(row) / uint32_t(p.rows_per_group)), 0.0f, 1.0f, 0.0f, 1.0f};
        if (p.y) scan_stats([&](int c) { return load1(p.y, row * p.ldy + c, p.dtype); }, p, p.post, sum, &o.my, &o.ky);
        if (p.n) scan_stats([&](int c) { return o.r(c); }, p, p.pre, sum, &o.mr, &o.kr);
        // r and n may be x and y themselves: a thread reads its element before it writes it
        for (int c = threadIdx.x; c < p.channels; c += blockDim.x) {
            const float r = o.r(c);
            if (p.n) {
                const float sh = o.param(p.shift, o.g * p.ldsh + c, 0.0f);
                store1(p.n, row * p.ldn + c, (r - o.mr) * o.kr * o.wq(c) * o.scale1(c) + sh, p.dtype);
            }
            if (p.r) store1(p.r, row * p.ldr + c, r, p.dtype);
        }
    }
}

// ---- backward, rows in registers ------------------------------------------------------------

// The rows [lo, hi) of chunk c.
__device__ __forceinline__ void chunk_range(const NormParams &p, int c, long long *lo, long long *hi) {
    if (p.groups_per_chunk) {   // whole groups
        *lo = (long long)c * p.groups_per_chunk * p.rows_per_group;
        *hi = min((long long)p.rows, *lo + (long long)p.groups_per_chunk * p.rows_per_group);
    } else {                    // a part of one group
        const int g = c / p.chunks_per_group, i = c - g * p.chunks_per_group;
        const long long first = (long long)g * p.rows_per_group;
        const long long end = min((long long)p.rows, first + p.rows_per_group);
        *lo = min(end, first + (long long)i * p.chunk_rows);
        *hi = min(end, *lo + p.chunk_rows);
    }
}

template <int kT, int kVecs, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 128 : 512)
block_norm_back_vec_kernel(const __grid_constant__ NormParams p) {
    constexpr int V = kPer<kT>, E = V * kVecs, kBytes = 16 / V;
    __shared__ float red[2 * 3 * 32];
    extern __shared__ float weight_sums[];   // [2][E][threads]: the weights' sums where a chunk is whole groups
    Sums<3, kWarp> sum{red, 0};
    const int size = kWarp ? 32 : int(blockDim.x), lane = kWarp ? int(threadIdx.x & 31) : int(threadIdx.x);
    const int teams = kWarp ? int(blockDim.x >> 5) : 1;
    const int n_vec = p.channels / V;
    const float inv_c = 1.0f / float(p.channels);
    bool real[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) real[j] = lane + j * size < n_vec;
    grid_wait();
    grid_release();
    for (int chunk = int(blockIdx.x) * teams + (kWarp ? int(threadIdx.x >> 5) : 0); chunk < p.chunks;
         chunk += int(gridDim.x) * teams) {
        long long lo, hi;
        chunk_range(p, chunk, &lo, &hi);
        float S[E], T[E], U[E];
#pragma unroll
        for (int i = 0; i < E; ++i) S[i] = T[i] = U[i] = 0.0f;
        if (p.groups_per_chunk && p.sums) {
#pragma unroll
            for (int i = 0; i < 2 * E; ++i) weight_sums[i * blockDim.x + threadIdx.x] = 0.0f;
        }
        int g = int(uint32_t(lo) / uint32_t(p.rows_per_group));
        long long group_end = (long long)(g + 1) * p.rows_per_group;
        for (long long row = lo; row < hi; ++row) {
            if (row == group_end) {
                ++g;
                group_end += p.rows_per_group;
            }
            uint4 xv[kVecs], yv[kVecs], rv[kVecs], nv[kVecs];
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                xv[j] = yv[j] = rv[j] = nv[j] = make_uint4(0, 0, 0, 0);
                const int c = (lane + j * size) * V;
                if (real[j]) {
                    if (p.y) yv[j] = ld_row(p.y, row * p.ldy + c, kBytes);
                    xv[j] = ld_row(p.x, row * p.ldx + c, kBytes);
                    if (p.dn) nv[j] = ld_row(p.dn, row * p.lddn + c, kBytes);
                    if (p.dr) rv[j] = ld_row(p.dr, row * p.lddr + c, kBytes);
                }
            }
            float my = 0.0f, ky = 1.0f;
            if (p.y) {
                float y[E];
#pragma unroll
                for (int j = 0; j < kVecs; ++j) unpack<kT>(yv[j], y + j * V);
                row_stats<E>(y, p.post, real, V, inv_c, p.eps, sum, &my, &ky);
            }
            // r and e of this thread's channels
            float r[E], e[E];
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                const int c = real[j] ? (lane + j * size) * V : 0;
                unpack<kT>(xv[j], r + j * V);
                if (p.y) {
                    float y[V], w[V], gt[V];
                    unpack<kT>(yv[j], y);
                    ld_weight<kT>(p.post_weight, c, p.param_f32, p.offset, w);
                    ld_param<kT>(p.gate, g * p.ldg + c, p.param_f32, 1.0f, gt);
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        r[j * V + i] = p.res * r[j * V + i] + gt[i] * ((y[i] - my) * ky * w[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) r[j * V + i] *= p.res;
                }
                float dn[V], w[V], sc[V];
                unpack<kT>(nv[j], dn);
                ld_weight<kT>(p.pre_weight, c, p.param_f32, p.offset, w);
                ld_param<kT>(p.scale, g * p.ldsc + c, p.param_f32, 0.0f, sc);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    e[j * V + i] = dn[i] * w[i] * (1.0f + sc[i]);
                    if (!real[j]) r[j * V + i] = e[j * V + i] = 0.0f;
                }
            }
            float mr = 0.0f, kr = 1.0f, me = 0.0f, mez = 0.0f;
            if (p.pre != ROPE3D_NORM_NONE) {
                if (p.pre == ROPE3D_NORM_LAYER) {
                    float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        s[0] += r[i];
                        s[1] += e[i];
                    }
                    sum(s);
                    mr = s[0] * inv_c;
                    me = s[1] * inv_c;
                }
                float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const float d = real[i / V] ? r[i] - mr : 0.0f;
                    s[0] += d * d;
                    s[1] += d * e[i];
                }
                sum(s);
                kr = rsqrtf(s[0] * inv_c + p.eps);
                mez = s[1] * inv_c * kr;
            }
            // the whole gradient of r, in e; the sums of n's parameters
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                float dr[V], dn[V];
                unpack<kT>(rv[j], dr);
                unpack<kT>(nv[j], dn);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float z = (r[j * V + i] - mr) * kr;
                    S[j * V + i] += dn[i] * z;
                    T[j * V + i] += dn[i];
                    e[j * V + i] = p.pre == ROPE3D_NORM_NONE ? dr[i] + e[j * V + i]
                                                             : dr[i] + kr * (e[j * V + i] - me - z * mez);
                }
                if (real[j]) {
                    float o[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) o[i] = p.res * e[j * V + i];
                    st_row(p.dx, row * p.lddx + (lane + j * size) * V, kBytes, pack<kT>(o));
                }
            }
            if (p.y) {
                // f, in r
                float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int j = 0; j < kVecs; ++j) {
                    const int c = real[j] ? (lane + j * size) * V : 0;
                    float y[V], w[V], gt[V];
                    unpack<kT>(yv[j], y);
                    ld_weight<kT>(p.post_weight, c, p.param_f32, p.offset, w);
                    ld_param<kT>(p.gate, g * p.ldg + c, p.param_f32, 1.0f, gt);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float yh = (y[i] - my) * ky, f = real[j] ? e[j * V + i] * gt[i] * w[i] : 0.0f;
                        U[j * V + i] += e[j * V + i] * yh;
                        r[j * V + i] = f;
                        s[0] += f;
                        s[1] += f * yh;
                    }
                }
                float mf = 0.0f, mfy = 0.0f;
                if (p.post != ROPE3D_NORM_NONE) {
                    sum(s);
                    mf = p.post == ROPE3D_NORM_LAYER ? s[0] * inv_c : 0.0f;
                    mfy = s[1] * inv_c;
                }
#pragma unroll
                for (int j = 0; j < kVecs; ++j) {
                    if (!real[j]) continue;
                    float y[V], o[V];
                    unpack<kT>(yv[j], y);
#pragma unroll
                    for (int i = 0; i < V; ++i) o[i] = ky * (r[j * V + i] - mf - (y[i] - my) * ky * mfy);
                    st_row(p.dy, row * p.lddy + (lane + j * size) * V, kBytes, pack<kT>(o));
                }
            }
            if (p.groups_per_chunk && p.sums && (row + 1 == group_end || row + 1 == hi)) {
                // a whole group is done: its gradients, and its part of the weights'
#pragma unroll
                for (int j = 0; j < kVecs; ++j) {
                    if (!real[j]) continue;
                    const int c = (lane + j * size) * V;
                    float wp[V], wq[V], gt[V], sc[V], o[V];
                    ld_weight<kT>(p.post_weight, c, p.param_f32, p.offset, wp);
                    ld_weight<kT>(p.pre_weight, c, p.param_f32, p.offset, wq);
                    ld_param<kT>(p.gate, g * p.ldg + c, p.param_f32, 1.0f, gt);
                    ld_param<kT>(p.scale, g * p.ldsc + c, p.param_f32, 0.0f, sc);
                    if (p.d_scale) {
#pragma unroll
                        for (int i = 0; i < V; ++i) o[i] = wq[i] * S[j * V + i];
                        st_param<kT>(p.d_scale, g * p.ldgrad + c, p.param_f32, o);
                    }
                    if (p.d_shift) st_param<kT>(p.d_shift, g * p.ldgrad + c, p.param_f32, T + j * V);
                    if (p.d_gate) {
#pragma unroll
                        for (int i = 0; i < V; ++i) o[i] = wp[i] * U[j * V + i];
                        st_param<kT>(p.d_gate, g * p.ldgrad + c, p.param_f32, o);
                    }
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        weight_sums[(j * V + i) * blockDim.x + threadIdx.x] += (1.0f + sc[i]) * S[j * V + i];
                        weight_sums[(E + j * V + i) * blockDim.x + threadIdx.x] += gt[i] * U[j * V + i];
                        S[j * V + i] = T[j * V + i] = U[j * V + i] = 0.0f;
                    }
                }
            }
        }
        if (p.part) {
            float *dst = p.part + (long long)chunk * 3 * p.channels;
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                if (!real[j]) continue;
                const int c = (lane + j * size) * V;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if (p.groups_per_chunk) {
                        S[j * V + i] = weight_sums[(j * V + i) * blockDim.x + threadIdx.x];
                        U[j * V + i] = weight_sums[(E + j * V + i) * blockDim.x + threadIdx.x];
                    }
                }
#pragma unroll
                for (int i = 0; i < V; i += 4) {
                    *reinterpret_cast<float4 *>(dst + c + i) =
                        make_float4(S[j * V + i], S[j * V + i + 1], S[j * V + i + 2], S[j * V + i + 3]);
                    *reinterpret_cast<float4 *>(dst + p.channels + c + i) =
                        make_float4(T[j * V + i], T[j * V + i + 1], T[j * V + i + 2], T[j * V + i + 3]);
                    *reinterpret_cast<float4 *>(dst + 2 * p.channels + c + i) =
                        make_float4(U[j * V + i], U[j * V + i + 1], U[j * V + i + 2], U[j * V + i + 3]);
                }
            }
        }
    }
}

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

// kLayer: one of the norms is a layer norm.
template <int kT, bool kLayer, bool kFull>
__global__ void __maxnreg__(80) block_norm_ring_kernel(const __grid_constant__ NormParams p) {
    using Team = RingTeam<kT, kFull>;
    constexpr int H = Team::H, kBytes = Team::kBytes;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(16) float2 red[2 * 16];
    __shared__ __align__(8) unsigned long long bars[kRingBars];
    const Team team(p, raw);
    const int tid = team.tid;
    const uint32_t row_bytes = uint32_t(p.channels) * kBytes;
    const int streams = p.y ? 2 : 1;
    const Ring ring{team.base + uint32_t(team.size) * 3 * 64, smem_u32(bars), row_bytes, row_bytes * uint32_t(streams), p.stages};
    const Kept km = team.kept(0), kq = team.kept(1), ks = team.kept(2);
    BlockSums sum{red, 0, ((team.size >> 5) + 1) & ~1};
    for (int i = tid; i < 2 * 16; i += team.size) red[i] = make_float2(0.0f, 0.0f);
    if (tid == 0) {
        for (int s = 0; s < p.stages; ++s) mbar_init(ring.bars + 8u * uint32_t(s), 1);
        mbar_fence_init();
    }
    __syncthreads();
    grid_wait();
    grid_release();
    const long long lo = (long long)p.rows * blockIdx.x / gridDim.x, hi = (long long)p.rows * (blockIdx.x + 1) / gridDim.x;
    auto fill = [&](int s, long long row) {
        const uint32_t bar = ring.bars + 8u * uint32_t(s), at = ring.base + uint32_t(s) * ring.stage_bytes;
        mbar_expect_tx(bar, ring.stage_bytes);
        bulk_row(at, static_cast<const char *>(p.x) + row * p.ldx * kBytes, row_bytes, bar);
        if (p.y) bulk_row(at + row_bytes, static_cast<const char *>(p.y) + row * p.ldy * kBytes, row_bytes, bar);
    };
    if (tid == 0)
        for (int s = 0; s < p.stages && lo + s < hi; ++s) fill(s, lo + s);
    bool dead = false;
    const float2 res = both(p.res);
    int g = int(uint32_t(lo) / uint32_t(p.rows_per_group)) - 1;
    long long group_end = lo;   // the first row starts a group
    int s = 0;
    uint32_t phase = 0;
    for (long long row = lo; row < hi; ++row) {
        if (row == group_end) {
            ++g;
            group_end = (long long)(g + 1) * p.rows_per_group;
            float m[kRingE], q[kRingE];
            team.group(g, m, q);
            km.store(m);   // read back by this thread alone
            kq.store(q);
#pragma unroll
            for (int j = 0; j < Team::kVecs; ++j)
                ld_param<kT>(p.shift, g * p.ldsh + (team.real(j) ? team.channel(j) : 0), p.param_f32, 0.0f, m + j * Team::V);
            ks.store(m);
        }
        mbar_wait(ring.bars + 8u * uint32_t(s), phase, dead, &g_norm_wait_timeouts);
        const uint32_t at = ring.base + uint32_t(s) * ring.stage_bytes;
        float2 v[H];
        team.unpack_row(at, v);
        bool synced = false;   // every thread has read its part of the stage
#pragma unroll
        for (int i = 0; i < H; ++i) v[i] = mul2(res, v[i]);
        if (p.y) {
            float2 y[H], m[H];
            team.unpack_row(at + row_bytes, y);
            if (p.post != ROPE3D_NORM_NONE) {
                team.template normalise<kLayer>(y, p.post, sum);
                synced = true;
            }
            km.load(m);
#pragma unroll
            for (int i = 0; i < H; ++i) v[i] = fma2(m[i], y[i], v[i]);
        }
        if (p.r) team.write(p.r, row * p.ldr, v);
        if (p.n) {
            if (p.pre != ROPE3D_NORM_NONE) {
                team.template normalise<kLayer>(v, p.pre, sum);
                synced = true;
            }
            float2 q[H], sh[H];
            kq.load(q);
            ks.load(sh);
#pragma unroll
            for (int i = 0; i < H; ++i) v[i] = fma2(v[i], q[i], sh[i]);
            team.write(p.n, row * p.ldn, v);
        }
        if (!synced) __syncthreads();
        if (tid == 0 && row + p.stages < hi && !dead) fill(s, row + p.stages);
        if (++s == p.stages) {
            s = 0;
            phase ^= 1;
        }
    }
}

// kShift: d_shift is wanted (its sums are one more array of registers).
template <int kT, bool kLayer, bool kFull, bool kShift>
__global__ void __launch_bounds__(512) block_norm_back_ring_kernel(const __grid_constant__ NormParams p) {
    using Team = RingTeam<kT, kFull>;
    constexpr int V = Team::V, kVecs = Team::kVecs, P = Team::P, H = Team::H, kBytes = Team::kBytes;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(16) float2 red[2 * 16];
    __shared__ __align__(8) unsigned long long bars[kRingBars];
    const Team team(p, raw);
    const int tid = team.tid;
    const uint32_t row_bytes = uint32_t(p.channels) * kBytes;
    // the arrays that a stage holds, in this order
    const uint32_t at_y = row_bytes, at_n = at_y + (p.y ? row_bytes : 0), at_r = at_n + (p.dn ? row_bytes : 0);
    const uint32_t stage_bytes = at_r + (p.dr ? row_bytes : 0);
    // m, q and, where a chunk is whole groups, the weights' sums
    const Ring ring{team.base + uint32_t(team.size) * (p.groups_per_chunk ? 4 : 2) * 64, smem_u32(bars), row_bytes,
                    stage_bytes, p.stages};
    const Kept km = team.kept(0), kq = team.kept(1), kwq = team.kept(2), kwp = team.kept(3);
    BlockSums sum{red, 0, ((team.size >> 5) + 1) & ~1};
    for (int i = tid; i < 2 * 16; i += team.size) red[i] = make_float2(0.0f, 0.0f);
    if (tid == 0) {
        for (int s = 0; s < p.stages; ++s) mbar_init(ring.bars + 8u * uint32_t(s), 1);
        mbar_fence_init();
    }
    __syncthreads();
    grid_wait();
    grid_release();
    const int chunk = int(blockIdx.x);
    long long lo, hi;
    chunk_range(p, chunk, &lo, &hi);
    auto fill = [&](int s, long long row) {
        const uint32_t bar = ring.bars + 8u * uint32_t(s), at = ring.base + uint32_t(s) * ring.stage_bytes;
        mbar_expect_tx(bar, ring.stage_bytes);
        bulk_row(at, static_cast<const char *>(p.x) + row * p.ldx * kBytes, row_bytes, bar);
        if (p.y) bulk_row(at + at_y, static_cast<const char *>(p.y) + row * p.ldy * kBytes, row_bytes, bar);
        if (p.dn) bulk_row(at + at_n, static_cast<const char *>(p.dn) + row * p.lddn * kBytes, row_bytes, bar);
        if (p.dr) bulk_row(at + at_r, static_cast<const char *>(p.dr) + row * p.lddr * kBytes, row_bytes, bar);
    };
    if (tid == 0)
        for (int s = 0; s < p.stages && lo + s < hi; ++s) fill(s, lo + s);
    bool dead = false;
    const float2 zero = make_float2(0.0f, 0.0f), res = both(p.res);
    float2 S[H], U[H], T[kShift ? H : 1];
#pragma unroll
    for (int i = 0; i < H; ++i) S[i] = U[i] = zero;
#pragma unroll
    for (int i = 0; i < (kShift ? H : 1); ++i) T[i] = zero;
    if (p.groups_per_chunk) {
        float z[kRingE] = {};
        kwq.store(z);
        kwp.store(z);
    }
    int g = int(uint32_t(lo) / uint32_t(p.rows_per_group)) - 1;
    long long group_end = lo;
    int s = 0;
    uint32_t phase = 0;
    for (long long row = lo; row < hi; ++row) {
        if (row == group_end) {
            ++g;
            group_end = (long long)(g + 1) * p.rows_per_group;
            float m[kRingE], q[kRingE];
            team.group(g, m, q);
            km.store(m);
            kq.store(q);
        }
        mbar_wait(ring.bars + 8u * uint32_t(s), phase, dead, &g_norm_wait_timeouts);
        const uint32_t at = ring.base + uint32_t(s) * ring.stage_bytes;
        // y normalised, r = res x + m y, dn
        float2 y[H], r[H], d[H];
        float ky = 1.0f;
        if (p.y) {
            team.unpack_row(at + at_y, y);
            if (p.post != ROPE3D_NORM_NONE) ky = team.template normalise<kLayer>(y, p.post, sum);
        }
        // (one vector at a time here and below: the sums leave few registers)
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
            float2 *rj = r + j * P;
            unpack2<kT>(team.read(at, j), rj);
#pragma unroll
            for (int i = 0; i < P; ++i) rj[i] = mul2(res, rj[i]);
            if (p.y) {
                float2 m[P];
                km.load_part<P>(j, m);
#pragma unroll
                for (int i = 0; i < P; ++i) rj[i] = fma2(m[i], y[j * P + i], rj[i]);
            }
            if (p.dn) {
                unpack2<kT>(team.read(at + at_n, j), d + j * P);
            } else {
#pragma unroll
                for (int i = 0; i < P; ++i) d[j * P + i] = zero;
            }
        }
        float kr = 1.0f, me = 0.0f, mez = 0.0f;
        if (p.pre != ROPE3D_NORM_NONE) {
            // 1 / std of r and the means of e = dn q and e z, from one pair of sums
            if (kLayer && p.pre == ROPE3D_NORM_LAYER) {
                float2 b = zero;
#pragma unroll
                for (int j = 0; j < kVecs; ++j) {
                    float2 q[P];
                    kq.load_part<P>(j, q);
#pragma unroll
                    for (int i = 0; i < P; ++i) b = fma2(d[j * P + i], q[i], b);
                }
                const float2 t = sum(Team::total(r), fold(b));
                team.center(r, t.x * team.inv_c);
                me = t.y * team.inv_c;
            }
            float2 a = zero, b = zero;
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                float2 q[P];
                kq.load_part<P>(j, q);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    a = fma2(r[j * P + i], r[j * P + i], a);
                    b = fma2(r[j * P + i], mul2(d[j * P + i], q[i]), b);
                }
            }
            const float2 t = sum(fold(a), fold(b));
            kr = rsqrtf(t.x * team.inv_c + p.eps);
            mez = t.y * team.inv_c * kr;
        }
        // d becomes the whole gradient of r
        {
            const float2 kr2 = both(kr), nme = both(-kr * me), nmez = both(-kr * mez);
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                float2 q[P], dr[P];
                kq.load_part<P>(j, q);
                if (p.dr) {
                    unpack2<kT>(team.read(at + at_r, j), dr);
                } else {
#pragma unroll
                    for (int i = 0; i < P; ++i) dr[i] = zero;
                }
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const int x = j * P + i;
                    const float2 z = mul2(r[x], kr2);
                    S[x] = fma2(d[x], z, S[x]);
                    if constexpr (kShift) T[x] = add2(T[x], d[x]);
                    if constexpr (kLayer) dr[i] = add2(dr[i], nme);
                    d[x] = fma2(kr2, mul2(d[x], q[i]), fma2(z, nmez, dr[i]));
                    dr[i] = mul2(res, d[x]);
                }
                if (team.real(j))
                    st_row(p.dx, row * p.lddx + team.channel(j), kBytes, pack<kT>(reinterpret_cast<const float *>(dr)));
            }
        }
        if (p.y) {
            float2 a = zero, b = zero;
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                float2 m[P];
                km.load_part<P>(j, m);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const int x = j * P + i;
                    U[x] = fma2(d[x], y[x], U[x]);
                    r[x] = mul2(d[x], m[i]);   // f; m is zero for absent channels
                    if constexpr (kLayer) a = add2(a, r[x]);
                    b = fma2(r[x], y[x], b);
                }
            }
            // the stage has been read by every thread once they meet in this sum
            if (p.post != ROPE3D_NORM_NONE) {
                float2 t = make_float2(0.0f, 0.0f);
                if (kLayer && p.post == ROPE3D_NORM_LAYER) t = sum(fold(a), fold(b));
                else t.y = sum.one(fold(b));
                if (tid == 0 && row + p.stages < hi && !dead) fill(s, row + p.stages);
                const float2 ky2 = both(ky), nmf = both(-ky * t.x * team.inv_c), nmfy = both(-ky * t.y * team.inv_c);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    if constexpr (kLayer) r[i] = fma2(ky2, r[i], fma2(y[i], nmfy, nmf));
                    else r[i] = fma2(ky2, r[i], mul2(y[i], nmfy));
                }
            } else {
                __syncthreads();
                if (tid == 0 && row + p.stages < hi && !dead) fill(s, row + p.stages);
            }
            team.write(p.dy, row * p.lddy, r);
        } else {
            __syncthreads();
            if (tid == 0 && row + p.stages < hi && !dead) fill(s, row + p.stages);
        }
        if (++s == p.stages) {
            s = 0;
            phase ^= 1;
        }
        if (p.groups_per_chunk && p.sums && (row + 1 == group_end || row + 1 == hi)) {
            // a whole group is done: its gradients, and its part of the weights'
            float wq[kRingE], wp[kRingE];
            float2 t[H];
            kwq.load(t);
            memcpy(wq, t, sizeof(wq));
            kwp.load(t);
            memcpy(wp, t, sizeof(wp));
#pragma unroll
            for (int j = 0; j < kVecs; ++j) {
                const int c = team.real(j) ? team.channel(j) : 0;
                const float *Sj = reinterpret_cast<const float *>(S + j * P), *Uj = reinterpret_cast<const float *>(U + j * P);
                float a[V], o[V];
                if (p.d_scale && team.real(j)) {
                    ld_weight<kT>(p.pre_weight, c, p.param_f32, p.offset, a);
#pragma unroll
                    for (int i = 0; i < V; ++i) o[i] = a[i] * Sj[i];
                    st_param<kT>(p.d_scale, g * p.ldgrad + c, p.param_f32, o);
                }
                if constexpr (kShift)
                    if (team.real(j))
                        st_param<kT>(p.d_shift, g * p.ldgrad + c, p.param_f32, reinterpret_cast<const float *>(T + j * P));
                if (p.d_gate && team.real(j)) {
                    ld_weight<kT>(p.post_weight, c, p.param_f32, p.offset, a);
#pragma unroll
                    for (int i = 0; i < V; ++i) o[i] = a[i] * Uj[i];
                    st_param<kT>(p.d_gate, g * p.ldgrad + c, p.param_f32, o);
                }
                ld_param<kT>(p.scale, g * p.ldsc + c, p.param_f32, 0.0f, a);
#pragma unroll
                for (int i = 0; i < V; ++i) wq[j * V + i] += (1.0f + a[i]) * Sj[i];
                ld_param<kT>(p.gate, g * p.ldg + c, p.param_f32, 1.0f, a);
#pragma unroll
                for (int i = 0; i < V; ++i) wp[j * V + i] += a[i] * Uj[i];
            }
            kwq.store(wq);
            kwp.store(wp);
#pragma unroll
            for (int i = 0; i < H; ++i) S[i] = U[i] = zero;
#pragma unroll
            for (int i = 0; i < (kShift ? H : 1); ++i) T[i] = zero;
        }
    }
    if (p.part) {
        if (p.groups_per_chunk) {
            kwq.load(S);
            kwp.load(U);
        }
        float *dst = p.part + (long long)chunk * 3 * p.channels;
        auto put = [&](float *to, const float2 *v) {
#pragma unroll
            for (int j = 0; j < kVecs; ++j)
                if (team.real(j))
#pragma unroll
                    for (int i = 0; i < P; i += 2)
                        *reinterpret_cast<float4 *>(to + team.channel(j) + 2 * i) =
                            make_float4(v[j * P + i].x, v[j * P + i].y, v[j * P + i + 1].x, v[j * P + i + 1].y);
        };
        put(dst, S);
        if constexpr (kShift) put(dst + p.channels, T);
        put(dst + 2ll * p.channels, U);
    }
}

// ---- backward, any row: dx, dy and the rows' statistics, then the columns --------------------

__global__ void __launch_bounds__(kGeneralThreads) block_norm_back_any_kernel(const __grid_constant__ NormParams p) {
    __shared__ float red[2 * 2 * 32];
    Sums<2, false> sum{red, 0};
    const float inv_c = 1.0f / float(p.channels);
    grid_wait();
    grid_release();
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        RowOps o{p, row, int(uint32_t(row) / uint32_t(p.rows_per_group)), 0.0f, 1.0f, 0.0f, 1.0f};
        if (p.y) scan_stats([&](int c) { return load1(p.y, row * p.ldy + c, p.dtype); }, p, p.post, sum, &o.my, &o.ky);
        scan_stats([&](int c) { return o.r(c); }, p, p.pre, sum, &o.mr, &o.kr);
        float me = 0.0f, mez = 0.0f, mf = 0.0f, mfy = 0.0f;
        if (p.pre != ROPE3D_NORM_NONE) {
            float s[2] = {0.0f, 0.0f};
            for (int c = threadIdx.x; c < p.channels; c += blockDim.x) {
                const float e = o.e(c);
                s[0] += e;
                s[1] += e * o.z(c);
            }
            sum(s);
            me = p.pre == ROPE3D_NORM_LAYER ? s[0] * inv_c : 0.0f;
            mez = s[1] * inv_c;
        }
        auto whole = [&](int c) {   // the whole gradient of r
            const float dr = p.dr ? load1(p.dr, row * p.lddr + c, p.dtype) : 0.0f;
            return dr + o.kr * (o.e(c) - me - o.z(c) * mez);
        };
        if (p.y && p.post != ROPE3D_NORM_NONE) {
            float s[2] = {0.0f, 0.0f};
            for (int c = threadIdx.x; c < p.channels; c += blockDim.x) {
                const float f = whole(c) * o.gate(c) * o.wp(c);
                s[0] += f;
                s[1] += f * o.yh(c);
            }
            sum(s);
            mf = p.post == ROPE3D_NORM_LAYER ? s[0] * inv_c : 0.0f;
            mfy = s[1] * inv_c;
        }
        if (p.stats && threadIdx.x == 0) {
            float *t = p.stats + row * 6;
            t[0] = o.my; t[1] = o.ky; t[2] = o.mr; t[3] = o.kr; t[4] = me; t[5] = mez;
        }
        if (!p.stats) {
            for (int c = threadIdx.x; c < p.channels; c += blockDim.x) {
                const float d = whole(c);
                const float f = p.y ? d * o.gate(c) * o.wp(c) : 0.0f;
                if (p.y) store1(p.dy, row * p.lddy + c, o.ky * (f - mf - o.yh(c) * mfy), p.dtype);
                store1(p.dx, row * p.lddx + c, p.res * d, p.dtype);
            }
        } else {
            // dx and dy may be dr and dn, which the columns' kernel still reads:
            // it writes them
            float *t = p.stats + (long long)p.rows * 6 + row * 2;
            if (threadIdx.x == 0) {
                t[0] = mf;
                t[1] = mfy;
            }
        }
    }
}

// One channel a thread over a chunk's rows: the sums, dx and dy.
__global__ void __launch_bounds__(kGeneralThreads) block_norm_back_cols_kernel(const __grid_constant__ NormParams p) {
    grid_wait();
    grid_release();
    const int c = int(blockIdx.x) * kGeneralThreads + int(threadIdx.x);
    if (c >= p.channels) return;
    const int param_type = p.param_f32 ? ROPE3D_F32 : p.dtype;
    for (int chunk = blockIdx.y; chunk < p.chunks; chunk += gridDim.y) {
        long long lo, hi;
        chunk_range(p, chunk, &lo, &hi);
        float S = 0.0f, T = 0.0f, U = 0.0f, Wq = 0.0f, Wp = 0.0f;
        RowOps o{p, lo, int(uint32_t(lo) / uint32_t(p.rows_per_group)), 0.0f, 1.0f, 0.0f, 1.0f};
        long long group_end = (long long)(o.g + 1) * p.rows_per_group;
        for (long long row = lo; row < hi; ++row) {
            if (row == group_end) {
                ++o.g;
                group_end += p.rows_per_group;
            }
            const float *t = p.stats + row * 6, *t2 = p.stats + (long long)p.rows * 6 + row * 2;
            o.row = row;
            o.my = t[0]; o.ky = t[1]; o.mr = t[2]; o.kr = t[3];
            const float z = o.z(c), dn = o.dn(c), e = o.e(c);
            const float dr = p.dr ? load1(p.dr, row * p.lddr + c, p.dtype) : 0.0f;
            const float d = dr + o.kr * (e - t[4] - z * t[5]);
            S += dn * z;
            T += dn;
            if (p.y) {
                const float yh = o.yh(c), f = d * o.gate(c) * o.wp(c);
                U += d * yh;
                store1(p.dy, row * p.lddy + c, o.ky * (f - t2[0] - yh * t2[1]), p.dtype);
            }
            store1(p.dx, row * p.lddx + c, p.res * d, p.dtype);
            if (p.groups_per_chunk && (row + 1 == group_end || row + 1 == hi)) {
                const long long at = o.g * p.ldgrad + c;
                if (p.d_scale) store1(p.d_scale, at, o.wq(c) * S, param_type);
                if (p.d_shift) store1(p.d_shift, at, T, param_type);
                if (p.d_gate) store1(p.d_gate, at, o.wp(c) * U, param_type);
                Wq += o.scale1(c) * S;
                Wp += o.gate(c) * U;
                S = T = U = 0.0f;
            }
        }
        if (p.part) {
            float *dst = p.part + (long long)chunk * 3 * p.channels + c;
            dst[0] = p.groups_per_chunk ? Wq : S;
            dst[p.channels] = T;
            dst[2ll * p.channels] = p.groups_per_chunk ? Wp : U;
        }
    }
}

// The chunks' partial sums of one group (blockIdx.y), or the weights' of all
// chunks, 32 channels a block: 16 rows of threads each add every 16th chunk,
// several loads in flight, then those sums in order. Where several groups make
// up the weights' gradients, their parts go to p.group_sums, [groups][2][channels],
// and block_norm_groups_kernel adds them.
constexpr int kFinishRows = 16;

__global__ void __launch_bounds__(32 * kFinishRows) block_norm_finish_kernel(const __grid_constant__ NormParams p) {
    __shared__ float part[3][kFinishRows][32];
    grid_wait();
    grid_release();
    const int lane = threadIdx.x & 31, ty = threadIdx.x >> 5, g = int(blockIdx.y);
    const int c = int(blockIdx.x) * 32 + lane;
    const int param_type = p.param_f32 ? ROPE3D_F32 : p.dtype;
    const int per = p.groups_per_chunk ? p.chunks : p.chunks_per_group;
    // which of the three sums exist: S with a pre weight or scale, and so on
    const bool want[3] = {p.d_pre_weight || p.d_scale, p.d_shift != nullptr, p.d_post_weight || p.d_gate};
    float s[3] = {0.0f, 0.0f, 0.0f};
    if (c < p.channels) {
        const float *src = p.part + (long long)g * per * 3 * p.channels + c;
        const long long step = 3ll * p.channels;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (!want[k]) continue;
            int i = ty;
            for (; i + 7 * kFinishRows < per; i += 8 * kFinishRows) {
                float v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) v[u] = __ldcs(src + (i + u * kFinishRows) * step + (long long)k * p.channels);
#pragma unroll
                for (int u = 0; u < 8; ++u) s[k] += v[u];
            }
            for (; i < per; i += kFinishRows) s[k] += __ldcs(src + i * step + (long long)k * p.channels);
        }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) part[k][ty][lane] = s[k];
    __syncthreads();
    if (ty != 0 || c >= p.channels) return;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        s[k] = 0.0f;
        for (int i = 0; i < kFinishRows; ++i) s[k] += part[k][i][lane];
    }
    float wq = s[0], wp = s[2];
    if (!p.groups_per_chunk) {
        const RowOps og{p, 0, g, 0.0f, 1.0f, 0.0f, 1.0f};
        const long long at = g * p.ldgrad + c;
        if (p.d_scale) store1(p.d_scale, at, og.wq(c) * s[0], param_type);
        if (p.d_shift) store1(p.d_shift, at, s[1], param_type);
        if (p.d_gate) store1(p.d_gate, at, og.wp(c) * s[2], param_type);
        wq *= og.scale1(c);
        wp *= og.gate(c);
        if (p.group_sums) {
            float *dst = p.group_sums + (long long)g * 2 * p.channels + c;
            dst[0] = wq;
            dst[p.channels] = wp;
            return;
        }
    }
    if (p.d_pre_weight) store1(p.d_pre_weight, c, wq, param_type);
    if (p.d_post_weight) store1(p.d_post_weight, c, wp, param_type);
}

__global__ void __launch_bounds__(128) block_norm_groups_kernel(const __grid_constant__ NormParams p) {
    grid_wait();
    grid_release();
    const int c = int(blockIdx.x * 128 + threadIdx.x);
    if (c >= p.channels) return;
    const int param_type = p.param_f32 ? ROPE3D_F32 : p.dtype;
    float wq = 0.0f, wp = 0.0f;
    for (int g = 0; g < p.groups; ++g) {
        wq += p.group_sums[(long long)g * 2 * p.channels + c];
        wp += p.group_sums[((long long)g * 2 + 1) * p.channels + c];
    }
    if (p.d_pre_weight) store1(p.d_pre_weight, c, wq, param_type);
    if (p.d_post_weight) store1(p.d_post_weight, c, wp, param_type);
}

// ---- host ------------------------------------------------------------------------------------

thread_local int t_norm_kernel = 0;

bool on_device(const void *p, int device) {
    cudaPointerAttributes attr{};
    if (cudaPointerGetAttributes(&attr, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    if (attr.type == cudaMemoryTypeManaged) return true;
    return attr.type == cudaMemoryTypeDevice && attr.device == device;
}

struct Span {
    const void *p;
    int64_t bytes, ld;
    int align;
};

Span span(const void *p, int64_t rows, int64_t cols, int64_t ld, int es) {
    return Span{p, p ? ((rows - 1) * ld + cols) * es : 0, ld, es};
}

bool overlap(const Span &a, const Span &b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && x < y + uint64_t(b.bytes) && y < x + uint64_t(a.bytes);
}

bool same(const Span &a, const Span &b) { return a.p == b.p && a.ld == b.ld; }

bool bad_ld(int64_t ld, int64_t cols) { return ld < cols || ld > (int64_t(1) << 31); }

// The GB300's SMs: the workspace's size, and with it the order of the column
// sums, is the same on every device and without one.
constexpr int64_t kSms = 152;

int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// The arguments that forward and backward share: everything but r, n and the
// gradients. Fills p and the input spans (7 of them).
int check_inputs(const rope3d_block_norm_args &a, NormParams &p, Span *in) {
    if (!a.x) return ROPE3D_ERR_NULL;
    const int64_t R = a.rows, C = a.channels;
    if (R <= 0 || C <= 0 || a.rows_per_group <= 0 || R > 0x7fffffff || C > ROPE3D_MAX_CHANNELS)
        return ROPE3D_ERR_SHAPE;
    if (a.dtype != ROPE3D_BF16 && a.dtype != ROPE3D_F32 && a.dtype != ROPE3D_F16) return ROPE3D_ERR_DTYPE;
    if (a.param_dtype != a.dtype && a.param_dtype != ROPE3D_F32) return ROPE3D_ERR_DTYPE;
    for (int kind : {a.post_kind, a.pre_kind})
        if (kind != ROPE3D_NORM_NONE && kind != ROPE3D_NORM_RMS && kind != ROPE3D_NORM_LAYER) return ROPE3D_ERR_ARG;
    if (!std::isfinite(a.eps) || a.eps < 0.0 || !std::isfinite(a.residual_scale) || !std::isfinite(a.weight_offset))
        return ROPE3D_ERR_ARG;
    if (!a.y && (a.post_weight || a.gate)) return ROPE3D_ERR_ARG;
    if (a.post_weight && a.post_kind == ROPE3D_NORM_NONE) return ROPE3D_ERR_ARG;
    const int64_t rpg = std::min(a.rows_per_group, R), G = (R + rpg - 1) / rpg;
    if (bad_ld(a.x_stride, C) || (a.y && bad_ld(a.y_stride, C))) return ROPE3D_ERR_SHAPE;
    if ((a.gate && bad_ld(a.gate_stride, C)) || (a.scale && bad_ld(a.scale_stride, C)) ||
        (a.shift && bad_ld(a.shift_stride, C)))
        return ROPE3D_ERR_SHAPE;
    const int es = a.dtype == ROPE3D_F32 ? 4 : 2, ps = a.param_dtype == ROPE3D_F32 ? 4 : 2;
    in[0] = span(a.x, R, C, a.x_stride, es);
    in[1] = span(a.y, R, C, a.y_stride, es);
    in[2] = span(a.post_weight, 1, C, C, ps);
    in[3] = span(a.pre_weight, 1, C, C, ps);
    in[4] = span(a.gate, G, C, a.gate_stride, ps);
    in[5] = span(a.scale, G, C, a.scale_stride, ps);
    in[6] = span(a.shift, G, C, a.shift_stride, ps);
    p = NormParams{};
    p.x = a.x; p.y = a.y; p.post_weight = a.post_weight; p.gate = a.gate; p.pre_weight = a.pre_weight;
    p.scale = a.scale; p.shift = a.shift;
    p.ldx = a.x_stride; p.ldy = a.y_stride; p.ldg = a.gate_stride; p.ldsc = a.scale_stride; p.ldsh = a.shift_stride;
    p.rows = int(R); p.channels = int(C); p.rows_per_group = int(rpg); p.groups = int(G);
    if (!a.gate && !a.scale && !a.shift) {   // no parameter of a group: one group
        p.rows_per_group = int(R);
        p.groups = 1;
    }
    p.eps = float(a.eps); p.res = float(a.residual_scale); p.offset = float(a.weight_offset);
    p.post = a.y ? a.post_kind : ROPE3D_NORM_NONE;
    p.pre = a.pre_kind;
    p.dtype = a.dtype;
    p.param_f32 = a.param_dtype == ROPE3D_F32;
    return ROPE3D_OK;
}

int check_align_device(const Span *const *all, int n, bool check_device) {
    for (int i = 0; i < n; ++i)
        if (all[i]->p && reinterpret_cast<uintptr_t>(all[i]->p) % uintptr_t(all[i]->align) != 0) return ROPE3D_ERR_ALIGN;
    if (!check_device) return ROPE3D_OK;
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) {
        cudaGetLastError();
        return ROPE3D_ERR_CUDA;
    }
    for (int i = 0; i < n; ++i)
        if (all[i]->p && !on_device(all[i]->p, device)) return ROPE3D_ERR_DEVICE;
    return ROPE3D_OK;
}

// Whether every row (and parameter row) is whole 16-byte vectors.
bool vectors(const Span *const *all, int n, int64_t channels, int vec) {
    if (channels % vec != 0) return false;
    for (int i = 0; i < n; ++i)
        if (all[i]->p && (reinterpret_cast<uintptr_t>(all[i]->p) % 16 != 0 || all[i]->ld % vec != 0)) return false;
    return true;
}

using NormFn = void (*)(NormParams);

int launch(NormFn fn, dim3 grid, dim3 block, size_t smem, const NormParams &p, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, fn, p) != cudaSuccess) {
        cudaGetLastError();
        return ROPE3D_ERR_CUDA;
    }
    return ROPE3D_OK;
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return n;
}

// A forward team: a warp up to 4 vectors a lane, else a block of 2 or 4 vectors
// a thread. kVecs 0: the general kernel.
struct Team {
    int vecs, threads;
    bool warp;
};

Team forward_team(int64_t n) {   // n: vectors of a row
    if (n <= 128) return Team{n <= 32 ? 1 : n <= 64 ? 2 : 4, 32, true};
    if (n <= 512) return Team{2, int(up((n + 1) / 2, 32)), false};
    if (n <= 2048) return Team{4, int(up((n + 3) / 4, 32)), false};
    return Team{0, 0, false};
}

template <int kT>
NormFn forward_fn(const Team &t) {
    if (t.warp)
        return t.vecs == 1   ? block_norm_vec_kernel<kT, 1, true>
               : t.vecs == 2 ? block_norm_vec_kernel<kT, 2, true>
                             : block_norm_vec_kernel<kT, 4, true>;
    return t.vecs == 2 ? block_norm_vec_kernel<kT, 2, false> : block_norm_vec_kernel<kT, 4, false>;
}

// A backward team: 8 or 16 elements a thread (the three sums of each stay in
// registers).
Team backward_team(int64_t n, int vec) {
    const int most = 16 / vec;   // vectors of 16 elements
    for (int v = vec == 4 ? 2 : 1; v <= most; v *= 2) {
        if (n <= 32 * v) return Team{v, 32, true};
        if (n <= 512 * v) return Team{v, int(up((n + v - 1) / v, 32)), false};
    }
    return Team{0, 0, false};
}

template <int kT>
NormFn backward_fn(const Team &t) {
    if constexpr (kT == ROPE3D_F32) {
        if (t.warp) return t.vecs == 2 ? block_norm_back_vec_kernel<kT, 2, true> : block_norm_back_vec_kernel<kT, 4, true>;
        return t.vecs == 2 ? block_norm_back_vec_kernel<kT, 2, false> : block_norm_back_vec_kernel<kT, 4, false>;
    } else {
        if (t.warp) return t.vecs == 1 ? block_norm_back_vec_kernel<kT, 1, true> : block_norm_back_vec_kernel<kT, 2, true>;
        return t.vecs == 1 ? block_norm_back_vec_kernel<kT, 1, false> : block_norm_back_vec_kernel<kT, 2, false>;
    }
}

// The ring kernels' shape for rows of `channels` elements of es bytes: threads of
// a block, blocks an SM, stages (0: the rows do not fit).
struct RingShape {
    int threads, per_sm, stages, smem;
};

RingShape ring_shape(int64_t channels, int es, int streams, int kept, int threads_per_sm) {
    RingShape r{};
    r.threads = int(up((channels + kRingE - 1) / kRingE, 32));
    if (r.threads > 512) return r;
    const int stage = int(channels) * es * streams, keep = r.threads * 64 * kept;
    for (r.per_sm = threads_per_sm / r.threads; r.per_sm >= 1; --r.per_sm) {
        r.stages = std::min(kRingBars, (227 * 1024 / r.per_sm - 1024 - 1024 - keep - 128) / stage);
        if (r.stages >= 2) break;
    }
    if (r.stages < 2) r.stages = 0;
    r.stages = std::min(r.stages, 4);
    r.smem = keep + r.stages * stage + 128;
    return r;
}

template <int kT>
NormFn ring_fn(bool layer, bool full) {
    if (layer) return full ? block_norm_ring_kernel<kT, true, true> : block_norm_ring_kernel<kT, true, false>;
    return full ? block_norm_ring_kernel<kT, false, true> : block_norm_ring_kernel<kT, false, false>;
}

template <int kT, bool kLayer>
NormFn ring_back_of(bool full, bool shift) {
    if (full)
        return shift ? block_norm_back_ring_kernel<kT, kLayer, true, true> : block_norm_back_ring_kernel<kT, kLayer, true, false>;
    return shift ? block_norm_back_ring_kernel<kT, kLayer, false, true> : block_norm_back_ring_kernel<kT, kLayer, false, false>;
}

template <int kT>
NormFn ring_back_fn(bool layer, bool full, bool shift) {
    return layer ? ring_back_of<kT, true>(full, shift) : ring_back_of<kT, false>(full, shift);
}

template <typename Fn>
int launch_ring(Fn fn, unsigned grid, const RingShape &shape, NormParams &p, cudaStream_t st) {
    p.stages = shape.stages;
    if (shape.smem > 48 * 1024 &&
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 226 * 1024) != cudaSuccess) {
        cudaGetLastError();
        return ROPE3D_ERR_CUDA;
    }
    return launch(fn, dim3(grid), dim3(unsigned(shape.threads)), size_t(shape.smem), p, st);
}

int forward(const rope3d_block_norm_args *a, bool run, bool check_device, cudaStream_t st) {
    if (!a || (!a->r && !a->n)) return ROPE3D_ERR_NULL;
    NormParams p;
    Span s[9];
    int rc = check_inputs(*a, p, s);
    if (rc != ROPE3D_OK) return rc;
    const int64_t R = a->rows, C = a->channels;
    if ((a->r && bad_ld(a->r_stride, C)) || (a->n && bad_ld(a->n_stride, C))) return ROPE3D_ERR_SHAPE;
    const int es = a->dtype == ROPE3D_F32 ? 4 : 2;
    s[7] = span(a->r, R, C, a->r_stride, es);
    s[8] = span(a->n, R, C, a->n_stride, es);
    const Span *all[9];
    for (int i = 0; i < 9; ++i) all[i] = &s[i];
    rc = check_align_device(all, 9, false);
    if (rc != ROPE3D_OK) return rc;
    for (int o = 7; o < 9; ++o)
        for (int i = 0; i < 7; ++i)
            if (overlap(s[o], s[i]) && !(i < 2 && same(s[o], s[i]))) return ROPE3D_ERR_ALIAS;
    if (overlap(s[7], s[8])) return ROPE3D_ERR_ALIAS;
    rc = check_align_device(all, 9, check_device);
    if (rc != ROPE3D_OK || !run) return rc;
    p.r = a->r; p.n = a->n; p.ldr = a->r_stride; p.ldn = a->n_stride;
    const int sms = sm_count();
    if (sms <= 0) return ROPE3D_ERR_CUDA;
    const int vec = 16 / es;
    const Team t = vectors(all, 9, C, vec) ? forward_team(C / vec) : Team{0, 0, false};
    if (t.vecs == 0) {
        t_norm_kernel = 2;
        return launch(block_norm_any_kernel, dim3(unsigned(std::min<int64_t>(R, int64_t(sms) * 8))),
                      dim3(kGeneralThreads), 0, p, st);
    }
    const RingShape shape = ring_shape(C, es, a->y ? 2 : 1, 3, 768);   // 80 registers a thread
    if (shape.stages && R >= int64_t(kSms) * shape.per_sm * 2) {
        t_norm_kernel = 3;
        const bool layer = p.post == ROPE3D_NORM_LAYER || p.pre == ROPE3D_NORM_LAYER, full = C == shape.threads * kRingE;
        const NormFn fn = a->dtype == ROPE3D_BF16 ? ring_fn<ROPE3D_BF16>(layer, full)
                          : a->dtype == ROPE3D_F16 ? ring_fn<ROPE3D_F16>(layer, full)
                                                   : ring_fn<ROPE3D_F32>(layer, full);
        return launch_ring(fn, unsigned(sms * shape.per_sm), shape, p, st);
    }
    t_norm_kernel = 1;
    const NormFn fn = a->dtype == ROPE3D_BF16 ? forward_fn<ROPE3D_BF16>(t)
                      : a->dtype == ROPE3D_F16 ? forward_fn<ROPE3D_F16>(t)
                                               : forward_fn<ROPE3D_F32>(t);
    const int block = t.warp ? 128 : t.threads;
    const int64_t teams = t.warp ? 4 : 1, need = (R + teams - 1) / teams;
    return launch(fn, dim3(unsigned(std::min<int64_t>(need, int64_t(sms) * (2048 / block)))), dim3(block), 0, p, st);
}

// One body for the call, its checks and its workspace query.
int backward(const rope3d_block_norm_backward_args *a, bool run, bool check_device, int64_t *need, cudaStream_t st) {
    if (!a || !a->dx || (!a->dr && !a->dn) || (a->fwd.y != nullptr) != (a->dy != nullptr)) return ROPE3D_ERR_NULL;
    const rope3d_block_norm_args &f = a->fwd;
    NormParams p;
    Span s[19];
    int rc = check_inputs(f, p, s);
    if (rc != ROPE3D_OK) return rc;
    if ((a->d_post_weight && !f.post_weight) || (a->d_gate && !f.gate) || (a->d_pre_weight && !f.pre_weight) ||
        (a->d_scale && !f.scale) || (a->d_shift && !f.shift))
        return ROPE3D_ERR_ARG;
    const int64_t R = f.rows, C = f.channels, G = p.groups;
    const bool group_grads = a->d_gate || a->d_scale || a->d_shift;
    if ((a->dr && bad_ld(a->dr_stride, C)) || (a->dn && bad_ld(a->dn_stride, C)) || bad_ld(a->dx_stride, C) ||
        (a->dy && bad_ld(a->dy_stride, C)) || (group_grads && bad_ld(a->grad_stride, C)))
        return ROPE3D_ERR_SHAPE;
    const int es = f.dtype == ROPE3D_F32 ? 4 : 2, ps = f.param_dtype == ROPE3D_F32 ? 4 : 2, vec = 16 / es;
    s[7] = span(a->dr, R, C, a->dr_stride, es);
    s[8] = span(a->dn, R, C, a->dn_stride, es);
    s[9] = span(a->dx, R, C, a->dx_stride, es);
    s[10] = span(a->dy, R, C, a->dy_stride, es);
    s[11] = span(a->d_post_weight, 1, C, C, ps);
    s[12] = span(a->d_pre_weight, 1, C, C, ps);
    s[13] = span(a->d_gate, G, C, a->grad_stride, ps);
    s[14] = span(a->d_scale, G, C, a->grad_stride, ps);
    s[15] = span(a->d_shift, G, C, a->grad_stride, ps);
    const Span *all[17];
    for (int i = 0; i < 16; ++i) all[i] = &s[i];
    rc = check_align_device(all, 16, false);
    if (rc != ROPE3D_OK) return rc;
    // the gradients are rows of dr and dn, which may be overwritten in place
    for (int o = 9; o < 16; ++o) {
        for (int i = 0; i < 9; ++i)
            if (overlap(s[o], s[i]) && !(o < 11 && i >= 7 && same(s[o], s[i]))) return ROPE3D_ERR_ALIAS;
        for (int q = o + 1; q < 16; ++q) {
            // gradients of one modulation tensor may interleave: rows of the same
            // stride, one behind the other
            const bool rows_of_one = o >= 13 && s[o].p && s[q].p &&
                                     std::abs(reinterpret_cast<intptr_t>(s[o].p) - reinterpret_cast<intptr_t>(s[q].p)) >= C * ps &&
                                     std::abs(reinterpret_cast<intptr_t>(s[o].p) - reinterpret_cast<intptr_t>(s[q].p)) <=
                                         (a->grad_stride - C) * ps;
            if (overlap(s[o], s[q]) && !rows_of_one) return ROPE3D_ERR_ALIAS;
        }
    }
    p.dr = a->dr; p.dn = a->dn; p.dx = a->dx; p.dy = a->dy;
    p.d_post_weight = a->d_post_weight; p.d_gate = a->d_gate; p.d_pre_weight = a->d_pre_weight;
    p.d_scale = a->d_scale; p.d_shift = a->d_shift;
    p.lddr = a->dr_stride; p.lddn = a->dn_stride; p.lddx = a->dx_stride; p.lddy = a->dy_stride;
    p.ldgrad = a->grad_stride;
    p.sums = group_grads || a->d_post_weight || a->d_pre_weight;
    const Team t = vectors(all, 16, C, vec) ? backward_team(C / vec, vec) : Team{0, 0, false};
    const int streams = 1 + (f.y != nullptr) + (a->dn != nullptr) + (a->dr != nullptr);
    RingShape shape = ring_shape(C, es, streams, 2, 512);   // 128 registers a thread
    bool ring = t.vecs && shape.stages && R >= kSms * shape.per_sm * 2;
    // Chunks: about as many as the GPU runs teams at once (or the general
    // kernel's column blocks), each of whole groups or a part of one.
    const int64_t target =
        ring     ? kSms * shape.per_sm
        : t.vecs ? (t.warp ? kSms * 16 : kSms * (t.threads > 256 ? 2 : t.threads > 128 ? 4 : 8))
               : std::max<int64_t>(1, kSms * 8 / ((C + kGeneralThreads - 1) / kGeneralThreads));
    const int64_t L = std::max<int64_t>(1, (R + target - 1) / target), rpg = p.rows_per_group;
    if (rpg >= L) {
        p.chunks_per_group = int((rpg + L - 1) / L);
        p.chunk_rows = int((rpg + p.chunks_per_group - 1) / p.chunks_per_group);
        p.chunks = int(G * p.chunks_per_group);
        p.groups_per_chunk = 0;
        if (p.chunks_per_group == 1) p.groups_per_chunk = 1;   // a chunk is one whole group
    } else {
        p.groups_per_chunk = int(L / rpg);
        p.chunks = int((G + p.groups_per_chunk - 1) / p.groups_per_chunk);
    }
    if (ring && p.groups_per_chunk) {   // the weights' sums take shared memory too
        shape = ring_shape(C, es, streams, 4, 512);
        ring = shape.stages > 0;
    }
    const bool partial = p.sums && (!p.groups_per_chunk || a->d_post_weight || a->d_pre_weight);
    const int64_t part_bytes = partial ? up(int64_t(p.chunks) * 3 * C * 4, 256) : 0;
    const int64_t stat_bytes = t.vecs || !p.sums ? 0 : up(R * 8 * 4, 256);
    const bool by_group = partial && !p.groups_per_chunk && G > 1 && (a->d_post_weight || a->d_pre_weight);
    const int64_t group_bytes = by_group ? up(G * 2 * C * 4, 256) : 0, bytes = part_bytes + stat_bytes + group_bytes;
    if (need) {
        *need = bytes;
        return ROPE3D_OK;
    }
    if (bytes) {
        if (!a->workspace) return ROPE3D_ERR_NULL;
        if (a->workspace_bytes < bytes) return ROPE3D_ERR_SCRATCH;
        s[16] = Span{a->workspace, bytes, 0, 256};
        for (int i = 0; i < 16; ++i)
            if (overlap(s[16], s[i])) return ROPE3D_ERR_ALIAS;
    } else {
        s[16] = Span{nullptr, 0, 0, 1};
    }
    all[16] = &s[16];
    rc = check_align_device(all, 17, check_device);
    if (rc != ROPE3D_OK || !run) return rc;
    char *ws = static_cast<char *>(a->workspace);
    p.part = partial ? reinterpret_cast<float *>(ws) : nullptr;
    p.group_sums = by_group ? reinterpret_cast<float *>(ws + part_bytes + stat_bytes) : nullptr;
    if (ring) {
        t_norm_kernel = 3;
        const bool layer = p.post == ROPE3D_NORM_LAYER || p.pre == ROPE3D_NORM_LAYER, full = C == shape.threads * kRingE;
        const NormFn fn = f.dtype == ROPE3D_BF16 ? ring_back_fn<ROPE3D_BF16>(layer, full, p.d_shift)
                          : f.dtype == ROPE3D_F16 ? ring_back_fn<ROPE3D_F16>(layer, full, p.d_shift)
                                                  : ring_back_fn<ROPE3D_F32>(layer, full, p.d_shift);
        rc = launch_ring(fn, unsigned(p.chunks), shape, p, st);
        if (rc != ROPE3D_OK) return rc;
    } else if (t.vecs) {
        t_norm_kernel = 1;
        const NormFn fn = f.dtype == ROPE3D_BF16 ? backward_fn<ROPE3D_BF16>(t)
                          : f.dtype == ROPE3D_F16 ? backward_fn<ROPE3D_F16>(t)
                                                  : backward_fn<ROPE3D_F32>(t);
        const int block = t.warp ? 128 : t.threads, teams = t.warp ? 4 : 1;
        const size_t smem = p.groups_per_chunk && p.sums ? size_t(2) * t.vecs * vec * block * 4 : 0;
        if (smem > 48 * 1024 &&
            cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 96 * 1024) != cudaSuccess) {
            cudaGetLastError();
            return ROPE3D_ERR_CUDA;
        }
        rc = launch(fn, dim3(unsigned((p.chunks + teams - 1) / teams)), dim3(block), smem, p, st);
        if (rc != ROPE3D_OK) return rc;
    } else {
        t_norm_kernel = 2;
        p.stats = p.sums ? reinterpret_cast<float *>(ws + part_bytes) : nullptr;
        rc = launch(block_norm_back_any_kernel, dim3(unsigned(std::min<int64_t>(R, kSms * 8))), dim3(kGeneralThreads), 0, p, st);
        if (rc != ROPE3D_OK) return rc;
        if (p.sums) {
            rc = launch(block_norm_back_cols_kernel,
                        dim3(unsigned((C + kGeneralThreads - 1) / kGeneralThreads), unsigned(std::min(p.chunks, 65535))),
                        dim3(kGeneralThreads), 0, p, st);
            if (rc != ROPE3D_OK) return rc;
        }
    }
    if (!partial) return ROPE3D_OK;
    // in split mode the groups are at most the chunks' target: far below 65535
    rc = launch(block_norm_finish_kernel, dim3(unsigned((C + 31) / 32), unsigned(p.groups_per_chunk ? 1 : G)),
                dim3(32 * kFinishRows), 0, p, st);
    if (rc != ROPE3D_OK || !by_group) return rc;
    return launch(block_norm_groups_kernel, dim3(unsigned((C + 127) / 128)), dim3(128), 0, p, st);
}

}  // namespace

extern "C" int rope3d_block_norm(const rope3d_block_norm_args *args, void *stream) {
    return forward(args, true, true, static_cast<cudaStream_t>(stream));
}

extern "C" int rope3d_block_norm_check(const rope3d_block_norm_args *args, int32_t check_device) {
    return forward(args, false, check_device != 0, nullptr);
}

extern "C" int rope3d_block_norm_backward(const rope3d_block_norm_backward_args *args, void *stream) {
    return backward(args, true, true, nullptr, static_cast<cudaStream_t>(stream));
}

extern "C" int rope3d_block_norm_backward_check(const rope3d_block_norm_backward_args *args, int32_t check_device) {
    return backward(args, false, check_device != 0, nullptr, nullptr);
}

extern "C" int rope3d_block_norm_backward_workspace(const rope3d_block_norm_backward_args *args, int64_t *bytes) {
    if (!bytes) return ROPE3D_ERR_NULL;
    return backward(args, false, false, bytes, nullptr);
}

extern "C" int rope3d_block_norm_last_kernel(void) { return t_norm_kernel; }

extern "C" int rope3d_testing_norm_wait_timeouts(int64_t *count, int32_t reset) {
    if (!count) return ROPE3D_ERR_NULL;
    unsigned int n = 0;
    if (cudaMemcpyFromSymbol(&n, g_norm_wait_timeouts, sizeof(n)) != cudaSuccess) {
        cudaGetLastError();
        return ROPE3D_ERR_CUDA;
    }
    if (reset) {
        const unsigned int zero = 0;
        if (cudaMemcpyToSymbol(g_norm_wait_timeouts, &zero, sizeof(zero)) != cudaSuccess) {
            cudaGetLastError();
            return ROPE3D_ERR_CUDA;
        }
    }
    *count = n;
    return ROPE3D_OK;
}
