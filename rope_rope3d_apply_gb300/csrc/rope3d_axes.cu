// rope3d_axes.cu -- rotary positions with several axes, given token by token:
// rope3d_apply_axes (and, with `inverse`, its gradient) and rope3d_cache_append,
// which writes the rotated keys and the values straight into the pages of a cache.
//
// Pair j of every head turns by angle = positions[axis(j)][token] * freqs[j]:
//     y_a = a cos - b sin,  y_b = a sin + b cos
// in fp32, each product and sum rounded by itself as in rope3d_apply_pair, then
// one cast. A rotation's transpose is the rotation by -angle, so the gradient
// is the same kernel with sin negated.
//
// The angle is never formed: what whole turns leave over, frac(position * freq / 2
// pi), is taken from a product with its error (freq / 2 pi split into two floats, the error by
// fma; two doubles where a position has no exact float or the turns are more than 2^21), and
// sincospi takes it from there. The error is that of sincospi, at position 2^20 as at 0.
//
// Each block takes tiles of a few tokens: cos and sin of the tile's tokens and pairs
// go into shared memory once (64 sincospi a token instead of 64 for each of its
// heads), then each thread moves 16-byte vectors at one place of head rows, four loads in
// flight; warps that are done with a tile prepare the next one's while the others move.
// Cosines and sines lie apart, so that a warp's 16-byte reads of either meet no bank twice.
// What bounds it is memory: 65,536 tokens of 2 x 16 heads of 128, bf16, out of a fused projection
// 172 us, 6,250 GB/s, 93 % of a copy on the same GPU; fp32 334 us, 6,450 GB/s. 5,138 new tokens of 8 / 4
// heads of 256 into pages take 20.3 us, 4,150 GB/s (16 where the inputs lie in L2): each block has one tile, whose
// loads wait for its cosines. Small calls: the launch. Single pairs are bound by their loads of single
// elements: the first of these with 63 pairs in halves 740 us, at odd addresses 554, in fp32 there 384.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "../../include/rope3d.h"
#include "rope3d_internal.h"
#include "rope3d_paged.h"
#include "rope3d_tc.cuh"

namespace {

using rope3d::FastDiv;
using rope3d::make_fastdiv;
using namespace rope3d_paged;

constexpr int kThreads = 256;
constexpr int kBlocks = 4;       // blocks that fit an SM beside one another
constexpr int kMaxTile = 32;     // tokens of a tile

__device__ __forceinline__ uint32_t fdiv(uint32_t n, const FastDiv &f) { return (__umulhi(n, f.mul) + n) >> f.shift; }

// Where a token's heads lie.
struct Rows {
    const char *p;
    int64_t token, head;   // bytes
};

struct AxesParams {
    Rows in[3], out[3];        // q, k, v; out of k and v: the caches (token unused) in an append
    int64_t slot[2], page[2];  // bytes: the caches' strides
    const void *positions;
    const float *freqs;
    int64_t positions_stride;
    int *invalid;
    Batch batch;
    int tokens, tile, pairs, head_dim;
    int end0, end1;            // pairs of axis 0; of axes 0 and 1
    int heads[3];              // q, k, v
    int per_head, rotating;    // units of a head row; those that rotate (the rest are copied)
    int heads_all;             // head rows of a token
    // How a block's threads divide a tile: `lanes` to a head row, `heads_step` head rows
    // of `tokens_step` tokens at a time.
    FastDiv lanes, heads_step;
    int tokens_step;
    int position_type;         // ROPE3D_POSITIONS_*; -1: the place in the sequence
    float sign;
};

// ---- angles ----------------------------------------------------------------------

constexpr double kInvTwoPi = 0.15915494309189535, kInvTwoPiLow = -9.839338337591243e-18;   // 1 / 2 pi
constexpr float kNear = 2097152.f;   // turns up to which two floats and the product's error do: 2^21

// cos and sin of 2 pi t, t = (whole turns +) a + e with a's whole turns taken off.
__device__ __forceinline__ float2 of_turns(float a, float e) {
    const float t = __fadd_rn(a, e);
    const float rest = __fsub_rn(e, __fsub_rn(t, a)) * 6.2831853f;
    float s, c;
    sincospif(2.0f * t, &s, &c);
    return make_float2(__fmaf_rn(-s, rest, c), __fmaf_rn(c, rest, s));
}

// The same of pos * freq / 2 pi in fp64, the product with what it drops.
__device__ __noinline__ float2 turn_far(double pos, float freq) {
    const double f = double(freq), c = f * kInvTwoPi, c_low = fma(f, kInvTwoPi, -c) + f * kInvTwoPiLow;
    const double a = pos * c, e = fma(pos, c, -a) + pos * c_low, r = a - rint(a);   // (r exact)
    const float hi = float(r);
    return of_turns(hi, float(r - double(hi) + e));
}

// cos and sin of 2 pi pos freq / (2 pi), from freq / 2 pi = hi + lo; false where it is too far.
__device__ __forceinline__ bool turn(float pos, float hi, float lo, float2 &cs) {
    const float a = __fmul_rn(pos, hi);
    const float e = __fmaf_rn(pos, lo, __fmaf_rn(pos, hi, -a));   // what the product dropped
    cs = of_turns(__fsub_rn(a, rintf(a)), e);                     // (the difference is exact)
    return fabsf(a) <= kNear;
}

// ---- elements --------------------------------------------------------------------

template <int kType>
__device__ __forceinline__ void widen(const uint4 &v, float *f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kType == ROPE3D_F32) {
            f[i] = __uint_as_float(w[i]);
        } else if constexpr (kType == ROPE3D_BF16) {
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

template <int kType>
__device__ __forceinline__ uint4 narrow(const float *f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kType == ROPE3D_F32) {
            w[i] = __float_as_uint(f[i]);
        } else if constexpr (kType == ROPE3D_BF16) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            memcpy(&w[i], &b, 4);
        } else {
            const __half2 b = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            memcpy(&w[i], &b, 4);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int kType>
__device__ __forceinline__ float load1(const char *p) {
    if constexpr (kType == ROPE3D_F32) return *reinterpret_cast<const float *>(p);
    else if constexpr (kType == ROPE3D_BF16) return __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(p));
    else return __half2float(*reinterpret_cast<const __half *>(p));
}

template <int kType>
__device__ __forceinline__ void store1(char *p, float v) {
    if constexpr (kType == ROPE3D_F32) *reinterpret_cast<float *>(p) = v;
    else if constexpr (kType == ROPE3D_BF16) *reinterpret_cast<__nv_bfloat16 *>(p) = __float2bfloat16_rn(v);
    else *reinterpret_cast<__half *>(p) = __float2half_rn(v);
}

__device__ __forceinline__ float2 rotate(float a, float b, float c, float s) {
    return make_float2(__fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)), __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c)));
}

// kN consecutive floats of shared memory, in the widest words that kN is whole in.
template <int kN>
__device__ __forceinline__ void load_floats(float *v, const float *from) {
    if constexpr (kN % 4 == 0) {
#pragma unroll
        for (int i = 0; i < kN; i += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(from + i);
            v[i] = f.x;
            v[i + 1] = f.y;
            v[i + 2] = f.z;
            v[i + 3] = f.w;
        }
    } else {
        static_assert(kN == 2, "two pairs of fp32");
        const float2 f = *reinterpret_cast<const float2 *>(from);
        v[0] = f.x;
        v[1] = f.y;
    }
}

__device__ __forceinline__ uint4 ld_stream(const char *p) {   // coherent: in place is allowed
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
    return r;
}

// ---- the kernel ------------------------------------------------------------------

// kVec: units of 16 bytes (kHalves: two of them, the parts of 16 bytes' worth of
// pairs), else single pairs and elements.
template <int kType, bool kHalves, bool kAppend, bool kVec>
__global__ void __launch_bounds__(kThreads, kBlocks) axes_kernel(const __grid_constant__ AxesParams p) {
    constexpr int kElem = kType == ROPE3D_F32 ? 4 : 2;
    constexpr int kV = kVec ? 16 / kElem : 1;   // elements of a vector
    constexpr int kInFlight = kVec && kHalves ? 2 : 4;   // units of a thread's loads in flight: 64 bytes
    // [2 buffers][cos, sin][tile][pairs], then freq / 2 pi as high and low parts [2][pairs]
    extern __shared__ __align__(16) float s_tiles[];
    const int tile_pairs = p.tile * p.pairs;
    float *s_freq = s_tiles + 4 * tile_pairs;
    __shared__ int64_t s_dst[2][2][kMaxTile];   // append: byte offsets in the caches, -1: nowhere
    __shared__ int s_live[2][kMaxTile];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    rope3d_tc::grid_release();
    rope3d_tc::grid_wait();
    for (int j = tid; j < p.pairs; j += kThreads) {
        const double f = double(p.freqs[j]) * kInvTwoPi;
        const float hi = float(f);
        s_freq[j] = hi;
        s_freq[p.pairs + j] = float(f - double(hi));
    }
    const int64_t second = int64_t(p.pairs) * kElem;
    const uint32_t row = fdiv(uint32_t(tid), p.lanes);
    const int token_at = int(fdiv(row, p.heads_step)), head_at = int(row - uint32_t(token_at) * p.heads_step.d);
    const int at0 = token_at < p.tokens_step ? tid - int(row * p.lanes.d) : p.per_head;   // (the last few have no row)

    // A warp's tokens of the tile at t0: their places, cosines and sines
    auto prepare = [&](int t0, int buf) {
        const int count = min(p.tile, p.tokens - t0);
        for (int i = warp; i < count; i += kThreads / 32) {
            const int t = t0 + i;
            int place = 0;
            if constexpr (kAppend) {
                const Batch &b = p.batch;
                int s = 0, lo, hi, len;
                if (b.starts) {   // the last sequence that starts at or before t
                    int above = b.seqs;
                    while (above - s > 1) {
                        const int mid = (s + above) >> 1;
                        if (b.starts[mid] <= t) s = mid;
                        else above = mid;
                    }
                } else {
                    s = t / (b.tokens / b.seqs);
                }
                sequence(b, s, lo, hi, len);
                const bool live = t >= lo && t < hi;
                place = len - hi + t;
                if (lane == 0) {
                    int64_t k = -1, v = -1;
                    if (live) {
                        const int page = place < 0 ? -1 : b.table[s * b.table_stride + place / b.page_size];
                        if (page >= 0 && page < b.pages) {
                            const int slot = place % b.page_size;
                            k = page * p.page[0] + slot * p.slot[0];
                            v = page * p.page[1] + slot * p.slot[1];
                        } else if (p.invalid) {
                            atomicAdd(p.invalid, 1);
                        }
                    }
                    s_dst[buf][0][i] = k;
                    s_dst[buf][1][i] = v;
                    s_live[buf][i] = live;
                }
                if (!live) continue;
            }
            // lane x has the position on axis x; as a float where that is exact
            int64_t whole = place;
            float near = float(place);
            bool exact = true;
            if (!kAppend || p.position_type >= 0) {
                const int axis = lane < 1 || p.end0 == p.pairs ? 0 : lane < 2 || p.end1 == p.pairs ? 1 : 2;   // (those that have pairs)
                const int64_t at = axis * p.positions_stride + t;
                if (p.position_type == ROPE3D_POSITIONS_F32) {
                    near = static_cast<const float *>(p.positions)[at];   // (`far` is made of it)
                } else {
                    whole = p.position_type == ROPE3D_POSITIONS_I64 ? static_cast<const int64_t *>(p.positions)[at]
                                                                    : static_cast<const int32_t *>(p.positions)[at];
                    exact = whole >= -(1 << 24) && whole <= (1 << 24);
                    near = exact ? float(int(whole)) : 0.f;
                }
            } else {
                exact = place >= -(1 << 24) && place <= (1 << 24);   // (below 0: a sequence shorter than its new tokens)
            }
            const bool all_near = __all_sync(0xffffffffu, exact);
            for (int j0 = 0; j0 < p.pairs; j0 += 32) {
                const int j = j0 + lane, axis = j < p.end0 ? 0 : j < p.end1 ? 1 : 2;
                const float at = __shfl_sync(0xffffffffu, near, axis);
                bool is_near = all_near || __shfl_sync(0xffffffffu, int(exact), axis);
                const int64_t far = __shfl_sync(0xffffffffu, whole, axis);
                if (j >= p.pairs) continue;
                float2 cs;
                is_near = turn(at, s_freq[j], s_freq[p.pairs + j], cs) && is_near;
                if (!is_near) {
                    const bool fractions = !(kAppend && p.position_type < 0) && p.position_type == ROPE3D_POSITIONS_F32;
                    cs = turn_far(fractions ? double(at) : double(far), p.freqs[j]);
                }
                float *to = s_tiles + 2 * buf * tile_pairs + i * p.pairs + j;
                to[0] = cs.x;
                to[tile_pairs] = cs.y * p.sign;
            }
        }
    };
    __syncthreads();   // s_freq is there
    const int step = int(gridDim.x) * p.tile;
    int t0 = blockIdx.x * p.tile;
    if (t0 < p.tokens) prepare(t0, 0);
    for (int buf = 0; t0 < p.tokens; t0 += step, buf ^= 1) {
        __syncthreads();   // this tile is prepared, and the one before moved
        const int count = min(p.tile, p.tokens - t0);
        const float *const s_cos = s_tiles + 2 * buf * tile_pairs;
        for (int at = at0; at < p.per_head; at += p.lanes.d) {
            // this thread's part of each of its rows: its first element and, where it turns, its
            // first pair (interleaved units lie in order; of halves', the first parts do, and behind
            // the second parts come the units that are copied)
            const bool turning = at < p.rotating;
            const int first = kHalves ? (turning ? at : at + p.rotating) * kV
                              : kVec  ? at * kV
                                      : (turning ? 2 * at : at + p.rotating);
            const int pair = kVec && !kHalves ? at * kV / 2 : at * kV;
            // both parts of a pair, where they are two loads
            const bool two = turning && (kHalves || !kVec);
            for (int head = head_at; head < p.heads_all; head += int(p.heads_step.d)) {
                int h = head, which = 0;
                if (h >= p.heads[0]) {
                    h -= p.heads[0];
                    which = 1;
                    if (kAppend && h >= p.heads[1]) {
                        h -= p.heads[1];
                        which = 2;
                    }
                }
                const Rows &in = p.in[which], &out = p.out[which];
                const char *const from = in.p + t0 * in.token + h * in.head + int64_t(first) * kElem;
                char *const to = const_cast<char *>(out.p) + t0 * out.token + h * out.head + int64_t(first) * kElem;
                const bool turns = turning && which < 2;
                const float *const of_pair = s_cos + pair;
                // token i's place; false where it has none
                auto place = [&](int i, char *&dst) {
                    if (kAppend && which > 0) {
                        const int64_t d = s_dst[buf][which - 1][i];
                        dst = to + d;   // (the caches' token strides are 0)
                        return d >= 0;
                    }
                    dst = to + i * out.token;
                    return !kAppend || s_live[buf][i] != 0;
                };
                for (int i0 = token_at; i0 < count; i0 += p.tokens_step * kInFlight) {
                    bool on[kInFlight];
                    char *dst;
                    if constexpr (kVec) {
                        uint4 a[kInFlight], b[kHalves ? kInFlight : 1];
#pragma unroll
                        for (int q = 0; q < kInFlight; ++q) {
                            const int i = i0 + q * p.tokens_step;
                            on[q] = i < count && place(i, dst);
                            if (on[q]) {
                                a[q] = ld_stream(from + i * in.token);
                                if constexpr (kHalves)
                                    if (two) b[q] = ld_stream(from + i * in.token + second);
                            }
                        }
#pragma unroll
                        for (int q = 0; q < kInFlight; ++q) {
                            if (!on[q]) continue;
                            const int i = i0 + q * p.tokens_step;
                            if (turns) {
                                // (a thread's pairs begin at 16 bytes: they are whole vectors of elements)
                                constexpr int kN = kHalves ? kV : kV / 2;
                                float x[kV], y[kV], c[kN], s[kN];
                                const float *at_pair = of_pair + i * p.pairs;
                                load_floats<kN>(c, at_pair);
                                load_floats<kN>(s, at_pair + tile_pairs);
                                widen<kType>(a[q], x);
                                if constexpr (kHalves) {
                                    widen<kType>(b[q], y);
#pragma unroll
                                    for (int e = 0; e < kV; ++e) {
                                        const float2 r = rotate(x[e], y[e], c[e], s[e]);
                                        x[e] = r.x;
                                        y[e] = r.y;
                                    }
                                    b[q] = narrow<kType>(y);
                                } else {
#pragma unroll
                                    for (int e = 0; e < kV; e += 2) {
                                        const float2 r = rotate(x[e], x[e + 1], c[e / 2], s[e / 2]);
                                        x[e] = r.x;
                                        x[e + 1] = r.y;
                                    }
                                }
                                a[q] = narrow<kType>(x);
                            }
                            place(i, dst);
                            __stcs(reinterpret_cast<uint4 *>(dst), a[q]);
                            if constexpr (kHalves)
                                if (two) __stcs(reinterpret_cast<uint4 *>(dst + second), b[q]);
                        }
                    } else {
                        const int64_t next = kHalves ? second : kElem;
                        float x[kInFlight], y[kInFlight];
#pragma unroll
                        for (int q = 0; q < kInFlight; ++q) {
                            const int i = i0 + q * p.tokens_step;
                            on[q] = i < count && place(i, dst);
                            if (on[q]) {
                                x[q] = load1<kType>(from + i * in.token);
                                if (two) y[q] = load1<kType>(from + i * in.token + next);
                            }
                        }
#pragma unroll
                        for (int q = 0; q < kInFlight; ++q) {
                            if (!on[q]) continue;
                            const int i = i0 + q * p.tokens_step;
                            if (turns) {
                                const float2 r = rotate(x[q], y[q], of_pair[i * p.pairs], of_pair[i * p.pairs + tile_pairs]);
                                x[q] = r.x;
                                y[q] = r.y;
                            }
                            place(i, dst);
                            store1<kType>(dst, x[q]);
                            if (two) store1<kType>(dst + next, y[q]);
                        }
                    }
                }
            }
        }
        if (t0 + step < p.tokens) prepare(t0 + step, buf ^ 1);   // while other warps still move this one
    }
}

using Kernel = void (*)(AxesParams);

template <bool kAppend, int kType>
Kernel kernel_of(bool halves, bool vec) {
    if (halves) return vec ? axes_kernel<kType, true, kAppend, true> : axes_kernel<kType, true, kAppend, false>;
    return vec ? axes_kernel<kType, false, kAppend, true> : axes_kernel<kType, false, kAppend, false>;
}

// ---- host --------------------------------------------------------------------------

thread_local int t_axes_kernel = 0;   // 1 vectors, 2 single pairs: this thread's last call

constexpr int64_t kMaxPairs = 1024;
constexpr int kTilePairs = 2048;      // tokens x pairs of a tile of more than one token
static_assert(kMaxPairs <= kTilePairs, "nor are a token's more");

// Shared memory of tiles of `tile` tokens: cosines and sines of two tiles, and a token's
// frequencies as two floats each.
constexpr size_t tile_bytes(int64_t tile, int64_t pairs) { return size_t(2 * tile + 1) * 2 * size_t(pairs) * sizeof(float); }
// (most where 2048 pairs are whole tiles: 40 KB, beside the kernel's static arrays)
static_assert(tile_bytes(kTilePairs / kMaxPairs, kMaxPairs) + 2 * 2 * kMaxTile * sizeof(int64_t) + 2 * kMaxTile * sizeof(int) <= 48 * 1024,
              "what a launch has without asking for more");

int elem_of(int32_t dtype) { return dtype == ROPE3D_F32 ? 4 : dtype == ROPE3D_BF16 || dtype == ROPE3D_F16 ? 2 : 0; }

int check_rotation(const int32_t *sections, int64_t head_dim, int32_t pairing, int *pairs) {
    int64_t n = 0;
    for (int i = 0; i < 3; ++i) {
        if (sections[i] < 0 || sections[i] > kMaxPairs) return ROPE3D_ERR_SHAPE;
        n += sections[i];
    }
    if (n <= 0 || n > kMaxPairs || 2 * n > head_dim) return ROPE3D_ERR_SHAPE;
    if (pairing != ROPE3D_PAIRS_INTERLEAVED && pairing != ROPE3D_PAIRS_HALVES) return ROPE3D_ERR_ARG;
    *pairs = int(n);
    return ROPE3D_OK;
}

int position_bytes(int32_t type) {
    return type == ROPE3D_POSITIONS_I64 ? 8 : type == ROPE3D_POSITIONS_I32 || type == ROPE3D_POSITIONS_F32 ? 4 : 0;
}

View positions_view(const void *p, int32_t type, const int32_t *sections, int64_t tokens, int64_t stride) {
    int axes = 1;   // rows that are read: up to the last axis that has pairs
    for (int i = 1; i < 3; ++i)
        if (sections[i]) axes = i + 1;
    return view(p, position_bytes(type), tokens, axes, stride);
}

Rows rows_of(const void *p, int64_t token, int64_t head, int elem) {
    return Rows{static_cast<const char *>(p), token * elem, head * elem};
}

template <bool kAppend>
int run(AxesParams &p, int32_t dtype, bool halves, bool vec, const int32_t *sections, cudaStream_t st) {
    const int sms = sm_count();
    if (sms <= 0) return ROPE3D_ERR_CUDA;
    const int v = vec ? 16 / elem_of(dtype) : 1;
    const int rest = (p.head_dim - 2 * p.pairs) / v;   // units that are only copied
    p.rotating = halves || !vec ? p.pairs / v : 2 * p.pairs / v;
    p.per_head = p.rotating + rest;
    p.heads_all = p.heads[0] + p.heads[1] + p.heads[2];
    p.lanes = make_fastdiv(uint32_t(std::min(p.per_head, kThreads)));
    const int rows = kThreads / int(p.lanes.d);
    p.heads_step = make_fastdiv(uint32_t(std::min(rows, p.heads_all)));
    p.tokens_step = rows / int(p.heads_step.d);
    p.end0 = sections[0];
    p.end1 = sections[0] + sections[1];
    // Tiles of one size for every resident block: cos and sin take 16 KB a tile at most, 32 KB with
    // the next one's, and the frequencies up to 8 KB.
    const int most = std::min(kMaxTile, kTilePairs / std::max(p.pairs, 1)), blocks = sms * kBlocks;
    const int rounds = int((int64_t(p.tokens) + int64_t(blocks) * most - 1) / (int64_t(blocks) * most));
    const int tile = int((int64_t(p.tokens) + int64_t(blocks) * rounds - 1) / (int64_t(blocks) * rounds));
    p.tile = tile;
    const size_t smem = tile_bytes(tile, p.pairs);
    const int tiles = (p.tokens + tile - 1) / tile;
    const Kernel fn = dtype == ROPE3D_BF16  ? kernel_of<kAppend, ROPE3D_BF16>(halves, vec)
                      : dtype == ROPE3D_F16 ? kernel_of<kAppend, ROPE3D_F16>(halves, vec)
                                            : kernel_of<kAppend, ROPE3D_F32>(halves, vec);
    const int rc = launch(fn, dim3(unsigned(std::min(tiles, blocks))), kThreads, smem, st, p);
    if (rc == ROPE3D_OK) t_axes_kernel = vec ? 1 : 2;
    return rc;
}

int apply(const rope3d_apply_axes_args *a, bool go, bool check_device, cudaStream_t st) {
    if (!a || !a->q || !a->q_out || !a->positions || !a->freqs || (a->k == nullptr) != (a->k_out == nullptr))
        return ROPE3D_ERR_NULL;
    const int64_t T = a->tokens, D = a->head_dim, H = a->q_heads, K = a->k ? a->k_heads : 0;
    if (T <= 0 || T > kMaxTokens || D <= 0 || D > ROPE3D_MAX_HEAD_DIM || H <= 0 || H > kMaxHeads || K < 0 || K > kMaxHeads ||
        (a->k && K == 0))
        return ROPE3D_ERR_SHAPE;
    const int es = elem_of(a->dtype);
    if (!es || !position_bytes(a->position_type)) return ROPE3D_ERR_DTYPE;
    AxesParams p{};
    int rc = check_rotation(a->sections, D, a->pairing, &p.pairs);
    if (rc != ROPE3D_OK) return rc;
    const View q = view(a->q, es, D, T, a->q_token_stride, H, a->q_head_stride);
    const View k = view(a->k, es, D, T, a->k_token_stride, K, a->k_head_stride);
    const View qo = view(a->q_out, es, D, T, a->q_out_token_stride, H, a->q_out_head_stride);
    const View ko = view(a->k_out, es, D, T, a->k_out_token_stride, K, a->k_out_head_stride);
    const View pos = positions_view(a->positions, a->position_type, a->sections, T, a->positions_stride);
    const View freqs = view(a->freqs, 4, p.pairs, 1, 0);
    if (bad_strides(q) || bad_strides(qo) || (a->k && (bad_strides(k) || bad_strides(ko))) || bad_strides(pos)) return ROPE3D_ERR_SHAPE;
    if (!rows_apart(qo) || (a->k && !rows_apart(ko))) return ROPE3D_ERR_SHAPE;
    for (const View *v : {&q, &k, &qo, &ko, &pos, &freqs})
        if (!aligned(v->p, v->elem)) return ROPE3D_ERR_ALIGN;
    for (const View *out : {&qo, &ko}) {
        const View &own = out == &qo ? q : k, &other = out == &qo ? k : q;
        if (may_meet(*out, own) && !same_view(*out, own)) return ROPE3D_ERR_ALIAS;
        if (may_meet(*out, other) || may_meet(*out, pos) || may_meet(*out, freqs)) return ROPE3D_ERR_ALIAS;
    }
    if (may_meet(qo, ko)) return ROPE3D_ERR_ALIAS;
    if (check_device) {
        const void *const all[] = {a->q, a->k, a->q_out, a->k_out, a->positions, a->freqs};
        if ((rc = on_current_device(all, 6)) != ROPE3D_OK) return rc;
    }
    if (!go) return ROPE3D_OK;
    const bool halves = a->pairing == ROPE3D_PAIRS_HALVES;
    const int v = 16 / es;
    const bool vec = vectors(q) && vectors(qo) && vectors(k) && vectors(ko) && (halves ? p.pairs : 2 * p.pairs) % v == 0;
    p.in[0] = rows_of(a->q, a->q_token_stride, a->q_head_stride, es);
    p.in[1] = rows_of(a->k, a->k_token_stride, a->k_head_stride, es);
    p.out[0] = rows_of(a->q_out, a->q_out_token_stride, a->q_out_head_stride, es);
    p.out[1] = rows_of(a->k_out, a->k_out_token_stride, a->k_out_head_stride, es);
    p.positions = a->positions;
    p.positions_stride = a->positions_stride;
    p.position_type = a->position_type;
    p.freqs = static_cast<const float *>(a->freqs);
    p.tokens = int(T);
    p.head_dim = int(D);
    p.heads[0] = int(H);
    p.heads[1] = int(K);
    p.sign = a->inverse ? -1.0f : 1.0f;
    return run<false>(p, a->dtype, halves, vec, a->sections, st);
}

int append(const rope3d_cache_append_args *a, bool go, bool check_device, cudaStream_t st) {
    if (!a || !a->k || !a->v || !a->k_cache || !a->v_cache || (a->q == nullptr) != (a->q_out == nullptr))
        return ROPE3D_ERR_NULL;
    const rope3d_paged_batch &b = a->batch;
    const int64_t T = a->tokens, D = a->head_dim, H = a->q ? a->q_heads : 0, K = a->kv_heads;
    if (T <= 0 || T > kMaxTokens || D <= 0 || D > ROPE3D_MAX_HEAD_DIM || H < 0 || H > kMaxHeads || K <= 0 || K > kMaxHeads ||
        (a->q && H == 0))
        return ROPE3D_ERR_SHAPE;
    int rc = check_batch(b, T);
    if (rc != ROPE3D_OK) return rc;
    const int es = elem_of(a->dtype);
    if (!es || (a->positions && !position_bytes(a->position_type))) return ROPE3D_ERR_DTYPE;
    AxesParams p{};
    if (a->freqs) {
        if ((rc = check_rotation(a->sections, D, a->pairing, &p.pairs)) != ROPE3D_OK) return rc;
    } else if (a->q || a->positions) {
        return ROPE3D_ERR_ARG;   // nothing to rotate by
    }
    const View q = view(a->q, es, D, T, a->q_token_stride, H, a->q_head_stride);
    const View qo = view(a->q_out, es, D, T, a->q_out_token_stride, H, a->q_out_head_stride);
    const View k = view(a->k, es, D, T, a->k_token_stride, K, a->k_head_stride);
    const View v = view(a->v, es, D, T, a->v_token_stride, K, a->v_head_stride);
    const View kc = view(a->k_cache, es, D, b.pages, a->k_page_stride, b.page_size, a->k_slot_stride, K, a->k_cache_head_stride);
    const View vc = view(a->v_cache, es, D, b.pages, a->v_page_stride, b.page_size, a->v_slot_stride, K, a->v_cache_head_stride);
    const View pos = a->positions ? positions_view(a->positions, a->position_type, a->sections, T, a->positions_stride)
                                  : View{nullptr, 1, {1, 1, 1}, {0, 0, 0}, 4};
    const View freqs = view(a->freqs, 4, std::max(p.pairs, 1), 1, 0);
    const View table = view(b.page_table, 4, b.table_width, b.seqs, b.table_stride), lens = view(b.seq_lens, 4, b.seqs, 1, 0),
               starts = view(b.q_starts, 4, b.seqs + 1, 1, 0), bad = view(a->invalid_count, 4, 1, 1, 0);
    for (const View *w : {&q, &qo, &k, &v, &kc, &vc, &pos})
        if (w->p && bad_strides(*w)) return ROPE3D_ERR_SHAPE;
    if ((a->q && !rows_apart(qo)) || !rows_apart(kc) || !rows_apart(vc)) return ROPE3D_ERR_SHAPE;
    for (const View *w : {&q, &qo, &k, &v, &kc, &vc, &pos, &freqs, &bad})
        if (!aligned(w->p, w->elem)) return ROPE3D_ERR_ALIGN;
    if (may_meet(qo, q) && !same_view(qo, q)) return ROPE3D_ERR_ALIAS;
    for (const View *out : {&qo, &kc, &vc, &bad}) {
        if (out != &qo && may_meet(*out, q)) return ROPE3D_ERR_ALIAS;
        for (const View *in : {&k, &v, &pos, &freqs, &table, &lens, &starts})
            if (may_meet(*out, *in)) return ROPE3D_ERR_ALIAS;
    }
    if (may_meet(qo, kc) || may_meet(qo, vc) || may_meet(kc, vc) || may_meet(bad, qo) || may_meet(bad, kc) || may_meet(bad, vc))
        return ROPE3D_ERR_ALIAS;
    if (check_device) {
        const void *const all[] = {a->q, a->q_out, a->k, a->v, a->k_cache, a->v_cache, a->positions, a->freqs,
                                   b.page_table, b.seq_lens, b.q_starts, a->invalid_count};
        if ((rc = on_current_device(all, 12)) != ROPE3D_OK) return rc;
    }
    if (!go) return ROPE3D_OK;
    const bool halves = a->freqs && a->pairing == ROPE3D_PAIRS_HALVES;
    const int n = 16 / es;
    const bool vec = vectors(q) && vectors(qo) && vectors(k) && vectors(v) && vectors(kc) && vectors(vc) &&
                     (halves ? p.pairs : 2 * p.pairs) % n == 0;
    p.in[0] = rows_of(a->q, a->q_token_stride, a->q_head_stride, es);
    p.in[1] = rows_of(a->k, a->k_token_stride, a->k_head_stride, es);
    p.in[2] = rows_of(a->v, a->v_token_stride, a->v_head_stride, es);
    p.out[0] = rows_of(a->q_out, a->q_out_token_stride, a->q_out_head_stride, es);
    p.out[1] = rows_of(a->k_cache, 0, a->k_cache_head_stride, es);
    p.out[2] = rows_of(a->v_cache, 0, a->v_cache_head_stride, es);
    p.page[0] = a->k_page_stride * es;
    p.page[1] = a->v_page_stride * es;
    p.slot[0] = a->k_slot_stride * es;
    p.slot[1] = a->v_slot_stride * es;
    p.positions = a->positions;
    p.positions_stride = a->positions_stride;
    p.position_type = a->positions ? a->position_type : -1;
    p.freqs = static_cast<const float *>(a->freqs);   // (none: no pairs, and none is read)
    p.invalid = a->invalid_count;
    p.batch = device_batch(b, T);
    p.tokens = int(T);
    p.head_dim = int(D);
    p.heads[0] = int(H);
    p.heads[1] = p.heads[2] = int(K);
    p.sign = 1.0f;
    const int32_t none[3] = {0, 0, 0};
    return run<true>(p, a->dtype, halves, vec, a->freqs ? a->sections : none, st);
}

}  // namespace

extern "C" int rope3d_apply_axes(const rope3d_apply_axes_args *args, void *stream) {
    return apply(args, true, true, static_cast<cudaStream_t>(stream));
}

extern "C" int rope3d_apply_axes_check(const rope3d_apply_axes_args *args, int32_t check_device) {
    return apply(args, false, check_device != 0, nullptr);
}

extern "C" int rope3d_cache_append(const rope3d_cache_append_args *args, void *stream) {
    return append(args, true, true, static_cast<cudaStream_t>(stream));
}

extern "C" int rope3d_cache_append_check(const rope3d_cache_append_args *args, int32_t check_device) {
    return append(args, false, check_device != 0, nullptr);
}

extern "C" int rope3d_apply_axes_last_kernel(void) { return t_axes_kernel; }
