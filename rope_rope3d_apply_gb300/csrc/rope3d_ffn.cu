// rope3d_ffn.cu -- the gated feed-forward of a transformer block and its
// backward pass: rope3d_gated_ffn, rope3d_gated_ffn_backward.
//
//   g = x Wg^T, u = x Wu^T, h = act(g) * u, y = h Wd^T
// with x [tokens, width], Wg and Wu [hidden, width], Wd [width, hidden]; and,
// for a gradient dy of y,
//   dh = dy Wd, dg = dh * u * act'(g), du = dh * act(g),
//   dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, dWd = dy^T h.
//
// Every product is one of three forms of C[i, j] = sum_k A(i, k) B(j, k):
//   x Wg^T | x Wu^T and h Wd^T     both operands K-major (rows along k)
//   dy Wd, dg Wg + du Wu           A K-major, B MN-major (rows across k)
//   dg^T x, du^T x, dy^T h         both MN-major
// which the fifth-generation tensor cores read as they lie in memory, so no
// matrix is ever transposed. Two kernels compute them:
//   ffn_tile_kernel    pairs of CTAs, 256-row tiles (many tokens; the weights'
//                      gradients always): bound by the tensor cores
//   ffn_stream_kernel  few tokens: a tile is 128 weight rows by all the tokens,
//                      its k range split over a cluster: bound by reading the
//                      weights from memory
// Products accumulate in fp32 in tensor memory; g and u reach the activation
// there without a rounding. The roundings to 16 bits are the operands of the
// next product (h, dg, du: the tensor cores take 16-bit operands) and the
// outputs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>

#include "../../include/rope3d.h"
#include "rope3d_internal.h"
#include "rope3d_tc.cuh"

namespace {

using namespace rope3d_tc;

// Bounded waits that ran out (rope3d_testing_ffn_wait_timeouts).
__device__ unsigned int g_ffn_wait_timeouts;

// ---- the element-wise part ---------------------------------------------------

__device__ __forceinline__ float rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float sigmoid(float v) { return rcp(1.0f + __expf(-v)); }

// act(g) and, where kGrad, act'(g). GELU's tanh form is g * sigmoid(2 z) with
// z = sqrt(2 / pi) (g + 0.044715 g^3), from 1 + tanh(z) = 2 sigmoid(2 z); past
// |g| = 50 the sigmoid is 0 or 1 and its slope 0 in fp32, and the clamp keeps
// g^3 finite.
template <int kAct, bool kGrad>
__device__ __forceinline__ float activation(float g, float *grad) {
    if constexpr (kAct == ROPE3D_ACT_SILU) {
        const float q = sigmoid(g);
        if constexpr (kGrad) *grad = q * (1.0f + g * (1.0f - q));
        return g * q;
    } else if constexpr (kAct == ROPE3D_ACT_GELU_TANH) {
        const float c = fminf(fmaxf(g, -50.0f), 50.0f);
        const float s = c * c;
        const float q = sigmoid(c * (1.5957691216f + 0.0713548163f * s));
        if constexpr (kGrad) *grad = q + g * (q * (1.0f - q) * (1.5957691216f + 0.2140644488f * s));
        return g * q;
    } else {
        // erfc(x) = (a1 t + ... + a5 t^5) exp(-x^2), t = 1 / (1 + p x), x >= 0:
        // Abramowitz and Stegun, Handbook of Mathematical Functions, 7.1.26, off by
        // at most 1.5e-7; here x = |g| / sqrt(2), and the slope needs the same
        // exp(-g^2 / 2)
        const float x = fabsf(g) * 0.7071067812f;
        const float t = rcp(1.0f + 0.3275911f * x), e = __expf(-x * x);
        const float poly = t * (0.254829592f + t * (-0.284496736f + t * (1.421413741f + t * (-1.453152027f + t * 1.061405429f))));
        const float tail = 0.5f * poly * e, cdf = g < 0.0f ? tail : 1.0f - tail;
        if constexpr (kGrad) *grad = cdf + g * (0.3989422804f * e);
        return g * cdf;
    }
}

template <bool kGrad>
__device__ __forceinline__ float activation_of(float g, int act, float *grad) {
    return act == ROPE3D_ACT_SILU        ? activation<ROPE3D_ACT_SILU, kGrad>(g, grad)
           : act == ROPE3D_ACT_GELU_TANH ? activation<ROPE3D_ACT_GELU_TANH, kGrad>(g, grad)
                                         : activation<ROPE3D_ACT_GELU_ERF, kGrad>(g, grad);
}

template <bool kF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    uint32_t w;
    if constexpr (kF16) {
        const __half2 h = __floats2half2_rn(a, b);
        memcpy(&w, &h, 4);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        memcpy(&w, &h, 4);
    }
    return w;
}

template <bool kF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (kF16) {
        __half2 h;
        memcpy(&h, &w, 4);
        return __half22float2(h);
    } else {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
}

__device__ __forceinline__ uint16_t pack1(float a, bool f16) {
    return f16 ? __half_as_ushort(__float2half_rn(a)) : __bfloat16_as_ushort(__float2bfloat16_rn(a));
}

// Two 16-bit loads in one word, and (unpack1) one value: without a shift right
// behind a 16-bit load, which makes the loads wait for one another.
__device__ __forceinline__ uint32_t word(uint32_t lo, uint32_t hi) { return __byte_perm(lo, hi, 0x5410); }

__device__ __forceinline__ float unpack1(uint16_t v, bool f16) {
    return f16 ? __half2float(__ushort_as_half(v)) : __bfloat162float(__ushort_as_bfloat16(v));
}

// ---- launch description ---------------------------------------------------------

enum Epi { kPlain = 0, kGated = 1, kBack = 2 };
// operand layouts: both K-major; A K-major and B MN-major; or (the gradients'
// launch) the latter for dx and both MN-major for the weights' gradients
constexpr int kKK = 0, kKM = 1, kGrads = 2;

// A matrix written by an epilogue: rows of 16-bit or fp32 elements.
struct Out {
    void *p;          // null: not written
    long long ld;     // elements from row to row
    int f32;
    int vec;          // rows start on 16-byte boundaries
    int tma_cols;     // the columns before this one are stored through the tensor map
    int word;         // else: bytes (2, 4 or 8) that base and rows are multiples of
};

struct Maps {
    CUtensorMap a[5], b[5];   // operands: segments 0 and 1 (gated: b = Wg, Wu), then the weights' gradients
    CUtensorMap c[4];         // outputs
};

// One product of a launch: its output's size, in elements and in tiles.
struct Sub {
    int m, n, tiles_m, tiles_n;
    __host__ __device__ int tiles() const { return tiles_m * tiles_n; }
};

struct Params {
    int m, n;                 // stream kernel: weight rows, tokens
    int nk0, nk1;             // 64-wide k blocks of the two segments
    int f16, act;
    Out out[4];               // gated: h, g, u; back: dg, du, h; else one a product
    const void *g, *u;        // back: the kept projections
    long long ldp;
    int pre_f32, pre_vec;     // they are fp32; their rows start on 32-byte boundaries
    int rows_n, stages;       // stream kernel: MMA N, ring slots
    // tile kernel: the products (gradients: dx, dWg, dWu, dWd); of the first
    // one the tiles computed by one pair each, then the rest, `split` units each
    // of a part of the k range; the units' fp32 sums
    Sub sub[4];
    int whole, split, units;
    float *part;
    // gradients: the weights' tiles and their k blocks; whether dx's units are
    // the longer ones, and how many of the shorter ones a longer one is worth
    int weight_units, nkw, dx_first, lag;
};

// 16 consecutive elements of a kept projection on their way: the bits as they
// lie in memory (32 bytes of 16-bit or 64 bytes of fp32 values).
struct Pre16 {
    uint32_t w[16];
    __device__ __forceinline__ void load8(int at, const void *src) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[at]), "=r"(w[at + 1]), "=r"(w[at + 2]), "=r"(w[at + 3]), "=r"(w[at + 4]),
                       "=r"(w[at + 5]), "=r"(w[at + 6]), "=r"(w[at + 7])
                     : "l"(src));
    }
    // elements off .. off + 15 of `base`, the first `valid` of which exist
    __device__ __forceinline__ void load(const void *base, long long off, int valid, const Params &p) {
        if (p.pre_vec && valid >= 16) {
            if (p.pre_f32) {
                load8(0, static_cast<const float *>(base) + off);
                load8(8, static_cast<const float *>(base) + off + 8);
            } else {
                load8(0, static_cast<const uint16_t *>(base) + off);
            }
            return;
        }
        if (p.pre_f32) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                w[i] = i < valid ? __float_as_uint(static_cast<const float *>(base)[off + i]) : 0u;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint16_t *s = static_cast<const uint16_t *>(base) + off + 2 * i;
                w[i] = word(2 * i < valid ? s[0] : 0u, 2 * i + 1 < valid ? s[1] : 0u);
            }
        }
    }
    template <bool kF16>
    __device__ __forceinline__ void values(float *v, const Params &p) const {
        if (p.pre_f32) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 f = unpack2<kF16>(w[i]);
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
};

// ---- many tokens: 256-row tiles of CTA pairs -------------------------------------
//
// A pair of CTAs (one cluster) computes 256 x kBN of C with cta_group::2 MMAs:
// each CTA holds 128 rows of A and kBN / 2 rows of B in shared memory, and the
// accumulators of its own 128 rows, kBN fp32 columns, in tensor memory. Both
// CTAs read both halves of B through the pair, so a stage costs each SM 16 KB
// of A and kBN / 2 * 128 B of B for 256 x kBN x 64 products of the pair.
// Gated: B's two halves are kBN / 2 rows of Wg and the same rows of Wu, so one
// thread finds g and u of an element in its own lane and no extra pass runs.
//
// Roles (384 threads): warp 0 TMA producer, warp 1 MMA issuer (of the pair's
// first CTA), warp 2 tensor memory, warps 4-11 the epilogue: warp w reads
// tensor memory lanes 32 (w % 4) + lane, half of the columns. Accumulators are
// double-buffered, so the epilogue of a tile runs under the next tile's MMAs.
// Persistent: cluster c computes tiles c, c + clusters, ... in an order that
// walks groups of 8 tile rows, so that the tiles in flight share operands in L2.
//
// The tiles that would leave most pairs idle in the last round are split along k
// where that is faster (launch_tile): `split` units each leave the fp32 sums of
// their part in the workspace, and ffn_finish_kernel adds them in order and runs
// the epilogue. No pair waits for another.
//
// Epilogue stores go through 2 KB staging boxes (32 rows x 64 bytes, the
// 64-byte swizzle keeps the writes free of bank conflicts) and TMA, four boxes
// in flight a warp; rows that TMA cannot address are stored in the widest words
// that they are aligned to.
//
// Measured (bf16, width 2048, hidden 8192): g and u of 8192 tokens 299 us, 1,840
// TFLOP/s (95 % of a cuBLAS product's burst), the tensor pipe busy for 83 % of the
// cycles, 300 MB read from memory; dx and the three weights' gradients of 2048
// tokens, one launch, 204 us, 1,680 TFLOP/s; dh with dg, du and h 79-86 us, 800-870
// TFLOP/s: there a CTA also reads 256 KB of kept projections a tile and writes
// 192 KB, and the epilogue's loads bound it (at the rate of the others the products
// would take 41 us).
constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kStages = 5;
constexpr int kABytes = 128 * 128;              // 128 rows x 64 elements
constexpr int kBoxBytes = 2048, kBoxes = 4;     // staging of one warp
constexpr int kGroupRows = 8;                   // tile rows of a raster group

template <int kBN>
constexpr int tile_smem() {
    return kStages * (kABytes + kBN / 2 * 128) + kEpiWarps * kBoxes * kBoxBytes + 256 + 1024;
}

struct Tile {
    int m0, n0;   // first row and first column, in tiles
};

__device__ __forceinline__ Tile tile_at(const Sub &p, int t) {
    const int group = t / (kGroupRows * p.tiles_n);
    const int first = group * kGroupRows;
    const int rows = min(kGroupRows, p.tiles_m - first);
    t -= first * p.tiles_n;
    return Tile{first + t % rows, t / rows};
}

// A unit of work: a tile of a product, or (part >= 0) a part of its k range.
struct Unit {
    int sub, tile, part, k_lo, k_hi;
};

__device__ __forceinline__ Unit unit_at(const Params &p, int u) {
    const int nk = p.nk0 + p.nk1;
    if (u < p.whole) return Unit{0, u, -1, 0, nk};
    const int i = u - p.whole, t = i / p.split, part = i - t * p.split;
    return Unit{0, p.whole + t, i, int((long long)nk * part / p.split), int((long long)nk * (part + 1) / p.split)};
}

// The i-th unit of this pair of CTAs; false past its last one. Units go to the
// pairs in turn. In the gradients' launch the longer kind goes first; the pairs
// that the last round of it leaves out start on the shorter kind at once and get
// as many of those more (`lag` each) as the others' last long unit takes.
template <int kLayout>
__device__ __forceinline__ bool next_unit(const Params &p, int i, Unit &un) {
    const int c = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    if constexpr (kLayout != kGrads) {
        const int u = c + i * pairs;
        if (u >= p.units) return false;
        un = unit_at(p, u);
        return true;
    } else {
        const int longs = p.dx_first ? p.units : p.weight_units, shorts = p.dx_first ? p.weight_units : p.units;
        const int r = longs % pairs, own = longs / pairs + (c < r);
        int u;
        bool dx = p.dx_first;
        if (i < own) {
            u = c + i * pairs;
        } else {
            int j = i - own;
            const int first = r ? min(shorts, p.lag * (pairs - r)) : 0;   // shared by pairs r ... alone
            const int mine = c >= r && first > c - r ? (first - (c - r) - 1) / (pairs - r) + 1 : 0;
            u = j < mine ? (c - r) + j * (pairs - r) : first + c + (j - mine) * pairs;
            if (u >= shorts) return false;
            dx = !dx;
        }
        if (dx) {
            un = unit_at(p, u);
        } else {
            int z = 1;
            while (z < 3 && u >= p.sub[z].tiles()) u -= p.sub[z++].tiles();
            un = Unit{z, u, -1, 0, p.nkw};
        }
        return true;
    }
}

// Epilogue stores of one warp.
struct Boxes {
    uint32_t base;   // shared-memory address of the warp's boxes
    int next;
    int lane;
};

// `bytes` of the first `rows` rows of a staging box to rows of `pitch` bytes at d,
// which start on multiples of kW bytes: 64 / kW lanes a row, words of kW bytes,
// eight loads in flight. (Gradients of 71 x 1546 x 4990 fp16, rows on multiples of
// 4 bytes: 34 us in words of 4 bytes, 56 in single elements.)
template <int kW>
__device__ __forceinline__ void copy_box(uint32_t box, char *d, long long pitch, int lane, int rows, int bytes) {
    constexpr int kLanes = 64 / kW, kRows = kW / 2;
    const int b = (lane % kLanes) * kW, first = lane / kLanes;
    d += first * pitch + b;
    for (int i = 0; i < rows; i += 8 * kRows) {
        uint64_t v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const uint32_t r = uint32_t(i + u * kRows + first);
            const uint32_t at = box + r * 64 + (((uint32_t(b) >> 4) ^ ((r >> 1) & 3)) << 4) + (uint32_t(b) & 15);
            if constexpr (kW == 8) {
                asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v[u]) : "r"(at) : "memory");
            } else if constexpr (kW == 4) {
                uint32_t w;
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(at) : "memory");
                v[u] = w;
            } else {
                uint16_t w;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(w) : "r"(at) : "memory");
                v[u] = w;
            }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (i + u * kRows + first >= rows) break;
            char *at = d + (i + u * kRows) * pitch;
            if (b + kW <= bytes) {
                if constexpr (kW == 8) *reinterpret_cast<uint64_t *>(at) = v[u];
                else if constexpr (kW == 4) *reinterpret_cast<uint32_t *>(at) = uint32_t(v[u]);
                else *reinterpret_cast<uint16_t *>(at) = uint16_t(v[u]);
            } else if constexpr (kW > 2) {   // the row ends inside the word
#pragma unroll
                for (int h = 0; h < kW / 2; ++h)
                    if (b + 2 * h < bytes) reinterpret_cast<uint16_t *>(at)[h] = uint16_t(v[u] >> (16 * h));
            }
        }
    }
}

// 16 words (64 bytes: 32 16-bit or 16 fp32 elements) of each lane's row, from
// column `col` of output o; the warp's rows are row0 .. row0 + 31. Through a
// staging box: a TMA store, or where TMA cannot address the rows or the box's last
// columns, the widest words that they are aligned to.
__device__ __forceinline__ void store_words(Boxes &bx, const uint32_t *w, const Out &o,
                                            const CUtensorMap *map, int row0, int col, int m, int n) {
    if (!o.p || row0 >= m || col >= n) return;
    const uint32_t box = bx.base + uint32_t(bx.next & (kBoxes - 1)) * kBoxBytes;
    ++bx.next;
    if (bx.lane == 0) bulk_wait_read<kBoxes - 1>();
    __syncwarp();
    const uint32_t row = box + uint32_t(bx.lane) * 64, sw = (uint32_t(bx.lane) >> 1) & 3;
#pragma unroll
    for (int c = 0; c < 4; ++c)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                     ::"r"(row + ((uint32_t(c) ^ sw) << 4)), "r"(w[4 * c]), "r"(w[4 * c + 1]),
                       "r"(w[4 * c + 2]), "r"(w[4 * c + 3]) : "memory");
    if (col < o.tma_cols) {
        fence_async_smem();
        __syncwarp();
        if (bx.lane == 0) tma_store2(map, box, col, row0);
    } else {
        __syncwarp();
        const int rows = min(32, m - row0), bytes = min(64, (n - col) << (o.f32 ? 2 : 1));
        char *d = static_cast<char *>(o.p) + ((row0 * o.ld + col) << (o.f32 ? 2 : 1));
        const long long pitch = o.ld << (o.f32 ? 2 : 1);
        if (o.word == 2) copy_box<2>(box, d, pitch, bx.lane, rows, bytes);
        else if (o.word == 4) copy_box<4>(box, d, pitch, bx.lane, rows, bytes);
        else copy_box<8>(box, d, pitch, bx.lane, rows, bytes);
        __syncwarp();
    }
    if (bx.lane == 0) bulk_commit();   // (an empty group where nothing was copied: boxes are counted by groups)
}

// A kept projection, 32 columns of each lane's row, in its own type.
template <bool kF16>
__device__ __forceinline__ void store_pre32(Boxes &bx, const float *v, const Out &o,
                                            const CUtensorMap *map, int row0, int col,
                                            const Sub &p) {
    if (!o.p) return;
    uint32_t w[16];
    if (o.f32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[16 * h + i]);
            store_words(bx, w, o, map, row0, col + 16 * h, p.m, p.n);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = pack2<kF16>(v[2 * i], v[2 * i + 1]);
        store_words(bx, w, o, map, row0, col, p.m, p.n);
    }
}

// The epilogues, on 32 columns of each lane's row (row0 + lane), from `col` on.
template <bool kF16>
__device__ __forceinline__ void finish_plain(Boxes &bx, const float *v, const Params &p, const CUtensorMap *c, int z,
                                             int row0, int col) {
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) w[e] = pack2<kF16>(v[2 * e], v[2 * e + 1]);
    store_words(bx, w, p.out[z], c + z, row0, col, p.sub[z].m, p.sub[z].n);
}

template <bool kF16, int kAct>
__device__ __forceinline__ void finish_gated(Boxes &bx, const float *g, const float *u, const Params &p,
                                             const CUtensorMap *c, int row0, int col) {
    store_pre32<kF16>(bx, g, p.out[1], c + 1, row0, col, p.sub[0]);
    store_pre32<kF16>(bx, u, p.out[2], c + 2, row0, col, p.sub[0]);
    if (!p.out[0].p) return;
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const float h0 = activation<kAct, false>(g[2 * e], nullptr) * u[2 * e];
        const float h1 = activation<kAct, false>(g[2 * e + 1], nullptr) * u[2 * e + 1];
        w[e] = pack2<kF16>(h0, h1);
    }
    store_words(bx, w, p.out[0], c, row0, col, p.sub[0].m, p.sub[0].n);
}

// dg, du and h of 16 columns, packed, from dh and the kept projections.
template <bool kF16, int kAct>
__device__ __forceinline__ void back16(const float *dh, const Pre16 &g, const Pre16 &u, const Params &p, uint32_t *wg,
                                       uint32_t *wu, uint32_t *wh) {
    float gv[16], uv[16];
    g.values<kF16>(gv, p);
    u.values<kF16>(uv, p);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float s0, s1;
        const float a0 = activation<kAct, true>(gv[2 * e], &s0), a1 = activation<kAct, true>(gv[2 * e + 1], &s1);
        wg[e] = pack2<kF16>(dh[2 * e] * uv[2 * e] * s0, dh[2 * e + 1] * uv[2 * e + 1] * s1);
        wu[e] = pack2<kF16>(dh[2 * e] * a0, dh[2 * e + 1] * a1);
        wh[e] = pack2<kF16>(a0 * uv[2 * e], a1 * uv[2 * e + 1]);
    }
}

__device__ __forceinline__ void store_back(Boxes &bx, const uint32_t *wg, const uint32_t *wu, const uint32_t *wh,
                                           const Params &p, const CUtensorMap *c, int row0, int col) {
    store_words(bx, wg, p.out[0], c, row0, col, p.sub[0].m, p.sub[0].n);
    store_words(bx, wu, p.out[1], c + 1, row0, col, p.sub[0].m, p.sub[0].n);
    store_words(bx, wh, p.out[2], c + 2, row0, col, p.sub[0].m, p.sub[0].n);
}

template <int kBN, int kLayout, int kEpi, bool kF16, int kAct>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
ffn_tile_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
    constexpr bool kBMn = kLayout != kKK;                 // (A: K-major but for the weights' gradients)
    constexpr int kBRows = kBN / 2;                       // rows of B in this CTA
    constexpr uint32_t kBBytes = kBRows * 128;
    constexpr uint32_t kStageBytes = kABytes + kBBytes;
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t boxes = base + kStages * kStageBytes;
    const uint32_t bars = boxes + kEpiWarps * kBoxes * kBoxBytes;
    auto full = [&](int s) { return bars + 8u * uint32_t(s); };
    auto empty = [&](int s) { return bars + 8u * uint32_t(kStages + s); };
    auto acc_full = [&](int b) { return bars + 8u * uint32_t(2 * kStages + b); };
    auto acc_empty = [&](int b) { return bars + 8u * uint32_t(2 * kStages + 2 + b); };
    const uint32_t slot = bars + 8u * (2 * kStages + 4);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full(b), 1);
            mbar_init(acc_empty(b), 2 * kEpiWarps);
        }
        mbar_fence_init();
        if (p.units > 0) {
            prefetch_map(&maps.a[0]);
            prefetch_map(&maps.b[0]);
        }
    }
    if (warp == 2) tmem_alloc<true>(slot, 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs' barriers exist before any copy or commit names them
    tc_fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(slot) : "memory");
    // results of earlier kernels are visible from here; only then may a later
    // kernel start (so that what runs beside this one has all older writes)
    grid_wait();
    grid_release();
    bool dead = false;

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            Unit un;
            for (int i = 0; !dead && next_unit<kLayout>(p, i, un); ++i) {
                const Tile x = tile_at(p.sub[un.sub], un.tile);
                const bool a_mn = kLayout == kGrads && un.sub > 0;
                const int m0 = x.m0 * 256 + int(rank) * 128;
                // gated: this CTA's rows are of Wg (rank 0) or Wu (rank 1)
                const int n0 = kEpi == kGated ? x.n0 * kBRows : x.n0 * kBN + int(rank) * kBRows;
                for (int kb = un.k_lo; kb < un.k_hi; ++kb, ++it) {
                    const int s = it % kStages;
                    const uint32_t use = uint32_t(it / kStages);
                    if (it >= kStages && !mbar_wait(empty(s), (use - 1) & 1u, dead, &g_ffn_wait_timeouts)) break;
                    const int seg = un.sub == 0 && kb >= p.nk0;
                    const int k = (seg ? kb - p.nk0 : kb) * 64;
                    const CUtensorMap *ma = &maps.a[un.sub ? 1 + un.sub : seg];
                    const CUtensorMap *mb = &maps.b[kEpi == kGated ? int(rank) : un.sub ? 1 + un.sub : seg];
                    const uint32_t sa = base + uint32_t(s) * kStageBytes, sb = sa + kABytes;
                    // the pair's copies complete on the first CTA's barrier
                    const uint32_t bar = map_rank(full(s), 0);
                    if (rank == 0) mbar_expect_tx(full(s), 2 * kStageBytes);
                    if (a_mn) {
                        tma_load2<true>(sa, ma, m0, k, bar);
                        tma_load2<true>(sa + 8192, ma, m0 + 64, k, bar);
                    } else {
                        tma_load2<true>(sa, ma, k, m0, bar);
                    }
                    if constexpr (kBMn) {
#pragma unroll
                        for (int j = 0; j < kBRows / 64; ++j)
                            tma_load2<true>(sb + 8192 * j, mb, n0 + 64 * j, k, bar);
                    } else {
                        tma_load2<true>(sb, mb, k, n0, bar);
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (rank == 0 && lane == 0) {
            int it = 0;
            Unit un;
            for (int i = 0; !dead && next_unit<kLayout>(p, i, un); ++i) {
                const bool a_mn = kLayout == kGrads && un.sub > 0;
                const uint32_t id = idesc(256, kBN, !kF16, a_mn, kBMn);
                // 16 elements of k: 32 bytes of a K-major row, 16 rows of an MN-major tile
                const uint32_t a_step = a_mn ? 2048 : 32, a_lbo = a_mn ? 8192 : 16;
                const int b = i & 1;
                if (i >= 2 && !mbar_wait(acc_empty(b), uint32_t(i / 2 - 1) & 1u, dead, &g_ffn_wait_timeouts)) break;
                tc_fence_after();
                const uint32_t d = tmem + uint32_t(b) * 256;
                for (int kb = un.k_lo; kb < un.k_hi; ++kb, ++it) {
                    const int s = it % kStages;
                    if (!mbar_wait(full(s), uint32_t(it / kStages) & 1u, dead, &g_ffn_wait_timeouts)) break;
                    tc_fence_after();
                    const uint32_t sa = base + uint32_t(s) * kStageBytes, sb = sa + kABytes;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint64_t da = sdesc(sa + j * a_step, a_lbo, 1024);
                        const uint64_t db = kBMn ? sdesc(sb + j * 2048, 8192, 1024) : sdesc(sb + j * 32, 16, 1024);
                        mma<true>(d, da, db, id, kb > un.k_lo || j > 0);
                    }
                    commit_pair(empty(s));
                }
                commit_pair(acc_full(b));
            }
            if (dead) drain(full, it, kStages, &g_ffn_wait_timeouts);   // (the pair's copies: the other CTA waits below)
        }
    } else if (warp >= 4) {
        const int quad = warp & 3, half = (warp - 4) >> 2;
        Boxes bx{boxes + uint32_t(warp - 4) * kBoxes * kBoxBytes, 0, lane};
        Unit un;
        for (int i = 0; !dead && next_unit<kLayout>(p, i, un); ++i) {
            const Tile x = tile_at(p.sub[un.sub], un.tile);
            const int b = i & 1;
            const int row0 = x.m0 * 256 + int(rank) * 128 + quad * 32;
            const uint32_t d = tmem + uint32_t(b) * 256 + (uint32_t(quad) << 21);
            constexpr int kCols = kEpi == kGated ? kBRows / 2 : kBN / 2;   // columns of this warp
            const int c0 = half * kCols;
            const int n0 = x.n0 * (kEpi == kGated ? kBRows : kBN) + c0;
            [[maybe_unused]] Pre16 g[2], u[2];
            [[maybe_unused]] auto fetch = [&](int c, int to) {   // the kept projections of 16 columns
                const int row = row0 + lane, col = n0 + c;
                const int valid = row < p.sub[0].m ? p.sub[0].n - col : 0;
                g[to].load(p.g, row * p.ldp + col, valid, p);
                u[to].load(p.u, row * p.ldp + col, valid, p);
            };
            // ... and 32 columns on their way to L2, two chunks before they are fetched
            [[maybe_unused]] auto ahead = [&](int c) {
                const int row = row0 + lane, col = n0 + c;
                if (c >= kCols || row >= p.sub[0].m || col >= p.sub[0].n) return;
                const long long off = (row * p.ldp + col) * (p.pre_f32 ? 4 : 2);
                asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char *>(p.g) + off));
                asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char *>(p.u) + off));
            };
            if (kEpi == kBack && un.part < 0) {   // on their way while the products finish
                fetch(0, 0);
                ahead(32);
                ahead(64);
            }
            // one answer for the warp: where a wait ran out for some of its lanes alone,
            // they would leave and the others wait for them in the next __syncwarp()
            const bool ready = mbar_wait(acc_full(b), uint32_t(i / 2) & 1u, dead, &g_ffn_wait_timeouts);
            if (!__all_sync(0xffffffffu, ready)) break;
            tc_fence_after();
            if (un.part >= 0) {
                // fp32 sums of this part: [8 groups of 32 rows][kBN columns][32 rows]
                float *dst = p.part + ((long long)un.part * 8 + rank * 4 + quad) * (kBN * 32) + lane;
#pragma unroll 1
                for (int c = 0; c < kBN / 2; c += 16) {
                    float v[16];
                    const int at = half * (kBN / 2) + c;
                    tmem_ld16(v, d + uint32_t(at));
                    tmem_wait();
                    tmem_tie16(v);
#pragma unroll
                    for (int e = 0; e < 16; ++e) dst[(at + e) * 32] = v[e];
                }
            } else if constexpr (kEpi == kBack) {
                // 16 columns at a time, the next ones' projections on their way
#pragma unroll 1
                for (int c = 0; c < kCols; c += 32) {
                    uint32_t wg[16], wu[16], wh[16];
                    ahead(c + 96);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float v[16];
                        tmem_ld16(v, d + uint32_t(c0 + c + 16 * q));
                        if (c + 16 * q + 16 < kCols) fetch(c + 16 * q + 16, 1 - q);
                        tmem_wait();
                        tmem_tie16(v);
                        back16<kF16, kAct>(v, g[q], u[q], p, wg + 8 * q, wu + 8 * q, wh + 8 * q);
                    }
                    store_back(bx, wg, wu, wh, p, maps.c, row0, n0 + c);
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < kCols; c += 32) {
                    float v[32];
                    tmem_ld16(v, d + uint32_t(c0 + c));
                    tmem_ld16(v + 16, d + uint32_t(c0 + c + 16));
                    if constexpr (kEpi == kGated) {
                        float w[32];
                        tmem_ld16(w, d + uint32_t(kBRows + c0 + c));
                        tmem_ld16(w + 16, d + uint32_t(kBRows + c0 + c + 16));
                        tmem_wait();
                        tmem_tie16(v);
                        tmem_tie16(v + 16);
                        tmem_tie16(w);
                        tmem_tie16(w + 16);
                        finish_gated<kF16, kAct>(bx, v, w, p, maps.c, row0, n0 + c);
                    } else {
                        tmem_wait();
                        tmem_tie16(v);
                        tmem_tie16(v + 16);
                        finish_plain<kF16>(bx, v, p, maps.c, un.sub, row0, n0 + c);
                    }
                }
            }
            // this warp's reads of the accumulators are done
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_rank(acc_empty(b), 0));
        }
        if (lane == 0) bulk_wait_all();
    }
    // neither CTA leaves while the other may still name its shared memory,
    // barriers or tensor memory
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    if (warp == 2) tmem_free<true>(tmem, 512);
}

// Eight values of each lane's row (row0 + lane) from column `col` of output o, the
// first `valid` of which exist. The block's four warps hold 32 consecutive columns:
// where rows do not start on 16-byte boundaries they are exchanged through shared
// memory and stored row by row, consecutive elements by consecutive lanes.
template <bool kF16>
__device__ __forceinline__ void store8(const Out &o, int row0, int col, int valid, const float *v, const Sub &sub,
                                       float (*stage)[33]) {
    if (!o.p) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (o.vec) {
        const long long at = (row0 + lane) * o.ld + col;
        if (valid >= 8 && o.f32) {
            float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(o.p) + at);
            d[0] = make_float4(v[0], v[1], v[2], v[3]);
            d[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else if (valid >= 8) {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(o.p) + at) =
                make_uint4(pack2<kF16>(v[0], v[1]), pack2<kF16>(v[2], v[3]), pack2<kF16>(v[4], v[5]), pack2<kF16>(v[6], v[7]));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < valid) {
                    if (o.f32) static_cast<float *>(o.p)[at + i] = v[i];
                    else static_cast<uint16_t *>(o.p)[at + i] = pack1(v[i], kF16);
                }
        }
        return;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) stage[lane][warp * 8 + i] = v[i];
    __syncthreads();
    const int c = col - warp * 8 + lane;
    if (c >= sub.n) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = row0 + warp * 8 + i;
        if (row >= sub.m) break;
        if (o.f32) static_cast<float *>(o.p)[row * o.ld + c] = stage[warp * 8 + i][lane];
        else static_cast<uint16_t *>(o.p)[row * o.ld + c] = pack1(stage[warp * 8 + i][lane], kF16);
    }
}

// The split tiles: each warp adds the parts' sums of 32 rows x 8 columns (of both
// halves where gated) in order and runs the epilogue on them, a row a lane. Bound
// by reading the sums from L2: 28 tiles of 256 x 256 in two parts, 14.7 MB, 6 us.
template <int kBN, int kEpi, bool kF16, int kAct>
__global__ void __launch_bounds__(128) ffn_finish_kernel(const __grid_constant__ Params p) {
    grid_wait();
    grid_release();
    constexpr int kTileCols = kEpi == kGated ? kBN / 2 : kBN, kChunks = kTileCols / 8;
    const int lane = threadIdx.x & 31;
    int w = int(blockIdx.x) * 4 + int(threadIdx.x >> 5);   // (split tile, group of rows, chunk of columns)
    const int chunk = w % kChunks;
    w /= kChunks;
    const int rows = w & 7, tile = w >> 3;
    const Tile x = tile_at(p.sub[0], p.whole + tile);
    const int row0 = x.m0 * 256 + rows * 32, row = row0 + lane, col = x.n0 * kTileCols + chunk * 8;
    __shared__ float stage[32][33];
    const int valid = row < p.sub[0].m ? p.sub[0].n - col : 0;
    auto sums = [&](float *v, int c) {
        const float *src = p.part + ((long long)tile * p.split * 8 + rows) * (kBN * 32) + c * 32 + lane;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.0f;
#pragma unroll 4
        for (int i = 0; i < p.split; ++i, src += 8ll * kBN * 32)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += __ldcs(src + e * 32);
    };
    float v[8];
    sums(v, chunk * 8);
    if constexpr (kEpi == kGated) {
        float u[8], h[8];
        sums(u, kBN / 2 + chunk * 8);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = activation<kAct, false>(v[i], nullptr) * u[i];
        store8<kF16>(p.out[0], row0, col, valid, h, p.sub[0], stage);
        store8<kF16>(p.out[1], row0, col, valid, v, p.sub[0], stage);
        store8<kF16>(p.out[2], row0, col, valid, u, p.sub[0], stage);
    } else if constexpr (kEpi == kBack) {
        float dg[8] = {}, du[8] = {}, h[8] = {};
        const long long at = row * p.ldp + col;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i >= valid) continue;
            const float g = p.pre_f32 ? static_cast<const float *>(p.g)[at + i]
                                      : unpack1(static_cast<const uint16_t *>(p.g)[at + i], kF16);
            const float u = p.pre_f32 ? static_cast<const float *>(p.u)[at + i]
                                      : unpack1(static_cast<const uint16_t *>(p.u)[at + i], kF16);
            float slope;
            const float a = activation<kAct, true>(g, &slope);
            dg[i] = v[i] * u * slope;
            du[i] = v[i] * a;
            h[i] = a * u;
        }
        store8<kF16>(p.out[0], row0, col, valid, dg, p.sub[0], stage);
        store8<kF16>(p.out[1], row0, col, valid, du, p.sub[0], stage);
        store8<kF16>(p.out[2], row0, col, valid, h, p.sub[0], stage);
    } else {
        store8<kF16>(p.out[0], row0, col, valid, v, p.sub[0], stage);
    }
}

// ---- few tokens: weights streamed once ---------------------------------------------
//
// With few tokens the weights' bytes bound every product, so a tile is turned
// over: 128 weight rows are the MMA's M and all the tokens (rounded up to 16)
// its N. A cluster of CTAs splits the k range of a tile, so that enough CTAs
// read at once also where the tiles are few; each leaves its fp32 partial sums
// in shared memory and the cluster adds them in rank order (always the same
// order) through distributed shared memory, with the activation on the way out.
// Warp 0: TMA, warp 1: MMAs, all eight warps: the epilogue (warps w and w + 4
// share tensor-memory lanes and take half of the columns each).
// The second product of a forward pass starts its weight copies while the first
// still runs, and waits for h alone.
// Measured (bf16, width 4096, hidden 16384): one token 65 us, 6,200 GB/s of weights
// (91 % of a copy's rate), the gated product 46.5 us of them; fp16, width 2048,
// hidden 8192, 24 tokens 21.6 us, 4,670 GB/s: filling and draining the rings of two
// products of 11 and 5 us.
constexpr int kStreamThreads = 256;
// Most tokens of this kernel: of the gated product (two accumulators to add up)
// and of the others. Measured, bf16, the whole forward pass: width 2048, hidden
// 8192: 96 tokens 30.3 us (gated product by tiles 34), 128: 33.6 (34); 320, 2944:
// 128: 18.2 (13.9). dx at 2048, 8192: 160 tokens 42.8 us (by tiles 54.8), 192:
// 63.4 (55.4).
constexpr int kStreamGated = 96, kStreamTokens = 160;
constexpr int kMaxSplit = 8;

template <bool kAMn, int kEpi>
__global__ void __launch_bounds__(kStreamThreads)
ffn_stream_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
    constexpr int kAcc = kEpi == kGated ? 2 : 1;
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
    const uint32_t stage_bytes = kAcc * kABytes + uint32_t(p.rows_n) * 128;
    const uint32_t bars = base + uint32_t(p.stages) * stage_bytes;
    auto full = [&](int s) { return bars + 16u * uint32_t(s); };
    auto empty = [&](int s) { return bars + 16u * uint32_t(s) + 8u; };
    const uint32_t done = bars + 16u * uint32_t(p.stages), slot = done + 8;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    uint32_t split;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(split));
    const int tile = blockIdx.x / split;
    const int f0 = tile * 128;
    const int nk = p.nk0 + p.nk1;
    const int k_lo = int(int64_t(nk) * rank / split), k_hi = int(int64_t(nk) * (rank + 1) / split);
    uint32_t cols = 32;
    while (cols < uint32_t(kAcc * p.rows_n)) cols *= 2;

    if (tid == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        mbar_init(done, 1);
        mbar_fence_init();
    }
    if (warp == 2) tmem_alloc<false>(slot, cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(slot) : "memory");
    bool dead = false;

    auto load_weights = [&](int kb, int s) {
        const int seg = kb >= p.nk0;
        const int k = (seg ? kb - p.nk0 : kb) * 64;
        const uint32_t sa = base + uint32_t(s) * stage_bytes;
        mbar_expect_tx(full(s), stage_bytes);
#pragma unroll
        for (int a = 0; a < kAcc; ++a) {
            const CUtensorMap *ma = &maps.a[kEpi == kGated ? a : seg];
            if constexpr (kAMn) {
                tma_load2<false>(sa + a * kABytes, ma, f0, k, full(s));
                tma_load2<false>(sa + a * kABytes + 8192, ma, f0 + 64, k, full(s));
            } else {
                tma_load2<false>(sa + a * kABytes, ma, k, f0, full(s));
            }
        }
    };
    auto load_tokens = [&](int kb, int s) {
        const int seg = kb >= p.nk0;
        const int k = (seg ? kb - p.nk0 : kb) * 64;
        tma_load2<false>(base + uint32_t(s) * stage_bytes + kAcc * kABytes, &maps.b[seg], k, 0, full(s));
    };

    if (warp == 0 && lane == 0) {
        const int n = k_hi - k_lo, ahead = min(n, p.stages);
        // the plain product's weights are no earlier kernel's output that may
        // still be in flight: the kernel before it waited for all older ones
        if constexpr (kEpi == kPlain && !kAMn) {
            for (int i = 0; i < ahead; ++i) load_weights(k_lo + i, i);
            grid_wait();
            for (int i = 0; i < ahead; ++i) load_tokens(k_lo + i, i);
        } else {
            grid_wait();
            for (int i = 0; i < ahead; ++i) {
                load_weights(k_lo + i, i);
                load_tokens(k_lo + i, i);
            }
        }
        for (int i = ahead; i < n; ++i) {
            const int s = i % p.stages;
            if (!mbar_wait(empty(s), uint32_t(i / p.stages - 1) & 1u, dead, &g_ffn_wait_timeouts)) break;
            load_weights(k_lo + i, s);
            load_tokens(k_lo + i, s);
        }
    } else if (warp == 1 && lane == 0) {
        const uint32_t id = idesc(128, uint32_t(p.rows_n), !p.f16, kAMn, false);
        // the tokens' copies start only then: a wait before it would spend its limit
        // on an earlier kernel's time
        grid_wait();
        int i = 0;
        for (; i < k_hi - k_lo; ++i) {
            const int s = i % p.stages;
            if (!mbar_wait(full(s), uint32_t(i / p.stages) & 1u, dead, &g_ffn_wait_timeouts)) break;
            tc_fence_after();
            const uint32_t sa = base + uint32_t(s) * stage_bytes, sb = sa + kAcc * kABytes;
#pragma unroll
            for (int a = 0; a < kAcc; ++a)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t w = sa + a * kABytes;
                    mma<false>(tmem + uint32_t(a * p.rows_n),
                               kAMn ? sdesc(w + j * 2048, 8192, 1024) : sdesc(w + j * 32, 16, 1024),
                               sdesc(sb + j * 32, 16, 1024), id, (i | j) != 0);
                }
            commit(empty(s));
        }
        commit(done);
        if (dead) drain(full, i, p.stages, &g_ffn_wait_timeouts);
    }
    if (warp >= 2) {
        // results of earlier kernels are visible from here; only then may a
        // later kernel start (so that what runs beside this one has all older
        // writes, and the one after may copy its weights early)
        grid_wait();
        grid_release();
    }
    __syncwarp();
    grid_wait();      // every thread: outputs of earlier kernels are read and overwritten below
    // all copies have landed and been read (each was waited for by its MMAs):
    // the ring's memory takes the partial sums, [accumulator][token][128 rows]
    // (one warp waits and the block meets behind it: eight warps that wait each for
    // themselves and then bring their lanes together cost 0.4 us a product)
    if (warp == 0) mbar_wait(done, 0, dead, &g_ffn_wait_timeouts);
    __syncthreads();
    tc_fence_after();
    const int row = (warp & 3) * 32 + lane;
    for (int c = (warp >> 2) * 16; c < kAcc * p.rows_n; c += 32) {
        float v[16];
        tmem_ld16(v, tmem + (uint32_t(warp & 3) << 21) + uint32_t(c));
        tmem_wait();
        tmem_tie16(v);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + uint32_t((c + i) * 128 + row) * 4), "f"(v[i]) : "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    // one token at a time, four weight rows a lane, shared out over the cluster's warps
    for (int tok = int(rank) * 8 + warp; tok < p.n; tok += int(split) * 8) {
        float acc[kAcc][4];
#pragma unroll
        for (int a = 0; a < kAcc; ++a) {
            const uint32_t at = base + uint32_t((a * p.rows_n + tok) * 128 + lane * 4) * 4;
            float4 part[kMaxSplit];
#pragma unroll
            for (int r = 0; r < kMaxSplit; ++r)
                part[r] = r < int(split) ? ld_cluster_v4(map_rank(at, uint32_t(r))) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[a][i] = 0.0f;
#pragma unroll
            for (int r = 0; r < kMaxSplit; ++r) {
                acc[a][0] += part[r].x;
                acc[a][1] += part[r].y;
                acc[a][2] += part[r].z;
                acc[a][3] += part[r].w;
            }
        }
        const int col = f0 + lane * 4, valid = min(4, p.m - col);
        if (valid <= 0) continue;
        auto put = [&](const Out &o, const float *v) {
            if (!o.p) return;
            const long long at = tok * o.ld + col;
            if (o.vec && valid == 4) {   // (four elements from a multiple of four on)
                if (o.f32) {
                    *reinterpret_cast<float4 *>(static_cast<float *>(o.p) + at) = make_float4(v[0], v[1], v[2], v[3]);
                } else {
                    const uint2 w = p.f16 ? make_uint2(pack2<true>(v[0], v[1]), pack2<true>(v[2], v[3]))
                                          : make_uint2(pack2<false>(v[0], v[1]), pack2<false>(v[2], v[3]));
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(o.p) + at) = w;
                }
                return;
            }
            for (int i = 0; i < valid; ++i) {
                if (o.f32) static_cast<float *>(o.p)[at + i] = v[i];
                else static_cast<uint16_t *>(o.p)[at + i] = pack1(v[i], p.f16);
            }
        };
        if constexpr (kEpi == kGated) {
            put(p.out[1], acc[0]);
            put(p.out[2], acc[1]);
            if (p.out[0].p) {
                float h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) h[i] = activation_of<false>(acc[0][i], p.act, nullptr) * acc[1][i];
                put(p.out[0], h);
            }
        } else if constexpr (kEpi == kBack) {
            const long long at = tok * p.ldp + col;
            float dg[4] = {}, du[4] = {}, h[4] = {};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i >= valid) break;
                const float g = p.pre_f32 ? static_cast<const float *>(p.g)[at + i]
                                          : unpack1(static_cast<const uint16_t *>(p.g)[at + i], p.f16);
                const float u = p.pre_f32 ? static_cast<const float *>(p.u)[at + i]
                                          : unpack1(static_cast<const uint16_t *>(p.u)[at + i], p.f16);
                float slope;
                const float a = activation_of<true>(g, p.act, &slope);
                dg[i] = acc[0][i] * u * slope;
                du[i] = acc[0][i] * a;
                h[i] = a * u;
            }
            put(p.out[0], dg);
            put(p.out[1], du);
            put(p.out[2], h);
        } else {
            put(p.out[0], acc[0]);
        }
    }
    cluster_sync();   // partial sums stay until every CTA of the cluster has read them
    if (warp == 2) tmem_free<false>(tmem, cols);
}

// ---- rows that TMA cannot address ----------------------------------------------------

// 16-bit matrices copied to rows that start on 16-byte boundaries (dst_ld a
// multiple of 8), up to five in one launch. A thread makes 8 elements of a row:
// loads of the widest words that the rows are aligned to (2, 4 or 8 bytes;
// consecutive threads read consecutive bytes), one 16-byte store; what a row has
// past its last column is not written. x and the weights of 777 x 1029 x 2731, in
// single elements: 10 us for 18.5 MB read and as much written (bound by L2 and the
// launch).
struct AlignJob {
    const uint16_t *src;
    uint16_t *dst;
    long long src_ld, dst_ld;
    int cols, vecs, word;        // vecs: 8-element vectors of a row; word: bytes of a load
    long long first, rows;       // the job's first vector in the launch
};

struct AlignJobs {
    AlignJob job[5];
    int count;
    long long total;
};

__global__ void __launch_bounds__(256) ffn_align_kernel(const __grid_constant__ AlignJobs jobs) {
    grid_wait();
    grid_release();
    const long long stride = (long long)gridDim.x * 256;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < jobs.total; i += stride) {
        int k = 0;
        while (k + 1 < jobs.count && i >= jobs.job[k + 1].first) ++k;
        const AlignJob &j = jobs.job[k];
        const long long v = i - j.first, row = v >> 32 ? v / j.vecs : uint32_t(v) / uint32_t(j.vecs);
        const int c = int(v - row * j.vecs) * 8;
        const uint16_t *s = j.src + row * j.src_ld + c;
        uint16_t *d = j.dst + row * j.dst_ld + c;
        if (c + 8 <= j.cols) {
            uint32_t w[4];
            if (j.word == 8) {
                const uint2 *t = reinterpret_cast<const uint2 *>(s);
                const uint2 lo = t[0], hi = t[1];
                w[0] = lo.x; w[1] = lo.y; w[2] = hi.x; w[3] = hi.y;
            } else if (j.word == 4) {
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = reinterpret_cast<const uint32_t *>(s)[e];
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = word(s[2 * e], s[2 * e + 1]);
            }
            *reinterpret_cast<uint4 *>(d) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            for (int e = 0; c + e < j.cols; ++e) d[e] = s[e];
        }
    }
}

// ---- host ---------------------------------------------------------------------------

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
    static const EncodeTiledFn fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return EncodeTiledFn(nullptr);
        }
        return reinterpret_cast<EncodeTiledFn>(ptr);
    }();
    return fn;
}

// The widest of 8, 4 and 2 bytes that rows of `pitch` bytes at p all start on
// multiples of.
int word_of(const void *p, int64_t pitch) {
    const uint64_t bits = reinterpret_cast<uintptr_t>(p) | uint64_t(pitch);
    return bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : 2;
}

// A row-major matrix of 16-bit elements in device memory.
struct Mat {
    const void *p;
    int64_t rows, cols, ld;
};

bool rows_on(const void *p, int64_t ld, int elem_bytes, int boundary) {
    return reinterpret_cast<uintptr_t>(p) % uintptr_t(boundary) == 0 && ld * elem_bytes % boundary == 0;
}

bool tma_ok(const void *p, int64_t ld, int elem_bytes) { return rows_on(p, ld, elem_bytes, 16); }

bool make_map(CUtensorMap *map, const void *p, int64_t rows, int64_t cols, int64_t ld, int elem_bytes,
              bool f16, int box_cols, int box_rows, bool swizzle128) {
    const EncodeTiledFn fn = encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(ld) * cuuint64_t(elem_bytes)};
    const cuuint32_t box[2] = {cuuint32_t(box_cols), cuuint32_t(box_rows)};
    const cuuint32_t elem[2] = {1, 1};
    const CUtensorMapDataType type = elem_bytes == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : f16           ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                     : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return fn(map, type, 2, const_cast<void *>(p), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
              swizzle128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An operand's map: boxes of 64 along the contiguous axis. K-major: `rows`
// rows of a tile; MN-major: 64 rows (of k).
bool operand_map(CUtensorMap *map, const Mat &x, bool mn, int rows, bool f16) {
    return make_map(map, x.p, x.rows, x.cols, x.ld, 2, f16, 64, mn ? 64 : rows, true);
}

// The outputs [rows, cols]; `maps_too`: with tensor maps for the tile kernel's
// stores (the stream kernel stores element by element).
int set_outs(Params &p, Maps &maps, const Out *outs, int first, int count, int64_t rows, int64_t cols, bool maps_too) {
    outs -= first;
    for (int i = first; i < first + count; ++i) {
        p.out[i] = outs[i];
        Out &o = p.out[i];
        const int es = o.f32 ? 4 : 2;
        o.vec = o.p && tma_ok(o.p, o.ld, es);
        // TMA stores whole 16-byte pieces: a last box that ends inside one goes without
        o.tma_cols = !maps_too || !o.vec ? 0 : int(cols * es % 16 == 0 ? cols : cols * es / 64 * 64 / es);
        o.word = word_of(o.p, o.ld * es);
        if (o.tma_cols && !make_map(&maps.c[i], o.p, rows, cols, o.ld, es, p.f16, o.f32 ? 16 : 32, 32, false))
            return ROPE3D_ERR_CUDA;
    }
    return ROPE3D_OK;
}

// How many pairs of CTAs the device holds at once (asked once a device).
template <int kBN, int kLayout, int kEpi, bool kF16, int kAct>
bool tile_ready(int *clusters) {
    static std::atomic<int> known[64];   // per device, 0 = not asked yet
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    int c = known[dev].load(std::memory_order_acquire);
    if (c == 0) {
        auto *fn = ffn_tile_kernel<kBN, kLayout, kEpi, kF16, kAct>;
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, tile_smem<kBN>()) != cudaSuccess) {
            cudaGetLastError();
            return false;
        }
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = tile_smem<kBN>();
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&c, fn, &cfg) != cudaSuccess || c < 1) {
            cudaGetLastError();
            return false;
        }
        known[dev].store(c, std::memory_order_release);
    }
    *clusters = c;
    return true;
}

// How a product of the tile kernel is divided: the tile's width, the tiles that
// one pair of CTAs computes each, and into how many parts of k the others are
// split.
struct Plan {
    int bn, cols;            // MMA N; columns of a tile (half of it where gated)
    int64_t tiles, whole;
    int split;
    int64_t units() const { return whole + (tiles - whole) * split; }
    int64_t part_bytes() const { return (tiles - whole) * split * 256 * bn * 4; }
};

// The fastest division by a model of the time in microseconds: `kPairs` pairs
// run rounds of tiles; 64 of k cost a pair 0.355 us at 256 columns and 0.28 us at
// 128 (4096 x 4096 of k = 16384, bf16: the narrow tile reads the operands from L2
// at the same rate for half of the products), a tile's start and end about 1.5;
// split tiles add a kernel (3) and their sums' bytes, written and read. Measured:
// 8192 x 2048 of k = 8192 takes 256 us at 128 columns in 7 rounds, 181 us at 256
// in 4 and 165 us with the last round's 28 tiles split in two.
// The GB300's 76 pairs are written here, not asked, so that the workspace's size
// is known without a device; the kernel's units run on any number of pairs.
constexpr int64_t kPairs = 76;
constexpr double kPerK256 = 0.355, kPerK128 = 0.28, kTileStart = 1.5, kFinish = 3.0;

int64_t tiles_of(int64_t m, int64_t n, int64_t cols) { return (m + 255) / 256 * ((n + cols - 1) / cols); }

Plan plan_tiles(int64_t m, int64_t n, int nk, bool gated) {
    Plan best{};
    double best_time = 1e30;
    for (int bn : {256, 128}) {
        Plan c{};
        c.bn = bn;
        c.cols = gated ? bn / 2 : bn;
        c.tiles = tiles_of(m, n, c.cols);
        const double per_k = bn == 256 ? kPerK256 : kPerK128;
        const int64_t rounds = c.tiles / kPairs, rest = c.tiles % kPairs;
        for (int s = 1; s <= 32; ++s) {
            if (s > 1 && (rest == 0 || nk / s < 4)) break;
            double t = double(rounds) * (nk * per_k + kTileStart);
            if (rest) t += double((rest * s + kPairs - 1) / kPairs) * (double((nk + s - 1) / s) * per_k + kTileStart);
            if (s > 1) t += kFinish + double(rest * s) * 256 * bn * 8 / 4.0e6;
            if (t < best_time) {
                best_time = t;
                best = c;
                best.split = s;
                best.whole = s > 1 ? c.tiles - rest : c.tiles;
            }
        }
    }
    return best;
}

// The gradients' launch: dx (where wanted) and the weights' gradients that are
// wanted. The model takes the whole work in equal shares, or the longest unit of dx
// where that is longer; dx is split where that pays. That is the time where units are
// many (2048 x 2048 x 8192: 207.7 us by the model, 208.1 by next_unit's order of the
// units at the same costs). It is too low where they are few or make one round and a
// little: the weights' tiles are not split, and their longest one, all tokens deep, is
// not in it (8192 x 256 x 1024, 12 such tiles: 12.9 us by the model, 46.9 by the
// units' order, 37.3 with the narrow tile that it then does not choose).
Plan plan_grads(int64_t tokens, int64_t width, int64_t hidden, bool dx, bool gate_up, bool down) {
    Plan best{};
    double best_time = 1e30;
    const int nk = int((hidden + 63) / 64) * 2, nkw = int((tokens + 63) / 64);
    for (int bn : {256, 128}) {
        Plan c{};
        c.bn = c.cols = bn;
        c.tiles = dx ? tiles_of(tokens, width, bn) : 0;
        const int64_t weights = (gate_up ? 2 * tiles_of(hidden, width, bn) : 0) + (down ? tiles_of(width, hidden, bn) : 0);
        const double per_k = bn == 256 ? kPerK256 : kPerK128;
        const int64_t rest = c.tiles % kPairs;
        for (int s = 1; s <= 32; ++s) {
            if (s > 1 && (rest == 0 || nk / s < 4)) break;
            const double work = double(c.tiles - rest) * (nk * per_k + kTileStart) +
                                double(rest * s) * (double(nk) / s * per_k + kTileStart) +
                                double(weights) * (nkw * per_k + kTileStart);
            double t = std::max(work / kPairs, rest ? double((nk + s - 1) / s) * per_k + kTileStart : 0.0);
            if (s > 1) t += kFinish + double(rest * s) * 256 * bn * 8 / 4.0e6;
            if (t < best_time) {
                best_time = t;
                best = c;
                best.split = s;
                best.whole = s > 1 ? c.tiles - rest : c.tiles;
            }
        }
    }
    return best;
}

Sub make_sub(int64_t m, int64_t n, int64_t cols) {
    return Sub{int(m), int(n), int((m + 255) / 256), int((n + cols - 1) / cols)};
}

// Launches the tile kernel (operands' and outputs' maps and p.sub are set) and,
// where tiles are split, the kernel that finishes them.
template <int kBN, int kLayout, int kEpi, bool kF16, int kAct>
int launch_tile_as(const Plan &plan, Params &p, const Maps &maps, void *part, cudaStream_t st) {
    int clusters = 0;
    if (!tile_ready<kBN, kLayout, kEpi, kF16, kAct>(&clusters)) return ROPE3D_ERR_CUDA;
    p.whole = int(plan.whole);
    p.split = plan.split;
    p.units = int(plan.units());
    p.part = static_cast<float *>(part);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(2 * std::min(clusters, p.units + p.weight_units)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = tile_smem<kBN>();
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, ffn_tile_kernel<kBN, kLayout, kEpi, kF16, kAct>, maps, p) != cudaSuccess) {
        cudaGetLastError();
        return ROPE3D_ERR_CUDA;
    }
    if (plan.whole == plan.tiles) return ROPE3D_OK;
    const int64_t warps = (plan.tiles - plan.whole) * 8 * (plan.cols / 8);
    cfg.gridDim = dim3(unsigned(warps / 4));
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, ffn_finish_kernel<kBN, kEpi, kF16, kAct>, p) != cudaSuccess) {
        cudaGetLastError();
        return ROPE3D_ERR_CUDA;
    }
    return ROPE3D_OK;
}

int sm_count() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return n;
}

template <int kValue>
struct Const {
    static constexpr int value = kValue;
};

template <int kLayout, int kEpi>
int launch_plan(const Plan &plan, Params &p, const Maps &maps, void *part, cudaStream_t st) {
    if (plan.units() + p.weight_units > (int64_t(1) << 30)) return ROPE3D_ERR_SHAPE;
    auto as = [&](auto bn, auto f16, auto act) {
        return launch_tile_as<decltype(bn)::value, kLayout, kEpi, decltype(f16)::value, decltype(act)::value>(
            plan, p, maps, part, st);
    };
    auto with_act = [&](auto bn, auto f16) {
        if constexpr (kEpi != kPlain) {   // (the plain product has no activation)
            if (p.act == ROPE3D_ACT_GELU_TANH) return as(bn, f16, Const<ROPE3D_ACT_GELU_TANH>{});
            if (p.act == ROPE3D_ACT_GELU_ERF) return as(bn, f16, Const<ROPE3D_ACT_GELU_ERF>{});
        }
        return as(bn, f16, Const<ROPE3D_ACT_SILU>{});
    };
    auto with_type = [&](auto bn) { return p.f16 ? with_act(bn, Const<1>{}) : with_act(bn, Const<0>{}); };
    return plan.bn == 128 ? with_type(Const<128>{}) : with_type(Const<256>{});
}

// One product of `m` rows and `n` columns (of each half where gated): a and b
// hold its operands, two of b where gated.
template <int kLayout, int kEpi>
int launch_tile(int64_t m, int64_t n, Params &p, Maps &maps, const Mat &a, const Mat *b, void *part, cudaStream_t st) {
    const Plan plan = plan_tiles(m, n, p.nk0 + p.nk1, kEpi == kGated);
    if (!operand_map(&maps.a[0], a, false, 128, p.f16)) return ROPE3D_ERR_CUDA;
    for (int i = 0; i < (kEpi == kGated ? 2 : 1); ++i)
        if (!operand_map(&maps.b[i], b[i], kLayout != kKK, plan.bn / 2, p.f16)) return ROPE3D_ERR_CUDA;
    p.sub[0] = make_sub(m, n, plan.cols);
    return launch_plan<kLayout, kEpi>(plan, p, maps, part, st);
}

// Few tokens. w: the weights (two where gated or of two segments), x: the
// tokens' rows; p.m = weight rows, p.n = tokens.
template <bool kAMn, int kEpi>
int launch_stream(Params &p, Maps &maps, const Mat *w, const Mat *x, int segs, cudaStream_t st) {
    constexpr int kAcc = kEpi == kGated ? 2 : 1;
    const int sms = sm_count();
    if (sms <= 0) return ROPE3D_ERR_CUDA;
    p.rows_n = (p.n + 15) / 16 * 16;
    for (int i = 0; i < (kEpi == kGated ? 2 : segs); ++i)
        if (!operand_map(&maps.a[i], w[i], kAMn, 128, p.f16)) return ROPE3D_ERR_CUDA;
    for (int i = 0; i < segs; ++i)
        if (!operand_map(&maps.b[i], x[i], false, p.rows_n, p.f16)) return ROPE3D_ERR_CUDA;
    // shared memory: two CTAs an SM where three slots of the ring fit half of
    // it (and the partial sums fit the ring), else one
    const int stage = kAcc * kABytes + p.rows_n * 128, sums = kAcc * p.rows_n * 512;
    const int extra = 1024 + 512;
    int stages = (112 * 1024 - extra) / stage, per_sm = 2;
    if (stages < 3 || stages * stage < sums) {
        stages = (226 * 1024 - extra) / stage;
        per_sm = 1;
    }
    stages = std::min(stages, 8);
    p.stages = stages;
    const int nk = p.nk0 + p.nk1;
    const int64_t tiles = (int64_t(p.m) + 127) / 128;
    int split = 1;
    while (split < kMaxSplit && tiles * split * 2 <= int64_t(sms) * per_sm && nk / (split * 2) >= 2) split *= 2;
    const int smem = stages * stage + extra;
    auto *fn = ffn_stream_kernel<kAMn, kEpi>;
    static std::atomic<int> set[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return ROPE3D_ERR_CUDA;
    if (!set[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess) {
            cudaGetLastError();
            return ROPE3D_ERR_CUDA;
        }
        set[dev].store(1, std::memory_order_release);
    }
    if (tiles * split > (int64_t(1) << 30)) return ROPE3D_ERR_SHAPE;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(tiles * split));
    cfg.blockDim = dim3(kStreamThreads);
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(split);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, fn, maps, p) != cudaSuccess) {
        cudaGetLastError();
        return ROPE3D_ERR_CUDA;
    }
    return ROPE3D_OK;
}

int blocks64(int64_t k) { return int((k + 63) / 64); }
int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// Workspace: pieces in a fixed order, each at a multiple of 256 bytes.
struct Carver {
    char *base;
    int64_t used = 0;
    void *take(int64_t bytes) {
        void *p = base ? base + used : nullptr;
        used += up(bytes, 256);
        return p;
    }
};

// x as TMA can read it: itself, or a copy in the workspace with its rows on
// 16-byte boundaries, added to `jobs`.
void aligned(Mat &x, Carver &ws, AlignJobs *jobs) {
    if (tma_ok(x.p, x.ld, 2)) return;
    const int64_t ld = up(x.cols, 8);
    void *dst = ws.take(x.rows * ld * 2);
    if (jobs) {
        jobs->job[jobs->count++] = AlignJob{static_cast<const uint16_t *>(x.p), static_cast<uint16_t *>(dst),
                                            x.ld, ld, int(x.cols), int(ld / 8), word_of(x.p, x.ld * 2), jobs->total, x.rows};
        jobs->total += x.rows * (ld / 8);
    }
    x.p = dst;
    x.ld = ld;
}

int launch_align(const AlignJobs &jobs, cudaStream_t st) {
    if (!jobs.count) return ROPE3D_OK;
    const int sms = sm_count();
    if (sms <= 0) return ROPE3D_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(std::min<int64_t>((jobs.total + 255) / 256, int64_t(sms) * 8)));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, ffn_align_kernel, jobs) != cudaSuccess) {
        cudaGetLastError();
        return ROPE3D_ERR_CUDA;
    }
    return ROPE3D_OK;
}

bool on_device(const void *p, int device) {
    cudaPointerAttributes attr{};
    if (cudaPointerGetAttributes(&attr, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    if (attr.type == cudaMemoryTypeManaged) return true;
    return attr.type == cudaMemoryTypeDevice && attr.device == device;
}

// One argument's memory: [p, p + bytes), bytes = 0 for an absent one.
struct Span {
    const void *p;
    int64_t bytes;
    int align;
};

Span span(const void *p, int64_t rows, int64_t cols, int64_t ld, int es) {
    return Span{p, p ? ((rows - 1) * ld + cols) * es : 0, es};
}

bool overlap(const Span &a, const Span &b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && x < y + uint64_t(b.bytes) && y < x + uint64_t(a.bytes);
}

// Alignment, overlap (outputs overlap nothing) and device memory.
int check_spans(const Span *in, int nin, const Span *out, int nout, bool check_device) {
    for (int i = 0; i < nin + nout; ++i) {
        const Span &s = i < nin ? in[i] : out[i - nin];
        if (s.p && reinterpret_cast<uintptr_t>(s.p) % uintptr_t(s.align) != 0) return ROPE3D_ERR_ALIGN;
    }
    for (int o = 0; o < nout; ++o) {
        for (int i = 0; i < nin; ++i)
            if (overlap(out[o], in[i])) return ROPE3D_ERR_ALIAS;
        for (int j = o + 1; j < nout; ++j)
            if (overlap(out[o], out[j])) return ROPE3D_ERR_ALIAS;
    }
    if (!check_device) return ROPE3D_OK;
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) {
        cudaGetLastError();
        return ROPE3D_ERR_CUDA;
    }
    for (int i = 0; i < nin + nout; ++i) {
        const Span &s = i < nin ? in[i] : out[i - nin];
        if (s.p && !on_device(s.p, device)) return ROPE3D_ERR_DEVICE;
    }
    return ROPE3D_OK;
}

constexpr int64_t kMaxDim = int64_t(1) << 20, kMaxTokens = int64_t(1) << 28, kMaxLd = int64_t(1) << 31;

bool bad_ld(int64_t ld, int64_t cols) { return ld < cols || ld > kMaxLd; }

int check_shape(int64_t tokens, int64_t width, int64_t hidden, int32_t dtype, int32_t act) {
    if (tokens <= 0 || width <= 0 || hidden <= 0 || tokens > kMaxTokens || width > kMaxDim || hidden > kMaxDim)
        return ROPE3D_ERR_SHAPE;
    if (dtype != ROPE3D_BF16 && dtype != ROPE3D_F16) return ROPE3D_ERR_DTYPE;
    if (act != ROPE3D_ACT_SILU && act != ROPE3D_ACT_GELU_TANH && act != ROPE3D_ACT_GELU_ERF) return ROPE3D_ERR_ARG;
    return ROPE3D_OK;
}

int check_pre(int32_t pre_dtype, int32_t dtype) {
    return pre_dtype == ROPE3D_F32 || pre_dtype == dtype ? ROPE3D_OK : ROPE3D_ERR_DTYPE;
}

Params base_params(int32_t dtype, int32_t act) {
    Params p{};
    p.f16 = dtype == ROPE3D_F16;
    p.act = act;
    return p;
}

thread_local int t_ffn_kernel = 0;   // 1 tile, 2 stream kernel: this thread's last forward or dx product

// h (may be null), g, u (may be null) of x.
int project(const Mat &x, const Mat &wg, const Mat &wu, Out h, Out g, Out u, int32_t dtype, int32_t act, void *part,
            cudaStream_t st) {
    Maps maps;
    Params p = base_params(dtype, act);
    const Out outs[3] = {h, g, u};
    const Mat w[2] = {wg, wu};
    p.nk0 = blocks64(x.cols);
    const int rc = set_outs(p, maps, outs, 0, 3, x.rows, wg.rows, x.rows > kStreamGated);
    if (rc != ROPE3D_OK) return rc;
    if (x.rows <= kStreamGated) {
        p.m = int(wg.rows);
        p.n = int(x.rows);
        return launch_stream<false, kGated>(p, maps, w, &x, 1, st);
    }
    return launch_tile<kKK, kGated>(x.rows, wg.rows, p, maps, x, w, part, st);
}

// One body for the call and for its workspace query (launch = false; *need
// receives the bytes).
int forward(const rope3d_gated_ffn_args *a, bool launch, bool check_device, int64_t *need, cudaStream_t st) {
    if (!a || !a->x || !a->w_gate || !a->w_up || !a->w_down || !a->y) return ROPE3D_ERR_NULL;
    if ((a->gate_pre == nullptr) != (a->up_pre == nullptr)) return ROPE3D_ERR_NULL;
    const int64_t M = a->tokens, D = a->width, F = a->hidden;
    int rc = check_shape(M, D, F, a->dtype, a->act);
    if (rc != ROPE3D_OK) return rc;
    if (a->gate_pre && (rc = check_pre(a->pre_dtype, a->dtype)) != ROPE3D_OK) return rc;
    if (bad_ld(a->x_stride, D) || bad_ld(a->w_gate_stride, D) || bad_ld(a->w_up_stride, D) ||
        bad_ld(a->w_down_stride, F) || bad_ld(a->y_stride, D) || (a->gate_pre && bad_ld(a->pre_stride, F)))
        return ROPE3D_ERR_SHAPE;
    const int pre_es = a->pre_dtype == ROPE3D_F32 ? 4 : 2;
    Mat x{a->x, M, D, a->x_stride}, wg{a->w_gate, F, D, a->w_gate_stride}, wu{a->w_up, F, D, a->w_up_stride},
        wd{a->w_down, D, F, a->w_down_stride};
    const int nkd = blocks64(D), nkf = blocks64(F);
    int64_t part_bytes = M <= kStreamGated ? 0 : plan_tiles(M, F, nkd, true).part_bytes();
    if (M > kStreamTokens) part_bytes = std::max(part_bytes, plan_tiles(M, D, nkf, false).part_bytes());
    Carver size{nullptr};
    {
        Mat t[4] = {x, wg, wu, wd};
        for (Mat &m : t) aligned(m, size, nullptr);
        size.take(M * up(F, 64) * 2);
        size.take(part_bytes);
    }
    if (need) *need = size.used;
    else if (!a->workspace) return ROPE3D_ERR_NULL;
    else if (a->workspace_bytes < size.used) return ROPE3D_ERR_SCRATCH;
    const Span in[4] = {span(x.p, M, D, x.ld, 2), span(wg.p, F, D, wg.ld, 2), span(wu.p, F, D, wu.ld, 2),
                        span(wd.p, D, F, wd.ld, 2)};
    Span out[4] = {span(a->y, M, D, a->y_stride, 2), span(a->gate_pre, M, F, a->pre_stride, pre_es),
                   span(a->up_pre, M, F, a->pre_stride, pre_es), Span{a->workspace, size.used, 256}};
    rc = check_spans(in, 4, out, need ? 3 : 4, check_device);
    if (rc != ROPE3D_OK || need || !launch) return rc;

    Carver ws{static_cast<char *>(a->workspace)};
    AlignJobs jobs{};
    for (Mat *m : {&x, &wg, &wu, &wd}) aligned(*m, ws, &jobs);
    if ((rc = launch_align(jobs, st)) != ROPE3D_OK) return rc;
    const int64_t hld = up(F, 64);
    void *hbuf = ws.take(M * hld * 2), *part = ws.take(part_bytes);
    const int f32 = a->gate_pre && a->pre_dtype == ROPE3D_F32;
    rc = project(x, wg, wu, Out{hbuf, hld, 0, 0, 0}, Out{a->gate_pre, a->pre_stride, f32, 0, 0},
                 Out{a->up_pre, a->pre_stride, f32, 0, 0}, a->dtype, a->act, part, st);
    if (rc != ROPE3D_OK) return rc;
    const Mat h{hbuf, M, F, hld};
    Maps maps;
    Params p = base_params(a->dtype, a->act);
    const Out y{a->y, a->y_stride, 0, 0, 0};
    p.nk0 = blocks64(F);
    if ((rc = set_outs(p, maps, &y, 0, 1, M, D, M > kStreamTokens)) != ROPE3D_OK) return rc;
    t_ffn_kernel = M <= kStreamGated ? 2 : 1;
    if (M <= kStreamTokens) {
        p.m = int(D);
        p.n = int(M);
        return launch_stream<false, kPlain>(p, maps, &wd, &h, 1, st);
    }
    return launch_tile<kKK, kPlain>(M, D, p, maps, h, &wd, part, st);
}

int backward(const rope3d_gated_ffn_backward_args *a, bool launch, bool check_device, int64_t *need,
             cudaStream_t st) {
    if (!a || !a->dy || !a->x || !a->w_gate || !a->w_up || !a->w_down) return ROPE3D_ERR_NULL;
    if ((a->gate_pre == nullptr) != (a->up_pre == nullptr)) return ROPE3D_ERR_NULL;
    if ((a->dw_gate == nullptr) != (a->dw_up == nullptr)) return ROPE3D_ERR_NULL;
    if (!a->dx && !a->dw_gate && !a->dw_down) return ROPE3D_ERR_NULL;
    const int64_t M = a->tokens, D = a->width, F = a->hidden;
    int rc = check_shape(M, D, F, a->dtype, a->act);
    if (rc != ROPE3D_OK) return rc;
    if (a->gate_pre && (rc = check_pre(a->pre_dtype, a->dtype)) != ROPE3D_OK) return rc;
    if (bad_ld(a->dy_stride, D) || bad_ld(a->x_stride, D) || bad_ld(a->w_gate_stride, D) ||
        bad_ld(a->w_up_stride, D) || bad_ld(a->w_down_stride, F) || (a->gate_pre && bad_ld(a->pre_stride, F)) ||
        (a->dx && bad_ld(a->dx_stride, D)) ||
        (a->dw_gate && (bad_ld(a->dw_gate_stride, D) || bad_ld(a->dw_up_stride, D))) ||
        (a->dw_down && bad_ld(a->dw_down_stride, F)))
        return ROPE3D_ERR_SHAPE;
    const bool again = !a->gate_pre;   // the projections are computed again, kept in fp32
    const int pre_es = again || a->pre_dtype == ROPE3D_F32 ? 4 : 2;
    Mat dy{a->dy, M, D, a->dy_stride}, x{a->x, M, D, a->x_stride}, wg{a->w_gate, F, D, a->w_gate_stride},
        wu{a->w_up, F, D, a->w_up_stride}, wd{a->w_down, D, F, a->w_down_stride};
    const int64_t hld = up(F, 64);
    const bool few = M <= kStreamTokens;
    // the split products' sums, one launch at a time
    const Plan grads = plan_grads(M, D, F, a->dx && !few, a->dw_gate != nullptr, a->dw_down != nullptr);
    int64_t part_bytes = grads.part_bytes();
    if (!few) part_bytes = std::max(part_bytes, plan_tiles(M, F, blocks64(D), false).part_bytes());
    if (again && M > kStreamGated) part_bytes = std::max(part_bytes, plan_tiles(M, F, blocks64(D), true).part_bytes());
    Carver size{nullptr};
    {
        Mat t[5] = {dy, x, wg, wu, wd};
        for (Mat &m : t) aligned(m, size, nullptr);
        for (int i = 0; i < 3; ++i) size.take(M * hld * 2);
        if (again)
            for (int i = 0; i < 2; ++i) size.take(M * hld * 4);
        size.take(part_bytes);
    }
    if (need) *need = size.used;
    else if (!a->workspace) return ROPE3D_ERR_NULL;
    else if (a->workspace_bytes < size.used) return ROPE3D_ERR_SCRATCH;
    const Span in[7] = {span(dy.p, M, D, dy.ld, 2), span(x.p, M, D, x.ld, 2), span(wg.p, F, D, wg.ld, 2),
                        span(wu.p, F, D, wu.ld, 2), span(wd.p, D, F, wd.ld, 2),
                        span(a->gate_pre, M, F, a->pre_stride, pre_es), span(a->up_pre, M, F, a->pre_stride, pre_es)};
    const Span out[5] = {span(a->dx, M, D, a->dx_stride, 2), span(a->dw_gate, F, D, a->dw_gate_stride, 2),
                         span(a->dw_up, F, D, a->dw_up_stride, 2), span(a->dw_down, D, F, a->dw_down_stride, 2),
                         Span{a->workspace, size.used, 256}};
    rc = check_spans(in, 7, out, need ? 4 : 5, check_device);
    if (rc != ROPE3D_OK || need || !launch) return rc;

    Carver ws{static_cast<char *>(a->workspace)};
    AlignJobs jobs{};
    for (Mat *m : {&dy, &x, &wg, &wu, &wd}) aligned(*m, ws, &jobs);
    if ((rc = launch_align(jobs, st)) != ROPE3D_OK) return rc;
    void *dgb = ws.take(M * hld * 2), *dub = ws.take(M * hld * 2), *hb = ws.take(M * hld * 2);
    const void *g = a->gate_pre, *u = a->up_pre;
    int64_t ldp = a->pre_stride;
    void *gb = again ? ws.take(M * hld * 4) : nullptr, *ub = again ? ws.take(M * hld * 4) : nullptr;
    void *part = ws.take(part_bytes);
    if (again) {
        rc = project(x, wg, wu, Out{nullptr, 0, 0, 0, 0}, Out{gb, hld, 1, 0, 0}, Out{ub, hld, 1, 0, 0}, a->dtype, a->act, part, st);
        if (rc != ROPE3D_OK) return rc;
        g = gb;
        u = ub;
        ldp = hld;
    }
    t_ffn_kernel = few ? 2 : 1;
    Maps maps;
    {
        // dh = dy Wd, and from it dg, du and h
        Params p = base_params(a->dtype, a->act);
        const Out outs[3] = {Out{dgb, hld, 0, 0, 0}, Out{dub, hld, 0, 0, 0},
                             Out{a->dw_down ? hb : nullptr, hld, 0, 0, 0}};
        if ((rc = set_outs(p, maps, outs, 0, 3, M, F, !few)) != ROPE3D_OK) return rc;
        p.nk0 = blocks64(D);
        p.g = g;
        p.u = u;
        p.ldp = ldp;
        p.pre_f32 = pre_es == 4;
        p.pre_vec = rows_on(g, ldp, pre_es, 32) && rows_on(u, ldp, pre_es, 32);
        p.m = int(F);
        p.n = int(M);
        rc = few ? launch_stream<true, kBack>(p, maps, &wd, &dy, 1, st)
                 : launch_tile<kKM, kBack>(M, F, p, maps, dy, &wd, part, st);
        if (rc != ROPE3D_OK) return rc;
    }
    const Mat dg{dgb, M, F, hld}, du{dub, M, F, hld}, h{hb, M, F, hld};
    const Out dx{a->dx, a->dx_stride, 0, 0, 0};
    if (a->dx && few) {
        Params p = base_params(a->dtype, a->act);
        const Mat t[2] = {dg, du}, w[2] = {wg, wu};
        if ((rc = set_outs(p, maps, &dx, 0, 1, M, D, false)) != ROPE3D_OK) return rc;
        p.nk0 = p.nk1 = blocks64(F);
        p.m = int(D);
        p.n = int(M);
        if ((rc = launch_stream<true, kPlain>(p, maps, w, t, 2, st)) != ROPE3D_OK) return rc;
    }
    const bool tile_dx = a->dx && !few;
    if (!tile_dx && !a->dw_gate && !a->dw_down) return ROPE3D_OK;
    // dx (of many tokens) and the weights' gradients in one launch
    Params p = base_params(a->dtype, a->act);
    p.nk0 = p.nk1 = blocks64(F);
    p.nkw = blocks64(M);
    if (tile_dx) {
        const Mat t[2] = {dg, du}, w[2] = {wg, wu};
        for (int i = 0; i < 2; ++i)
            if (!operand_map(&maps.a[i], t[i], false, 128, p.f16) || !operand_map(&maps.b[i], w[i], true, 64, p.f16))
                return ROPE3D_ERR_CUDA;
        if ((rc = set_outs(p, maps, &dx, 0, 1, M, D, true)) != ROPE3D_OK) return rc;
        p.sub[0] = make_sub(M, D, grads.cols);
    }
    if (a->dw_gate) {
        const Mat t[2] = {dg, du};
        const Out o[2] = {Out{a->dw_gate, a->dw_gate_stride, 0, 0, 0}, Out{a->dw_up, a->dw_up_stride, 0, 0, 0}};
        for (int i = 0; i < 2; ++i) {
            if (!operand_map(&maps.a[2 + i], t[i], true, 64, p.f16) || !operand_map(&maps.b[2 + i], x, true, 64, p.f16))
                return ROPE3D_ERR_CUDA;
            p.sub[1 + i] = make_sub(F, D, grads.cols);
        }
        if ((rc = set_outs(p, maps, o, 1, 2, F, D, true)) != ROPE3D_OK) return rc;
    }
    if (a->dw_down) {
        const Out o{a->dw_down, a->dw_down_stride, 0, 0, 0};
        if (!operand_map(&maps.a[4], dy, true, 64, p.f16) || !operand_map(&maps.b[4], h, true, 64, p.f16))
            return ROPE3D_ERR_CUDA;
        if ((rc = set_outs(p, maps, &o, 3, 1, D, F, true)) != ROPE3D_OK) return rc;
        p.sub[3] = make_sub(D, F, grads.cols);
    }
    int64_t weight_units = 0;
    for (int z = 1; z < 4; ++z) weight_units += int64_t(p.sub[z].tiles_m) * p.sub[z].tiles_n;
    if (weight_units > (int64_t(1) << 30)) return ROPE3D_ERR_SHAPE;
    p.weight_units = int(weight_units);
    // the length of the last round's units of dx against a tile of the weights'
    const int last = (p.nk0 + p.nk1) / (grads.whole == grads.tiles ? 1 : grads.split);
    p.dx_first = last >= p.nkw;
    p.lag = p.dx_first ? (last + p.nkw / 2) / p.nkw : (p.nkw + last / 2) / last;
    return launch_plan<kGrads, kPlain>(grads, p, maps, part, st);
}

}  // namespace

extern "C" int rope3d_gated_ffn(const rope3d_gated_ffn_args *args, void *stream) {
    return forward(args, true, true, nullptr, static_cast<cudaStream_t>(stream));
}

extern "C" int rope3d_gated_ffn_check(const rope3d_gated_ffn_args *args, int32_t check_device) {
    return forward(args, false, check_device != 0, nullptr, nullptr);
}

extern "C" int rope3d_gated_ffn_workspace(const rope3d_gated_ffn_args *args, int64_t *bytes) {
    if (!bytes) return ROPE3D_ERR_NULL;
    return forward(args, false, false, bytes, nullptr);
}

extern "C" int rope3d_gated_ffn_backward(const rope3d_gated_ffn_backward_args *args, void *stream) {
    return backward(args, true, true, nullptr, static_cast<cudaStream_t>(stream));
}

extern "C" int rope3d_gated_ffn_backward_check(const rope3d_gated_ffn_backward_args *args, int32_t check_device) {
    return backward(args, false, check_device != 0, nullptr, nullptr);
}

extern "C" int rope3d_gated_ffn_backward_workspace(const rope3d_gated_ffn_backward_args *args, int64_t *bytes) {
    if (!bytes) return ROPE3D_ERR_NULL;
    return backward(args, false, false, bytes, nullptr);
}

extern "C" int rope3d_gated_ffn_last_kernel(void) { return t_ffn_kernel; }

extern "C" int rope3d_testing_ffn_wait_timeouts(int64_t *count, int32_t reset) {
    if (!count) return ROPE3D_ERR_NULL;
    unsigned int n = 0;
    if (cudaMemcpyFromSymbol(&n, g_ffn_wait_timeouts, sizeof(n)) != cudaSuccess) {
        cudaGetLastError();
        return ROPE3D_ERR_CUDA;
    }
    if (reset) {
        const unsigned int zero = 0;
        if (cudaMemcpyToSymbol(g_ffn_wait_timeouts, &zero, sizeof(zero)) != cudaSuccess) {
            cudaGetLastError();
            return ROPE3D_ERR_CUDA;
        }
    }
    *count = n;
    return ROPE3D_OK;
}
