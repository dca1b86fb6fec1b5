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
// Rows that are not whole aligned 16-byte vectors are read element by element
// (consecutive threads, consecutive elements); rows too long for registers take
// general kernels that read a row once for each of its sums.
// This file: the forward kernels and the entry points; rope3d_norm_back.cu: the
// backward kernels.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/rope3d.h"
#include "rope3d_internal.h"
#include "rope3d_norm.cuh"

namespace {

using namespace rope3d_norm;

// ---- rows in registers -----------------------------------------------------------------

// Bound by the latency of a row's loads and sums while the rows are few: one row of
// 4096 bf16 3.5 us, 1021 x 1157 fp32 7.5 us (124 registers a thread: four blocks an
// SM, 608 rows at once, so two rounds); by memory past that (fp32 9528 x 1790
// 53 us, 5,100 GB/s), except where 16-bit elements go one by one (bf16 9728 x 4001
// 134 us, 2,300 GB/s: too few bytes in flight a thread).
template <int kT, bool kVec, int kE, int kTeam>
__global__ void __launch_bounds__(kTeam > 32 ? kTeam : kTeam ? 128 : 512)
block_norm_team_kernel(const __grid_constant__ NormParams p) {
    using Part = RowPart<kT, kVec, kE>;
    constexpr int W = Part::W, B = kE / 8;
    __shared__ float red[2 * 2 * 32];
    Sums<kTeam> sum{red, 0};
    const TeamOf<kTeam> t;
    const int C = p.channels;
    const float inv_c = 1.0f / float(C);
    auto real_e = [&](int i) { return Part::chan(t.lane, t.size, i / W) < C; };
    grid_wait();
    grid_release();
    for (long long row = (long long)blockIdx.x * t.teams + t.team; row < p.rows; row += (long long)gridDim.x * t.teams) {
        Part x, y;
        x.load(p.x, row * p.ldx, t.lane, t.size, C);
        if (p.y) y.load(p.y, row * p.ldy, t.lane, t.size, C);
        const int g = int(uint32_t(row) / uint32_t(p.rows_per_group));
        float v[kE];
#pragma unroll
        for (int b = 0; b < B; ++b) x.get(b, v + 8 * b);
        if (p.y) {
            float yv[kE], mean, k;
#pragma unroll
            for (int b = 0; b < B; ++b) y.get(b, yv + 8 * b);
            row_stats<kE>(yv, p.post, real_e, inv_c, p.eps, sum, &mean, &k);
#pragma unroll
            for (int b = 0; b < B; ++b) {
                float w[8], gt[8];
                Part::weight(p.post_weight, p.param_f32, p.offset, t.lane, t.size, C, b, w);
                Part::param(p.gate, g * p.ldg, p.param_f32, 1.0f, t.lane, t.size, C, b, gt);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int e = 8 * b + i;
                    v[e] = real_e(e) ? p.res * v[e] + gt[i] * ((yv[e] - mean) * k * w[i]) : 0.0f;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kE; ++i) v[i] *= p.res;
        }
        if (p.r) {
#pragma unroll
            for (int b = 0; b < B; ++b) Part::put(p.r, row * p.ldr, t.lane, t.size, C, b, v + 8 * b);
        }
        if (p.n) {
            float mean, k;
            row_stats<kE>(v, p.pre, real_e, inv_c, p.eps, sum, &mean, &k);
#pragma unroll
            for (int b = 0; b < B; ++b) {
                float w[8], sc[8], sh[8];
                Part::weight(p.pre_weight, p.param_f32, p.offset, t.lane, t.size, C, b, w);
                Part::param(p.scale, g * p.ldsc, p.param_f32, 0.0f, t.lane, t.size, C, b, sc);
                Part::param(p.shift, g * p.ldsh, p.param_f32, 0.0f, t.lane, t.size, C, b, sh);
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = (v[8 * b + i] - mean) * k * w[i] * (1.0f + sc[i]) + sh[i];
                Part::put(p.n, row * p.ldn, t.lane, t.size, C, b, w);
            }
        }
    }
}

// ---- any row ------------------------------------------------------------------------------

// A row longer than a block's registers is read again for each of its sums, from
// L2 mostly: bf16 1000 x 20000 with two RMS norms 238 us, 670 GB/s of the bytes that
// have to move.

__global__ void __launch_bounds__(kGeneralThreads) block_norm_any_kernel(const __grid_constant__ NormParams p) {
    __shared__ float red[2 * 2 * 32];
    Sums<0> sum{red, 0};
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

// ---- many rows ----------------------------------------------------------------------------

// kLayer: one of the norms is a layer norm. Bound by memory: 16384 x 2048 bf16 with
// y, gate and modulation 47 us, 5,700 GB/s (84 % of a copy's rate); five blocks of
// 128 threads an SM, two to four rows each on the way.
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
    int lost = -1;   // the first row whose wait ran out
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
        if (!mbar_wait(ring.bars + 8u * uint32_t(s), phase, dead, &g_norm_wait_timeouts) && lost < 0) lost = int(row - lo);
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
    if (tid == 0 && dead)
        drain([&](int i) { return ring.bars + 8u * uint32_t(i); }, lost, p.stages, &g_norm_wait_timeouts);
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
    // as the kernels have them, in fp32: not infinite there, nor an eps turned to zero
    if (!std::isfinite(float(a.eps)) || a.eps < 0.0 || (a.eps > 0.0 && float(a.eps) == 0.0f) ||
        !std::isfinite(float(a.residual_scale)) || !std::isfinite(float(a.weight_offset)))
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

// Elements of a thread, threads of a block, team (8 or 32 lanes, a fixed block, 0:
// the block). elems 0: the general kernels.
struct Team {
    int elems, threads, team;
};

// Single elements: fp32 8000 x 1790 takes 53 us of the general kernel's 145, 8000 x
// 4001 113 of 265; bf16 8 x 4001 4.5 of 20, 1216 x 8003 34 of 75, 9728 x 4001 134 of
// 316; fp16 4864 x 4001 without y 41 of 96.
Team forward_team(int64_t c, bool vec) {
    if (c <= 64) return Team{8, 128, 8};
    if (c <= 256) return Team{8, 128, 32};
    if (c <= 512) return Team{16, 128, 32};
    if (!vec) {
        for (int t : {128, 256, 512})
            if (c <= 16 * t) return Team{16, t, t};
        return c <= 32 * 512 ? Team{32, 512, 512} : Team{0, 0, 0};
    }
    for (int e : {16, 32})
        if (c <= 512 * e) return Team{e, int(up((c + e - 1) / e, 32)), 0};
    return Team{0, 0, 0};
}

// The backward pass holds three column sums of each element too. Single elements:
// 8000 rows of 4001 channels: fp32 189 us of the general kernels' 892, bf16 193.
Team backward_team(int64_t c, bool vec) {
    if (c <= 64) return Team{8, 128, 8};
    if (c <= 256) return Team{8, 128, 32};
    if (!vec) {
        for (int t : {128, 256, 512})
            if (c <= 8 * t) return Team{8, t, t};
        return c <= 16 * 512 ? Team{16, 512, 512} : Team{0, 0, 0};
    }
    if (c <= 512) return Team{16, 128, 32};
    for (int e : {8, 16})
        if (c <= 512 * e) return Team{e, int(up((c + e - 1) / e, 32)), 0};
    return Team{0, 0, 0};
}

template <int kT>
NormFn team_fn(const Team &t, bool vec) {
    if (vec) {
        if (t.team == 8) return block_norm_team_kernel<kT, true, 8, 8>;
        if (t.team == 32) return t.elems == 8 ? block_norm_team_kernel<kT, true, 8, 32> : block_norm_team_kernel<kT, true, 16, 32>;
        return t.elems == 16 ? block_norm_team_kernel<kT, true, 16, 0> : block_norm_team_kernel<kT, true, 32, 0>;
    }
    switch (t.team) {
        case 8: return block_norm_team_kernel<kT, false, 8, 8>;
        case 32: return t.elems == 8 ? block_norm_team_kernel<kT, false, 8, 32> : block_norm_team_kernel<kT, false, 16, 32>;
        case 128: return block_norm_team_kernel<kT, false, 16, 128>;
        case 256: return block_norm_team_kernel<kT, false, 16, 256>;
        default: return t.elems == 16 ? block_norm_team_kernel<kT, false, 16, 512> : block_norm_team_kernel<kT, false, 32, 512>;
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

// Narrower rows leave most of a ring block's warp idle: teams of lanes take them.
constexpr int64_t kRingChannels = 384;

template <typename Fn>
int launch_ring(Fn fn, unsigned grid, const RingShape &shape, NormParams &p, cudaStream_t st) {
    p.stages = shape.stages;
    if (shape.smem > 40 * 1024 &&
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
    const bool vec = vectors(all, 9, C, 16 / es);
    const Team t = forward_team(C, vec);
    if (t.elems == 0) {
        t_norm_kernel = 2;
        return launch(block_norm_any_kernel, dim3(unsigned(std::min<int64_t>(R, int64_t(sms) * 8))),
                      dim3(kGeneralThreads), 0, p, st);
    }
    const RingShape shape = ring_shape(C, es, a->y ? 2 : 1, 3, 768);   // 80 registers a thread
    if (vec && C >= kRingChannels && shape.stages && R >= int64_t(kSms) * shape.per_sm * 2) {
        t_norm_kernel = 3;
        const bool layer = p.post == ROPE3D_NORM_LAYER || p.pre == ROPE3D_NORM_LAYER, full = C == shape.threads * kRingE;
        const NormFn fn = a->dtype == ROPE3D_BF16 ? ring_fn<ROPE3D_BF16>(layer, full)
                          : a->dtype == ROPE3D_F16 ? ring_fn<ROPE3D_F16>(layer, full)
                                                   : ring_fn<ROPE3D_F32>(layer, full);
        return launch_ring(fn, unsigned(sms * shape.per_sm), shape, p, st);
    }
    t_norm_kernel = 1;
    const NormFn fn = a->dtype == ROPE3D_BF16 ? team_fn<ROPE3D_BF16>(t, vec)
                      : a->dtype == ROPE3D_F16 ? team_fn<ROPE3D_F16>(t, vec)
                                               : team_fn<ROPE3D_F32>(t, vec);
    const int64_t teams = is_block(t.team) ? 1 : t.threads / t.team, need = (R + teams - 1) / teams;
    return launch(fn, dim3(unsigned(std::min<int64_t>(need, int64_t(sms) * (2048 / t.threads)))), dim3(t.threads), 0, p, st);
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
    const int es = f.dtype == ROPE3D_F32 ? 4 : 2, ps = f.param_dtype == ROPE3D_F32 ? 4 : 2;
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
    const bool vec = vectors(all, 16, C, 16 / es);
    const Team t = backward_team(C, vec);
    const int streams = 1 + (f.y != nullptr) + (a->dn != nullptr) + (a->dr != nullptr);
    RingShape shape = ring_shape(C, es, streams, 2, 512);   // 128 registers a thread
    bool ring = vec && C >= kRingChannels && shape.stages && R >= kSms * shape.per_sm * 2;
    // Chunks: about as many as the GPU runs teams at once (or the general
    // kernel's column blocks), each of whole groups or a part of one.
    const int64_t target =
        ring     ? kSms * shape.per_sm
        : t.elems ? kSms * (!is_block(t.team) ? 6 : t.threads > 256 ? 2 : t.threads > 128 ? 4 : 8)
                  : std::max<int64_t>(1, kSms * 8 / ((C + kGeneralThreads - 1) / kGeneralThreads));
    // Rows in registers: four rows at least for each of a block's teams, and for a team
    // of a block as many up to four as leave one chunk an SM: fewer partial sums to
    // add. (bf16, two RMS norms, rows a chunk: 600 x 4096 1 or 2: 32.7 us, 4: 23.9,
    // 6: 25.0; 1000 x 2048 36.5, 25.3, 28.7; 300 x 2048 1: 22.1, 2: 20.5; 128 x 4096
    // 1: 17.2, 2: 18.1.)
    const int64_t least = ring || !t.elems      ? 1
                          : !is_block(t.team) ? 4 * t.threads / t.team
                                              : std::min<int64_t>(4, (R + kSms - 1) / kSms);
    const int64_t L = std::max<int64_t>(least, (R + target - 1) / target), rpg = p.rows_per_group;
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
    const int64_t stat_bytes = ring || t.elems || !p.sums ? 0 : up(R * 8 * 4, 256);
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
        const NormFn fn = back_ring_fn(f.dtype, layer, full, p.d_shift != nullptr);
        rc = launch_ring(fn, unsigned(p.chunks), shape, p, st);
        if (rc != ROPE3D_OK) return rc;
    } else if (t.elems) {
        t_norm_kernel = 1;
        const NormFn fn = back_team_fn(f.dtype, vec, t.elems, t.team);
        // the teams' sums, or the weights' where a chunk is whole groups
        const size_t smem = p.sums && (p.groups_per_chunk || !is_block(t.team)) ? size_t(3) * t.elems * t.threads * 4 : 0;
        if (smem > 40 * 1024 &&   // (with the kernel's own, past the default limit of 48 KB)
            cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 100 * 1024) != cudaSuccess) {
            cudaGetLastError();
            return ROPE3D_ERR_CUDA;
        }
        rc = launch(fn, dim3(unsigned(p.chunks)), dim3(t.threads), smem, p, st);
        if (rc != ROPE3D_OK) return rc;
    } else {
        t_norm_kernel = 2;
        p.stats = p.sums ? reinterpret_cast<float *>(ws + part_bytes) : nullptr;
        rc = launch(back_any_fn(), dim3(unsigned(std::min<int64_t>(R, kSms * 8))), dim3(kGeneralThreads), 0, p, st);
        if (rc != ROPE3D_OK) return rc;
        if (p.sums) {
            rc = launch(back_cols_fn(),
                        dim3(unsigned((C + kGeneralThreads - 1) / kGeneralThreads), unsigned(std::min(p.chunks, 65535))),
                        dim3(kGeneralThreads), 0, p, st);
            if (rc != ROPE3D_OK) return rc;
        }
    }
    if (!partial) return ROPE3D_OK;
    // in split mode the groups are at most the chunks' target: far below 65535
    const int per = p.groups_per_chunk ? p.chunks : p.chunks_per_group;
    // measured with the whole backward pass: 2223 chunks of one group (20000 x 512 bf16)
    // 43 us at 16 rows, 38 at 32; 147 of each of 4 (8192 x 2048 fp16) 49 at 16
    const int rows = per <= 64 ? 8 : per <= 512 ? 16 : 32;
    rc = launch(finish_fn(rows), dim3(unsigned((C + 31) / 32), unsigned(p.groups_per_chunk ? 1 : G)), dim3(32 * rows), 0, p, st);
    if (rc != ROPE3D_OK || !by_group) return rc;
    return launch(groups_fn(), dim3(unsigned((C + 127) / 128)), dim3(128), 0, p, st);
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
    unsigned int n = 0, back = 0;
    const unsigned int zero = 0;
    if (cudaMemcpyFromSymbol(&n, g_norm_wait_timeouts, sizeof(n)) != cudaSuccess ||
        (reset && cudaMemcpyToSymbol(g_norm_wait_timeouts, &zero, sizeof(zero)) != cudaSuccess) ||
        back_wait_timeouts(&back, reset != 0) != 0) {
        cudaGetLastError();
        return ROPE3D_ERR_CUDA;
    }
    *count = int64_t(n) + back;
    return ROPE3D_OK;
}
