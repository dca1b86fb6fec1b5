// rope3d_norm_back.cu -- the backward kernels of the norms around a transformer
// block (the mathematics and the division of the work: rope3d_norm.cu).
#include "rope3d_norm.cuh"

namespace rope3d_norm {
namespace {

// ---- rows in registers -----------------------------------------------------------------

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

// Bound by latency (three sums a row, one after the other) and, at 16 elements, by
// spilled registers: 8000 x 4001 189 us in fp32 (4,070 GB/s), 193 in bf16; 20000 x
// 256 bf16, warps, 31 us with the finish (2,000 GB/s).
template <int kT, bool kVec, int kE, int kTeam>
__global__ void __launch_bounds__(kTeam > 32 ? kTeam : kTeam ? 128 : 512)
block_norm_back_team_kernel(const __grid_constant__ NormParams p) {
    using Part = RowPart<kT, kVec, kE>;
    constexpr int W = Part::W, B = kE / 8;
    __shared__ float red[2 * 2 * 32];
    extern __shared__ float kept[];   // [3][kE][threads]: the teams' sums, or (whole groups) the weights' in 0 and 2
    Sums<kTeam> sum{red, 0};
    const TeamOf<kTeam> t;
    const int C = p.channels;
    const float inv_c = 1.0f / float(C);
    auto real_e = [&](int i) { return Part::chan(t.lane, t.size, i / W) < C; };
    const bool whole = p.groups_per_chunk != 0;
    grid_wait();
    grid_release();
    const int chunk = int(blockIdx.x);
    long long lo, hi;
    chunk_range(p, chunk, &lo, &hi);
    float S[kE], T[kE], U[kE];
#pragma unroll
    for (int i = 0; i < kE; ++i) S[i] = T[i] = U[i] = 0.0f;
    if (whole && p.sums) {
#pragma unroll
        for (int i = 0; i < kE; ++i) kept[i * blockDim.x + threadIdx.x] = kept[(2 * kE + i) * blockDim.x + threadIdx.x] = 0.0f;
    }
    // one span: the team's rows of the chunk; whole groups: a span a group
    for (int span = whole ? t.team : 0; span < (whole ? p.groups_per_chunk : 1); span += t.teams) {
        const long long first = whole ? lo + (long long)span * p.rows_per_group : lo + t.team;
        const long long end = whole ? min(hi, first + p.rows_per_group) : hi;
        if (first >= end) break;
        const int step = whole ? 1 : t.teams;
        const int g = int(uint32_t(first) / uint32_t(p.rows_per_group));
        // the group's m = gate * wp and q = wq * (1 + scale); zero for absent channels
        float m[kE], q[kE];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            float f[8];
            Part::weight(p.post_weight, p.param_f32, p.offset, t.lane, t.size, C, b, m + 8 * b);
            Part::param(p.gate, g * p.ldg, p.param_f32, 1.0f, t.lane, t.size, C, b, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) m[8 * b + i] = real_e(8 * b + i) ? m[8 * b + i] * f[i] : 0.0f;
            Part::weight(p.pre_weight, p.param_f32, p.offset, t.lane, t.size, C, b, q + 8 * b);
            Part::param(p.scale, g * p.ldsc, p.param_f32, 0.0f, t.lane, t.size, C, b, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) q[8 * b + i] = real_e(8 * b + i) ? q[8 * b + i] * (1.0f + f[i]) : 0.0f;
        }
        for (long long row = first; row < end; row += step) {
            Part xv, yv, rv, nv;
            if (p.y) yv.load(p.y, row * p.ldy, t.lane, t.size, C);
            xv.load(p.x, row * p.ldx, t.lane, t.size, C);
            nv.load(p.dn, row * p.lddn, t.lane, t.size, C);
            rv.load(p.dr, row * p.lddr, t.lane, t.size, C);
            float my = 0.0f, ky = 1.0f;
            if (p.y) {
                float y[kE];
#pragma unroll
                for (int b = 0; b < B; ++b) yv.get(b, y + 8 * b);
                row_stats<kE>(y, p.post, real_e, inv_c, p.eps, sum, &my, &ky);
            }
            // r, and e = dn q
            float r[kE], e[kE];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                float *rb = r + 8 * b, *eb = e + 8 * b;
                xv.get(b, rb);
                nv.get(b, eb);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    rb[i] *= p.res;
                    eb[i] *= q[8 * b + i];
                }
                if (p.y) {
                    float y[8];
                    yv.get(b, y);
#pragma unroll
                    for (int i = 0; i < 8; ++i) rb[i] += m[8 * b + i] * ((y[i] - my) * ky);
                }
            }
            float mr = 0.0f, kr = 1.0f, me = 0.0f, mez = 0.0f;
            if (p.pre != ROPE3D_NORM_NONE) {
                if (p.pre == ROPE3D_NORM_LAYER) {
                    float s[2] = {0.0f, 0.0f};
#pragma unroll
                    for (int i = 0; i < kE; ++i) {
                        s[0] += r[i];
                        s[1] += e[i];
                    }
                    sum(s);
                    mr = s[0] * inv_c;
                    me = s[1] * inv_c;
                }
                float s[2] = {0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < kE; ++i) {
                    const float d = real_e(i) ? r[i] - mr : 0.0f;
                    s[0] += d * d;
                    s[1] += d * e[i];
                }
                sum(s);
                kr = rsqrtf(s[0] * inv_c + p.eps);
                mez = s[1] * inv_c * kr;
            }
            // the whole gradient of r, in e; the sums of n's parameters
#pragma unroll
            for (int b = 0; b < B; ++b) {
                float dr[8], dn[8];
                rv.get(b, dr);
                nv.get(b, dn);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int x = 8 * b + i;
                    const float z = (r[x] - mr) * kr;
                    S[x] += dn[i] * z;
                    T[x] += dn[i];
                    e[x] = p.pre == ROPE3D_NORM_NONE ? dr[i] + e[x] : dr[i] + kr * (e[x] - me - z * mez);
                    dr[i] = p.res * e[x];
                }
                Part::put(p.dx, row * p.lddx, t.lane, t.size, C, b, dr);
            }
            if (p.y) {
                // f, in r (m is zero for absent channels)
                float s[2] = {0.0f, 0.0f};
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    float y[8];
                    yv.get(b, y);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int x = 8 * b + i;
                        const float yh = (y[i] - my) * ky;
                        U[x] += e[x] * yh;
                        r[x] = e[x] * m[x];
                        s[0] += r[x];
                        s[1] += r[x] * yh;
                    }
                }
                float mf = 0.0f, mfy = 0.0f;
                if (p.post != ROPE3D_NORM_NONE) {
                    sum(s);
                    mf = p.post == ROPE3D_NORM_LAYER ? s[0] * inv_c : 0.0f;
                    mfy = s[1] * inv_c;
                }
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    float y[8];
                    yv.get(b, y);
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = ky * (r[8 * b + i] - mf - (y[i] - my) * ky * mfy);
                    Part::put(p.dy, row * p.lddy, t.lane, t.size, C, b, y);
                }
            }
        }
        if (whole && p.sums) {
            // a whole group is done: its gradients, and its part of the weights'
#pragma unroll
            for (int b = 0; b < B; ++b) {
                float w[8], o[8];
                if (p.d_scale) {
                    Part::weight(p.pre_weight, p.param_f32, p.offset, t.lane, t.size, C, b, w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = w[i] * S[8 * b + i];
                    Part::put_param(p.d_scale, g * p.ldgrad, p.param_f32, t.lane, t.size, C, b, o);
                }
                if (p.d_shift) Part::put_param(p.d_shift, g * p.ldgrad, p.param_f32, t.lane, t.size, C, b, T + 8 * b);
                if (p.d_gate) {
                    Part::weight(p.post_weight, p.param_f32, p.offset, t.lane, t.size, C, b, w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = w[i] * U[8 * b + i];
                    Part::put_param(p.d_gate, g * p.ldgrad, p.param_f32, t.lane, t.size, C, b, o);
                }
                Part::param(p.scale, g * p.ldsc, p.param_f32, 0.0f, t.lane, t.size, C, b, w);
                Part::param(p.gate, g * p.ldg, p.param_f32, 1.0f, t.lane, t.size, C, b, o);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int x = 8 * b + i;
                    kept[x * blockDim.x + threadIdx.x] += (1.0f + w[i]) * S[x];
                    kept[(2 * kE + x) * blockDim.x + threadIdx.x] += o[i] * U[x];
                    S[x] = T[x] = U[x] = 0.0f;
                }
            }
        }
    }
    if (!p.part) return;
    float *dst = p.part + (long long)chunk * 3 * p.channels;
    if (!whole && is_block(kTeam)) {
        // one team: straight from the registers
#pragma unroll
        for (int i = 0; i < kE; ++i) {
            if (!real_e(i)) continue;
            const int c = Part::chan(t.lane, t.size, i / W) + i % W;
            dst[c] = S[i];
            dst[p.channels + c] = T[i];
            dst[2ll * p.channels + c] = U[i];
        }
        return;
    }
    if (!whole) {
#pragma unroll
        for (int i = 0; i < kE; ++i) {
            kept[i * blockDim.x + threadIdx.x] = S[i];
            kept[(kE + i) * blockDim.x + threadIdx.x] = T[i];
            kept[(2 * kE + i) * blockDim.x + threadIdx.x] = U[i];
        }
    }
    __syncthreads();
    // the teams' sums in order
    for (int q = int(threadIdx.x); q < 3 * kE * t.size; q += int(blockDim.x)) {
        const int lane = q % t.size, ki = q / t.size, k = ki / kE, i = ki % kE;
        const int c = (lane + i / W * t.size) * W + i % W;
        if (c >= p.channels || (whole && k == 1)) continue;
        float v = 0.0f;
        for (int team = 0; team < t.teams; ++team) v += kept[ki * int(blockDim.x) + team * t.size + lane];
        dst[(long long)k * p.channels + c] = v;
    }
}

// ---- many rows ----------------------------------------------------------------------------

// kShift: d_shift is wanted (its sums are one more array of registers). Bound by
// memory at one group: 16384 x 4096 bf16 135 us, 5,960 GB/s, 142 us with the finish;
// 8192 x 2048 fp16 with a layer norm and four groups' modulation 50 us, 4,000 GB/s of
// the bytes that have to move: its 588 chunks of 14 rows leave 14.4 MB of partial sums,
// written and read again, and a row's two sums (of two values each) and barrier come
// in turn.
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
    int lost = -1;   // the first row whose wait ran out
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
        if (!mbar_wait(ring.bars + 8u * uint32_t(s), phase, dead, &g_norm_wait_timeouts) && lost < 0) lost = int(row - lo);
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
    if (tid == 0 && dead)
        drain([&](int i) { return ring.bars + 8u * uint32_t(i); }, lost, p.stages, &g_norm_wait_timeouts);
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
// (bf16 1000 x 20000 with two RMS norms: 717 us, 330 GB/s of the bytes that have to
// move: every sum reads the row again, and the columns a third time.)

__global__ void __launch_bounds__(kGeneralThreads) block_norm_back_any_kernel(const __grid_constant__ NormParams p) {
    __shared__ float red[2 * 2 * 32];
    Sums<0> sum{red, 0};
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
// chunks, 32 channels a block: n rows of threads each add every n-th chunk, then the
// rows' sums in order. Few chunks: all of a thread's in flight, of all three sums;
// many: 16 of one sum in flight (2223 chunks of 20000 x 512 bf16: 38 us with the
// rows' kernel, 49 with eight of each sum). Where several
// groups make up the weights' gradients, their parts go to p.group_sums,
// [groups][2][channels], and block_norm_groups_kernel adds them. 304 chunks of 4096
// channels, 10 MB, take 7 us: the latency of two rounds of loads and of the launch.
template <int n>
__global__ void __launch_bounds__(32 * n) block_norm_finish_kernel(const __grid_constant__ NormParams p) {
    __shared__ float part[3][n][32], param[4][32];
    grid_wait();
    grid_release();
    const int lane = threadIdx.x & 31, ty = threadIdx.x >> 5, g = int(blockIdx.y);
    const int c = int(blockIdx.x) * 32 + lane;
    const int param_type = p.param_f32 ? ROPE3D_F32 : p.dtype;
    const int per = p.groups_per_chunk ? p.chunks : p.chunks_per_group;
    // which of the three sums are needed: chunks of whole groups have written their
    // groups' gradients and left the weights' sums alone
    const bool split = !p.groups_per_chunk;
    const bool want[3] = {p.d_pre_weight || (split && p.d_scale), split && p.d_shift, p.d_post_weight || (split && p.d_gate)};
    float s[3] = {0.0f, 0.0f, 0.0f};
    if (c < p.channels) {
        if (ty < 4 && !p.groups_per_chunk) {   // a group's parameters, one a warp
            const RowOps og{p, 0, g, 0.0f, 1.0f, 0.0f, 1.0f};
            param[ty][lane] = ty == 0 ? og.scale1(c) : ty == 1 ? og.gate(c) : ty == 2 ? (p.d_scale ? og.wq(c) : 1.0f)
                                                                                      : (p.d_gate ? og.wp(c) : 1.0f);
        }
        const float *src = p.part + (long long)g * per * 3 * p.channels + c;
        const long long step = 3ll * p.channels;
        if constexpr (n < 32) {
            constexpr int kU = n == 8 ? 8 : 10;
            for (int i = ty; i < per; i += kU * n) {
                float v[3][kU];
#pragma unroll
                for (int u = 0; u < kU; ++u)
#pragma unroll
                    for (int k = 0; k < 3; ++k)
                        v[k][u] = want[k] && i + u * n < per ? __ldcs(src + (i + u * n) * step + (long long)k * p.channels) : 0.0f;
#pragma unroll
                for (int u = 0; u < kU; ++u)
#pragma unroll
                    for (int k = 0; k < 3; ++k) s[k] += v[k][u];
            }
        } else {
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                if (!want[k]) continue;
                const float *col = src + (long long)k * p.channels;
                int i = ty;
                for (; i + 15 * n < per; i += 16 * n) {
                    float v[16];
#pragma unroll
                    for (int u = 0; u < 16; ++u) v[u] = __ldcs(col + (i + u * n) * step);
#pragma unroll
                    for (int u = 0; u < 16; ++u) s[k] += v[u];
                }
#pragma unroll 4
                for (; i < per; i += n) s[k] += __ldcs(col + i * step);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) part[k][ty][lane] = s[k];
    __syncthreads();
    if (ty != 0 || c >= p.channels) return;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        s[k] = 0.0f;
        for (int i = 0; i < n; ++i) s[k] += part[k][i][lane];
    }
    float wq = s[0], wp = s[2];
    if (!p.groups_per_chunk) {
        const long long at = g * p.ldgrad + c;
        if (p.d_scale) store1(p.d_scale, at, param[2][lane] * s[0], param_type);
        if (p.d_shift) store1(p.d_shift, at, s[1], param_type);
        if (p.d_gate) store1(p.d_gate, at, param[3][lane] * s[2], param_type);
        wq *= param[0][lane];
        wp *= param[1][lane];
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

template <int kT>
NormFn team_fn(bool vec, int elems, int team) {
    if (vec) {
        if (team == 8) return block_norm_back_team_kernel<kT, true, 8, 8>;
        if (team == 32) return elems == 8 ? block_norm_back_team_kernel<kT, true, 8, 32> : block_norm_back_team_kernel<kT, true, 16, 32>;
        return elems == 8 ? block_norm_back_team_kernel<kT, true, 8, 0> : block_norm_back_team_kernel<kT, true, 16, 0>;
    }
    switch (team) {
        case 8: return block_norm_back_team_kernel<kT, false, 8, 8>;
        case 32: return block_norm_back_team_kernel<kT, false, 8, 32>;
        case 128: return block_norm_back_team_kernel<kT, false, 8, 128>;
        case 256: return block_norm_back_team_kernel<kT, false, 8, 256>;
        default: return elems == 8 ? block_norm_back_team_kernel<kT, false, 8, 512> : block_norm_back_team_kernel<kT, false, 16, 512>;
    }
}

template <int kT, bool kLayer>
NormFn ring_of(bool full, bool shift) {
    if (full)
        return shift ? block_norm_back_ring_kernel<kT, kLayer, true, true> : block_norm_back_ring_kernel<kT, kLayer, true, false>;
    return shift ? block_norm_back_ring_kernel<kT, kLayer, false, true> : block_norm_back_ring_kernel<kT, kLayer, false, false>;
}

template <int kT>
NormFn ring(bool layer, bool full, bool shift) {
    return layer ? ring_of<kT, true>(full, shift) : ring_of<kT, false>(full, shift);
}

}  // namespace

NormFn back_team_fn(int dtype, bool vec, int elems, int team) {
    return dtype == ROPE3D_BF16  ? team_fn<ROPE3D_BF16>(vec, elems, team)
           : dtype == ROPE3D_F16 ? team_fn<ROPE3D_F16>(vec, elems, team)
                                 : team_fn<ROPE3D_F32>(vec, elems, team);
}

NormFn back_ring_fn(int dtype, bool layer, bool full, bool shift) {
    return dtype == ROPE3D_BF16  ? ring<ROPE3D_BF16>(layer, full, shift)
           : dtype == ROPE3D_F16 ? ring<ROPE3D_F16>(layer, full, shift)
                                 : ring<ROPE3D_F32>(layer, full, shift);
}

NormFn back_any_fn() { return block_norm_back_any_kernel; }
NormFn back_cols_fn() { return block_norm_back_cols_kernel; }
NormFn finish_fn(int rows) { return rows == 8 ? block_norm_finish_kernel<8> : rows == 16 ? block_norm_finish_kernel<16> : block_norm_finish_kernel<32>; }
NormFn groups_fn() { return block_norm_groups_kernel; }

int back_wait_timeouts(unsigned int *count, bool reset) {
    const unsigned int zero = 0;
    cudaError_t rc = cudaMemcpyFromSymbol(count, g_norm_wait_timeouts, sizeof(*count));
    if (rc == cudaSuccess && reset) rc = cudaMemcpyToSymbol(g_norm_wait_timeouts, &zero, sizeof(zero));
    return int(rc);
}

}  // namespace rope3d_norm
