// rope3d_api.cpp -- host side of the fused paired 3D RoPE library: the C ABI,
// the axis-table builder and its FIFO cache, the preflight checks, the
// first-seen bit-exact gate, and the host-buffer pipeline.
//
// Sources (sglang PR #35698 review, "fused LTX-2.5 decoder 3D RoPE"):
//   "实现拆解" step 1  -- _axis_tables / _tables: per-axis (cos, sin) tables of
//                        shape [length, dim/2], cached in a module-level dict
//                        keyed on the grid, the split and the base, FIFO, 16 max;
//   "实现拆解" step 3  -- one launch writes Q_out and K_out; the preflight
//                        can_use_ltx25_decoder_rope ("关键源码片段");
//   "实现拆解" step 4  -- BitExactFusionGate: the first call of a configuration is
//                        compared bit for bit with the eager order, and the
//                        verdict is kept for the life of the process.
// Differences from the pages: a mismatch does not fall back to an eager path
// (there is none); the configuration is refused with ROPE3D_ERR_PARITY.
//
// Build with -ffp-contract=off: the gate's CPU rotation must round every
// product and sum on its own, like the kernel.
#include <algorithm>
#include <array>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <deque>
#include <map>
#include <memory>
#include <mutex>
#include <thread>
#include <tuple>
#include <vector>

#include <cuda_runtime.h>

#include "../../include/rope3d.h"
#include "rope3d_internal.h"

using rope3d::FastDiv;
using rope3d::LaunchArgs;
using rope3d::LaunchInfo;

// ============================================================================
// table handles and the cache
// ============================================================================

struct rope3d_tables {
    // key
    int device;
    int64_t dims[3];
    int32_t split[3];
    double base;
    // host copy, per axis: cos and sin [L_X][d_X/2]
    std::vector<float> cos_host[3];
    std::vector<float> sin_host[3];
    // device buffer: float2 (cos, sin) entries, T | H | W, each table starting
    // at a multiple of 4 entries
    float2 *dev = nullptr;
    bool host_backed = false;  // test mode: dev points to host memory
    bool pooled = false;       // dev comes from the stream-ordered allocator
    uint32_t offset[3] = {0, 0, 0};
    uint32_t len = 0;          // float2 entries including padding
    std::atomic<int64_t> refs{0};
    // Events recorded after the launches that read `dev` and have not been
    // seen complete yet (oldest first).
    std::mutex use_mutex;
    std::deque<cudaEvent_t> uses;
};

namespace {

std::mutex g_mutex;  // guards the cache, the gate map and the scratch

struct CacheState {
    std::deque<rope3d_tables *> fifo;
    int64_t hits = 0, misses = 0, evictions = 0;
    bool host_tables = false;
} g_cache;

// ---- releasing table memory in stream order --------------------------------
// A launch that reads a handle's tables records an event on its stream; when
// the handle's last reference goes, its buffer is retired and freed only once
// every one of those events has completed. Nothing waits for the device:
// retired buffers are checked (and freed) on later calls into the cache.

std::mutex g_event_mutex;                               // guards g_event_pool
std::map<int, std::vector<cudaEvent_t>> g_event_pool;   // spare events per device

cudaEvent_t take_event(int device) {
    {
        std::lock_guard<std::mutex> lock(g_event_mutex);
        std::vector<cudaEvent_t> &spare = g_event_pool[device];
        if (!spare.empty()) {
            cudaEvent_t e = spare.back();
            spare.pop_back();
            return e;
        }
    }
    cudaEvent_t e = nullptr;
    if (cudaEventCreateWithFlags(&e, cudaEventDisableTiming) != cudaSuccess) {
        cudaGetLastError();
        return nullptr;
    }
    return e;
}

void give_event(int device, cudaEvent_t e) {
    std::lock_guard<std::mutex> lock(g_event_mutex);
    g_event_pool[device].push_back(e);
}

// True once the work the event captured has finished. A failed query also
// counts as finished: the context is then unusable and nothing runs on it.
bool event_done(cudaEvent_t e) {
    const cudaError_t rc = cudaEventQuery(e);
    if (rc == cudaSuccess) return true;
    cudaGetLastError();  // clear cudaErrorNotReady (or the failure) from the thread's last error
    return rc != cudaErrorNotReady;
}

// Drop the completed events of t (all of them when `all`, else from the front
// up to the first pending one); returns whether none is left. Caller holds
// t->use_mutex.
bool prune_uses(rope3d_tables *t, bool all) {
    for (auto it = t->uses.begin(); it != t->uses.end();) {
        if (event_done(*it)) {
            give_event(t->device, *it);
            it = t->uses.erase(it);
        } else if (all) {
            ++it;
        } else {
            break;
        }
    }
    return t->uses.empty();
}

std::mutex g_retire_mutex;                 // guards g_retired and g_release_streams
std::vector<rope3d_tables *> g_retired;    // released, waiting for their last launches
std::map<int, cudaStream_t> g_release_streams;

// Free t's memory now (its launches have all completed). Caller holds
// g_retire_mutex when t is device-backed and pooled.
void free_now(rope3d_tables *t) {
    for (cudaEvent_t e : t->uses) give_event(t->device, e);
    t->uses.clear();
    if (t->dev) {
        if (t->host_backed) {
            std::free(t->dev);
        } else {
            int cur = -1;
            cudaGetDevice(&cur);
            if (cur != t->device) cudaSetDevice(t->device);
            if (t->pooled) {
                // on a stream of the library's own, so that no caller's stream
                // is ordered behind the free
                cudaStream_t &rs = g_release_streams[t->device];
                if (!rs && cudaStreamCreateWithFlags(&rs, cudaStreamNonBlocking) != cudaSuccess) {
                    rs = nullptr;
                    cudaGetLastError();
                }
                if (!rs || cudaFreeAsync(t->dev, rs) != cudaSuccess) cudaGetLastError();
            } else {
                cudaFree(t->dev);
            }
            if (cur >= 0 && cur != t->device) cudaSetDevice(cur);
        }
    }
    delete t;
}

// Free every retired buffer whose launches have completed; returns how many
// are still waiting.
int64_t drain_retired() {
    std::lock_guard<std::mutex> lock(g_retire_mutex);
    for (auto it = g_retired.begin(); it != g_retired.end();) {
        rope3d_tables *t = *it;
        bool done;
        {
            std::lock_guard<std::mutex> ul(t->use_mutex);
            done = prune_uses(t, true);
        }
        if (done) {
            free_now(t);
            it = g_retired.erase(it);
        } else {
            ++it;
        }
    }
    return static_cast<int64_t>(g_retired.size());
}

void retire(rope3d_tables *t) {
    std::lock_guard<std::mutex> lock(g_retire_mutex);
    bool done;
    {
        std::lock_guard<std::mutex> ul(t->use_mutex);
        done = t->host_backed || prune_uses(t, true);
    }
    if (done)
        free_now(t);
    else
        g_retired.push_back(t);
}

void drop_ref(rope3d_tables *t) {
    if (t->refs.fetch_sub(1) == 1) retire(t);
}

bool valid_base(double base) { return std::isfinite(base) && base > 0.0; }

int check_grid(int64_t T, int64_t H, int64_t W, const int32_t split[3]) {
    if (T <= 0 || H <= 0 || W <= 0) return ROPE3D_ERR_SHAPE;
    const int64_t lim = (int64_t(1) << 31) - 1;
    if (T > lim || H > lim || W > lim) return ROPE3D_ERR_SHAPE;
    if (T * H > lim || T * H * W > lim) return ROPE3D_ERR_SHAPE;
    int64_t sum = 0;
    for (int a = 0; a < 3; ++a) {
        if (split[a] <= 0 || (split[a] % 2) != 0) return ROPE3D_ERR_SHAPE;
        sum += split[a];
    }
    if (sum > ROPE3D_MAX_HEAD_DIM) return ROPE3D_ERR_SHAPE;
    // the table buffer is indexed with 32-bit entries
    const int64_t entries = T * (split[0] / 2) + H * (split[1] / 2) + W * (split[2] / 2) + 12;
    if (entries > lim) return ROPE3D_ERR_SHAPE;
    return ROPE3D_OK;
}

}  // namespace

// ----------------------------------------------------------------------------
// the table builder: standard per-axis RoPE angles in double, one rounding to
// float at the end (the pages give the table's shape and inputs, not its
// formula).
// ----------------------------------------------------------------------------
extern "C" int rope3d_axis_table_host(int64_t length, int64_t dim, double base,
                                      float *cos_out, float *sin_out) {
    if (!cos_out || !sin_out) return ROPE3D_ERR_NULL;
    if (length <= 0 || dim <= 0 || (dim % 2) != 0) return ROPE3D_ERR_SHAPE;
    if (!valid_base(base)) return ROPE3D_ERR_ARG;
    const int64_t half = dim / 2;
    std::vector<double> inv_freq(static_cast<size_t>(half));
    for (int64_t j = 0; j < half; ++j)
        inv_freq[j] = std::pow(base, -(2.0 * static_cast<double>(j)) / static_cast<double>(dim));
    for (int64_t p = 0; p < length; ++p) {
        const double pos = static_cast<double>(p);
        for (int64_t j = 0; j < half; ++j) {
            const double angle = pos * inv_freq[j];
            cos_out[p * half + j] = static_cast<float>(std::cos(angle));
            sin_out[p * half + j] = static_cast<float>(std::sin(angle));
        }
    }
    return ROPE3D_OK;
}

// ----------------------------------------------------------------------------
// The LTX DiT's RoPE frequency vector: n = dim / num_rope_elems exponents
// evenly spaced over [0, 1], theta to each power, times pi, halved, cast to
// float. Every step in double (double_precision) or in float; the float power
// is the double power rounded once, i.e. correctly rounded except within a
// double ulp of a float rounding boundary.
// ----------------------------------------------------------------------------
extern "C" int rope3d_dit_freqs_host(int64_t dim, int64_t num_rope_elems, double theta,
                                     int32_t double_precision, float *out) {
    if (!out) return ROPE3D_ERR_NULL;
    if (dim <= 0 || num_rope_elems <= 0 || dim / num_rope_elems == 0) return ROPE3D_ERR_SHAPE;
    if (dim / num_rope_elems > (int64_t(1) << 24)) return ROPE3D_ERR_SHAPE;
    if (!valid_base(theta)) return ROPE3D_ERR_ARG;
    const int64_t n = dim / num_rope_elems;
    const double last = static_cast<double>(n - 1);
    const double kPi = 3.14159265358979323846;
    for (int64_t i = 0; i < n; ++i) {
        // exponent i / (n - 1), rounded once in the working precision
        const double exponent = n == 1 ? 0.0 : static_cast<double>(i) / last;
        if (double_precision) {
            const double scaled = std::pow(theta, exponent) * kPi;
            out[i] = static_cast<float>(scaled / 2.0);
        } else {
            const float exponent_f = static_cast<float>(exponent);
            const float theta_f = static_cast<float>(theta);
            const float power_f = static_cast<float>(
                std::pow(static_cast<double>(theta_f), static_cast<double>(exponent_f)));
            const float scaled_f = power_f * static_cast<float>(kPi);
            out[i] = scaled_f / 2.0f;
        }
    }
    return ROPE3D_OK;
}

extern "C" int rope3d_build_tables(int64_t T, int64_t H, int64_t W, const int32_t split[3],
                                   double base, void *stream, rope3d_tables **out) {
    if (!split || !out) return ROPE3D_ERR_NULL;
    *out = nullptr;
    int rc = check_grid(T, H, W, split);
    if (rc != ROPE3D_OK) return rc;
    if (!valid_base(base)) return ROPE3D_ERR_ARG;

    drain_retired();
    int device = -1;
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!g_cache.host_tables) {
        if (cudaGetDevice(&device) != cudaSuccess) return ROPE3D_ERR_CUDA;
    }
    const int64_t dims[3] = {T, H, W};
    for (rope3d_tables *t : g_cache.fifo) {
        if (t->device == device && t->base == base &&
            std::equal(dims, dims + 3, t->dims) && std::equal(split, split + 3, t->split)) {
            ++g_cache.hits;
            t->refs.fetch_add(1);
            *out = t;
            return ROPE3D_OK;
        }
    }
    ++g_cache.misses;

    std::unique_ptr<rope3d_tables> t(new rope3d_tables());
    t->device = device;
    std::copy(dims, dims + 3, t->dims);
    std::copy(split, split + 3, t->split);
    t->base = base;
    uint32_t off = 0;
    for (int a = 0; a < 3; ++a) {
        const size_t n = static_cast<size_t>(dims[a]) * (split[a] / 2);
        t->cos_host[a].resize(n);
        t->sin_host[a].resize(n);
        rc = rope3d_axis_table_host(dims[a], split[a], base, t->cos_host[a].data(),
                                    t->sin_host[a].data());
        if (rc != ROPE3D_OK) return rc;
        t->offset[a] = off;
        off += static_cast<uint32_t>((n + 3) / 4 * 4);
    }
    t->len = off;
    std::vector<float2> packed(t->len, float2{0.f, 0.f});
    for (int a = 0; a < 3; ++a)
        for (size_t i = 0; i < t->cos_host[a].size(); ++i)
            packed[t->offset[a] + i] = float2{t->cos_host[a][i], t->sin_host[a][i]};
    const size_t bytes = packed.size() * sizeof(float2);
    if (g_cache.host_tables) {
        t->dev = static_cast<float2 *>(std::malloc(bytes));
        if (!t->dev) return ROPE3D_ERR_NOMEM;
        std::memcpy(t->dev, packed.data(), bytes);
        t->host_backed = true;
    } else {
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        // the stream-ordered allocator, so that a later free waits for no one
        if (cudaMallocAsync(reinterpret_cast<void **>(&t->dev), bytes, s) == cudaSuccess) {
            t->pooled = true;
        } else {
            cudaGetLastError();
            if (cudaMalloc(&t->dev, bytes) != cudaSuccess) {
                t->dev = nullptr;
                cudaGetLastError();
                return ROPE3D_ERR_NOMEM;
            }
        }
        if (cudaMemcpyAsync(t->dev, packed.data(), bytes, cudaMemcpyHostToDevice, s) != cudaSuccess ||
            cudaStreamSynchronize(s) != cudaSuccess) {
            std::lock_guard<std::mutex> rl(g_retire_mutex);
            free_now(t.release());
            return ROPE3D_ERR_CUDA;
        }
    }
    // insert: the cache holds one reference, the caller another
    t->refs.store(2);
    if (static_cast<int>(g_cache.fifo.size()) >= ROPE3D_TABLE_CACHE_CAP) {
        rope3d_tables *old = g_cache.fifo.front();
        g_cache.fifo.pop_front();
        ++g_cache.evictions;
        drop_ref(old);
    }
    g_cache.fifo.push_back(t.get());
    *out = t.release();
    return ROPE3D_OK;
}

extern "C" int rope3d_release_tables(rope3d_tables *tables) {
    if (!tables) return ROPE3D_ERR_NULL;
    drop_ref(tables);
    drain_retired();
    return ROPE3D_OK;
}

extern "C" int rope3d_cache_retired(int64_t *waiting) {
    const int64_t n = drain_retired();
    if (waiting) *waiting = n;
    return ROPE3D_OK;
}

// Record that a launch on `stream` reads t's tables (see retire()). Launches
// into a capturing stream are not tracked: a graph keeps using the tables'
// memory on every replay, so its owner keeps a reference for the graph's life.
int rope3d::tables_note_use(const rope3d_tables *tc, cudaStream_t stream) {
    rope3d_tables *t = const_cast<rope3d_tables *>(tc);
    if (!t) return ROPE3D_ERR_NULL;
    if (t->host_backed) return ROPE3D_OK;
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(stream, &cap) != cudaSuccess) {
        cudaGetLastError();
        return ROPE3D_ERR_CUDA;
    }
    if (cap != cudaStreamCaptureStatusNone) return ROPE3D_OK;
    std::lock_guard<std::mutex> lock(t->use_mutex);
    prune_uses(t, t->uses.size() > 64);
    cudaEvent_t e = take_event(t->device);
    if (!e) return ROPE3D_ERR_CUDA;
    if (cudaEventRecord(e, stream) != cudaSuccess) {
        cudaGetLastError();
        give_event(t->device, e);
        return ROPE3D_ERR_CUDA;
    }
    t->uses.push_back(e);
    return ROPE3D_OK;
}

extern "C" int rope3d_retain_tables(rope3d_tables *tables) {
    if (!tables) return ROPE3D_ERR_NULL;
    tables->refs.fetch_add(1);
    return ROPE3D_OK;
}

extern "C" int rope3d_tables_info(const rope3d_tables *t, int64_t dims[3], int32_t split[3],
                                  double *base) {
    if (!t) return ROPE3D_ERR_NULL;
    if (dims) std::copy(t->dims, t->dims + 3, dims);
    if (split) std::copy(t->split, t->split + 3, split);
    if (base) *base = t->base;
    return ROPE3D_OK;
}

extern "C" int rope3d_tables_read(const rope3d_tables *t, int32_t axis, int32_t from_device,
                                  float *cos_out, float *sin_out) {
    if (!t || !cos_out || !sin_out) return ROPE3D_ERR_NULL;
    if (axis < 0 || axis > 2) return ROPE3D_ERR_ARG;
    const size_t n = t->cos_host[axis].size();
    if (!from_device) {
        std::memcpy(cos_out, t->cos_host[axis].data(), n * sizeof(float));
        std::memcpy(sin_out, t->sin_host[axis].data(), n * sizeof(float));
        return ROPE3D_OK;
    }
    std::vector<float2> buf(n);
    if (t->host_backed) {
        std::memcpy(buf.data(), t->dev + t->offset[axis], n * sizeof(float2));
    } else if (cudaMemcpy(buf.data(), t->dev + t->offset[axis], n * sizeof(float2),
                          cudaMemcpyDeviceToHost) != cudaSuccess) {
        return ROPE3D_ERR_CUDA;
    }
    for (size_t i = 0; i < n; ++i) {
        cos_out[i] = buf[i].x;
        sin_out[i] = buf[i].y;
    }
    return ROPE3D_OK;
}

// The device layout of a handle, for kernels outside this file.
int rope3d::tables_layout(const rope3d_tables *t, const float2 **dev, uint32_t *len,
                          uint32_t offsets[3], int64_t dims[3], int32_t split[3], int *device,
                          bool *host_backed) {
    if (!t) return ROPE3D_ERR_NULL;
    *dev = t->dev;
    *len = t->len;
    std::copy(t->offset, t->offset + 3, offsets);
    std::copy(t->dims, t->dims + 3, dims);
    std::copy(t->split, t->split + 3, split);
    *device = t->device;
    *host_backed = t->host_backed;
    return ROPE3D_OK;
}

extern "C" int rope3d_cache_stats(int64_t *entries, int64_t *hits, int64_t *misses,
                                  int64_t *evictions) {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (entries) *entries = static_cast<int64_t>(g_cache.fifo.size());
    if (hits) *hits = g_cache.hits;
    if (misses) *misses = g_cache.misses;
    if (evictions) *evictions = g_cache.evictions;
    return ROPE3D_OK;
}

extern "C" int rope3d_cache_clear(void) {
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        while (!g_cache.fifo.empty()) {
            rope3d_tables *t = g_cache.fifo.front();
            g_cache.fifo.pop_front();
            drop_ref(t);
        }
        g_cache.hits = g_cache.misses = g_cache.evictions = 0;
    }
    drain_retired();
    rope3d::na3d_scratch_trim();
    return ROPE3D_OK;
}

extern "C" int rope3d_testing_host_tables(int32_t on) {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!g_cache.fifo.empty()) return ROPE3D_ERR_ARG;
    g_cache.host_tables = on != 0;
    return ROPE3D_OK;
}

// ============================================================================
// geometry and preflight
// ============================================================================

namespace {

struct Geom {
    int64_t B, T, H, W, heads, head_dim;
    int32_t split[3];
    int32_t dtype;
    int64_t esize;
    int64_t rows() const { return B * T * H * W; }
    int64_t row_elems() const { return heads * head_dim; }
    int64_t numel() const { return rows() * row_elems(); }
    int64_t bytes() const { return numel() * esize; }
};

int check_geom(const Geom &g) {
    if (g.dtype != ROPE3D_BF16 && g.dtype != ROPE3D_F32 && g.dtype != ROPE3D_F16)
        return ROPE3D_ERR_DTYPE;
    if (g.B <= 0 || g.heads <= 0 || g.head_dim <= 0) return ROPE3D_ERR_SHAPE;
    int rc = check_grid(g.T, g.H, g.W, g.split);
    if (rc != ROPE3D_OK) return rc;
    if (g.head_dim > ROPE3D_MAX_HEAD_DIM) return ROPE3D_ERR_SHAPE;
    if (int64_t(g.split[0]) + g.split[1] + g.split[2] != g.head_dim) return ROPE3D_ERR_SHAPE;
    if (g.heads > 65536 || g.B > (int64_t(1) << 31) - 1) return ROPE3D_ERR_SHAPE;
    // every byte offset, for all four buffers together, must fit in 62 bits
    const double total = double(g.B) * double(g.T) * double(g.H) * double(g.W) *
                         double(g.heads) * double(g.head_dim) * double(g.esize);
    if (total > 1.0e18) return ROPE3D_ERR_SHAPE;
    return ROPE3D_OK;
}

bool overlaps(const void *a, const void *b, int64_t bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a);
    const uintptr_t y = reinterpret_cast<uintptr_t>(b);
    return x < y + static_cast<uintptr_t>(bytes) && y < x + static_cast<uintptr_t>(bytes);
}

int check_pointers(const void *q, const void *k, const void *qo, const void *ko, int64_t bytes) {
    if (!q || !k || !qo || !ko) return ROPE3D_ERR_NULL;
    for (const void *p : {q, k, qo, ko})
        if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return ROPE3D_ERR_ALIGN;
    if (overlaps(qo, q, bytes) || overlaps(qo, k, bytes) || overlaps(ko, q, bytes) ||
        overlaps(ko, k, bytes) || overlaps(qo, ko, bytes))
        return ROPE3D_ERR_ALIAS;
    return ROPE3D_OK;
}

int check_tables(const rope3d_tables *t, const Geom &g) {
    if (!t) return ROPE3D_ERR_NULL;
    const int64_t dims[3] = {g.T, g.H, g.W};
    if (!std::equal(dims, dims + 3, t->dims) || !std::equal(g.split, g.split + 3, t->split))
        return ROPE3D_ERR_TABLES;
    return ROPE3D_OK;
}

// Device memory of the current device (or managed memory)?
bool is_device_ptr(const void *p, int device) {
    cudaPointerAttributes attr{};
    if (cudaPointerGetAttributes(&attr, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    if (attr.type == cudaMemoryTypeManaged) return true;
    return attr.type == cudaMemoryTypeDevice && attr.device == device;
}

bool is_host_ptr(const void *p) {
    cudaPointerAttributes attr{};
    if (cudaPointerGetAttributes(&attr, p) != cudaSuccess) {
        cudaGetLastError();
        return true;  // unknown to CUDA: plain pageable host memory
    }
    return attr.type == cudaMemoryTypeHost || attr.type == cudaMemoryTypeUnregistered;
}

Geom make_geom(int64_t B, int64_t T, int64_t H, int64_t W, int64_t heads, int64_t head_dim,
               const int32_t split[3], int32_t dtype) {
    Geom g{B, T, H, W, heads, head_dim, {0, 0, 0}, dtype, dtype == ROPE3D_F32 ? 4 : 2};
    if (split) std::copy(split, split + 3, g.split);
    return g;
}

int preflight(const void *q, const void *k, const void *qo, const void *ko,
              const rope3d_tables *tables, const Geom &g, const int32_t split[3]) {
    if (!split) return ROPE3D_ERR_NULL;
    int rc = check_geom(g);
    if (rc != ROPE3D_OK) return rc;
    rc = check_pointers(q, k, qo, ko, g.bytes());
    if (rc != ROPE3D_OK) return rc;
    return check_tables(tables, g);
}

}  // namespace

extern "C" int rope3d_preflight(const void *q, const void *k, const void *q_out,
                                const void *k_out, const rope3d_tables *tables, int64_t B,
                                int64_t T, int64_t H, int64_t W, int64_t heads,
                                int64_t head_dim, const int32_t split[3], int32_t dtype,
                                int32_t check_device) {
    const Geom g = make_geom(B, T, H, W, heads, head_dim, split, dtype);
    int rc = preflight(q, k, q_out, k_out, tables, g, split);
    if (rc != ROPE3D_OK || !check_device) return rc;
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return ROPE3D_ERR_CUDA;
    if (tables->host_backed || tables->device != device) return ROPE3D_ERR_DEVICE;
    for (const void *p : {q, k, q_out, k_out})
        if (!is_device_ptr(p, device)) return ROPE3D_ERR_DEVICE;
    return ROPE3D_OK;
}

// Checks of an entry point that takes no table handle: everything
// rope3d_preflight checks except the tables, plus the device query. Allocates
// nothing.
int rope3d::check_call_without_tables(const void *q, const void *k, const void *q_out,
                                      const void *k_out, int64_t B, int64_t T, int64_t H,
                                      int64_t W, int64_t heads, int64_t head_dim,
                                      const int32_t split[3], int32_t dtype) {
    if (!split) return ROPE3D_ERR_NULL;
    const Geom g = make_geom(B, T, H, W, heads, head_dim, split, dtype);
    int rc = check_geom(g);
    if (rc != ROPE3D_OK) return rc;
    rc = check_pointers(q, k, q_out, k_out, g.bytes());
    if (rc != ROPE3D_OK) return rc;
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return ROPE3D_ERR_CUDA;
    for (const void *p : {q, k, q_out, k_out})
        if (!is_device_ptr(p, device)) return ROPE3D_ERR_DEVICE;
    return ROPE3D_OK;
}

// ============================================================================
// the gate: CPU eager order, compared element by element
// ============================================================================

namespace {

using GateKey = std::tuple<int, int32_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t,
                           int32_t, int32_t, int32_t, double>;

std::map<GateKey, int> g_verdicts;  // 1 verified, 2 refused
std::atomic<int> g_gate_mode{ROPE3D_GATE_FIRST};
std::atomic<int> g_corrupt{0};

GateKey gate_key(int device, const Geom &g, double base) {
    return GateKey{device, g.dtype, g.B, g.T, g.H, g.W, g.heads, g.head_dim,
                   g.split[0], g.split[1], g.split[2], base};
}

// bf16 <-> float for the gate, from the formats' layouts.
inline float widen_bf16(uint16_t v) {
    const uint32_t u = static_cast<uint32_t>(v) << 16;
    float f;
    std::memcpy(&f, &u, 4);
    return f;
}

inline uint16_t narrow_bf16(float f) {
    uint32_t u;
    std::memcpy(&u, &f, 4);
    const uint32_t exp_bits = u & 0x7f800000u;
    const uint32_t frac = u & 0x007fffffu;
    if (exp_bits == 0x7f800000u && frac != 0) return static_cast<uint16_t>((u >> 16) | 0x40u);
    uint32_t upper = u >> 16;
    const uint32_t lower = u & 0xffffu;
    // nearest; on an exact half, the even neighbour
    if (lower > 0x8000u || (lower == 0x8000u && (upper & 1u))) upper += 1;
    return static_cast<uint16_t>(upper);
}

// binary16 <-> float for the gate, from the format's layout (5 exponent bits
// biased by 15, 10 fraction bits, subnormals fraction * 2^-24).
inline float widen_f16(uint16_t h) {
    const uint32_t sign = static_cast<uint32_t>(h & 0x8000u) << 16;
    const uint32_t e = (h >> 10) & 0x1fu;
    const uint32_t m = h & 0x3ffu;
    uint32_t bits;
    if (e == 0x1fu) {
        bits = sign | 0x7f800000u | (m << 13);
    } else if (e != 0) {
        bits = sign | ((e + 112u) << 23) | (m << 13);
    } else if (m == 0) {
        bits = sign;
    } else {
        // subnormal: normalise the fraction
        uint32_t mm = m;
        uint32_t shift = 0;
        while (!(mm & 0x400u)) {
            mm <<= 1;
            ++shift;
        }
        bits = sign | ((113u - shift) << 23) | ((mm & 0x3ffu) << 13);
    }
    float f;
    std::memcpy(&f, &bits, 4);
    return f;
}

inline uint16_t narrow_f16(float f) {
    uint32_t u;
    std::memcpy(&u, &f, 4);
    const uint32_t sign = (u >> 16) & 0x8000u;
    const int32_t exp = static_cast<int32_t>((u >> 23) & 0xffu);
    const uint32_t mant = u & 0x7fffffu;
    if (exp == 0xff) return static_cast<uint16_t>(sign | 0x7c00u | (mant ? 0x200u | (mant >> 13) : 0u));
    if (exp == 0) return static_cast<uint16_t>(sign);  // far below the smallest binary16
    const int32_t e16 = exp - 112;                     // binary16 biased exponent
    const uint32_t sig = mant | 0x800000u;             // 24-bit significand
    const int32_t shift = e16 >= 1 ? 13 : 14 - e16;    // bits dropped from sig
    if (shift >= 25) return static_cast<uint16_t>(sign);  // below half the smallest subnormal
    uint32_t kept = sig >> shift;
    const uint32_t dropped = sig & ((1u << shift) - 1u);
    const uint32_t halfway = 1u << (shift - 1);
    if (dropped > halfway || (dropped == halfway && (kept & 1u))) ++kept;
    const uint32_t result = e16 >= 1 ? (static_cast<uint32_t>(e16) << 10) + (kept - 0x400u) : kept;
    if (result >= 0x7c00u) return static_cast<uint16_t>(sign | 0x7c00u);
    return static_cast<uint16_t>(sign | result);
}

inline bool same_or_both_nan_f16(uint16_t a, uint16_t b) {
    if (a == b) return true;
    return (a & 0x7fffu) > 0x7c00u && (b & 0x7fffu) > 0x7c00u;
}

inline bool same_or_both_nan_f32(uint32_t a, uint32_t b) {
    if (a == b) return true;
    return (a & 0x7fffffffu) > 0x7f800000u && (b & 0x7fffffffu) > 0x7f800000u;
}

inline bool same_or_both_nan_bf16(uint16_t a, uint16_t b) {
    if (a == b) return true;
    return (a & 0x7fffu) > 0x7f80u && (b & 0x7fffu) > 0x7f80u;
}

// Per-pair plan of one head: axis and column of each pair.
struct PairPlan {
    std::vector<uint8_t> axis;
    std::vector<uint32_t> col;
};

PairPlan make_plan(const Geom &g) {
    PairPlan p;
    for (int a = 0; a < 3; ++a)
        for (int j = 0; j < g.split[a] / 2; ++j) {
            p.axis.push_back(static_cast<uint8_t>(a));
            p.col.push_back(static_cast<uint32_t>(j));
        }
    return p;
}

// Compare rows [r0, r1) of the given host buffers (whose row 0 is global row
// `base_row`) against the eager order. Returns the number of mismatching
// elements.
int64_t verify_rows(const Geom &g, const rope3d_tables *t, const PairPlan &plan,
                    const void *in, const void *out, int64_t base_row, int64_t r0, int64_t r1) {
    const int64_t N = g.T * g.H * g.W;
    const int64_t re = g.row_elems();
    const int64_t pairs = g.head_dim / 2;
    int64_t bad = 0;
    for (int64_t r = r0; r < r1; ++r) {
        const int64_t tok = (base_row + r) % N;
        const int64_t pos[3] = {tok / (g.H * g.W), (tok / g.W) % g.H, tok % g.W};
        const float *cs[3], *sn[3];
        for (int a = 0; a < 3; ++a) {
            const int64_t half = g.split[a] / 2;
            cs[a] = t->cos_host[a].data() + pos[a] * half;
            sn[a] = t->sin_host[a].data() + pos[a] * half;
        }
        for (int64_t hd = 0; hd < g.heads; ++hd) {
            const int64_t e0 = r * re + hd * g.head_dim;
            for (int64_t p = 0; p < pairs; ++p) {
                const int a = plan.axis[p];
                const float c = cs[a][plan.col[p]];
                const float s = sn[a][plan.col[p]];
                const int64_t i = e0 + 2 * p;
                float ev, od;
                if (g.dtype == ROPE3D_BF16) {
                    ev = widen_bf16(static_cast<const uint16_t *>(in)[i]);
                    od = widen_bf16(static_cast<const uint16_t *>(in)[i + 1]);
                } else if (g.dtype == ROPE3D_F16) {
                    ev = widen_f16(static_cast<const uint16_t *>(in)[i]);
                    od = widen_f16(static_cast<const uint16_t *>(in)[i + 1]);
                } else {
                    ev = static_cast<const float *>(in)[i];
                    od = static_cast<const float *>(in)[i + 1];
                }
                const float ec = ev * c;
                const float os = od * s;
                const float es = ev * s;
                const float oc = od * c;
                const float y0 = ec - os;
                const float y1 = es + oc;
                if (g.dtype == ROPE3D_BF16) {
                    const uint16_t *o = static_cast<const uint16_t *>(out);
                    bad += !same_or_both_nan_bf16(narrow_bf16(y0), o[i]);
                    bad += !same_or_both_nan_bf16(narrow_bf16(y1), o[i + 1]);
                } else if (g.dtype == ROPE3D_F16) {
                    const uint16_t *o = static_cast<const uint16_t *>(out);
                    bad += !same_or_both_nan_f16(narrow_f16(y0), o[i]);
                    bad += !same_or_both_nan_f16(narrow_f16(y1), o[i + 1]);
                } else {
                    const uint32_t *o = static_cast<const uint32_t *>(out);
                    uint32_t b0, b1;
                    std::memcpy(&b0, &y0, 4);
                    std::memcpy(&b1, &y1, 4);
                    bad += !same_or_both_nan_f32(b0, o[i]);
                    bad += !same_or_both_nan_f32(b1, o[i + 1]);
                }
            }
        }
    }
    return bad;
}

// Verify `rows` rows of (q, k) -> (qo, ko) host buffers, in parallel.
int64_t verify_host(const Geom &g, const rope3d_tables *t, const void *q, const void *k,
                    const void *qo, const void *ko, int64_t base_row, int64_t rows) {
    const PairPlan plan = make_plan(g);
    unsigned nt = std::max(1u, std::min(32u, std::thread::hardware_concurrency()));
    if (rows * g.row_elems() < (int64_t(1) << 16)) nt = 1;
    std::vector<int64_t> bad(nt, 0);
    std::vector<std::thread> pool;
    const int64_t per = (rows + nt - 1) / nt;
    for (unsigned w = 0; w < nt; ++w) {
        const int64_t r0 = std::min<int64_t>(rows, int64_t(w) * per);
        const int64_t r1 = std::min<int64_t>(rows, r0 + per);
        auto job = [&, w, r0, r1] {
            bad[w] = verify_rows(g, t, plan, q, qo, base_row, r0, r1) +
                     verify_rows(g, t, plan, k, ko, base_row, r0, r1);
        };
        if (nt == 1) job(); else pool.emplace_back(job);
    }
    for (auto &th : pool) th.join();
    int64_t total = 0;
    for (int64_t b : bad) total += b;
    return total;
}

// Flip one bit of the first output element if a corruption was requested.
void maybe_corrupt(void *qo_host) {
    int c = g_corrupt.load();
    while (c > 0 && !g_corrupt.compare_exchange_weak(c, c - 1)) {}
    if (c > 0) static_cast<uint8_t *>(qo_host)[0] ^= 1u;
}

// Pinned staging for the device-buffer gate.
struct GateStage {
    void *buf[4] = {nullptr, nullptr, nullptr, nullptr};
    size_t bytes = 0;
    cudaStream_t stream = nullptr;
    int device = -1;
} g_gate_stage;

constexpr size_t kGateChunkBytes = size_t(64) << 20;

// Copy back and verify device buffers; returns mismatch count or -1 on a CUDA error.
int64_t verify_device(const Geom &g, const rope3d_tables *t, const void *q, const void *k,
                      const void *qo, const void *ko, int device) {
    const int64_t row_bytes = g.row_elems() * g.esize;
    const size_t need = static_cast<size_t>(std::max<int64_t>(row_bytes, int64_t(kGateChunkBytes)));
    GateStage &st = g_gate_stage;
    if (st.device != device || st.bytes < need) {
        for (void *&b : st.buf) {
            if (b) cudaFreeHost(b);
            b = nullptr;
        }
        if (st.stream && st.device >= 0) cudaStreamDestroy(st.stream);
        st.stream = nullptr;
        st.bytes = 0;
        st.device = device;
        for (void *&b : st.buf)
            if (cudaMallocHost(&b, need) != cudaSuccess) return -1;
        if (cudaStreamCreateWithFlags(&st.stream, cudaStreamNonBlocking) != cudaSuccess) return -1;
        st.bytes = need;
    }
    const int64_t rows_per = std::max<int64_t>(1, static_cast<int64_t>(st.bytes) / row_bytes);
    const int64_t rows = g.rows();
    int64_t bad = 0;
    bool corrupted_once = false;
    for (int64_t r = 0; r < rows; r += rows_per) {
        const int64_t n = std::min(rows_per, rows - r);
        const size_t off = static_cast<size_t>(r * row_bytes);
        const size_t len = static_cast<size_t>(n * row_bytes);
        const void *src[4] = {q, k, qo, ko};
        for (int i = 0; i < 4; ++i)
            if (cudaMemcpyAsync(st.buf[i], static_cast<const char *>(src[i]) + off, len,
                                cudaMemcpyDeviceToHost, st.stream) != cudaSuccess)
                return -1;
        if (cudaStreamSynchronize(st.stream) != cudaSuccess) return -1;
        if (!corrupted_once) {
            maybe_corrupt(st.buf[2]);
            corrupted_once = true;
        }
        bad += verify_host(g, t, st.buf[0], st.buf[1], st.buf[2], st.buf[3], r, n);
    }
    return bad;
}

thread_local LaunchInfo t_last{0, 0, 0};

bool vec16_ok(const Geom &g, const void *q, const void *k, const void *qo, const void *ko) {
    const int64_t vec = 16 / g.esize;
    if (g.head_dim % vec != 0) return false;
    for (int a = 0; a < 3; ++a)
        if (g.split[a] % vec != 0) return false;
    for (const void *p : {q, k, qo, ko})
        if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return false;
    return true;
}

// Debug builds' test hook: launches see the tables this many entries shorter
// than they are (the memory stays valid), so the kernels' table-index checks
// must fire.
std::atomic<uint32_t> g_debug_shrink{0};

LaunchArgs make_launch(const Geom &g, const rope3d_tables *t, const void *q, const void *k,
                       void *qo, void *ko, int64_t rows, int64_t row0, bool vec16) {
    LaunchArgs a{};
    a.q = q;
    a.k = k;
    a.q_out = qo;
    a.k_out = ko;
    a.tables = t->dev;
    a.table_len = t->len;
    if (ROPE3D_DEBUG_BOUNDS) {   // test hook: see rope3d_testing_debug_shrink_tables
        const uint32_t shrink = g_debug_shrink.load(std::memory_order_relaxed);
        a.table_len = shrink < a.table_len ? a.table_len - shrink : 0;
    }
    a.offH = t->offset[1];
    a.offW = t->offset[2];
    a.pT = static_cast<uint32_t>(g.split[0] / 2);
    a.pH = static_cast<uint32_t>(g.split[1] / 2);
    a.pW = static_cast<uint32_t>(g.split[2] / 2);
    a.T = static_cast<uint32_t>(g.T);
    a.H = static_cast<uint32_t>(g.H);
    a.W = static_cast<uint32_t>(g.W);
    a.heads = static_cast<uint32_t>(g.heads);
    a.head_dim = static_cast<uint32_t>(g.head_dim);
    a.rows = static_cast<uint64_t>(rows);
    a.row0 = static_cast<uint64_t>(row0);
    a.dtype = g.dtype;
    a.vec16 = vec16;
    return a;
}

// Gate lookup before a launch: ROPE3D_ERR_PARITY for a refused configuration;
// *verify = true when this call must verify.
int gate_before(const GateKey &key, bool *verify) {
    *verify = false;
    std::lock_guard<std::mutex> lock(g_mutex);
    auto it = g_verdicts.find(key);
    if (it != g_verdicts.end() && it->second == 2) return ROPE3D_ERR_PARITY;
    *verify = g_gate_mode.load() == ROPE3D_GATE_FIRST && it == g_verdicts.end();
    return ROPE3D_OK;
}

int gate_record(const GateKey &key, int64_t bad) {
    std::lock_guard<std::mutex> lock(g_mutex);
    g_verdicts[key] = bad == 0 ? 1 : 2;
    return bad == 0 ? ROPE3D_OK : ROPE3D_ERR_PARITY;
}

}  // namespace

extern "C" int rope3d_apply_pair(const void *q, const void *k, void *q_out, void *k_out,
                                 const rope3d_tables *tables, int64_t B, int64_t T, int64_t H,
                                 int64_t W, int64_t heads, int64_t head_dim,
                                 const int32_t split[3], int32_t dtype, void *stream) {
    const int rc = rope3d_preflight(q, k, q_out, k_out, tables, B, T, H, W, heads, head_dim,
                                    split, dtype, 1);
    if (rc != ROPE3D_OK) return rc;
    const Geom g = make_geom(B, T, H, W, heads, head_dim, split, dtype);
    const GateKey key = gate_key(tables->device, g, tables->base);
    bool verify = false;
    int grc = gate_before(key, &verify);
    if (grc != ROPE3D_OK) return grc;

    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool vec16 = vec16_ok(g, q, k, q_out, k_out);
    LaunchArgs a = make_launch(g, tables, q, k, q_out, k_out, g.rows(), 0, vec16);
    a.pdl = true;
    LaunchInfo info{};
    if (rope3d::launch_rope3d(a, s, &info) != cudaSuccess) return ROPE3D_ERR_CUDA;
    t_last = info;
    if (rope3d::tables_note_use(tables, s) != ROPE3D_OK) return ROPE3D_ERR_CUDA;
    if (!verify) return ROPE3D_OK;

    if (cudaStreamSynchronize(s) != cudaSuccess) return ROPE3D_ERR_CUDA;
    int64_t bad;
    {
        std::lock_guard<std::mutex> lock(g_mutex);  // the staging is shared
        bad = verify_device(g, tables, q, k, q_out, k_out, tables->device);
    }
    if (bad < 0) return ROPE3D_ERR_CUDA;
    return gate_record(key, bad);
}

// ============================================================================
// strided views and rotation in place
// ============================================================================

namespace {

// A strided view of logical shape [B, T, H, W, heads, head_dim]: element
// strides of the six dimensions (the channel stride is 1).
struct View {
    uintptr_t base;
    int64_t n[6];
    int64_t s[6];
    int64_t esize;
    uintptr_t lo() const { return base; }
    uintptr_t hi() const {  // one past the last byte
        int64_t last = 0;
        for (int i = 0; i < 6; ++i) last += (n[i] - 1) * s[i];
        return base + static_cast<uintptr_t>((last + 1) * esize);
    }
};

View make_view(const void *p, const Geom &g, const int64_t st[5]) {
    View v{reinterpret_cast<uintptr_t>(p), {g.B, g.T, g.H, g.W, g.heads, g.head_dim},
           {st[0], st[1], st[2], st[3], st[4], 1}, g.esize};
    return v;
}

// Is delta (elements) a difference of two element offsets of one view, i.e.
// delta = sum_i d_i * s_i with |d_i| <= n_i - 1? Depth-first over the
// dimensions by decreasing stride, bounding each d_i by what the smaller
// dimensions can still reach. Gives up (answers yes) past `budget` nodes.
bool reachable(int64_t delta, const std::vector<std::pair<int64_t, int64_t>> &dims, size_t k,
               const std::vector<int64_t> &reach, int64_t *budget) {
    if (--*budget < 0) return true;
    if (k == dims.size()) return delta == 0;
    const int64_t s = dims[k].first, n = dims[k].second;
    const int64_t m = reach[k + 1];
    if (s == 0) return reachable(delta, dims, k + 1, reach, budget);
    // d * s in [delta - m, delta + m]
    auto floor_div = [](int64_t a, int64_t b) { return a >= 0 ? a / b : -((-a + b - 1) / b); };
    const int64_t lo = std::max(-(n - 1), -floor_div(-(delta - m), s));
    const int64_t hi = std::min(n - 1, floor_div(delta + m, s));
    for (int64_t d = lo; d <= hi; ++d)
        if (reachable(delta - d * s, dims, k + 1, reach, budget)) return true;
    return false;
}

std::vector<std::pair<int64_t, int64_t>> sorted_dims(const View &v) {
    std::vector<std::pair<int64_t, int64_t>> dims;
    for (int i = 0; i < 6; ++i)
        if (v.n[i] > 1) dims.emplace_back(v.s[i], v.n[i]);
    std::sort(dims.begin(), dims.end(), [](auto &a, auto &b) { return a.first > b.first; });
    return dims;
}

// Could the two views share an element? Exact for views with identical
// strides and sizes whose bases differ by a whole number of elements;
// otherwise answered from the byte ranges.
bool may_share(const View &a, const View &b) {
    if (a.hi() <= b.lo() || b.hi() <= a.lo()) return false;
    if (!std::equal(a.s, a.s + 6, b.s) || !std::equal(a.n, a.n + 6, b.n) || a.esize != b.esize)
        return true;
    const int64_t diff = static_cast<int64_t>(b.base) - static_cast<int64_t>(a.base);
    if (diff % a.esize != 0) return true;
    const auto dims = sorted_dims(a);
    std::vector<int64_t> reach(dims.size() + 1, 0);
    for (size_t k = dims.size(); k-- > 0;) reach[k] = reach[k + 1] + (dims[k].second - 1) * dims[k].first;
    int64_t budget = 1 << 16;
    return reachable(diff / a.esize, dims, 0, reach, &budget);
}

// Is there a nonzero (d_i), |d_i| <= n_i - 1, with sum_i d_i * s_i == delta?
// Same search as reachable(), tracking whether some d_i is nonzero.
bool reachable_nonzero(int64_t delta, const std::vector<std::pair<int64_t, int64_t>> &dims,
                       size_t k, const std::vector<int64_t> &reach, bool nonzero,
                       int64_t *budget) {
    if (--*budget < 0) return true;
    if (k == dims.size()) return delta == 0 && nonzero;
    const int64_t s = dims[k].first, n = dims[k].second;
    if (s == 0) return true;  // two indices along this dimension meet (n > 1)
    const int64_t m = reach[k + 1];
    auto floor_div = [](int64_t a, int64_t b) { return a >= 0 ? a / b : -((-a + b - 1) / b); };
    const int64_t lo = std::max(-(n - 1), -floor_div(-(delta - m), s));
    const int64_t hi = std::min(n - 1, floor_div(delta + m, s));
    for (int64_t d = lo; d <= hi; ++d)
        if (reachable_nonzero(delta - d * s, dims, k + 1, reach, nonzero || d != 0, budget))
            return true;
    return false;
}

// Does the view map two different indices to one element? Exact (a nonzero
// index difference whose offset is zero), answering yes if the search runs
// past its budget.
bool self_overlapping(const View &v) {
    const auto dims = sorted_dims(v);
    std::vector<int64_t> reach(dims.size() + 1, 0);
    for (size_t k = dims.size(); k-- > 0;) reach[k] = reach[k + 1] + (dims[k].second - 1) * dims[k].first;
    int64_t budget = 1 << 16;
    return reachable_nonzero(0, dims, 0, reach, false, &budget);
}

bool same_view(const View &a, const View &b) {
    return a.base == b.base && std::equal(a.s, a.s + 6, b.s) && std::equal(a.n, a.n + 6, b.n);
}

int check_strided(const void *q, const void *k, const void *qo, const void *ko, const Geom &g,
                  const int64_t *const st[4]) {
    const void *ptrs[4] = {q, k, qo, ko};
    for (int i = 0; i < 4; ++i)
        if (!ptrs[i] || !st[i]) return ROPE3D_ERR_NULL;
    const int64_t extents[5] = {g.B, g.T, g.H, g.W, g.heads};
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 5; ++j) {
            if (st[i][j] < 0 || st[i][j] > (int64_t(1) << 50)) return ROPE3D_ERR_SHAPE;
            if (g.esize == 2 && extents[j] > 1 && (st[i][j] % 2) != 0) return ROPE3D_ERR_ALIGN;
        }
    for (const void *p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return ROPE3D_ERR_ALIGN;
    View v[4];
    for (int i = 0; i < 4; ++i) v[i] = make_view(ptrs[i], g, st[i]);
    // the whole footprint must stay inside the address space
    for (int i = 0; i < 4; ++i)
        if (v[i].hi() < v[i].lo()) return ROPE3D_ERR_SHAPE;
    for (int o = 2; o < 4; ++o)
        if (self_overlapping(v[o])) return ROPE3D_ERR_ALIAS;
    // each output against each input (exact in-place identity allowed for its
    // own input) and against the other output
    const bool inplace_q = same_view(v[2], v[0]);
    const bool inplace_k = same_view(v[3], v[1]);
    if (!inplace_q && may_share(v[2], v[0])) return ROPE3D_ERR_ALIAS;
    if (!inplace_k && may_share(v[3], v[1])) return ROPE3D_ERR_ALIAS;
    if (may_share(v[2], v[1]) || may_share(v[3], v[0]) || may_share(v[2], v[3]))
        return ROPE3D_ERR_ALIAS;
    return ROPE3D_OK;
}

int preflight_strided(const void *q, const void *k, const void *qo, const void *ko,
                      const rope3d_tables *tables, const Geom &g, const int32_t split[3],
                      const int64_t *const st[4], bool check_device) {
    if (!split) return ROPE3D_ERR_NULL;
    int rc = check_geom(g);
    if (rc != ROPE3D_OK) return rc;
    rc = check_strided(q, k, qo, ko, g, st);
    if (rc != ROPE3D_OK) return rc;
    rc = check_tables(tables, g);
    if (rc != ROPE3D_OK || !check_device) return rc;
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return ROPE3D_ERR_CUDA;
    if (tables->host_backed || tables->device != device) return ROPE3D_ERR_DEVICE;
    for (const void *p : {q, k, qo, ko})
        if (!is_device_ptr(p, device)) return ROPE3D_ERR_DEVICE;
    return ROPE3D_OK;
}

using StridedKey = std::pair<GateKey, std::array<int64_t, 20>>;
std::map<StridedKey, int> g_verdicts_strided;  // 1 verified, 2 refused

bool vec16_strided_ok(const Geom &g, const void *const ptrs[4], const int64_t *const st[4]) {
    const int64_t vec = 16 / g.esize;
    if (g.head_dim % vec != 0) return false;
    for (int a = 0; a < 3; ++a)
        if (g.split[a] % vec != 0) return false;
    const int64_t extents[5] = {g.B, g.T, g.H, g.W, g.heads};
    for (int i = 0; i < 4; ++i) {
        if (reinterpret_cast<uintptr_t>(ptrs[i]) % 16 != 0) return false;
        for (int j = 0; j < 5; ++j)
            if (extents[j] > 1 && st[i][j] % vec != 0) return false;
    }
    return true;
}

}  // namespace

extern "C" int rope3d_preflight_strided(const void *q, const void *k, const void *q_out,
                                        const void *k_out, const rope3d_tables *tables,
                                        int64_t B, int64_t T, int64_t H, int64_t W,
                                        int64_t heads, int64_t head_dim, const int32_t split[3],
                                        int32_t dtype, const int64_t q_strides[5],
                                        const int64_t k_strides[5],
                                        const int64_t q_out_strides[5],
                                        const int64_t k_out_strides[5], int32_t check_device) {
    const Geom g = make_geom(B, T, H, W, heads, head_dim, split, dtype);
    const int64_t *const st[4] = {q_strides, k_strides, q_out_strides, k_out_strides};
    return preflight_strided(q, k, q_out, k_out, tables, g, split, st, check_device != 0);
}

extern "C" int rope3d_apply_pair_strided(const void *q, const void *k, void *q_out, void *k_out,
                                         const rope3d_tables *tables, int64_t B, int64_t T,
                                         int64_t H, int64_t W, int64_t heads, int64_t head_dim,
                                         const int32_t split[3], int32_t dtype,
                                         const int64_t q_strides[5], const int64_t k_strides[5],
                                         const int64_t q_out_strides[5],
                                         const int64_t k_out_strides[5], void *stream) {
    const Geom g = make_geom(B, T, H, W, heads, head_dim, split, dtype);
    const int64_t *const st[4] = {q_strides, k_strides, q_out_strides, k_out_strides};
    int rc = preflight_strided(q, k, q_out, k_out, tables, g, split, st, true);
    if (rc != ROPE3D_OK) return rc;

    StridedKey key{gate_key(tables->device, g, tables->base), {}};
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 5; ++j) key.second[i * 5 + j] = st[i][j];
    bool verify = false;
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        auto it = g_verdicts_strided.find(key);
        if (it != g_verdicts_strided.end() && it->second == 2) return ROPE3D_ERR_PARITY;
        verify = g_gate_mode.load() == ROPE3D_GATE_FIRST && it == g_verdicts_strided.end();
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t bytes = static_cast<size_t>(g.bytes());
    void *copy[4] = {nullptr, nullptr, nullptr, nullptr};
    auto free_copies = [&] {
        for (void *&c : copy)
            if (c) cudaFree(c), c = nullptr;
    };
    if (verify) {
        // the inputs are gathered before the kernel runs: in-place calls overwrite them
        for (void *&c : copy)
            if (cudaMalloc(&c, bytes) != cudaSuccess) {
                c = nullptr;
                cudaGetLastError();
                free_copies();
                return ROPE3D_ERR_NOMEM;
            }
        for (int i = 0; i < 2; ++i)
            if (rope3d::launch_gather(i == 0 ? q : k, st[i], copy[i], static_cast<int>(g.esize),
                                      g.B, g.T, g.H, g.W, g.heads, g.head_dim, s) != cudaSuccess) {
                free_copies();
                return ROPE3D_ERR_CUDA;
            }
    }
    const void *ptrs[4] = {q, k, q_out, k_out};
    LaunchArgs a = make_launch(g, tables, q, k, q_out, k_out, g.rows(), 0,
                               vec16_strided_ok(g, ptrs, st));
    a.strided = true;
    a.pdl = !verify;  // the gate's gathers precede the kernel on this stream
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 5; ++j) a.strides[i][j] = st[i][j];
    LaunchInfo info{};
    if (rope3d::launch_rope3d(a, s, &info) != cudaSuccess) {
        free_copies();
        return ROPE3D_ERR_CUDA;
    }
    t_last = info;
    if (rope3d::tables_note_use(tables, s) != ROPE3D_OK) {
        free_copies();
        return ROPE3D_ERR_CUDA;
    }
    if (!verify) return ROPE3D_OK;

    for (int i = 0; i < 2; ++i)
        if (rope3d::launch_gather(i == 0 ? q_out : k_out, st[2 + i], copy[2 + i],
                                  static_cast<int>(g.esize), g.B, g.T, g.H, g.W, g.heads,
                                  g.head_dim, s) != cudaSuccess) {
            free_copies();
            return ROPE3D_ERR_CUDA;
        }
    if (cudaStreamSynchronize(s) != cudaSuccess) {
        free_copies();
        return ROPE3D_ERR_CUDA;
    }
    int64_t bad;
    {
        std::lock_guard<std::mutex> lock(g_mutex);  // the staging is shared
        bad = verify_device(g, tables, copy[0], copy[1], copy[2], copy[3], tables->device);
    }
    free_copies();
    if (bad < 0) return ROPE3D_ERR_CUDA;
    std::lock_guard<std::mutex> lock(g_mutex);
    g_verdicts_strided[key] = bad == 0 ? 1 : 2;
    return bad == 0 ? ROPE3D_OK : ROPE3D_ERR_PARITY;
}

// ============================================================================
// host-buffer pipeline
// ============================================================================

namespace {

constexpr int kSlots = 3;
constexpr size_t kSlotBytes = size_t(64) << 20;  // per tensor per slot

struct HostPipe {
    int device = -1;
    size_t slot_bytes = 0;
    void *buf[kSlots][4] = {};
    cudaStream_t s_h2d = nullptr, s_comp = nullptr, s_d2h = nullptr;
    cudaEvent_t ev_h2d[kSlots] = {}, ev_comp[kSlots] = {}, ev_d2h[kSlots] = {};
    cudaEvent_t ev_start = nullptr;
    bool used[kSlots] = {};
};

std::mutex g_pipe_mutex;
std::map<int, HostPipe> g_pipes;

void destroy_pipe(HostPipe &p) {
    if (p.device < 0) return;
    int cur = 0;
    cudaGetDevice(&cur);
    cudaSetDevice(p.device);
    cudaDeviceSynchronize();
    for (auto &slot : p.buf)
        for (void *&b : slot) {
            if (b) cudaFree(b);
            b = nullptr;
        }
    for (cudaStream_t *s : {&p.s_h2d, &p.s_comp, &p.s_d2h})
        if (*s) cudaStreamDestroy(*s), *s = nullptr;
    for (int i = 0; i < kSlots; ++i)
        for (cudaEvent_t *e : {&p.ev_h2d[i], &p.ev_comp[i], &p.ev_d2h[i]})
            if (*e) cudaEventDestroy(*e), *e = nullptr;
    if (p.ev_start) cudaEventDestroy(p.ev_start), p.ev_start = nullptr;
    p.slot_bytes = 0;
    cudaSetDevice(cur);
}

int ensure_pipe(HostPipe &p, int device, size_t slot_bytes) {
    if (p.device == device && p.slot_bytes >= slot_bytes) return ROPE3D_OK;
    destroy_pipe(p);
    p.device = device;
    for (auto &slot : p.buf)
        for (void *&b : slot)
            if (cudaMalloc(&b, slot_bytes) != cudaSuccess) {
                b = nullptr;
                cudaGetLastError();
                destroy_pipe(p);
                p.device = -1;
                return ROPE3D_ERR_NOMEM;
            }
    bool ok = true;
    for (cudaStream_t *s : {&p.s_h2d, &p.s_comp, &p.s_d2h})
        ok = ok && cudaStreamCreateWithFlags(s, cudaStreamNonBlocking) == cudaSuccess;
    for (int i = 0; i < kSlots; ++i)
        for (cudaEvent_t *e : {&p.ev_h2d[i], &p.ev_comp[i], &p.ev_d2h[i]})
            ok = ok && cudaEventCreateWithFlags(e, cudaEventDisableTiming) == cudaSuccess;
    ok = ok && cudaEventCreateWithFlags(&p.ev_start, cudaEventDisableTiming) == cudaSuccess;
    if (!ok) {
        destroy_pipe(p);
        p.device = -1;
        return ROPE3D_ERR_CUDA;
    }
    p.slot_bytes = slot_bytes;
    for (bool &u : p.used) u = false;
    return ROPE3D_OK;
}

}  // namespace

extern "C" int rope3d_apply_pair_host(const void *q, const void *k, void *q_out, void *k_out,
                                      const rope3d_tables *tables, int64_t B, int64_t T,
                                      int64_t H, int64_t W, int64_t heads, int64_t head_dim,
                                      const int32_t split[3], int32_t dtype, void *stream) {
    const Geom g = make_geom(B, T, H, W, heads, head_dim, split, dtype);
    int rc = preflight(q, k, q_out, k_out, tables, g, split);
    if (rc != ROPE3D_OK) return rc;
    int device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return ROPE3D_ERR_CUDA;
    if (tables->host_backed || tables->device != device) return ROPE3D_ERR_DEVICE;
    for (const void *p : {q, k, static_cast<const void *>(q_out), static_cast<const void *>(k_out)})
        if (!is_host_ptr(p)) return ROPE3D_ERR_DEVICE;
    const GateKey key = gate_key(device, g, tables->base);
    bool verify = false;
    rc = gate_before(key, &verify);
    if (rc != ROPE3D_OK) return rc;

    const int64_t row_bytes = g.row_elems() * g.esize;
    const size_t slot = std::max(kSlotBytes, static_cast<size_t>((row_bytes + 255) / 256 * 256));
    std::lock_guard<std::mutex> lock(g_pipe_mutex);
    HostPipe &p = g_pipes[device];
    rc = ensure_pipe(p, device, slot);
    if (rc != ROPE3D_OK) return rc;
    const int64_t rows_per = std::max<int64_t>(1, static_cast<int64_t>(p.slot_bytes) / row_bytes);
    const bool vec16 = vec16_ok(g, p.buf[0][0], p.buf[0][1], p.buf[0][2], p.buf[0][3]);

    // order after earlier work on the caller's stream
    cudaStream_t user = static_cast<cudaStream_t>(stream);
    if (cudaEventRecord(p.ev_start, user) != cudaSuccess ||
        cudaStreamWaitEvent(p.s_h2d, p.ev_start, 0) != cudaSuccess)
        return ROPE3D_ERR_CUDA;

    const char *src[2] = {static_cast<const char *>(q), static_cast<const char *>(k)};
    char *dst[2] = {static_cast<char *>(q_out), static_cast<char *>(k_out)};
    LaunchInfo info{};
    int64_t chunk = 0;
    for (int64_t r = 0; r < g.rows(); r += rows_per, ++chunk) {
        const int s = static_cast<int>(chunk % kSlots);
        const int64_t n = std::min(rows_per, g.rows() - r);
        const size_t off = static_cast<size_t>(r * row_bytes);
        const size_t len = static_cast<size_t>(n * row_bytes);
        if (p.used[s] && cudaStreamWaitEvent(p.s_h2d, p.ev_d2h[s], 0) != cudaSuccess)
            return ROPE3D_ERR_CUDA;
        for (int i = 0; i < 2; ++i)
            if (cudaMemcpyAsync(p.buf[s][i], src[i] + off, len, cudaMemcpyHostToDevice,
                                p.s_h2d) != cudaSuccess)
                return ROPE3D_ERR_CUDA;
        if (cudaEventRecord(p.ev_h2d[s], p.s_h2d) != cudaSuccess ||
            cudaStreamWaitEvent(p.s_comp, p.ev_h2d[s], 0) != cudaSuccess)
            return ROPE3D_ERR_CUDA;
        const LaunchArgs a = make_launch(g, tables, p.buf[s][0], p.buf[s][1], p.buf[s][2],
                                         p.buf[s][3], n, r, vec16);
        if (rope3d::launch_rope3d(a, p.s_comp, &info) != cudaSuccess ||
            rope3d::tables_note_use(tables, p.s_comp) != ROPE3D_OK)
            return ROPE3D_ERR_CUDA;
        if (cudaEventRecord(p.ev_comp[s], p.s_comp) != cudaSuccess ||
            cudaStreamWaitEvent(p.s_d2h, p.ev_comp[s], 0) != cudaSuccess)
            return ROPE3D_ERR_CUDA;
        for (int i = 0; i < 2; ++i)
            if (cudaMemcpyAsync(dst[i] + off, p.buf[s][2 + i], len, cudaMemcpyDeviceToHost,
                                p.s_d2h) != cudaSuccess)
                return ROPE3D_ERR_CUDA;
        if (cudaEventRecord(p.ev_d2h[s], p.s_d2h) != cudaSuccess) return ROPE3D_ERR_CUDA;
        p.used[s] = true;
    }
    if (cudaStreamSynchronize(p.s_d2h) != cudaSuccess) return ROPE3D_ERR_CUDA;
    t_last = info;
    if (!verify) return ROPE3D_OK;
    // the test hook flips a bit of the caller's output only for the comparison
    const uint8_t first = *static_cast<const uint8_t *>(q_out);
    maybe_corrupt(q_out);
    const int64_t bad = verify_host(g, tables, q, k, q_out, k_out, 0, g.rows());
    *static_cast<uint8_t *>(q_out) = first;
    return gate_record(key, bad);
}

extern "C" int rope3d_debug_bounds(int64_t *errors, int32_t reset) {
    if (!errors) return ROPE3D_ERR_NULL;
    int64_t total = 0;
    for (int64_t n : {rope3d::kernels_bound_errors(reset != 0), rope3d::patchify_bound_errors(reset != 0),
                      rope3d::neox_bound_errors(reset != 0), rope3d::na3d_bound_errors(reset != 0)}) {
        if (n < 0) return ROPE3D_ERR_CUDA;
        total += n;
    }
    *errors = total;
    return ROPE3D_DEBUG_BOUNDS ? 1 : 0;
}

extern "C" int rope3d_testing_debug_shrink_tables(int32_t n) {
    if (!ROPE3D_DEBUG_BOUNDS) return ROPE3D_ERR_ARG;
    if (n < 0) return ROPE3D_ERR_ARG;
    g_debug_shrink.store(static_cast<uint32_t>(n));
    return ROPE3D_OK;
}

extern "C" int rope3d_release_scratch(void) {
    std::lock_guard<std::mutex> lock(g_pipe_mutex);
    for (auto &kv : g_pipes) destroy_pipe(kv.second);
    g_pipes.clear();
    return ROPE3D_OK;
}

// ============================================================================
// gate controls, introspection
// ============================================================================

extern "C" int rope3d_gate_set_mode(int32_t mode) {
    if (mode != ROPE3D_GATE_OFF && mode != ROPE3D_GATE_FIRST) return ROPE3D_ERR_ARG;
    g_gate_mode.store(mode);
    return ROPE3D_OK;
}

extern "C" int rope3d_gate_get_mode(void) { return g_gate_mode.load(); }

extern "C" int rope3d_gate_reset(void) {
    std::lock_guard<std::mutex> lock(g_mutex);
    g_verdicts.clear();
    g_verdicts_strided.clear();
    g_corrupt.store(0);
    return ROPE3D_OK;
}

extern "C" int rope3d_gate_verdict(int64_t B, int64_t T, int64_t H, int64_t W, int64_t heads,
                                   int64_t head_dim, const int32_t split[3], double base,
                                   int32_t dtype) {
    if (!split) return ROPE3D_ERR_NULL;
    int device = -1;
    {
        std::lock_guard<std::mutex> lock(g_mutex);
        if (!g_cache.host_tables && cudaGetDevice(&device) != cudaSuccess) return ROPE3D_ERR_CUDA;
    }
    const Geom g = make_geom(B, T, H, W, heads, head_dim, split, dtype);
    std::lock_guard<std::mutex> lock(g_mutex);
    auto it = g_verdicts.find(gate_key(device, g, base));
    return it == g_verdicts.end() ? 0 : it->second;
}

extern "C" int rope3d_testing_corrupt_gate(int32_t count) {
    if (count < 0) return ROPE3D_ERR_ARG;
    g_corrupt.store(count);
    return ROPE3D_OK;
}

extern "C" int rope3d_last_launch(int32_t *grid, int32_t *block) {
    if (grid) *grid = t_last.grid;
    if (block) *block = t_last.block;
    return t_last.kernel;
}

extern "C" int64_t rope3d_testing_fastdiv(int64_t n, int64_t d) {
    if (d < 1 || d >= (int64_t(1) << 31) || n < 0 || n >= (int64_t(1) << 31)) return -1;
    const FastDiv f = rope3d::make_fastdiv(static_cast<uint32_t>(d));
    return rope3d::fastdiv_host(static_cast<uint32_t>(n), f);
}

extern "C" int rope3d_testing_max_units_per_launch(int64_t n) {
    if (n < 0 || n > int64_t(rope3d::kMaxUnitsPerLaunch)) return ROPE3D_ERR_ARG;
    rope3d::set_max_units_per_launch(static_cast<uint32_t>(n));
    rope3d::na3d_set_max_units_per_launch(static_cast<uint32_t>(n));
    return ROPE3D_OK;
}

extern "C" int rope3d_abi_version(void) { return ROPE3D_ABI_VERSION; }

extern "C" const char *rope3d_status_string(int status) {
    switch (status) {
        case ROPE3D_OK: return "ROPE3D_OK";
        case ROPE3D_ERR_NULL: return "ROPE3D_ERR_NULL: a required pointer is NULL";
        case ROPE3D_ERR_SHAPE: return "ROPE3D_ERR_SHAPE: invalid sizes or split";
        case ROPE3D_ERR_DTYPE: return "ROPE3D_ERR_DTYPE: dtype must be ROPE3D_BF16, ROPE3D_F32 or ROPE3D_F16";
        case ROPE3D_ERR_ALIGN: return "ROPE3D_ERR_ALIGN: a pointer is not 4-byte aligned";
        case ROPE3D_ERR_ALIAS: return "ROPE3D_ERR_ALIAS: an output overlaps another buffer";
        case ROPE3D_ERR_DEVICE: return "ROPE3D_ERR_DEVICE: a pointer is not memory of the expected kind on the current device";
        case ROPE3D_ERR_PARITY: return "ROPE3D_ERR_PARITY: the bit-exact gate refused this configuration";
        case ROPE3D_ERR_CUDA: return "ROPE3D_ERR_CUDA: a CUDA call failed";
        case ROPE3D_ERR_TABLES: return "ROPE3D_ERR_TABLES: the tables do not match (T, H, W, split)";
        case ROPE3D_ERR_NOMEM: return "ROPE3D_ERR_NOMEM: an allocation failed";
        case ROPE3D_ERR_ARG: return "ROPE3D_ERR_ARG: an argument is out of range";
        case ROPE3D_ERR_SCRATCH: return "ROPE3D_ERR_SCRATCH: the tables exceed the 64 KiB static table area of rope3d_apply_pair_noalloc, or a workspace is too small";
        default: return "ROPE3D: unknown status";
    }
}
