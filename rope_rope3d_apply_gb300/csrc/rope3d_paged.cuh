// rope3d_paged.cuh -- how the attention over pages divides its work; shared by its
// kernels (rope3d_paged.cu, rope3d_paged_tc.cu).
//
// An item is a tile of query rows of one sequence and key/value head: row
// g of the sequence's tokens * group rows is query head g % group of the group, of
// token g / group, so the heads that share keys share their loads. An item's keys are
// those that some row of it sees, in blocks of kKeys places (at least one, where there
// are none zeros have to be written); its cost is their number and a constant for
// beginning and ending an item. The items in order (sequence, key/value head, tile)
// make a line that is cut into as many equal parts as there are thread blocks, wherever
// the cuts fall: a prompt, one token over a long cache and ragged mixtures are
// divided alike, and nothing has to be known on the host. An item that a cut divides
// leaves partial results (sums not yet divided, with the row's maximum and sum) in
// the workspace, which a second kernel adds in order.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "rope3d_internal.h"
#include "rope3d_paged.h"

namespace rope3d_paged {

struct AttnParams {
    const char *q, *k, *v;
    char *out;
    float *lse;
    Batch batch;
    rope3d::FastDiv group;          // query heads of a key/value head
    rope3d::FastDiv page;           // places of a page
    rope3d::FastDiv span;           // kKeys * group / kRows: tiles whose rows' keys end in one block
    rope3d::FastDiv cuts;           // parts
    int item_cost;                  // what an item costs besides its blocks, in blocks
    int kv_heads, head_dim;
    int causal, window;             // window 0: none
    int64_t q_token, q_head, out_token, out_head, lse_token;   // bytes; lse_token in floats
    int64_t k_page, k_slot, k_head, v_page, v_slot, v_head;    // bytes
    float scale_log2;               // scale * log2(e), positive
    int parts;                      // thread blocks the line of blocks is cut for
    float *partial;                 // workspace: two slots a part
    struct PartNote *notes;         // workspace: where each part's first cut fell
};

// What a part leaves for the kernel that adds the partial results: where its
// range begins, and the item that the cut falls into.
struct PartNote {
    long long begin, end;           // the part's range of the line
    long long item, cost;           // where the item at `begin` begins, and its cost
    int s, h, t, pad;
};

// (The arithmetic of the division is compiled for the host too, where tests run it.)
__host__ __device__ __forceinline__ uint32_t udiv(uint32_t n, const rope3d::FastDiv &f) {
#ifdef __CUDA_ARCH__
    return (__umulhi(n, f.mul) + n) >> f.shift;
#else
    return rope3d::fastdiv_host(n, f);
#endif
}

// A sequence as the line of blocks sees it.
struct Seq {
    int lo, n, len, tiles;
};

template <int kRows>
__host__ __device__ __forceinline__ Seq seq_of(const AttnParams &p, int s) {
    Seq q;
    int hi;
    sequence(p.batch, s, q.lo, hi, q.len);
    q.n = hi - q.lo;
    q.tiles = int((int64_t(q.n) * p.group.d + kRows - 1) / kRows);
    return q;
}

// Blocks [b0, b1) of tile t; the places [k0, k1) that its rows see.
struct Tile {
    int b0, b1, k0, k1;
    __host__ __device__ int blocks() const { return max(b1 - b0, 1); }
};

template <int kRows, int kKeys>
__host__ __device__ __forceinline__ Tile tile_of(const AttnParams &p, const Seq &q, int t) {
    const uint32_t rows = uint32_t(q.n) * p.group.d, last = min(rows, uint32_t(t + 1) * kRows) - 1;
    const int past = q.len - q.n;   // place of the first new token; negative where the length is too short
    Tile r;
    r.k1 = p.causal ? min(max(past + int(udiv(last, p.group)) + 1, 0), q.len) : q.len;
    r.k0 = p.window ? min(max(past + int(udiv(uint32_t(t) * kRows, p.group)) - p.window + 1, 0), r.k1) : 0;
    r.b0 = r.k0 / kKeys;
    r.b1 = r.k1 > r.k0 ? (r.k1 + kKeys - 1) / kKeys : r.b0;
    return r;
}

// The cost of tiles 0 .. t - 1 (t below the tiles) of one key/value head, without a
// loop over them. With T rows a tile, K places a block, G rows a token and `past` places
// before the new tokens, the last row of tile u < t sees ceil((past + 1 + floor((u T + T -
// 1) / G)) / K) = floor((a + u) / D) blocks from place 0 on, where D = K G / T and a =
// floor((G (past + K) + T - 1) / T), and a window leaves out floor((c + u) / D) of
// them, c = floor(G (past - window + 1) / T): sums of floors in a row.
template <typename T>
__host__ __device__ __forceinline__ T floors(T n, const rope3d::FastDiv &f) {   // sum of floor(i / d) over 0 <= i < n
    const T d = T(f.d), q = sizeof(T) == 4 || n < 0x7fffffff ? T(udiv(uint32_t(n), f)) : n / d;
    return q * (q - 1) / 2 * d + q * (n - q * d);
}

// What the cost of a sequence's tiles depends on, in T: in 32 bits where every number stays
// below 2^31 (a call of microseconds feels the others).
template <typename T, int kRows, int kKeys>
struct Costs {
    T a, c, each;   // each: blocks of a tile that is not causal

    __host__ __device__ __forceinline__ Costs(const AttnParams &p, const Seq &q) {
        static_assert(kKeys % kRows == 0 && (kRows == 256 || kRows == 128 || kRows == 16), "D is whole");
        constexpr int kShift = kRows == 256 ? 8 : kRows == 128 ? 7 : 4;
        const T group = T(p.group.d), past = T(q.len - q.n);
        a = (group * (past + kKeys) + kRows - 1) >> kShift;
        c = group * (past - p.window + 1) >> kShift;
        each = T(max((q.len + kKeys - 1) / kKeys, 1));
    }

    // of tiles 0 .. t - 1
    __host__ __device__ __forceinline__ T at(const AttnParams &p, int t) const {
        const T d = T(p.span.d);
        T sum = each * t;
        if (p.causal) {   // at least 1 each
            const T ones = min(max(d - a, T(0)), T(t));
            sum = ones + (T(t) > ones ? floors<T>(a + t, p.span) - floors<T>(a + ones, p.span) : T(0));
        }
        if (p.window && c + t > 0) sum -= floors<T>(c + t, p.span) - floors<T>(max(c, T(0)), p.span);
        return sum + T(t) * p.item_cost;
    }

    // The last of `tiles` that begins at or before place `in` of the line, and where it begins.
    __host__ __device__ __forceinline__ int find(const AttnParams &p, int tiles, T in, T &begins) const {
        int t = 0, above = tiles;
        begins = 0;
#pragma unroll 1
        while (above - t > 1) {
            const int mid = (t + above) >> 1;
            const T v = at(p, mid);
            if (v <= in) {
                t = mid;
                begins = v;
            } else {
                above = mid;
            }
        }
        return t;
    }
};

// Whether 32 bits do: with fewer than 64 rows a token, and tokens and places times those below
// 2^17, n in floors() is below 2^15 and every sum of theirs below 2^31 (16 rows a tile; larger
// tiles less).
__host__ __device__ __forceinline__ bool small_costs(const AttnParams &p, const Seq &q) {
    const int most = (1 << 17) / int(p.group.d);
    return p.group.d < 64 && q.len < most && q.n < most && p.window < (1 << 17);
}

// The cost of one key/value head of a sequence.
template <int kRows, int kKeys>
__host__ __device__ __forceinline__ long long seq_cost(const AttnParams &p, const Seq &q) {
    if (q.tiles == 0) return 0;
    const long long last = tile_of<kRows, kKeys>(p, q, q.tiles - 1).blocks() + p.item_cost;
    if (q.tiles == 1) return last;
    if (small_costs(p, q)) return last + Costs<int, kRows, kKeys>(p, q).at(p, q.tiles - 1);
    return last + Costs<long long, kRows, kKeys>(p, q).at(p, q.tiles - 1);
}

// Where part `part` begins (one answer for all threads of the block, by way of
// shared memory): its range of the line and the item there.
struct Start {
    long long begin, end, item, cost;
    int s, h, t, off;
};

// floor(total * part / parts)
__host__ __device__ __forceinline__ long long cut(const AttnParams &p, long long total, int part) {
    if (total < (1 << 21)) return udiv(uint32_t(total) * uint32_t(part), p.cuts);   // (fewer than 1024 parts)
    const long long whole = total < 0x7fffffff ? (long long)udiv(uint32_t(total), p.cuts) : total / p.parts;
    return whole * part + udiv(uint32_t(total - whole * p.parts) * uint32_t(part), p.cuts);
}

// The item at place `begin` of the line, in a sequence whose first is `before` and whose
// heads cost `head` each.
template <int kRows, int kKeys>
__host__ __device__ __forceinline__ void start_in(const AttnParams &p, int s, const Seq &q, long long before, long long head, long long begin,
                                         Start *out) {
    const long long in = begin - before;
    out->s = s;
    out->h = in < 0x7fffffff && head < 0x7fffffff ? int(uint32_t(in) / uint32_t(head)) : int(in / head);
    before += out->h * head;
    int t = 0;
    if (q.tiles > 1) {
        if (small_costs(p, q)) {
            int at;
            t = Costs<int, kRows, kKeys>(p, q).find(p, q.tiles, int(begin - before), at);
            before += at;
        } else {
            long long at;
            t = Costs<long long, kRows, kKeys>(p, q).find(p, q.tiles, begin - before, at);
            before += at;
        }
    }
    out->t = t;
    out->off = int(begin - before);
    out->item = before;
    out->cost = tile_of<kRows, kKeys>(p, q, t).blocks() + p.item_cost;
}

// Sequences [first, end) of a thread, which begin at `before` and cost `sum` together: the item
// at place `begin` of the line, if it is one of theirs. (q and head: the last of them.)
template <int kRows, int kKeys>
__host__ __device__ __forceinline__ void start_among(const AttnParams &p, int first, int end, Seq q, long long before, long long sum,
                                                     long long head, long long begin, long long stop, Start *out) {
    if (begin >= stop || begin < before || begin >= before + sum) return;
    int s = first;
    while (end - first > 1) {   // which of the thread's sequences
        q = seq_of<kRows>(p, s);
        head = seq_cost<kRows, kKeys>(p, q);
        if (begin < before + head * p.kv_heads) break;
        before += head * p.kv_heads;
        ++s;
    }
    start_in<kRows, kKeys>(p, s, q, before, head, begin, out);
}

template <int kRows, int kKeys, int kThreads>
__device__ void find_start(const AttnParams &p, int part, Start *out, long long *s_sums) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int seqs = p.batch.seqs, each = (seqs + kThreads - 1) / kThreads;
    const int first = min(tid * each, seqs), end = min(first + each, seqs);
    Seq q{0, 0, 0, 0};
    long long sum = 0, head = 0;
    for (int s = first; s < end; ++s) {
        q = seq_of<kRows>(p, s);
        head = seq_cost<kRows, kKeys>(p, q);
        sum += head * p.kv_heads;
    }
    long long inc = sum;
#pragma unroll 1
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == 31) s_sums[warp] = inc;
    if (tid == 0) out->s = -1;
    __syncthreads();
    long long before = inc - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += s_sums[w];
        total += s_sums[w];
    }
    const long long begin = cut(p, total, part), stop = cut(p, total, part + 1);
    start_among<kRows, kKeys>(p, first, end, q, before, sum, head, begin, stop, out);
    if (tid == 0) {
        out->begin = begin;
        out->end = stop;
    }
    __syncthreads();
}

// One item, as far as a part computes it.
struct Item {
    int s, h, t;
    Seq q;
    Tile tile;
    int begin, end;      // blocks this part computes
    int rows;            // rows of the tile
    bool whole;          // all of the item's blocks
    bool head;           // an earlier part began it: the first of the part's two slots
};

// Walks the items of a part; every thread that does so takes the same steps. An item's
// constant cost comes before its blocks: a cut within it leaves the item to the later part.
template <int kRows, int kKeys>
struct Walker {
    const AttnParams &p;
    long long left;
    int s, h, t, off;
    Seq q;

    __host__ __device__ Walker(const AttnParams &params, const Start &st)
        : p(params), left(st.s < 0 ? 0 : st.end - st.begin), s(st.s), h(st.h), t(st.t), off(st.off) {
        if (left) q = seq_of<kRows>(p, s);
    }

    __host__ __device__ bool next(Item &it) {
        while (left > 0) {
            while (t >= q.tiles) {   // the next head, or the next sequence with tokens
                t = 0;
                if (q.tiles == 0 || ++h >= p.kv_heads) {
                    h = 0;
                    if (++s >= p.batch.seqs) return false;
                    q = seq_of<kRows>(p, s);
                }
            }
            it.tile = tile_of<kRows, kKeys>(p, q, t);
            const int blocks = it.tile.blocks(), cost = blocks + p.item_cost, take = int(min(left, (long long)(cost - off)));
            const int from = max(off - p.item_cost, 0), to = max(off + take - p.item_cost, 0);
            it.s = s;
            it.h = h;
            it.t = t;
            it.q = q;
            it.begin = it.tile.b0 + from;
            it.end = min(it.tile.b0 + to, it.tile.b1);
            it.rows = int(min(uint32_t(kRows), uint32_t(q.n) * p.group.d - uint32_t(t) * kRows));
            it.whole = from == 0 && to == blocks;
            it.head = from > 0;
            left -= take;
            off = 0;
            ++t;
            if (to > from) return true;
        }
        return false;
    }
};

// The places [lo, hi) that row r of an item sees, its token and query head.
struct RowOf {
    int token, head, lo, hi;
};

template <int kRows>
__host__ __device__ __forceinline__ RowOf row_of(const AttnParams &p, const Item &it, int r) {
    const uint32_t g = uint32_t(it.t) * kRows + uint32_t(r), i = udiv(g, p.group);
    RowOf o;
    o.token = it.q.lo + int(i);
    o.head = it.h * int(p.group.d) + int(g - i * p.group.d);
    const int place = it.q.len - it.q.n + int(i);
    o.hi = p.causal ? min(max(place + 1, 0), it.q.len) : it.q.len;
    o.lo = p.window ? max(place - p.window + 1, 0) : 0;
    if (r >= it.rows) o.hi = o.lo = 0;
    return o;
}

// A slot of partial results: [head_dim / 4][kRows] vectors of sums, then the
// rows' maxima and sums.
template <int kRows>
__host__ __device__ inline int64_t slot_floats(int head_dim) { return int64_t(kRows) * (((head_dim + 3) & ~3) + 2); }

template <int kRows>
__device__ __forceinline__ float *slot_of(const AttnParams &p, int part, bool head) {
    return p.partial + (2 * int64_t(part) + (head ? 0 : 1)) * slot_floats<kRows>(p.head_dim);
}

__device__ __forceinline__ void write_note(const AttnParams &p, int part, const Start &st) {
    PartNote n;
    n.begin = st.begin;
    n.end = st.end;
    n.item = st.item;
    n.cost = st.cost;
    n.s = st.s;
    n.h = st.h;
    n.t = st.t;
    n.pad = 0;
    p.notes[part] = n;
}

constexpr int kFewRows = 16;     // rows of an item of the kernel for few rows
constexpr int kTileRows = 128;   // rows of an item of one block on the tensor cores
constexpr int kPairRows = 256;   // rows of an item of a pair of blocks
constexpr int kTileParts = 152;  // parts of the line for single blocks: the GB300's SMs
constexpr int kPairParts = 76;   // and for pairs

// Launches of rope3d_paged_tc.cu: items of kTileRows, or of kPairRows.
int launch_tiles(const AttnParams &p, const rope3d_paged_attention_args &a, bool pair, cudaStream_t st);
bool tiles_fit(const rope3d_paged_attention_args &a);
bool pairs_fit(const rope3d_paged_attention_args &a);
int tiles_wait_timeouts(unsigned int *count, bool reset);

}  // namespace rope3d_paged
