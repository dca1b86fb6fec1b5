// The division of the attention over pages (rope3d_paged.cuh) run on the host against
// brute force: the cost of every tile from what its rows see, the line's cuts in 128 bits,
// where each part begins, and the items that every part walks. Prints how often each
// branch of the arithmetic was taken; ends with 1 and a message where something differs.
//
//     paged_line <seed> <calls of each kind>
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <string>
#include <vector>

#include "rope3d_paged.cuh"

using namespace rope3d_paged;
typedef long long ll;
typedef __int128 lll;

static std::mt19937_64 rng;
static std::map<std::string, ll> taken;

static ll pick(ll lo, ll hi) { return lo + ll(rng() % uint64_t(hi - lo + 1)); }
template <typename T> static T one_of(std::initializer_list<T> v) { return v.begin()[rng() % v.size()]; }

#define EXPECT(x)                                                        \
    do {                                                                 \
        if (!(x)) {                                                      \
            std::printf("line %d: %s\n", __LINE__, #x);                  \
            std::exit(1);                                                \
        }                                                                \
    } while (0)

struct Call {
    std::vector<int> lens, starts;
    bool given;   // starts
    int width, page, tokens, heads, group, parts, item_cost, causal, window;
};

struct Want {
    int s, h, t, rows;
    ll k0, k1, b0, b1, at;   // at: where it begins on the line
    ll blocks() const { return std::max<ll>(b1 - b0, 1); }
};

// What the rows of tile t see, from the definition.
template <int kRows, int kKeys>
static Want tile_by_rows(const Call &c, int s, int h, int t, ll n, ll len) {
    Want w{s, h, t, 0, 0, 0, 0, 0, 0};
    const ll rows = n * c.group, g0 = ll(t) * kRows, g1 = std::min<ll>(rows, g0 + kRows);
    w.rows = int(g1 - g0);
    bool any = false;
    for (ll i = g0 / c.group; i <= (g1 - 1) / c.group; ++i) {
        const ll place = len - n + i;
        const ll hi = c.causal ? std::min(std::max<ll>(place + 1, 0), len) : len, lo = c.window ? std::max<ll>(place - c.window + 1, 0) : 0;
        if (lo >= hi) continue;
        w.k0 = any ? std::min(w.k0, lo) : lo;
        w.k1 = any ? std::max(w.k1, hi) : hi;
        any = true;
    }
    w.b0 = w.k0 / kKeys;
    w.b1 = any ? (w.k1 + kKeys - 1) / kKeys : w.b0;
    return w;
}

template <int kRows, int kKeys, int kThreads>
static void check(const Call &c) {
    const int seqs = int(c.lens.size());
    AttnParams p{};
    std::vector<int> table(1, 0);
    p.batch = Batch{table.data(), c.lens.data(), c.given ? c.starts.data() : nullptr, c.width, seqs, c.width, 1 << 20, c.page, c.tokens};
    p.group = rope3d::make_fastdiv(uint32_t(c.group));
    p.page = rope3d::make_fastdiv(uint32_t(c.page));
    p.span = rope3d::make_fastdiv(uint32_t(c.group) * (kKeys / kRows));
    p.cuts = rope3d::make_fastdiv(uint32_t(c.parts));
    p.item_cost = c.item_cost;
    p.kv_heads = c.heads;
    p.causal = c.causal;
    p.window = c.window;
    p.parts = c.parts;

    // the line, item by item
    std::vector<Want> line;
    std::vector<ll> costs(seqs, 0);
    std::vector<Seq> of(seqs);
    ll total = 0;
    for (int s = 0; s < seqs; ++s) {
        const ll len = std::min<ll>(std::max(c.lens[s], 0), ll(c.width) * c.page);
        ll lo = ll(s) * (c.tokens / seqs), hi = lo + c.tokens / seqs;
        if (c.given) {
            lo = std::min<ll>(std::max(c.starts[s], 0), c.tokens);
            hi = std::min<ll>(std::max<ll>(c.starts[s + 1], lo), c.tokens);
        }
        const ll n = hi - lo, tiles = (n * c.group + kRows - 1) / kRows;
        const Seq q = of[s] = seq_of<kRows>(p, s);
        EXPECT(q.lo == lo && q.n == n && q.len == len && q.tiles == tiles);
        std::vector<Want> head;
        std::vector<ll> prefix(1, 0);
        for (ll t = 0; t < tiles; ++t) {
            head.push_back(tile_by_rows<kRows, kKeys>(c, s, 0, int(t), n, len));
            const Want &w = head.back();
            const Tile got = tile_of<kRows, kKeys>(p, q, int(t));
            EXPECT(got.blocks() == w.blocks());
            if (w.b1 > w.b0) EXPECT(got.k0 == w.k0 && got.k1 == w.k1 && got.b0 == w.b0 && got.b1 == w.b1);
            else EXPECT(got.k0 >= got.k1 && got.b0 >= got.b1);
            prefix.push_back(prefix.back() + w.blocks() + c.item_cost);
        }
        costs[s] = prefix.back();
        EXPECT((seq_cost<kRows, kKeys>(p, q)) == prefix.back());
        if (tiles > 1) {   // the closed form, at every tile
            const Costs<ll, kRows, kKeys> wide(p, q);
            const bool small = small_costs(p, q);
            ++taken[std::string(small ? "32 bits" : "64 bits") + (c.window ? ", window" : "") + (c.causal ? ", causal" : "")];
            for (ll t = 0; t < tiles; ++t) EXPECT(wide.at(p, int(t)) == prefix[t]);
            if (small) {
                const Costs<int, kRows, kKeys> narrow(p, q);
                for (ll t = 0; t < tiles; ++t) EXPECT(narrow.at(p, int(t)) == prefix[t]);
            }
            for (int i = 0; i < 20; ++i) {
                const ll in = pick(0, prefix.back() - 1);
                ll begins;
                const int t = wide.find(p, int(tiles), in, begins);
                EXPECT(prefix[t] <= in && in < prefix[t + 1] && begins == prefix[t]);
            }
            if (prefix.back() >= 0x7fffffff) ++taken["heads of 2^31"];
        }
        for (int h = 0; h < c.heads; ++h)
            for (ll t = 0; t < tiles; ++t) {
                Want w = head[t];
                w.h = h;
                w.at = total + h * prefix.back() + prefix[t];
                line.push_back(w);
            }
        total += prefix.back() * c.heads;
    }
    ++taken[total < (1 << 21) ? "lines below 2^21" : total < 0x7fffffff ? "lines below 2^31" : "lines of 2^31"];

    struct Piece {
        int part;
        ll from, to;
        bool head, whole;
    };
    std::vector<std::vector<Piece>> done(line.size());
    std::vector<ll> begins(c.parts), ends(c.parts);
    const int each = (seqs + kThreads - 1) / kThreads;
    for (int part = 0; part < c.parts; ++part) {
        // what find_start's threads do, one after the other
        const ll begin = cut(p, total, part), stop = cut(p, total, part + 1);
        EXPECT(begin == ll(lll(total) * part / c.parts) && stop == ll(lll(total) * (part + 1) / c.parts));
        begins[part] = begin;
        ends[part] = stop;
        Start st{};
        st.s = -1;
        int found = 0;
        ll before = 0;
        for (int tid = 0; tid < kThreads; ++tid) {
            const int first = std::min(tid * each, seqs), end = std::min(first + each, seqs);
            Seq q{0, 0, 0, 0};
            ll sum = 0, head = 0;
            for (int s = first; s < end; ++s) {
                q = of[s];
                head = costs[s];   // (seq_cost's, as seen above)
                sum += head * c.heads;
            }
            const int was = st.s;
            st.s = -1;
            start_among<kRows, kKeys>(p, first, end, q, before, sum, head, begin, stop, &st);
            if (st.s >= 0) ++found;
            else st.s = was;
            before += sum;
        }
        EXPECT(found == (begin < stop ? 1 : 0));
        st.begin = begin;
        st.end = stop;
        size_t i = line.size();
        if (found) {
            i = size_t(std::upper_bound(line.begin(), line.end(), begin, [](ll v, const Want &w) { return v < w.at; }) - line.begin()) - 1;
            EXPECT(st.s == line[i].s && st.h == line[i].h && st.t == line[i].t && st.item == line[i].at);
            EXPECT(st.off == begin - line[i].at && st.cost == line[i].blocks() + c.item_cost);
        }
        Walker<kRows, kKeys> walk(p, st);
        Item it;
        while (walk.next(it)) {
            while (i < line.size() && (line[i].s != it.s || line[i].h != it.h || line[i].t != it.t)) ++i;
            EXPECT(i < line.size());
            const Want &w = line[i];
            EXPECT(it.rows == w.rows && it.q.lo == of[it.s].lo);
            // a piece of the item: its blocks from..to (an item without keys has one that is empty)
            const ll from = std::max<ll>(begin - w.at - c.item_cost, 0), to = std::min<ll>(stop - w.at - c.item_cost, w.blocks());
            EXPECT(to > from);
            if (w.b1 > w.b0) EXPECT(it.begin == w.b0 + from && it.end == w.b0 + to);
            else EXPECT(it.begin >= it.end && it.whole && !it.head);
            done[i].push_back(Piece{part, from, to, it.head, it.whole});
            for (int r = 0; r < it.rows; r += std::max(1, it.rows - 1)) {   // the first row and the last
                const RowOf o = row_of<kRows>(p, it, r);
                const ll g = ll(it.t) * kRows + r, place = of[it.s].len - of[it.s].n + g / c.group;
                EXPECT(o.token == of[it.s].lo + g / c.group && o.head == it.h * c.group + g % c.group);
                EXPECT(o.hi == (c.causal ? std::min<ll>(std::max<ll>(place + 1, 0), of[it.s].len) : of[it.s].len));
                EXPECT(o.lo == (c.window ? std::max<ll>(place - c.window + 1, 0) : 0));
            }
        }
    }
    // every item's blocks once and in order; the parts of a divided one as the joining kernel lists them
    for (size_t i = 0; i < line.size(); ++i) {
        const Want &w = line[i];
        ll next = 0;
        for (const Piece &d : done[i]) {
            EXPECT(d.from == next && d.head == (d.from > 0) && d.whole == (d.from == 0 && d.to == w.blocks()));
            next = d.to;
        }
        EXPECT(next == w.blocks());
        if (done[i].size() < 2) continue;
        ++taken["divided items"];
        const ll first = w.at + c.item_cost;
        std::vector<int> want(1, 0);
        const int near = int(std::lower_bound(begins.begin(), begins.end(), w.at) - begins.begin());
        for (int q = 0; q < c.parts && begins[q] <= first; ++q)
            if (begins[q] < ends[q]) want[0] = q;
        for (int q = std::max(near - 1, 0); q < c.parts && begins[q] < w.at + w.blocks() + c.item_cost; ++q)
            if (begins[q] > first && begins[q] < ends[q]) want.push_back(q);
        EXPECT(want.size() == done[i].size());
        for (size_t k = 0; k < want.size(); ++k) EXPECT(want[k] == done[i][k].part && done[i][k].head == (k > 0));
    }
}

static void check(int kind, const Call &c) {
    if (kind == 0) check<16, 64, 128>(c);
    else if (kind == 1) check<128, 128, 512>(c);
    else check<256, 256, 512>(c);
}

static Call call(int kind, int seqs, ll most_new, ll most_len, int group, int heads) {
    Call c;
    c.group = group;
    c.heads = heads;
    c.page = one_of<int>({1, 5, 8, 16, 128});
    c.causal = rng() % 3 != 0;
    c.window = one_of<int>({0, 0, 0, 1, 5, 64, int(pick(1, most_len + 1)), int(std::min<ll>(2 * most_len, 1 << 30))});
    c.parts = one_of<int>({1, 2, 7, kind == 0 ? int(pick(1, 456)) : int(pick(1, 152)), kind == 0 ? 456 : kind == 1 ? kTileParts : kPairParts});
    c.item_cost = int(pick(0, 3));
    c.given = rng() % 4 != 0;
    c.width = int((most_len + c.page - 1) / c.page);
    int at = 0;
    const int same = int(pick(1, most_new));
    for (int s = 0; s < seqs; ++s) {
        const int n = c.given ? one_of<int>({0, 1, int(pick(1, most_new)), int(pick(1, most_new)), int(most_new)}) : same;
        c.starts.push_back(at);
        at += n;
        // longer than the new tokens, as long, shorter, empty, damaged
        c.lens.push_back(one_of<int>({int(std::min<ll>(n + pick(0, most_len), most_len)), int(std::min<ll>(n + pick(0, most_len), most_len)), n,
                                      int(pick(0, n)), int(most_len), rng() % 8 ? n : one_of<int>({-5, 0x7fffffff})}));
    }
    c.starts.push_back(at);
    c.tokens = std::max(at, 1) + (c.given ? int(pick(0, 3)) : 0);
    if (c.given && rng() % 8 == 0)   // damaged starts
        for (int k = 0; k < 2; ++k) c.starts[rng() % c.starts.size()] = one_of<int>({-3, 0x7fffffff, int(pick(0, c.tokens)), 0});
    return c;
}

int main(int argc, char **argv) {
    rng.seed(argc > 1 ? strtoull(argv[1], nullptr, 10) : 1);
    const int count = argc > 2 ? atoi(argv[2]) : 100;
    // divisions: n / d for n below 2^31, and sums of floors past 32 bits
    for (int i = 0; i < 200 * count; ++i) {
        const uint32_t d = uint32_t(one_of<ll>({pick(1, 5000), pick(1, 0x7fffffff), ll(1) << pick(0, 30)}));
        const uint32_t n = uint32_t(one_of<ll>({pick(0, 0x7fffffff), 0x7fffffff, ll(d) - 1, std::min<ll>(ll(d) * pick(0, 9), 0x7fffffff)}));
        const auto f = rope3d::make_fastdiv(d);
        EXPECT(udiv(n, f) == n / d);
        if (d > (1u << 20)) continue;
        const ll m = one_of<ll>({pick(0, 1 << 15), pick(0, ll(1) << 34), 0x7ffffffe, 0x7fffffff, 0x80000000ll}), q = m / d;
        const lll want = lll(q) * (q - 1) / 2 * d + lll(q) * (m - q * d);
        if (want < (lll(1) << 62)) EXPECT(floors<ll>(m, f) == ll(want));
    }
    // cuts of lines of any length
    for (int i = 0; i < 200 * count; ++i) {
        AttnParams p{};
        p.parts = int(pick(1, 456));
        p.cuts = rope3d::make_fastdiv(uint32_t(p.parts));
        const ll base = one_of<ll>({1 << 21, 0x7fffffff, ll(1) << 40, pick(0, ll(1) << 50), pick(0, 1 << 22)});
        const ll total = std::max<ll>(base + pick(-3, 3), 0);
        const int part = int(one_of<ll>({0, p.parts, pick(0, p.parts)}));
        EXPECT(cut(p, total, part) == ll(lll(total) * part / p.parts));
    }
    for (int i = 0; i < count; ++i)
        for (int kind = 0; kind < 3; ++kind) {
            const int group = one_of<int>({1, 2, 3, 4, 6, 7, 8, 16, 40, 63, 64, 200});
            check(kind, call(kind, int(pick(1, 40)), one_of<ll>({1, 2, 40, 700}), one_of<ll>({3, 300, 5000}), group, int(pick(1, 4))));
            if (i % 4 == 0) check(kind, call(kind, int(pick(400, 3000)), one_of<ll>({1, 3, 30}), one_of<ll>({40, 3000}), group, int(pick(1, 3))));
            // about the border between 32 and 64 bits: 2^17 rows
            const ll border = (1 << 17) / group;
            check(kind, call(kind, int(pick(1, 3)), std::max<ll>(border + pick(-2, 2), 1), border + pick(-2, 2) + one_of<ll>({0, 0, border}), group, 1));
            if (i % 4 == 1)
                check(kind, call(kind, int(pick(1, 4)), one_of<ll>({1, 17, 900}), pick(1 << 17, 1 << 23), one_of<int>({group, 1, 2}), int(pick(1, 20))));
            // long lines: many rows over far places
            if (i % 10 == 2) check(kind, call(kind, 1, pick(1 << 15, 1 << 17), pick(1 << 18, 1 << 24), one_of<int>({8, 16, 70}), int(pick(1, 2))));
            if (i % 10 == 7) check(kind, call(kind, 2, pick(1, 1 << 12), (ll(1) << 30) - pick(0, 5), one_of<int>({1, 16, 100}), 1));
        }
    for (const auto &t : taken) std::printf("%s: %lld\n", t.first.c_str(), t.second);
    return 0;
}
