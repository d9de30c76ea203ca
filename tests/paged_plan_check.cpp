// Host check of the paged attention's division of work (csrc/paged_walk.cuh): reads
// "tokens block grid start_cost snap whole least Hkv causal window n" and n pairs "q_len kv_len",
// plays the plan kernel, and checks every range.  Prints "ok <ranges> <longest> <mean>"
// (cost of the longest range and the mean) or the first fault found.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <tuple>
#include <vector>

#include "paged_walk.cuh"

using namespace xs;

static void fault(const char* what, long long a, long long b) {
    std::printf("%s %lld %lld\n", what, a, b);
    std::exit(1);
}

int main() {
    PagedTiling g;
    int Hkv, causal, window, n;
    while (std::scanf("%d %d %d %d %d %d %d %d %d %d %d", &g.tokens, &g.block, &g.grid, &g.start_cost, &g.snap, &g.whole,
                      &g.least, &Hkv, &causal, &window, &n) == 11) {
        std::vector<PagedSeq> seqs;
        for (int i = 0; i < n; ++i) {
            PagedSeq s{0, 0, 0, i};
            if (std::scanf("%d %d", &s.q_len, &s.kv_len) != 2) fault("input", i, 0);
            if (s.q_len > 0) seqs.push_back(s);
        }
        const int kept = static_cast<int>(seqs.size());
        std::vector<long long> prefix(kept + 1, 0);
        for (int i = 0; i < kept; ++i) {
            // the closed form against the sum over tiles
            long long sum = 0;
            const int tiles = paged_tiles(seqs[i], g.tokens);
            for (int t = 0; t < tiles; ++t) {
                if (paged_cost(seqs[i], t, g, causal, window) != sum) fault("cost", i, t);
                int lo, hi, b0, nb;
                paged_tile_keys(seqs[i], t, g.tokens, causal, window, lo, hi);
                paged_tile_blocks(seqs[i], t, g, causal, window, b0, nb);
                if (lo < 0 || hi <= lo || nb < 1) fault("tile", i, t);
                // brute force over the tile's rows
                long long rlo = 1ll << 40, rhi = 0;
                for (int j = t * g.tokens; j < (t + 1) * g.tokens && j < seqs[i].q_len; ++j) {
                    const long long p = static_cast<long long>(seqs[i].kv_len) - seqs[i].q_len + j;
                    const long long h = causal ? p + 1 : seqs[i].kv_len;
                    const long long l = window > 0 && p - window + 1 > 0 ? p - window + 1 : 0;
                    if (h > l) {
                        if (l < rlo) rlo = l;
                        if (h > rhi) rhi = h;
                    }
                }
                if (rhi > 0 && (rlo < lo || rhi > hi)) fault("keys", i, t);
                sum += hi - lo + g.start_cost;
            }
            if (paged_cost(seqs[i], tiles, g, causal, window) != sum) fault("cost", i, tiles);
            prefix[i + 1] = prefix[i] + Hkv * sum;
        }
        const long long total = prefix[kept];
        long long all_tiles = 0;
        for (const PagedSeq& s : seqs) all_tiles += static_cast<long long>(Hkv) * paged_tiles(s, g.tokens);
        long long ranges = total / g.least;
        if (ranges < all_tiles) ranges = all_tiles;
        if (ranges > g.grid) ranges = g.grid;
        if (ranges > total / (2 * g.block)) ranges = total / (2 * g.block);
        if (ranges < 1) ranges = kept > 0 ? 1 : 0;
        std::vector<PagedPos> cut(ranges + 1);
        for (int c = 0; c <= ranges && ranges > 0; ++c) {
            PagedPos p{kept, 0, 0, 0};
            if (c == 0) p.seq = 0;
            if (c > 0 && c < ranges) {
                const long long x = total / ranges * c + total % ranges * c / ranges;   // (without waves)
                int i = 0;
                while (prefix[i + 1] <= x) ++i;
                p = paged_locate(seqs[i], i, x - prefix[i], (prefix[i + 1] - prefix[i]) / Hkv, g, Hkv, causal, window);
            }
            cut[c] = p;
        }
        // walk every range as the attention kernels do
        std::map<std::tuple<int, int, int>, std::vector<std::tuple<int, int, int>>> pieces;   // tile -> (k0, k1, cta)
        double longest = 0, all = 0;
        for (int c = 0; c < ranges; ++c) {
            const PagedPos end = cut[c + 1];
            if (paged_before(end, cut[c])) fault("order", c, 0);
            double cost = 0;
            for (PagedPos p = cut[c]; paged_before(p, end);) {
                if (p.seq >= kept) fault("past the end", c, p.seq);
                const PagedSeq& s = seqs[p.seq];
                int b0, count;
                paged_tile_blocks(s, p.tile, g, causal, window, b0, count);
                const bool cut_end = paged_same_tile(p, end);
                const int k1 = cut_end && end.k < count ? end.k : count;
                if (k1 <= p.k) fault("empty piece", c, p.k);
                pieces[{p.seq, p.head, p.tile}].push_back({p.k, k1, c});
                cost += (k1 - p.k) * g.block + g.start_cost;
                if (cut_end) break;
                paged_next(p, s, g.tokens, Hkv);
            }
            all += cost;
            if (cost > longest) longest = cost;
        }
        long long tiles = 0;
        for (int i = 0; i < kept; ++i) tiles += static_cast<long long>(Hkv) * paged_tiles(seqs[i], g.tokens);
        if (tiles != static_cast<long long>(pieces.size())) fault("tiles", tiles, pieces.size());
        auto first_at = [&](const PagedPos& p) {
            int c = 0;
            while (c < ranges && paged_before(cut[c], p)) ++c;
            return c;
        };
        for (auto& kv : pieces) {
            int i, h, t, b0, count, at = 0;
            std::tie(i, h, t) = kv.first;
            paged_tile_blocks(seqs[i], t, g, causal, window, b0, count);
            int cta = std::get<2>(kv.second[0]);
            const int c_first = cta, c_last = std::get<2>(kv.second.back());
            for (auto& p : kv.second) {
                if (std::get<0>(p) != at || std::get<2>(p) != cta) fault("pieces", i, t);   // no CTA between has none
                // what the range record says of the tile's CTAs
                PagedPos q{i, h, t, 1};
                if (at > 0 && first_at(q) - 1 != c_first) fault("c0", i, cta);
                q.k = 0x7fffffff;
                if ((at > 0 || cta != c_last) && first_at(q) - 1 != c_last) fault("c1", i, cta);
                at = std::get<1>(p);
                ++cta;
            }
            if (at != count) fault("end", i, t);
        }
        std::printf("ok %lld %.0f %.0f\n", ranges, longest, ranges ? all / ranges : 0.0);
    }
    return 0;
}
