// Walks the stretches of all blocks of one paged-attention call on the host,
// with the kernel's own arithmetic (csrc/w4_attn_plan.cuh), and checks that
// they are in order, take every record once and agree on the pieces to join.
// Returns 0, or what is wrong (see test_attn_division.py).
#include "w4_attn_plan.cuh"

#include <vector>

using namespace w4;

namespace {

struct Written {                       // what a block leaves in one of its two slots
    int b = -1, item = -1;
};

}  // namespace

extern "C" int walk(int D, int record_bytes, int group, int kv_heads, int tokens, int window,
                    int seqs, const int *lens, int sms, int *shape) {
    const int rows = tokens * group, NT = tiles_a_warp(D, rows);
    const Plan plan = plan_of(D, NT, rows, record_bytes);
    const int grid = sms < kMaxGrid ? sms : kMaxGrid;
    if (plan.KG < 1 || plan.stages < 3 || plan.QG * plan.KG > compute_warps(D, NT) ||
        8 * NT * plan.QG * plan.row_tiles < rows || 8 * NT * plan.QG > kRowsMax)
        return 1;                      // a plan that does not hold the rows or three records
    Division d;
    d.extra = plan.extra;
    d.per_seq = kv_heads * plan.row_tiles;
    std::vector<int> records(seqs), before(seqs + 1, 0);
    long long longest = 0;
    for (int b = 0; b < seqs; ++b) {
        records[b] = seen_records(lens[b], tokens, window).records;
        before[b + 1] = before[b] + (records[b] + d.extra) * d.per_seq;
        if ((lens[b] + 15) / 16 > longest) longest = (lens[b] + 15) / 16;
    }
    d.divide(plan, seqs, before[seqs], grid);
    if (shape) shape[0] = d.blocks, shape[1] = plan.KG, shape[2] = d.least, shape[3] = d.extra;
    const auto cut = [&](int u) {
        for (int b = 0; b < seqs; ++b)
            if (u >= before[b] && u < before[b + 1])
                return d.cut_inside(b, u - before[b], records[b]);
        return Cut{seqs, 0, 0};
    };

    std::vector<std::vector<int>> taken(seqs * d.per_seq);
    for (int b = 0; b < seqs; ++b)
        for (int i = 0; i < d.per_seq; ++i) taken[b * d.per_seq + i].assign(records[b] + 1, 0);
    std::vector<Written> slot(2 * grid);
    std::vector<int> pieces(grid, 0), started(grid, -1);
    bool any_cut = false;
    for (int block = 0; block < d.blocks; ++block) {
        Cut c = cut(d.start(block));
        const Cut to = cut(d.start(block + 1));
        int starts = 0, goes_on = 0;
        while (has_more(c, to, seqs)) {
            if (c.b < 0 || c.b >= seqs || c.item < 0 || c.item >= d.per_seq) return 2;   // outside
            const int n = records[c.b], item = c.b * d.per_seq + c.item;
            const bool last = c.b == to.b && c.item == to.item;
            const int stop = last ? to.u : n;
            if (c.u < 0 || stop > n || (n > 0 && c.u >= stop)) return 3;   // an empty piece
            for (int u = c.u; u < stop; ++u) ++taken[item][u];
            ++taken[item][n];          // visits
            if (c.u > 0 || stop != n) {
                any_cut = true;
                slot[2 * block + (c.u == 0)] = {c.b, c.item};
                if (c.u == 0 ? starts++ : goes_on++) return 4;             // a slot used twice
                if (c.u == 0)
                    started[block] = item,
                    pieces[block] = d.pieces(before[c.b] + c.item * (n + d.extra), n);
            }
            if (last)
                c = to;
            else
                d.advance(c);
        }
    }
    int joined = 0;
    for (int block = 0; block < grid; ++block)
        for (int x = 0; x < pieces[block]; ++x) {
            if (block + x >= grid) return 5;                               // past the workspace
            const Written &w = slot[2 * (block + x) + (x == 0)];
            if (w.b * d.per_seq + w.item != started[block]) return 6;      // another head's piece
            ++joined;
        }
    int written = 0;
    for (const Written &w : slot) written += w.b >= 0;
    if (joined != written) return 7;                                       // a piece is left over
    for (int b = 0; b < seqs; ++b)
        for (int i = 0; i < d.per_seq; ++i) {
            const auto &t = taken[b * d.per_seq + i];
            for (int u = 0; u < records[b]; ++u)
                if (t[u] != 1) return 8;                                   // left out, or twice
            if (t[records[b]] < 1) return 9;                               // a head never visited
        }
    if (any_cut && nothing_to_join(plan, seqs, kv_heads, longest, grid)) return 10;
    return 0;
}
