// How the paged attention divides its work: what a launch chooses on the host,
// and which records of which heads each block takes.  Integer arithmetic alone
// and no CUDA header, so that tests compile it for the host and walk every
// block's stretch there.  Internal to libw4.
#pragma once

#ifdef __CUDACC__
#define W4_HD __host__ __device__ __forceinline__
#else
#define W4_HD inline
#endif

namespace w4 {

constexpr int kRecTokens = 16;         // tokens of a record = keys of one tensor-core tile
constexpr int kRowsMax = 64;           // rows of a block
// What a head's start and end cost, in records of one tile of rows.  Ragged
// batches: 64 x 8k int8 64 us at 0, 50.8 at 28, 49.7 at 40, 50.5 at 56; 8 new
// tokens over 8 x 8k bf16 44.1, 33.8, 30.4, 30.7; 64 x 8k int4 57.6, 43.6, 41.4,
// 40.2; even ones lose a little (8 x 2k bf16 12.0, 13.5, 12.6, 12.7).  One number
// for all formats: the three ragged ones want about the same.
constexpr int kHeadRecords = 40;
constexpr int kMaxStages = 16;         // of one group's ring
constexpr int kMaxGrid = 256;
constexpr int kSharedBytes = 224256;   // rings and join: 219 of the 227 KB of a block

// Warps that compute, of NT row tiles each; with the two that copy 20 of 96
// registers, 16 of 128 or 12 of 168, by the values that a warp holds.
constexpr int kCopyWarps = 2;
W4_HD constexpr int compute_warps(int D, int NT) {
    return D * NT == 64 ? 18 : D * NT == 128 ? 14 : 10;
}

// Two tiles a warp where that makes a third as many groups again: the operands
// of a record serve both tiles, but fewer warps are there to wait.  Measured, in
// us with one and with two tiles a warp:
//   tiles               2           3           4           5           6           7
//   48 x 4 k of 64
//     bf16                  -       27.9, 29.3  36.1, 29.7  42.3, 39.1      -       54.0, 48.5
//     4 bits           24.9, 20.7  29.3, 28.7  38.1, 28.9  45.0, 37.6      -       55.9, 47.3
//   8 x 8 k of 128
//     bf16             30.6, 31.4  31.1, 33.9  35.4, 34.2  43.1, 45.0  46.2, 45.8  48.8, 55.4
//   32 x 4 k of 128
//     4 bits           38.8, 33.4  53.2, 51.5  68.0, 52.0  85.4, 75.2  92.7, 76.7  101.8, 95.7
//     8 bits                -       51.4, 55.7      -       81.0, 80.9      -       98.8, 97.7
// The rule is bf16's; 4-bit caches, whose conversion a second tile shares, would
// gain by two from 2 tiles on, and at 7 of 128.
inline int tiles_a_warp(int D, int rows) {
    const int tiles = (rows < kRowsMax ? rows + 7 : kRowsMax) / 8;
    const int one = compute_warps(D, 1) / tiles, two = compute_warps(D, 2) / ((tiles + 1) / 2);
    return tiles > 2 && 3 * two >= 4 * one ? 2 : 1;
}

// How a launch divides a block.
struct Plan {
    int row_tiles;     // blocks of rows per key/value head
    int QG, KG;        // warps on a record, groups of them
    int stages;        // records of a group's ring
    int ring_bytes;    // of all rings
    int extra;         // what a head costs beside its records
    int part;          // records of a group that a part of a head has at least
    int least;         // records that are not cut off a head
};

constexpr int kPart = 4;               // of the whole attention

// Of listed blocks, whose lists are short: how many records a part has costs more or
// less latency.  Measured, in us with 4, 3, 2, 1 records a group: 64 blocks of one
// sequence, of 64 tokens in bf16 10.2, 10.5, 10.9, 10.9, in 4 bits 12.6, 12.1, 10.3,
// 11.1, of 32 tokens in bf16 of 64 11.3, 11.3, 9.7, 8.9; of four sequences in 8 bits
// 13.8, 13.5, 12.1, 11.2; of two with 4 new tokens in bf16 15.5, 14.2, 14.1, 14.8; 64
// of 4096 tokens in 8 bits 50.7 whatever it is.  One sequence's short lists, where two
// records cut a head and four do not: 80 records in 4 bits 11.5 and 10.8, 111 12.1 and
// 12.6, 103 in 8 bits 11.9 and 12.1, 39 for 4 new tokens 13.2 and 14.7, 143 of 64 in 4
// bits 10.2 and 12.0.
inline int listed_part(bool bf16, int D) { return bf16 && D == 128 ? 3 : 2; }

inline Plan plan_of(int D, int NT, int rows, int record_bytes, int part = kPart) {
    const int warps = compute_warps(D, NT);
    const int tiles = (rows + 8 * NT - 1) / (8 * NT), most = kRowsMax / (8 * NT);
    Plan p;
    p.row_tiles = (tiles + most - 1) / most;
    p.QG = (tiles + p.row_tiles - 1) / p.row_tiles;
    // groups: as many as the warps allow with three records in a ring
    const int join_row = 8 * NT * p.QG * (D + 4) * 4;
    p.KG = warps / p.QG;
    while (p.KG > 1 && p.KG * (join_row + 3 * record_bytes) > kSharedBytes) --p.KG;
    p.stages = (kSharedBytes - p.KG * join_row) / (p.KG * record_bytes);
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    p.ring_bytes = p.KG * p.stages * record_bytes;
    p.extra = kHeadRecords / ((p.QG * NT + 1) / 2);
    p.part = part;
    p.least = p.KG > p.extra / 2 ? p.KG : p.extra / 2;
    return p;
}

// Whether no head of a call of one sequence is cut, however few of the records that
// there is room for it has, so that there is nothing to join.  By Division::divide a
// head makes k parts from k * part * KG records on; by Division::cut_inside the last of
// its cuts, at (k - 1) / k of what it costs, stays in it if `least` records are ahead
// of it.
inline bool nothing_to_join(const Plan &p, int seqs, int kv_heads, long long table_records,
                            int grid) {
    const long long heads = (long long)kv_heads * p.row_tiles, each = (long long)p.part * p.KG;
    if (seqs != 1 || heads > grid) return false;
    for (long long k = 2; k * each <= table_records; ++k) {
        const long long cut = (k * (p.least + p.extra) + k - 2) / (k - 1) - p.extra;
        const long long first = cut > k * each ? cut : k * each;
        if (k * heads > grid || (first < (k + 1) * each && first <= table_records)) return false;
    }
    return true;
}

// The records of a sequence that a call looks at.
struct Seq {
    int len;           // visible tokens
    int first;         // first record with a visible key
    int records;       // records from there on (0: none)
};

W4_HD Seq seen_records(int len, int tokens, int window) {
    Seq s;
    s.len = len;
    const long long lo = (long long)len - tokens + 1 - window;
    s.first = window > 0 && lo > 0 ? (int)(lo / kRecTokens) : 0;
    s.records = (len + kRecTokens - 1) / kRecTokens - s.first;
    return s;
}

// A place in the list of records (the host refuses lists of 2^31).
struct Cut {
    int b, item, u;        // sequence, head (x row tile) of it, record of that
};

// Whether there is anything from c on that a block whose stretch ends at `to`
// takes (in the list's order; never past the last sequence).
W4_HD bool has_more(const Cut &c, const Cut &to, int seqs) {
    if (c.b >= seqs) return false;
    if (c.b != to.b) return c.b < to.b;
    return c.item != to.item ? c.item < to.item : c.u < to.u;
}

// The list (sequence, head, record), an item costing its records and `extra`,
// cut into stretches of like cost.
struct Division {
    int extra, per_seq;    // heads (x row tiles) of a sequence
    int work;              // what all items cost
    int blocks, least;     // blocks that have a stretch; as the plan has it
    int q, rest;           // work / blocks and its remainder
    unsigned magic;        // 2^32 / blocks, rounded up

    // As many blocks as heads, or that many times the parts of at least `part`
    // records a group that the mean head has (so heads of one length are cut
    // alike), while there are blocks.
    W4_HD void divide(const Plan &plan, int seqs, int all, int grid) {
        work = all;
        const int heads = seqs * per_seq, parts = (work / heads - extra) / (plan.part * plan.KG);
        const int want = heads * (parts > 1 ? parts : 1);
        blocks = grid < want ? grid : want;
        q = work / blocks, rest = work - q * blocks;
        magic = 0xFFFFFFFFu / (unsigned)blocks + 1;
        least = plan.least;
    }

    // Start of block c's stretch.  rest * c < 2^16, so the product with magic
    // gives rest * c / blocks exactly (blocks = 1: rest is 0).
    W4_HD int start(int c) const {
        return q * c + (int)(((unsigned long long)(unsigned)(rest * c) * magic) >> 32);
    }

    // The cut at cost `in` of sequence b's items, each of `records` records;
    // moved to its head's border where fewer than `least` records would be cut
    // off: the border on that side, or in a head too short for a cut the nearer
    // one.  Both ways a later `in` gives no earlier cut, which is what makes the
    // blocks' stretches follow one another.
    W4_HD Cut cut_inside(int b, int in, int records) const {
        const int n = records + extra;
        Cut c;
        c.b = b, c.item = in / n, c.u = in - c.item * n - extra;
        const bool to_end =
            records < 2 * least ? 2 * (c.u + extra) > n : records - c.u < least;
        if (to_end)
            advance(c);
        else if (records < 2 * least || c.u < least)
            c.u = 0;
        return c;
    }

    // First block c with start(c) >= u (u > 0).
    W4_HD int block_from(int u) const {
        int c = (int)((float)u * ((float)blocks / (float)work));
        if (c > blocks) c = blocks;
        while (c > 0 && start(c) >= u) --c;
        while (start(c) < u) ++c;
        return c;
    }

    // Pieces of an item of `records` records that starts at cost `head` of the
    // list and is cut: the cuts inside it are at least `least` records from its
    // borders.
    W4_HD int pieces(int head, int records) const {
        const int lo = block_from(head + extra + least);
        const int hi = block_from(head + extra + records - least + 1) - 1;
        return hi - lo + 2;
    }

    // The next item, of the next sequence where b's are done.
    W4_HD void advance(Cut &c) const {
        c.u = 0;
        if (++c.item == per_seq) c.item = 0, ++c.b;
    }
};

}  // namespace w4
