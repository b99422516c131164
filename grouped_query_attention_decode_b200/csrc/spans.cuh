// Work partition of the span kernels: groups of query rows, each group against one span of
// cached rows.
//
// A span is either a shared one -- the tokens of a group of sequences (or of one encoder
// sequence) against the rows they all attend -- or one sequence's own rows.  Per key/value head
// a span's query rows are (token, query head of the group) pairs; they are cut into units of up
// to `blk` tokens and rb heads, and a unit's cached rows into tiles of T.  As in schedule.cuh
// the tiles of all units form one line, CTA i of G (of as many as there are tiles, if fewer) takes
// the tiles
//     [floor(i * total / G), floor((i + 1) * total / G)),
// and every CTA derives its range from the lengths on the device.  A unit that lies in one CTA's
// range is whole; the pieces of the others go to workspace slots (two per CTA: only a range's
// first and last piece can be partial) and are joined by the kernel launched behind
// (span_merge.cu):  out = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c over the pieces c.
#pragma once

#include <cstdint>

#include "device.cuh"
#include "gqa.h"
#include "schedule.cuh"
#include "span_device.cuh"

namespace gqa {

struct SpanParams {
    // shared spans: group g holds the members [gstart[g], gstart[g + 1]) and attends glen[g] rows
    const int32_t *gstart, *glen;
    int P, g_max;
    int g_step;  // glen has to be a multiple of this (the page size; 1 for contiguous caches)
    // own spans, none when B = 0: sequence b attends lens[b] rows of its own cache, or, with
    // own_after (paged), the rows [glen[its group], lens[b]) of its block table
    const int32_t *lens;
    int B, own_max, own_after;
    int s_begin, s_end;  // spans that take part: [0, P) are the shared ones, [P, P + B) the own ones
    int Q, N;  // tokens per member (1 for cross attention), tokens in all
    int H_q, H_kv, d, r;
    int rb, HB, tb;  // heads per row tile, head blocks = ceil(r / rb), tokens per row tile
    int blk;         // tokens per unit: one or two row tiles
    int nblkQ;       // units of one own span and head block: ceil(Q / blk)
    int T, RT;       // cached rows per tile, query rows per row tile
    int G;
    const int32_t *block_table;  // nullptr: contiguous caches
    int max_pages, page_size, n_pages;
    float scale_log2;  // softmax scale * log2(e); the bf16 kernel takes its magnitude ...
    int negate;        // ... and the sign here
    unsigned long long wait_ns;
    float *out;
    int32_t *status;
    // workspace
    int4 *uinfo;           // own spans present: [unit] (first CTA, its slot, last CTA, 0)
    struct SpanRecord *rec;  // no own spans: [CTA] the cut unit that starts there
    float *slots;          // [2 * G][slot_floats]
    long long slot_floats;
    float *res, *res_ml;   // [2][N * H_q][d] sums and [2][N * H_q][2] (m, l) of whole units
    int behind_shared;     // few rows: launched behind the launch over the shared spans (span_few.cu)
    int u1;                // number of the own spans' first token block, after the shared spans'
    int unit_rows;         // query rows of a slot
    int spread;            // cross attention: units are cut into many pieces (span_merge.cu)
};

struct SpanRecord {
    int valid, tok0, ntok, kvh, hb, k0, c1;
    int cont;  // with `spread`: the worker that starts the cut unit which this one's first piece goes on
               // with, or -1
};

// The group that member i belongs to, -1 for none: the last g with gstart[g] <= i.
__device__ __forceinline__ int group_of(const SpanParams &p, int i) {
    int lo = 0, hi = p.P + 1;  // first index whose start is past i lies in [lo, hi]
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.gstart + mid) > i) hi = mid;
        else lo = mid + 1;
    }
    return lo - 1 < p.P ? lo - 1 : -1;
}

// Rows group g shares, or -1 when the entry is out of range.
__device__ __forceinline__ int shared_rows_of(const SpanParams &p, int g) {
    const int n = __ldg(p.glen + g);
    return n < 0 || n > p.g_max || (p.g_step > 1 && n % p.g_step != 0) ? -1 : n;
}

// First own row and number of own rows of sequence b; false when its length (or its group's) is
// out of range.
__device__ __forceinline__ bool own_rows_of(const SpanParams &p, int b, int &row0, int &rows) {
    const int n = __ldg(p.lens + b);
    row0 = rows = 0;
    if (p.own_after) {
        if (n == 0 && p.Q == 1) return true;  // an empty sequence attends nothing, shared rows neither
        const int g = group_of(p, b);
        if (g >= 0) row0 = shared_rows_of(p, g);
        if (row0 < 0) return row0 = 0, false;
    }
    if (n < row0 || n > p.own_max || (p.Q > 1 && n - row0 < p.Q)) return false;
    rows = n - row0;
    return true;
}

// Paged caches: the first sequence of [a, e) whose length is one that own_rows_of takes behind `shared`
// rows, so its table holds them; -1 for none (all have ended).  One length at a time: the kernels inline
// this in many places, and longer code, fetched once a call, costs more than it saves (four at a time:
// 131 us for 127 at 128 conversations under 12032 rows).
__device__ __forceinline__ int holder_of(const int32_t *lens, int a, int e, int least, int most) {
#pragma unroll 1
    for (int i = a; i < e; ++i) {
        const int n = __ldg(lens + i);
        if (n >= least && n <= most) return i;
    }
    return -1;
}

struct Span {
    int tok0, ntok;  // its tokens
    int row0, rows;  // its cached rows within the source
    int src;         // contiguous: prefix / encoder sequence / sequence; paged: block-table row
};

// `table`: false where the span's block-table row is not asked for; then the shared rows of a group that
// has ended are counted too.
__device__ inline Span span_at(const SpanParams &p, int s, bool flag, bool table = true) {
    Span sp = {0, 0, 0, 0, 0};
    int bad = 0;
    if (s < p.P) {
        // all three reads at once: every caller waits for them
        const int a = __ldg(p.gstart + s), e = __ldg(p.gstart + s + 1), n = shared_rows_of(p, s);
        if (a < 0 || e < a || e > (p.B > 0 ? p.B : p.N)) {
            bad = GQA_STATUS_GROUP_RANGE;
        } else {
            if (n < 0) bad = GQA_STATUS_SEQLEN_RANGE;
            sp.tok0 = a * p.Q;
            sp.ntok = (e - a) * p.Q;
            sp.rows = max(n, 0);
            sp.src = s;
            if (p.block_table != nullptr && table && sp.rows > 0) {
                sp.src = holder_of(p.lens, a, e, sp.rows + (p.Q > 1 ? p.Q : 0), p.own_max);
                if (sp.src < 0) sp.src = sp.rows = 0;
            }
        }
    } else if (s < p.P + p.B) {
        const int b = s - p.P;
        if (!own_rows_of(p, b, sp.row0, sp.rows)) bad = GQA_STATUS_SEQLEN_RANGE;
        sp.tok0 = b * p.Q;
        sp.ntok = p.Q;
        sp.src = b;
    }
    if (flag && bad != 0 && p.status != nullptr) atomicOr(p.status, bad);
    return sp;
}

__device__ __forceinline__ int span_blocks(const SpanParams &p, const Span &sp) { return (sp.ntok + p.blk - 1) / p.blk; }

__device__ __forceinline__ long long span_tiles(const SpanParams &p, const Span &sp) {
    return static_cast<long long>(tiles_of(sp.rows, p.T)) * span_blocks(p, sp) * p.H_kv * p.HB;
}

// Number of a span's unit `block` of key/value head kvh and head block hb.  Token blocks of shared
// spans are numbered by their first token / blk + group: that grows along the line by at least the
// span's blocks, so no two share a number, and unit numbers grow along the line.
__device__ __forceinline__ int unit_number(const SpanParams &p, int s, const Span &sp, int block, int kvh, int hb) {
    const int base = s < p.P ? sp.tok0 / p.blk + s : p.u1 + (s - p.P) * p.nblkQ;
    return base * p.H_kv * p.HB + (kvh * p.HB + hb) * span_blocks(p, sp) + block;
}

struct SpanRange {
    long long begin, end, total, off0;
    int s0;
    int parts;  // CTAs that have tiles, the first of them: min(G, total)
    Span span;  // span s0
};

// Worker `cta`'s share of `total` tiles.
__device__ __forceinline__ void share_of(const SpanParams &p, int cta, SpanRange &r) {
    r.parts = static_cast<int>(r.total < p.G ? r.total : p.G);
    const bool some = cta < r.parts;
    r.begin = some ? cta_range_begin(cta, r.total, r.parts) : 0;
    r.end = some ? cta_range_begin(cta + 1, r.total, r.parts) : 0;
    r.s0 = 0;
    r.off0 = 0;
    r.span = Span{0, 0, 0, 0, 0};
}

// Whole CTA of NT threads: the total number of tiles, this CTA's range and the span it starts
// in.  `scratch`: NT / 32 long longs of shared memory; `res`: shared.
template <int NT>
__device__ void locate_span_range(const SpanParams &p, int cta, long long *scratch, SpanRange *res) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.s_end - p.s_begin + NT - 1) / NT;
    const int s0 = p.s_begin + tid * per, s1 = min(p.s_end, s0 + per);
    long long mine = 0;
    Span sp = {0, 0, 0, 0, 0};
    for (int s = s0; s < s1; ++s) {
        sp = span_at(p, s, cta == 0);
        mine += span_tiles(p, sp);
    }
    const long long incl = warp_incl_scan(mine, lane);
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    long long off = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) off += scratch[w];
        total += scratch[w];
    }
    SpanRange mine_r;
    mine_r.total = total;
    share_of(p, cta, mine_r);
    const long long begin = mine_r.begin;
    if (tid == 0 && begin >= mine_r.end) *res = mine_r;
    if (begin < mine_r.end && off <= begin && begin < off + mine) {
        for (int s = s0; s < s1; ++s) {
            if (per > 1) sp = span_at(p, s, false);
            const long long v = span_tiles(p, sp);
            if (begin < off + v) {
                mine_r.s0 = s;
                mine_r.off0 = off;
                mine_r.span = sp;
                *res = mine_r;
                break;
            }
            off += v;
        }
    }
    __syncthreads();
}

// The same for a CTA whose warps are workers of their own: called by all NT threads, it gives every
// warp the range of its worker.  `before`: NT long longs of shared memory, `scratch` NT / 32.
template <int NT>
__device__ SpanRange locate_warp_ranges(const SpanParams &p, int worker, bool flag, long long *before, long long *scratch) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.s_end - p.s_begin + NT - 1) / NT;
    const int s0 = p.s_begin + tid * per, s1 = min(p.s_end, s0 + per);
    long long mine = 0;
    for (int s = s0; s < s1; ++s) mine += span_tiles(p, span_at(p, s, flag));
    const long long incl = warp_incl_scan(mine, lane);
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    long long off = incl - mine;
    SpanRange r = {};
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) off += scratch[w];
        r.total += scratch[w];
    }
    before[tid] = off;
    __syncthreads();
    share_of(p, worker, r);
    if (r.begin >= r.end) return r;
    // the last thread whose spans start at or before the range's first tile holds it (of several
    // that start there, all but the last are empty)
    int t = -1;
    for (int b = 0; b < NT; b += 32) {
        const uint32_t m = __ballot_sync(kFullMask, before[b + lane] <= r.begin);
        if (m != 0) t = b + 31 - __clz(m);
        if (m != kFullMask) break;
    }
    r.off0 = before[t];
    for (int s = p.s_begin + t * per; s < min(p.s_end, p.s_begin + (t + 1) * per); ++s) {
        r.span = span_at(p, s, false);
        const long long v = span_tiles(p, r.span);
        r.s0 = s;
        if (r.begin < r.off0 + v) break;
        r.off0 += v;
    }
    return r;
}

// One CTA-range piece of one unit.
struct SpanSegment {
    int s, src;
    int tok0, ntok;   // tokens of the unit
    int kvh, hb;
    int row0, rows;   // cached rows of the span within its source
    int j0, len, nt;  // first tile and tiles of the piece, tiles of the unit
    int unit;
    long long uoff;   // line position of the unit's first tile
    bool first;       // the piece opens the CTA's range (its slot is 0, else 1)
    __device__ __forceinline__ bool whole() const { return len == nt; }
};

struct SpanWalker {
    long long t, end, off;
    int s, nt, nblk;
    Span sp;
    bool opened;

    __device__ void open(const SpanParams &p) {
        nt = tiles_of(sp.rows, p.T);
        nblk = span_blocks(p, sp);
    }
    __device__ void init(const SpanParams &p, const SpanRange &cr) {
        t = cr.begin;
        end = cr.end;
        off = cr.off0;
        s = cr.s0;
        opened = false;
        nt = nblk = 0;
        sp = cr.span;
        if (t < end) open(p);
    }
    __device__ bool next(const SpanParams &p, SpanSegment &g) {
        if (t >= end) return false;
        const int hv = p.H_kv * p.HB;
        while (t >= off + static_cast<long long>(nt) * nblk * hv) {
            off += static_cast<long long>(nt) * nblk * hv;
            if (++s >= p.s_end) {  // cannot happen while t < total
                t = end;
                return false;
            }
            sp = span_at(p, s, false);
            open(p);
        }
        const long long rel = t - off;
        const int k = static_cast<int>(udiv(rel, nt));
        const int h = nblk == 1 ? k : k / nblk, block = k - h * nblk;
        g.s = s;
        g.src = sp.src;
        g.tok0 = sp.tok0 + block * p.blk;
        g.ntok = min(p.blk, sp.ntok - block * p.blk);
        g.kvh = p.HB == 1 ? h : h / p.HB;
        g.hb = h - g.kvh * p.HB;
        g.row0 = sp.row0;
        g.rows = sp.rows;
        g.j0 = static_cast<int>(rel - static_cast<long long>(k) * nt);
        const long long left = end - t;
        g.len = static_cast<int>(left < nt - g.j0 ? left : nt - g.j0);
        g.nt = nt;
        g.unit = unit_number(p, s, sp, block, g.kvh, g.hb);
        g.uoff = off + static_cast<long long>(k) * nt;
        g.first = !opened;
        opened = true;
        t += g.len;
        return true;
    }
};

// Row of q and out that row i of a unit's row tile stands for, -1 for padding.  `token` gets the
// row's token.
__device__ __forceinline__ long long span_row(const SpanParams &p, const SpanSegment &g, int tile, int i, int &token) {
    const int tl = tile * p.tb + i / p.rb, h = g.hb * p.rb + i % p.rb;
    token = g.tok0 + tl;
    if (i >= p.tb * p.rb || tl >= g.ntok || h >= p.r) return -1;
    return static_cast<long long>(token) * p.H_q + g.kvh * p.r + h;
}

// Own rows that token `token` of its sequence sees: the Q tokens are the last Q of the rows and
// token j sees one fewer than token j + 1.
__device__ __forceinline__ int seen_rows(const SpanParams &p, const SpanSegment &g, int token) {
    return g.s < p.P || p.Q == 1 ? g.rows : g.rows - p.Q + 1 + token % p.Q;
}

// One thread of worker `cta` (a CTA, or a warp of span_few.cu), before its segments.
__device__ __forceinline__ void open_notes(const SpanParams &p, int cta) {
    if (p.B == 0) {
        p.rec[cta].valid = 0;
        p.rec[cta].cont = -1;  // not read without `spread`
    }
}

// The same thread, once per segment: what the merge needs to find the unit's pieces.
__device__ inline void note_unit(const SpanParams &p, const SpanSegment &g, const SpanRange &cr, int c0) {
    if (g.j0 != 0) {
        if (p.spread) p.rec[c0].cont = static_cast<int>(cta_of_tile(g.uoff, cr.total, cr.parts));
        return;
    }
    const int c1 = g.whole() ? c0 : static_cast<int>(cta_of_tile(g.uoff + g.nt - 1, cr.total, cr.parts));
    if (p.B > 0) {  // there are own rows to join with, here or in another launch
        p.uinfo[g.unit] = make_int4(c0, g.first ? 0 : 1, c1, 0);
    } else if (!g.whole()) {
        SpanRecord &u = p.rec[c0];
        u.tok0 = g.tok0;
        u.ntok = g.ntok;
        u.kvh = g.kvh;
        u.hb = g.hb;
        u.k0 = g.first ? 0 : 1;
        u.c1 = c1;
        u.valid = 1;
    }
}

// TMA descriptors of one bf16 call: q in boxes of a shared span's row tile (tb tokens) and of an
// own span's (min(tb, Q) tokens); K and V of the shared rows and of the own rows, each in boxes
// of a tile (or a page) and of 8 rows.
struct SpanMaps {
    CUtensorMap q_shared, q_own;
    CUtensorMap k_shared, k_shared8, v_shared, v_shared8;
    CUtensorMap k_own, k_own8, v_own, v_own8;
};

int launch_span_tc(const SpanMaps &maps, const SpanParams &p, cudaStream_t stream);
int launch_span_f32(const SpanParams &p, const float *q, const float *ks, const float *vs, const float *ko,
                    const float *vo, cudaStream_t stream);
// Joins the pieces of one launch over the shared spans and one over the own ones (the same launch,
// or none: own.B = 0).
int launch_span_merge(const SpanParams &shared, const SpanParams &own, cudaStream_t stream);
// The kernel for few query rows per span; p.G is the number of warps (span_few_warps a CTA), K and V
// are copied in boxes of 8 rows.
struct SpanFewMaps {
    CUtensorMap kv[4];  // K and V of the shared rows, K and V of the own ones
};
int launch_span_few(const SpanParams &p, const SpanFewMaps &maps, const void *q, cudaStream_t stream);
int span_few_warps(int d);

}  // namespace gqa
