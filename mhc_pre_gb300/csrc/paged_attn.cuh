// paged_attn.cuh -- what the paged-attention kernels share: the plan that
// splits a ragged batch evenly over the CTAs, the masks, and the joining of
// partial results.
//
// Work.  For each sequence and key head, the query heads that share the key
// head and the sequence's new tokens form one list of rows (row r is token
// r / G, head r % G of the group, G = Hq/Hk); a tile is up to `tile_rows`
// consecutive rows, and it reads the keys that any of its rows sees in blocks
// of `block_keys`.  The unit of work is one block of one tile of one key head.
// A tile of a key head begins with `lead` units that stand for its fixed costs
// (queries in, sums out), so that many short tiles weigh what they take.
// All units are laid end to end (tiles, then key heads, then blocks) and CTA c
// takes the `per_cta` consecutive units from c * per_cta: every CTA has the
// same share whatever the lengths are, a long sequence is split over as many
// CTAs as it needs, and at most two of a CTA's pieces (its first and its last)
// are incomplete.  A tile of a key head that costs at most 1/8 of a share is
// not split: the border moves to its nearer end, which unbalances the shares
// by less than joining its parts would take (14 tiles of 7 units a CTA: 216 ->
// 203 us).  Incomplete pieces go to the workspace as unnormalised sums
// with their row maxima, and the CTA that finishes a tile last joins them in
// the order of the CTAs, so that results do not depend on timing.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mhc_common.cuh"

namespace mhc {

constexpr unsigned ATTN_ERR_TIMEOUT = 1u, ATTN_ERR_RANGE = 2u;

// Most new tokens of a sequence that is a tree.
constexpr int TREE_MOST = 1024;

// Tiles below 1/8 of a CTA's share are not split.  Of trees, whose parts have many
// rows to write and join, those below 1/3, and a tile's fixed cost counts as 3 units:
// 64 sequences of 8 drafted and 1000 cached tokens take 60 us, 70 with 1/4 or 1/6
// (47 and 60 with heads of 64); fixed costs of 1, 2 and 5 are 0 to 6 % slower or
// faster, case by case.  On the CUDA cores, where a block takes much longer, 1 unit:
// 4 sequences of 30 and 2000 in float32 119 us, 123, 134 and 134 with 0, 2 and 3.
constexpr int ATTN_SMALL_TILE = 8, TREE_SMALL_TILE = 3, TREE_LEAD = 3, TREE_LEAD_CC = 1;

// Join counters of a tile and key head: each warp's rows are joined by
// themselves.
constexpr int JOINS = 8;

// One tile of rows of one sequence, for every key head.
struct alignas(16) AttnTile {
    int64_t start;      // its first unit
    int64_t q0;         // the sequence's first row of q
    int seq;
    int qlen, kvlen;    // new tokens; cached tokens including them
    int row0;           // first row of the tile in the sequence's list
    int blk0, nblk;     // key blocks that any of its rows sees
    int cnt;            // index of its join counters (JOINS per key head)
    int pad;
};
static_assert(sizeof(AttnTile) == 48, "AttnTile is read as three 16-byte words");

struct AttnHead {       // start of the plan
    int64_t per_cta;    // units of a CTA
    int64_t T;          // this and the sizes below: for the check that plan and call agree
    int64_t max_q, max_kv;
    int ntiles;
    int ncta;
    int Hq, Hk, B, tile_rows, block_keys, window, lead;
    int spent;          // a wait ran out in a call with this plan: parts of its tiles never
                        // came, and their join counters stand where the next call would
                        // take them for its own
};
static_assert(sizeof(AttnHead) <= 256, "the header has 256 bytes");

// Sizes both the host and the device need.
struct AttnPlan {
    int ncta;           // CTAs of the launch
    int tile_rows, block_keys;
    int lane_rows;      // rows of one softmax lane (tensor cores): whole tokens
    int lead;           // fixed cost of a tile, in blocks
    int slot_rows;      // rows a partial result can have
    int64_t max_tiles;
    size_t start_off, tile_off, count_off, part_off, part_slot_bytes, total;
};

struct AttnParams {
    const void *q, *k_cache, *v_cache;
    void* o;
    float* lse;                    // may be null
    const int32_t* page_table;     // [B, table_stride]
    const uint32_t* tree;          // [T, tree_stride]: bit i of a row, the sequence's i-th new token is seen
    const int32_t *cu_q, *kv_lens; // of trees only, which have no plan
    unsigned char* ws;
    int64_t q_stride, table_stride, num_pages, tree_stride;
    int64_t k_page_stride, k_slot_stride, k_head_stride;
    int64_t v_page_stride, v_slot_stride, v_head_stride;
    int64_t T, max_q, max_kv;
    int B, Hq, Hk, G, Dh, page_size, page_shift, window;
    unsigned g_mul, g_shift;       // r / G = umulhi(r, g_mul) >> g_shift for 0 <= r < 2^31
    float scale, softcap;
    unsigned force_timeout;
    AttnPlan plan;
};

// A CTA's share: its units, tile, key head and unit of the tile, and the tile itself
// (one read instead of two on the way to the first queries and keys).
struct alignas(16) AttnStart {
    int64_t begin, end;     // the CTA's units
    int tile, head, unit;
    int after;              // of trees, while it is looked for: `t` is the last tile before it
    AttnTile t;
};
static_assert(sizeof(AttnStart) == 80, "AttnStart is read as five 16-byte words");

__device__ __forceinline__ const AttnHead* attn_head(const AttnParams& p) {
    return reinterpret_cast<const AttnHead*>(p.ws);
}
__device__ __forceinline__ const AttnStart* attn_starts(const AttnParams& p) {
    return reinterpret_cast<const AttnStart*>(p.ws + p.plan.start_off);
}
__device__ __forceinline__ const AttnTile* attn_tiles(const AttnParams& p) {
    return reinterpret_cast<const AttnTile*>(p.ws + p.plan.tile_off);
}
__device__ __forceinline__ int* attn_counts(const AttnParams& p) {
    return reinterpret_cast<int*>(p.ws + p.plan.count_off);
}

// Whether the plan in the workspace is the one that this call's sizes ask for (a
// larger max_q would overrun the parts, a larger max_kv the page table) and its
// counters are at zero.
__device__ __forceinline__ bool attn_plan_agrees(const AttnParams& p) {
    const AttnHead* h = attn_head(p);
    return h->T == p.T && h->max_q == p.max_q && h->max_kv == p.max_kv && h->Hq == p.Hq && h->Hk == p.Hk &&
           h->B == p.B && h->tile_rows == p.plan.tile_rows && h->block_keys == p.plan.block_keys &&
           h->window == p.window && h->ncta == p.plan.ncta && h->lead == p.plan.lead && h->ntiles >= 0 &&
           h->ntiles <= p.plan.max_tiles && h->per_cta > 0 && h->spent == 0;
}
__device__ __forceinline__ void attn_plan_spent(const AttnParams& p) { reinterpret_cast<AttnHead*>(p.ws)->spent = 1; }

// The token of row r.
__device__ __forceinline__ int attn_token(const AttnParams& p, int r) {
    return p.G == 1 ? r : static_cast<int>(__umulhi(static_cast<unsigned>(r), p.g_mul) >> p.g_shift);
}

// Keys [lo, hi) that token i of the sequence's new ones sees.  A token before the
// cached ones has end = 0: end - window stays in 32 bits for every window.
template <typename T>
__device__ __forceinline__ void attn_token_keys(const T& t, int i, int window, int& lo, int& hi) {
    const int end = max(0, t.kvlen - t.qlen + i + 1);
    hi = min(t.kvlen, end);
    lo = window > 0 ? max(0, end - window) : 0;
}

// A tree's new tokens see the cached ones before them (with a window the last
// ones of these) and, of each other, those whose bits they have.  Keys [lo, hi)
// of which any of the sequence's tokens may see some: a path has at least one
// token, which a window counts.
template <typename T>
__device__ __forceinline__ void attn_tree_keys(const T& t, int window, int& lo, int& hi) {
    const int ctx = t.kvlen - t.qlen;   // a sequence of fewer cached than new tokens sees nothing
    hi = ctx >= 0 ? t.kvlen : 0;
    lo = window > 0 && ctx >= window ? ctx - window + 1 : 0;
}
// Keys that some row of a tile, from `first` to `last`, may see.
template <bool TREE, typename T>
__device__ __forceinline__ void attn_tile_keys(const T& t, int first, int last, int window, int& lo, int& hi) {
    if (TREE) {
        attn_tree_keys(t, window, lo, hi);
    } else {
        int unused;
        attn_token_keys(t, first, window, lo, unused);
        attn_token_keys(t, last, window, unused, hi);
    }
}

// What one token of a tree sees: keys [lo, ctx), and of those from ctx on the
// ones whose bits it has.  `words` are the bits of the sequence's new tokens;
// those past them count for nothing.
struct AttnNode {
    const uint32_t* words;
    int lo, ctx, nodes;
    __device__ __forceinline__ uint32_t word(int i) const {
        const int left = nodes - 32 * i;   // of the sequence's tokens from this word on
        if (i < 0 || left <= 0) return 0u;
        const uint32_t w = __ldg(words + i);
        return left < 32 ? w & ((1u << left) - 1u) : w;
    }
    template <typename T>
    __device__ __forceinline__ void init(const AttnParams& p, const T& t, int token) {
        words = p.tree + (t.q0 + token) * p.tree_stride;
        ctx = t.kvlen - t.qlen;
        nodes = ctx >= 0 ? t.qlen : 0;
        lo = 0;
        if (p.window > 0 && t.kvlen > p.window && ctx >= 0) {
            int path = 0;
            for (int i = 0; 32 * i < nodes; ++i) path += __popc(word(i));
            lo = max(0, min(ctx, ctx - p.window + max(path, 1)));
        }
    }
    // Which of the 32 N keys from g that lie at ctx or later it sees (bits of keys
    // before ctx are 0).  The words come in one round of loads.
    template <int N>
    __device__ __forceinline__ void drafted(int g, uint32_t (&out)[N]) const {
        const int from = g - ctx, w0 = from >> 5;   // rounded down: the first word may be one before the first
        uint32_t w[N + 1];
#pragma unroll
        for (int i = 0; i <= N; ++i) w[i] = word(w0 + i);
#pragma unroll
        for (int i = 0; i < N; ++i) out[i] = __funnelshift_r(w[i], w[i + 1], from & 31);
    }
};

// A sequence of drafted tokens as tiles.  They see the same keys, so they have the
// same blocks; the last one may have fewer rows than the others, and its blocks then
// take less time.
struct TreeSeq {
    int64_t q0;
    int qlen, kvlen, blk0, nblk, tiles;   // no tiles: no new tokens, or numbers that do not fit the call
    bool fits;
    __device__ __forceinline__ AttnTile tile(const AttnParams& p, int seq, int i, int64_t start) const {
        AttnTile t = {};
        t.start = start;
        t.q0 = q0;
        t.seq = seq;
        t.qlen = qlen;
        t.kvlen = kvlen;
        t.row0 = i * p.plan.tile_rows;
        t.blk0 = blk0;
        t.nblk = nblk;
        return t;
    }
};
__device__ __forceinline__ TreeSeq tree_seq(const AttnParams& p, int b) {
    const int q0 = p.cu_q[b], qlen = p.cu_q[b + 1] - q0, kvlen = p.kv_lens[b];
    TreeSeq s;
    s.fits = q0 >= 0 && qlen >= 0 && qlen <= p.max_q && q0 + static_cast<int64_t>(qlen) <= p.T && kvlen >= 0 &&
             kvlen <= p.max_kv;
    s.q0 = q0;
    s.qlen = s.fits ? qlen : 0;
    s.kvlen = kvlen;
    s.tiles = (s.qlen * p.G + p.plan.tile_rows - 1) / p.plan.tile_rows;
    int lo, hi;
    attn_tree_keys(s, p.window, lo, hi);
    // rows that see nothing still get their zeros written: one masked block
    s.blk0 = hi > lo ? lo / p.plan.block_keys : 0;
    s.nblk = hi > lo ? (hi + p.plan.block_keys - 1) / p.plan.block_keys - s.blk0 : 1;
    return s;
}
// The tile after `t`: of its sequence, or the first of the next that has any
// (seq = B: there is none).  All lanes of a warp call it, and look through the
// sequences without new tokens together (8 of 11 new tokens on 3200 keys among 8184
// without, float32: 126 us, one after the other 535).
__device__ __forceinline__ void tree_next_tile(const AttnParams& p, AttnTile& t) {
    t.start += static_cast<int64_t>(p.Hk) * (t.nblk + p.plan.lead);
    t.row0 += p.plan.tile_rows;
    if (t.row0 < t.qlen * p.G) return;
    int b = t.seq + 1;
    while (b < p.B) {
        const TreeSeq s = tree_seq(p, b);
        if (s.tiles > 0) {
            t = s.tile(p, b, 0, t.start);
            return;
        }
        // on to the next one with rows, whether they fit the call or not
        ++b;
        unsigned found = 0u;
        for (; found == 0u && b < p.B; b += found != 0u ? __ffs(found) - 1 : 32) {
            const int at = b + static_cast<int>(threadIdx.x & 31);
            found = __ballot_sync(0xffffffffu, at < p.B && p.cu_q[at] != p.cu_q[at + 1]);
        }
    }
    t.seq = p.B;
}

// a / b for a >= 0, b > 0 with a quotient of 32 bits: the 64-bit division is a long subroutine.
__device__ __forceinline__ int tree_divide(int64_t a, int64_t b) {
    if (((a | b) >> 31) == 0) return static_cast<int>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
    return static_cast<int>(a / b);
}

// What the CTAs of a launch leave for the joins, and how a CTA finds its share: in
// place of a plan, each CTA sums up the units, the weights and the tiles of all
// sequences and finds its two borders among them.  That takes a microsecond more than
// reading a plan, and a launch of five less.
struct TreeShare {
    AttnStart start;
    int64_t sums[16][3];   // of a warp each
    int most[16], kinds[16];
};
// How shares are cut.
struct TreeCut {
    int least;          // weight of a CTA's share, at least: a block or more, so that none in a tile is empty
    int join;           // what splitting tiles costs a call, in weight
    int full, part;     // weight of a block: of a tile of more rows than one lane holds, of fewer
};
struct TreeSums {
    int64_t units, weight, tiles;   // tiles: of a key head each
};
// The tiles' weights.
struct TreeWeights {
    int lead, full, last;   // of the fixed cost; of a tile (of a key head), all but the last and the last one
    int block;              // of a block of the last one
    __device__ __forceinline__ TreeWeights(const AttnParams& p, const TreeSeq& s, const TreeCut& cut) {
        block = s.qlen * p.G - (s.tiles - 1) * p.plan.tile_rows <= p.plan.lane_rows ? cut.part : cut.full;
        lead = p.plan.lead * cut.part;
        full = lead + s.nblk * cut.full;
        last = lead + s.nblk * block;
    }
};
__device__ __forceinline__ TreeSums tree_sums(const AttnParams& p, const TreeSeq& s, const TreeWeights& w) {
    if (s.tiles == 0) return {0, 0, 0};
    const int64_t t = static_cast<int64_t>(s.tiles) * p.Hk;
    return {t * (s.nblk + p.plan.lead), static_cast<int64_t>(p.Hk) * (static_cast<int64_t>(s.tiles - 1) * w.full + w.last), t};
}
// The border before the sequence's i-th tile and head (behind its last where there is
// no such one), whose first unit is `base` units.
__device__ __forceinline__ AttnStart tree_border_whole(const AttnParams& p, const TreeSeq& s, int b, int64_t base, int i,
                                                       int64_t units) {
    const int cost = s.nblk + p.plan.lead, tile = i / p.Hk;
    const int64_t start = base + static_cast<int64_t>(tile) * p.Hk * cost;
    AttnStart a = {};
    a.head = i - tile * p.Hk;
    a.begin = start + static_cast<int64_t>(a.head) * cost;
    a.t = s.tile(p, b, tile, start);
    if (tile == s.tiles && a.begin < units) {   // the next sequence's first one
        const TreeSeq next = tree_seq(p, b + 1);
        a.after = next.tiles == 0;              // far: looked for by a warp
        a.t = a.after ? s.tile(p, b, tile - 1, start - static_cast<int64_t>(p.Hk) * cost) : next.tile(p, b + 1, 0, start);
    }
    return a;
}
// The border at weight `in` of a sequence, moved to the nearer end of a tile that is
// not to be split (`per`: a CTA's share of the weight), else between two blocks.
__device__ __forceinline__ AttnStart tree_border(const AttnParams& p, const TreeSeq& s, const TreeWeights& w,
                                                 const TreeCut& cut, int b, int64_t base, int64_t in, int64_t per,
                                                 int64_t units) {
    const int64_t before = static_cast<int64_t>(s.tiles - 1) * p.Hk * w.full;   // of all tiles but the last
    const bool last = in >= before;
    const int64_t cost = last ? w.last : w.full, block = last ? w.block : cut.full;
    const int i = last ? (s.tiles - 1) * p.Hk + tree_divide(in - before, cost) : tree_divide(in, cost);
    const int off = static_cast<int>(last ? in - before - static_cast<int64_t>(i - (s.tiles - 1) * p.Hk) * cost
                                          : in - static_cast<int64_t>(i) * cost);
    const bool small = cost * TREE_SMALL_TILE <= per;
    AttnStart a = tree_border_whole(p, s, b, base, small && 2 * off >= cost ? i + 1 : i, units);
    if (!small) {
        a.unit = off < w.lead ? off / cut.part : p.plan.lead + (off - w.lead) / static_cast<int>(block);
        a.begin += a.unit;
    }
    return a;
}
// All threads of CTA `cta`: its share, into shared memory and the workspace.  Where
// whole tiles dealt out by their number take no more than cut.join above an even
// share, none is split.
template <int THREADS>
__device__ __forceinline__ void tree_share(const AttnParams& p, int cta, const TreeCut& cut, TreeShare& out,
                                           unsigned* error_word) {
    static_assert(THREADS <= 512, "TreeShare has 16 warps");
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    // each thread has sequences that follow each other (32 of 16 and 4096 among 8160
    // without new tokens: 124 us, in rounds of a sequence a thread 218; without those 104)
    const int each = (p.B + THREADS - 1) / THREADS, first = tid * each, last = min(p.B, first + each);
    TreeSeq s = {};
    TreeSums mine = {0, 0, 0}, upto, all = {0, 0, 0};
    int most = 0;               // weight of the heaviest tile
    int kinds = 0;              // of blocks: 1, of tiles of fewer rows; 2, of more
    for (int b = first; b < last; ++b) {
        s = tree_seq(p, b);
        if (!s.fits && cta == 0) atomicOr(error_word, ATTN_ERR_RANGE);
        if (s.tiles == 0) continue;
        const TreeWeights tw(p, s, cut);
        const TreeSums sum = tree_sums(p, s, tw);
        mine = {mine.units + sum.units, mine.weight + sum.weight, mine.tiles + sum.tiles};
        most = max(most, s.tiles > 1 ? tw.full : tw.last);
        kinds |= (s.tiles > 1 || tw.block == cut.full ? 2 : 0) | (tw.block == cut.part ? 1 : 0);
    }
    // inclusive sums over the block
    upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto.units, o), y = __shfl_up_sync(0xffffffffu, upto.weight, o);
        const int64_t z = __shfl_up_sync(0xffffffffu, upto.tiles, o);
        if (lane >= o) upto = {upto.units + x, upto.weight + y, upto.tiles + z};
    }
    most = __reduce_max_sync(0xffffffffu, most);
    kinds = __reduce_or_sync(0xffffffffu, kinds);
    if (lane == 31) {
        out.sums[w][0] = upto.units;
        out.sums[w][1] = upto.weight;
        out.sums[w][2] = upto.tiles;
        out.most[w] = most;
        out.kinds[w] = kinds;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        if (i == w) upto = {upto.units + all.units, upto.weight + all.weight, upto.tiles + all.tiles};
        all = {all.units + out.sums[i][0], all.weight + out.sums[i][1], all.tiles + out.sums[i][2]};
        most = max(most, out.most[i]);
        kinds |= out.kinds[i];
    }
    const int ncta = p.plan.ncta;
    // where all blocks weigh the same a multiple of that, so that borders leave no remainders
    const int grain = kinds == 1 ? cut.part : kinds == 2 ? cut.full : 1;
    const int64_t even = static_cast<int64_t>(ncta) * grain;
    int64_t per = all.weight >> 31 == 0 ? static_cast<int64_t>(tree_divide(all.weight + even - 1, even))
                                        : (all.weight + even - 1) / even;
    per *= grain;
    if (per < cut.least) per = cut.least;
    // (more than 31 bits of them only if sequences overlap)
    const int n = all.tiles >> 31 == 0 ? static_cast<int>(all.tiles) : 0, deal = n / ncta, rest = n - deal * ncta;
    const bool whole = n > 0 && static_cast<int64_t>(deal + (rest > 0 ? 1 : 0)) * most <= per + cut.join;
    // in weight, or in tiles: the first `rest` CTAs have one more
    const int64_t end = whole ? all.tiles : all.weight;
    const int64_t u0 = whole ? static_cast<int64_t>(cta) * deal + min(cta, rest) : min(cta * per, end);
    const int64_t u1 = cta + 1 == ncta ? end : whole ? u0 + deal + (cta < rest ? 1 : 0) : min(u0 + per, end);
    if (tid == 0) {
        out.start = AttnStart{};
        out.start.begin = out.start.end = all.units;
    }
    __syncthreads();
    // the thread whose sequences a border is among finds it
    const int64_t high = whole ? upto.tiles : upto.weight, low = high - (whole ? mine.tiles : mine.weight);
    if ((u0 < end && low <= u0 && u0 < high) || (u1 < end && low <= u1 && u1 < high)) {
        int64_t lo = low, base = upto.units - mine.units;
        for (int b = first; b < last; ++b) {
            if (each > 1) s = tree_seq(p, b);   // (the only one is still there)
            if (s.tiles == 0) continue;
            const TreeWeights tw(p, s, cut);
            const TreeSums sum = tree_sums(p, s, tw);
            const int64_t hi = lo + (whole ? sum.tiles : sum.weight);
            auto border = [&](int64_t u) {
                return whole ? tree_border_whole(p, s, b, base, static_cast<int>(u - lo), all.units)
                             : tree_border(p, s, tw, cut, b, base, u - lo, per, all.units);
            };
            // the end in its own field, which the start's thread does not touch
            if (u1 < end && lo <= u1 && u1 < hi) out.start.end = border(u1).begin;
            if (u0 < end && lo <= u0 && u0 < hi) {
                const AttnStart a = border(u0);
                out.start.begin = a.begin;
                out.start.head = a.head;
                out.start.unit = a.unit;
                out.start.after = a.after;
                out.start.t = a.t;
            }
            lo = hi;
            base += sum.units;
        }
    }
    __syncthreads();
    if (out.start.after != 0) {   // (past 7400 sequences without new tokens: 2200 us by one thread, 15 by a warp)
        if (w == 0) {
            AttnTile t = out.start.t;
            tree_next_tile(p, t);
            __syncwarp();
            if (lane == 0) out.start.t = t;
        }
        __syncthreads();
    }
    if (tid == 0) reinterpret_cast<AttnStart*>(p.ws + p.plan.start_off)[cta] = out.start;
}

// A CTA's pieces one after the other.
struct AttnPiece {
    int64_t q0;
    int seq, qlen, kvlen, row0, head;
    int blk, nb;                // first key block and number of blocks (0: there is no piece)
    int whole;                  // the tile's only piece
    int cnt, slot;              // join counters; where a partial result goes
    int first_cta, last_cta;    // the CTAs with a part of the tile (unless whole)
    int lo, hi;                 // keys [lo, hi) that any row of the tile sees
};
struct AttnWalk {
    int64_t at, end, per;
    int tile, head, unit;
    AttnTile t;
    __device__ __forceinline__ bool begin(const AttnParams& p, int cta) {
        return begin(attn_starts(p)[cta], attn_head(p)->per_cta);
    }
    __device__ __forceinline__ bool begin(const AttnStart& s, int64_t per_cta = 0) {   // (of trees it is not asked for)
        per = per_cta;
        at = s.begin;
        end = s.end;
        tile = s.tile;
        head = s.head;
        unit = s.unit;
        t = s.t;
        return at < end;
    }
    // The next piece that has blocks; false when the CTA's share is done.
    template <bool TREE>
    __device__ __forceinline__ bool next(const AttnParams& p, int cta, AttnPiece& out) {
        while (at < end) {
            const int lead = p.plan.lead, cost = t.nblk + lead;
            const int64_t left = end - at;
            const int n = left < cost - unit ? static_cast<int>(left) : cost - unit;
            const int b0 = max(0, unit - lead), b1 = max(0, unit + n - lead);
            out.q0 = t.q0;
            out.seq = t.seq;
            out.qlen = t.qlen;
            out.kvlen = t.kvlen;
            out.row0 = t.row0;
            out.head = head;
            out.blk = t.blk0 + b0;
            out.nb = b1 - b0;
            out.whole = b0 == 0 && b1 == t.nblk;
            attn_tile_keys<TREE>(t, attn_token(p, t.row0), attn_token(p, min(t.row0 + p.plan.tile_rows, t.qlen * p.G) - 1),
                                 p.window, out.lo, out.hi);
            out.cnt = (t.cnt + head) * JOINS;
            out.slot = 2 * cta + (b0 > 0 ? 0 : 1);
            if (!TREE && !out.whole) {   // who joins a tile's parts
                const int64_t u0 = t.start + static_cast<int64_t>(head) * cost + lead, u1 = u0 + t.nblk - 1;
                if (u1 >> 31 == 0) {   // the 64-bit division is a long subroutine
                    out.first_cta = static_cast<int>(static_cast<uint32_t>(u0) / static_cast<uint32_t>(per));
                    out.last_cta = static_cast<int>(static_cast<uint32_t>(u1) / static_cast<uint32_t>(per));
                } else {
                    out.first_cta = static_cast<int>(u0 / per);
                    out.last_cta = static_cast<int>(u1 / per);
                }
            }
            at += n;
            unit += n;
            if (unit == cost) {
                unit = 0;
                if (++head == p.Hk) {
                    head = 0;
                    ++tile;
                    if (at < end) {
                        if (TREE) tree_next_tile(p, t);
                        else t = attn_tiles(p)[tile];
                    }
                }
            }
            if (b1 > b0) return true;
        }
        out.nb = 0;
        return false;
    }
};

// Partial result of one piece: rows of `dp` sums, then the maxima (in the
// scores' own unit times log2 e), then the sums of the exponentials.
__device__ __forceinline__ float* attn_slot(const AttnParams& p, int slot) {
    return reinterpret_cast<float*>(p.ws + p.plan.part_off + static_cast<size_t>(slot) * p.plan.part_slot_bytes);
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// One row's log sum exp from its maximum in base 2 and its sum.
__device__ __forceinline__ float attn_lse(float m2, float l) {
    return l != 0.0f ? fmaf(m2, LN2, logf(l)) : -INFINITY;
}

// Joins the partial results of rows [begin, end) of a tile (one warp, after the
// last part has arrived), R rows at a time.  Lane c first takes the maximum and
// the sum of part c for each row, so that the parts' weights come from one round
// of loads; then the lanes take 4 values of a row each and add the parts in
// order, the loads of U parts in flight together.  More than 32 parts go in
// rounds of 32 with a running maximum.
template <typename TA, int DP, int R, int U>
__device__ __forceinline__ void attn_join(const AttnParams& p, const AttnPiece& pc, int begin, int end, int lane) {
    constexpr int LPR = DP < 128 ? DP / 4 : 32;   // lanes of a row
    constexpr int NV = DP / 4 / LPR;              // pieces of 4 values a lane has of a row
    constexpr int RW = 32 / LPR;                  // rows side by side
    const int sub = lane % LPR, side = lane / LPR, sr = p.plan.slot_rows;
    auto part = [&](int c) { return attn_slot(p, 2 * c + (c == pc.first_cta ? 1 : 0)); };
    for (int r0 = begin; r0 < end; r0 += RW * R) {
        float M[RW * R], l[RW * R];
        float4 a[R][NV];
#pragma unroll
        for (int i = 0; i < RW * R; ++i) {
            M[i] = -INFINITY;
            l[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int v = 0; v < NV; ++v) a[i][v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int c0 = pc.first_cta; c0 <= pc.last_cta; c0 += 32) {
            const int n = min(32, pc.last_cta - c0 + 1);
            float w[RW * R], pl[RW * R];
#pragma unroll
            for (int i = 0; i < RW * R; ++i) {
                const float* s = part(c0 + min(lane, n - 1)) + static_cast<int64_t>(sr) * DP + min(r0 + i, end - 1);
                w[i] = lane < n ? __ldcg(s) : -INFINITY;
                pl[i] = lane < n ? __ldcg(s + sr) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < RW * R; ++i) {
                float top = w[i];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                top = fmaxf(top, M[i]);
                const float base = top == -INFINITY ? 0.0f : top, keep = ex2(M[i] - base);
                w[i] = ex2(w[i] - base);
                l[i] = fmaf(l[i], keep, warp_sum(pl[i] * w[i]));
                if (c0 > pc.first_cta) {
#pragma unroll
                    for (int v = 0; v < NV; ++v)
                        if (i % RW == side) {
                            float4& x = a[i / RW][v];
                            x = make_float4(x.x * keep, x.y * keep, x.z * keep, x.w * keep);
                        }
                }
                M[i] = top;
            }
            for (int c = 0; c < n; c += U) {
                float4 pv[U][R][NV];
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        const float* s = part(c0 + min(c + u, n - 1));
                        const int row = min(r0 + i * RW + side, end - 1);
#pragma unroll
                        for (int v = 0; v < NV; ++v)
                            pv[u][i][v] = __ldcg(reinterpret_cast<const float4*>(s + static_cast<int64_t>(row) * DP) +
                                                 v * LPR + sub);
                    }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        float f = 0.0f;
#pragma unroll
                        for (int q = 0; q < RW; ++q) {
                            const float x = __shfl_sync(0xffffffffu, w[i * RW + q], min(c + u, 31));
                            if (q == side) f = x;
                        }
                        if (c + u < n) {
#pragma unroll
                            for (int v = 0; v < NV; ++v) {
                                a[i][v].x = fmaf(pv[u][i][v].x, f, a[i][v].x);
                                a[i][v].y = fmaf(pv[u][i][v].y, f, a[i][v].y);
                                a[i][v].z = fmaf(pv[u][i][v].z, f, a[i][v].z);
                                a[i][v].w = fmaf(pv[u][i][v].w, f, a[i][v].w);
                            }
                        }
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int row = r0 + i * RW + side;
            if (row >= end) continue;
            float ml = M[i * RW], ll = l[i * RW];
#pragma unroll
            for (int q = 1; q < RW; ++q)
                if (q == side) {
                    ml = M[i * RW + q];
                    ll = l[i * RW + q];
                }
            const float inv = ll != 0.0f ? 1.0f / ll : 0.0f;
            const int r = pc.row0 + row, tok = attn_token(p, r);
            const int64_t out = (pc.q0 + tok) * p.Hq + pc.head * p.G + (r - tok * p.G);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int d = (v * LPR + sub) * 4;
                if (d >= p.Dh) continue;
                TA* o = static_cast<TA*>(p.o) + out * p.Dh + d;
                if (sizeof(TA) == 2) {
                    const __nv_bfloat162 x = __floats2bfloat162_rn(a[i][v].x * inv, a[i][v].y * inv);
                    const __nv_bfloat162 y = __floats2bfloat162_rn(a[i][v].z * inv, a[i][v].w * inv);
                    *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&x),
                                                              *reinterpret_cast<const uint32_t*>(&y));
                } else {
                    *reinterpret_cast<float4*>(o) = make_float4(a[i][v].x * inv, a[i][v].y * inv, a[i][v].z * inv,
                                                                a[i][v].w * inv);
                }
            }
            if (sub == 0 && p.lse != nullptr) p.lse[out] = attn_lse(ml, ll);
        }
    }
}

}  // namespace mhc
