// plan.cu -- the metadata step of one attention call, as a single-CTA kernel.
//
// From query_lens / seq_lens ("Ascend dual-stream parallel" article, section 3.1:
// seq_lens = history plus current tokens, query_lens = current tokens) it builds
//   cu_q      exclusive scan of query_lens (row offset of every request in q/out),
//   checks    seq_len >= query_len >= 0, seq_len fits the block_table row, and
//             sum(query_lens) == num_tokens,
//   pieces    the stream-K cut of all prefill units' KV tiles into one run per
//             chunk-kernel CTA (see plan.cuh), decode items, combine items,
//             (the merge counters of split units need no zeroing: they carry
//             the call's epoch, see the chunk kernel),
// and stores the counts that the persistent kernels read.
// Pass 1 sums tokens, prefill tiles (W) and decode partial rows and finds the
// shortest and longest unit, which fix the run length, whether the partials fit
// the workspace (if not, nothing is split) and whether units are cut at all (see
// choose_split). Pass 2 gives each request its token and tile offsets, counts its
// entries (in closed form, and for the units that run boundaries cut a thread a
// boundary), gives it its list offsets, and a warp per request then writes its
// entries: plan_kernel for any number of requests, 1024 at a time by block scans;
// plan_warps_kernel for at most 32, by one warp's scans. Batches of very few requests
// take a one-warp kernel that builds the same lists in one walk.
#include "common.cuh"
#include "plan.cuh"

namespace cpsa {

namespace {

constexpr int kPlanThreads = 1024;
static_assert(kPlanThreads == 32 * 32, "the block's scans and totals are of 32 warps, a lane each");
constexpr int kScan = 6;

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

struct Req {
    bool valid;
    int q, s, hist;
};

__device__ Req make_req(const PlanParams &p, int query_len, int seq_len)
{
    Req q;
    q.q = query_len;
    q.s = seq_len;
    q.valid = !(q.q < 0 || q.s < q.q) && fits_table(q.s, p.max_blocks, p.page_size);
    q.hist = q.s - q.q;
    return q;
}

__device__ Req load_req(const PlanParams &p, int r) { return make_req(p, p.query_lens[r], p.seq_lens[r]); }

// KV tiles of one unit of query tile qt (rows [128 qt, 128 qt + rows)); see the
// tile grids in plan.cuh.
__device__ __forceinline__ int unit_tiles(const PlanParams &p, const Req &rq, int qt, int rows)
{
    return p.fused ? ceil_div(rq.hist, kTileN) + qt + 1 : ceil_div(rq.hist + qt * kTileM + rows, kTileN);
}

// Stream-K positions of all prefill units of one request: their KV tiles plus
// unit_cost per unit (0 for decode / invalid / empty). I: in 64 bits until it is
// known that all requests' together pass kMaxPlanTiles.
template <typename I = int>
__device__ I prefill_tiles(const PlanParams &p, const Req &rq)
{
    if (!rq.valid || rq.q < 2)
        return 0;
    // query tile qt has hb + qt + 1 tiles, but for the last, which may be short
    const int nqt = ceil_div(rq.q, kTileM), hb = ceil_div(rq.hist, kTileN);
    const int last = unit_tiles(p, rq, nqt - 1, rq.q - (nqt - 1) * kTileM);
    return (I)(p.Hkv * (p.group / p.nq)) *
           (last + (I)(nqt - 1) * (hb + 1) + (I)(nqt - 1) * (nqt - 2) / 2 + nqt * p.unit_cost);
}

// Positions of the request's longest unit (its last query tile), 0 for decode /
// invalid / empty requests.
__device__ int longest_unit(const PlanParams &p, const Req &rq)
{
    if (!rq.valid || rq.q < 2)
        return 0;
    const int nqt = ceil_div(rq.q, kTileM);
    return unit_tiles(p, rq, nqt - 1, rq.q - (nqt - 1) * kTileM) + p.unit_cost;
}

// Positions of the request's shortest unit (its first query tile), INT_MAX for
// decode / invalid / empty requests.
__device__ int shortest_unit(const PlanParams &p, const Req &rq)
{
    if (!rq.valid || rq.q < 2)
        return 0x7fffffff;
    return unit_tiles(p, rq, 0, min(kTileM, rq.q)) + p.unit_cost;
}

__device__ int decode_splits(const Req &rq, int max_splits, int dec_keys)
{
    const int nch = ceil_div(rq.s, kDecodeChunk);
    int ns = ceil_div(rq.s, dec_keys);
    ns = min(ns, max_splits);
    ns = min(ns, nch);
    return max(ns, 1);
}

// pieces; partial rows; combine units and combine items (split decode rows);
// decode items; split prefill units
struct Counts {
    int pieces, prows, cunits, citems, ditems, sunits;
};

__device__ __forceinline__ int warp_excl_scan(int x, int lane, int &total)
{
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    total = __shfl_sync(0xffffffffu, incl, 31);
    return incl - x;
}

// A request's counts as long as no run boundary cuts a unit (see add_cuts).
__device__ Counts request_counts(const PlanParams &p, const Req &rq, int max_splits)
{
    Counts c{0, 0, 0, 0, 0, 0};
    if (!rq.valid || rq.q == 0)
        return c;
    if (rq.q > 1) {
        c.pieces = ceil_div(rq.q, kTileM) * p.Hkv * (p.group / p.nq);
    } else if (!p.dec_stream) {   // (streamed rows: decode_stream_work)
        const int ns = decode_splits(rq, max_splits, p.dec_keys);
        c.ditems = p.Hkv / p.dec_heads * ns;   // decode items per split, times the splits
        if (ns > 1) {
            c.prows = p.Hq * ns;
            c.citems = 1;
            c.cunits = p.Hq;
        }
    }
    return c;
}

// The first position of the a-th query tile from the last, behind the request's own: the tiles of
// query tiles nqt - 1 .. nqt - a (nkv_last, then hb + nqt - a' for a' = 1 .. a - 1) and their units' costs.
__device__ __forceinline__ int query_tile_pos(const PlanParams &p, int a, int upq, int nqt, int hb, int nkv_last)
{
    const int before = a == 0 ? 0 : nkv_last + (a - 1) * (hb + nqt) - (a - 1) * a / 2;
    return upq * (before + a * p.unit_cost);
}

// Where run boundaries cut units, without a walk over the units: there is a boundary a CTA, and a
// thread finds the request and the unit that it falls into by bisection. Of the n requests with
// lengths q, s and first tiles tile_off, up to tile `end`, cuts[r] (zero before) gets the
// boundaries inside a unit's tiles, and in its upper half the units that hold them. By the block.
__device__ void count_cuts(const PlanParams &p, const int *q, const int *s, const int *tile_off, int n, int end, int run,
                           int *cuts)
{
    const int lane = threadIdx.x & 31, k0 = tile_off[0] / run + 1, nb = (end - 1) / run - k0 + 1;
    for (int i0 = threadIdx.x - lane; i0 < nb; i0 += blockDim.x) {
        int r = -1;
        bool inside = false, first = false;   // inside a unit's tiles; and the first one there
        if (i0 + lane < nb) {
            const int x = (k0 + i0 + lane) * run;
            int hi = n - 1;                   // the last request that starts at x or ahead of it
            r = 0;
            while (r < hi) {
                const int mid = (r + hi + 1) / 2;
                if (tile_off[mid] <= x)
                    r = mid;
                else
                    hi = mid - 1;
            }
            const Req rq = make_req(p, q[r], s[r]);
            const int upq = p.Hkv * (p.group / p.nq), nqt = ceil_div(rq.q, kTileM), hb = ceil_div(rq.hist, kTileN);
            const int nkv_last = unit_tiles(p, rq, nqt - 1, rq.q - (nqt - 1) * kTileM), y = x - tile_off[r];
            int a = 0;                        // the last of its query tiles that starts at y or ahead of it
            hi = nqt - 1;
            while (a < hi) {
                const int mid = (a + hi + 1) / 2;
                if (query_tile_pos(p, mid, upq, nqt, hb, nkv_last) <= y)
                    a = mid;
                else
                    hi = mid - 1;
            }
            const int z = (y - query_tile_pos(p, a, upq, nqt, hb, nkv_last)) %
                          ((a == 0 ? nkv_last : hb + nqt - a) + p.unit_cost);
            inside = z > p.unit_cost;
            first = inside && z - run <= p.unit_cost;
        }
        const uint32_t alike = __match_any_sync(0xffffffffu, r);   // the warp's boundaries of the same request
        const uint32_t in = __ballot_sync(0xffffffffu, inside) & alike, units = __ballot_sync(0xffffffffu, first) & alike;
        if (in != 0 && lane == __ffs(alike) - 1)
            atomicAdd(&cuts[r], __popc(in) | __popc(units) << 16);
    }
}

__device__ __forceinline__ void add_cuts(const PlanParams &p, int cuts, Counts &c)
{
    const int in = cuts & 0xffff, units = cuts >> 16;
    c.pieces += in;
    c.sunits += units;
    c.prows += kTileM * p.nq * (in + units);
}

// One request's work, walked by a whole warp (all arguments warp-uniform): its
// entries are written at the given offsets, lane l of each pass taking one unit
// and placing its pieces by a warp scan. Returns their counts.
// tile_off: global index of the request's first prefill tile; run: tiles per CTA
// run; cut: whether a run boundary may split a unit (else a unit goes whole to
// the run that holds its first tile).
__device__ Counts request_work(const PlanParams &p, int r, const Req &rq, int tile_off, int run, bool cut,
                               int max_splits, int q_off, const Counts &off, int lane)
{
    Counts c{0, 0, 0, 0, 0, 0};
    if (!rq.valid || rq.q == 0)
        return c;
    if (rq.q == 1 && p.dec_stream)   // see DecodeStream
        return c;
    if (rq.q == 1) {
        const int ns = decode_splits(rq, max_splits, p.dec_keys);
        const int nch = ceil_div(rq.s, kDecodeChunk);
        const int ngroups = p.Hkv / p.dec_heads;   // decode items per split
        c = request_counts(p, rq, max_splits);
        for (int k = lane; k < c.ditems; k += 32) {
            const int sp = k / ngroups, kvh = k % ngroups;
            const int c0 = sp * nch / ns, c1 = (sp + 1) * nch / ns;
            const int key1 = min(c1 * kDecodeChunk, rq.s);
            p.ditems[off.ditems + k] = DecodeItem{r, kvh, c0 * kDecodeChunk, key1, sp, ns,
                                                  ns > 1 ? off.prows : -1, q_off};
        }
        if (ns > 1 && lane == 0)
            p.citems[off.citems] = CombineItem{q_off, 1, 0, p.Hq, off.prows, ns, off.cunits, 0};
        return c;
    }
    // prefill units in order: query tiles (longest KV range first), kv heads, head
    // pairs. Lane l of pass g0 takes unit g = g0 + l, the a-th query tile from the
    // last; its first tile is found in closed form (unit_tiles is hb + qt + 1 for
    // every query tile but the last, which may be short).
    static_assert(kTileM == kTileN, "unit tile counts assume square tiles");
    const int pairs = p.group / p.nq;
    const int upq = p.Hkv * pairs;            // units per query tile
    const int nqt = ceil_div(rq.q, kTileM);
    const int hb = ceil_div(rq.hist, kTileN);
    const int nkv_last = unit_tiles(p, rq, nqt - 1, rq.q - (nqt - 1) * kTileM);
    const int prow_unit = kTileM * p.nq;      // partial rows of one piece of a split unit
    const unsigned lanes_below = (1u << lane) - 1u;
    for (int g0 = 0; g0 < nqt * upq; g0 += 32) {
        const int g = g0 + lane;
        const bool active = g < nqt * upq;
        const int a = g / upq, j = g - a * upq;
        const int qt = nqt - 1 - a;
        const int nkv = a == 0 ? nkv_last : hb + qt + 1;
        // the unit's positions [u0, u1): unit_cost of fixed cost, then its tiles from t0
        const int u0 = tile_off + query_tile_pos(p, a, upq, nqt, hb, nkv_last) + j * (nkv + p.unit_cost);
        const int t0 = u0 + p.unit_cost, u1 = t0 + nkv;
        const int first = t0 / run;
        const int np = active ? (cut ? (u1 - 1) / run - first + 1 : 1) : 0;
        const bool split = np > 1;
        // one scan for two sums: pieces (low word) and pieces of split units (high word)
        long long sc = (long long)np | ((long long)(split ? np : 0) << 32);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, sc, o);
            if (lane >= o) sc += y;
        }
        const long long tot = __shfl_sync(0xffffffffu, sc, 31);
        const long long ex = sc - ((long long)np | ((long long)(split ? np : 0) << 32));
        const unsigned split_lanes = __ballot_sync(0xffffffffu, split);
        if (active) {
            const int kvh = j / pairs, hp = j - kvh * pairs;
            const int i0 = qt * kTileM;
            const int pi = off.pieces + c.pieces + (int)(ex & 0xffffffffll);
            // with cuts, every run starts a piece: the piece holding position c *
            // run (or the first one after it when that position is a unit's fixed
            // cost) is the first of CTA c's run
            if (!split) {
                p.pitems[pi] = PrefillItem{r, i0, kvh | (hp << 16), 0, nkv, (1 << 16), -1, first};
                if (cut && u0 <= first * run)
                    p.run_first[first] = pi;
            } else {
                // a split unit's partials: kTileM rows x nq heads x np pieces (see the chunk kernel's merge)
                const int pbase = off.prows + c.prows + prow_unit * (int)(ex >> 32);
                const int sunit = off.sunits + c.sunits + __popc(split_lanes & lanes_below);
                int x = t0;
                for (int pc = 0; pc < np; ++pc) {
                    const int owner = first + pc;
                    const int end = min(u1, (owner + 1) * run);
                    p.pitems[pi + pc] =
                        PrefillItem{r, i0, kvh | (hp << 16), x - t0, end - t0, pc | (np << 16), pbase, sunit};
                    if (pc > 0 || u0 <= owner * run)
                        p.run_first[owner] = pi + pc;
                    x = end;
                }
            }
        }
        c.pieces += (int)(tot & 0xffffffffll);
        c.sunits += __popc(split_lanes);
        c.prows += prow_unit * (int)(tot >> 32);
    }
    return c;
}

// Stream-K run length; cuts inside units only when splitting is allowed and the
// partials' bound fits the workspace (else nothing is split and the flag is set).
// A cut costs the run that holds it a second item and, at its end, a merge
// (about kCutCostTiles tiles of work, measured). When every unit is at least a
// run long, whole units land one per CTA (no run holds two unit starts) and cost
// the longest unit's length: then, if that is within kCutCostTiles of the run,
// nothing is cut.
struct SplitChoice {
    int run, max_splits;
    bool split_prefill, clamped;
};

__device__ SplitChoice choose_split(const PlanParams &p, long long tiles, int shortest, int longest,
                                    long long dprows)
{
    const int grid = max(1, p.chunk_grid);
    SplitChoice c;
    c.run = max((int)((tiles + grid - 1) / grid), kMinRunTiles);
    c.max_splits = p.max_splits;
    c.split_prefill = p.max_splits > 1;
    c.clamped = false;
    const long long pbound = (long long)2 * grid * kTileM * p.nq;
    if (p.max_splits > 1 && pbound + dprows > p.prow_capacity) {
        c.max_splits = 1;
        c.split_prefill = false;
        c.clamped = true;
    }
    if (c.split_prefill && !cut_units(shortest, longest, c.run))
        c.split_prefill = false;
    return c;
}

// run_first[c] = first piece whose owner is >= c (pieces are sorted by owner);
// threads tid, tid + nthreads, ... of the caller share the entries. With cuts the
// emission already wrote the entries of runs holding tiles (runs [0, ceil(W /
// run))), and only the rest are set here; without cuts they are read back from
// the pieces' owners.
__device__ void fill_run_first(const PlanParams &p, int n_pieces, int grid, bool cut, long long tiles, int run,
                               int tid, int nthreads)
{
    if (cut) {
        const int first_empty = (int)((tiles + run - 1) / run);
        for (int c = first_empty + tid; c <= grid; c += nthreads) p.run_first[c] = n_pieces;
        return;
    }
    for (int i = tid; i <= n_pieces; i += nthreads) {
        const int lo = i == 0 ? 0 : p.pitems[i - 1].aux + 1;   // without cuts, aux is the owner CTA
        const int hi = i == n_pieces ? grid : p.pitems[i].aux;
        for (int c = lo; c <= hi; ++c) p.run_first[c] = i;
    }
}

// Block-wide exclusive scan of N ints; returns the totals.
template <int N, typename T>
__device__ void block_scan(T (&v)[N], T (&tot)[N])
{
    __shared__ T warp_sums[kPlanThreads / 32][N];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T incl[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        T x = v[j];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        incl[j] = x;
    }
    if (lane == 31)
        for (int j = 0; j < N; ++j) warp_sums[warp][j] = incl[j];
    __syncthreads();
    if (warp == 0) {
        for (int j = 0; j < N; ++j) {
            T x = warp_sums[lane][j];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const T y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            warp_sums[lane][j] = x;   // inclusive over warps
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const T before = warp > 0 ? warp_sums[warp - 1][j] : 0;
        tot[j] = warp_sums[kPlanThreads / 32 - 1][j];
        v[j] = before + incl[j] - v[j];
    }
    __syncthreads();
}

// Decode rows cut stream-K style (dec_stream, see plan.cuh): a unit is a row and one item's
// heads; a request's units follow one another from tile u0 on. One thread does one request.
struct DecodeStream {
    long long tiles;   // of all units
    int run;           // tiles per CTA
    bool cut;          // whether a run boundary may split a unit (else a unit goes whole to the run of its first tile)
};

__device__ __forceinline__ int decode_tiles(const PlanParams &p, const Req &rq)
{
    return p.dec_stream && rq.valid && rq.q == 1 ? ceil_div(rq.s, kDecodeChunk) : 0;
}

// Partial rows that a request's units can take, before the run is known (a bound: max_splits each).
__device__ __forceinline__ int decode_stream_rows(const PlanParams &p, int tiles)
{
    return tiles > 1 ? p.Hq * p.max_splits : 0;
}

// The bound of all: a boundary between two runs leaves two more pieces of one unit at most.
__device__ __forceinline__ long long decode_stream_bound(const PlanParams &p, long long rows)
{
    return min(rows, (long long)2 * p.dec_grid * p.dec_heads * p.group);
}

__device__ DecodeStream decode_stream(const PlanParams &p, long long tiles, int longest, int max_splits)
{
    DecodeStream d;
    d.tiles = tiles;
    d.cut = max_splits > 1;
    d.run = (int)max((tiles + p.dec_grid - 1) / p.dec_grid, (long long)kMinDecodeRun);
    if (d.cut)
        d.run = max(d.run, ceil_div(longest - 1, max_splits - 1));
    return d;
}

// A request's counts; with emit its items at the given offsets.
__device__ Counts decode_stream_work(const PlanParams &p, const DecodeStream &d, int r, const Req &rq, long long u0,
                                     bool emit, int q_off, const Counts &off)
{
    Counts c{0, 0, 0, 0, 0, 0};
    const int n = decode_tiles(p, rq);
    if (n == 0)
        return c;
    const int ngroups = p.Hkv / p.dec_heads, nh = p.dec_heads * p.group;
    for (int g = 0; g < ngroups; ++g, u0 += n) {
        const long long first = u0 / d.run;
        const int np = d.cut ? (int)((u0 + n - 1) / d.run - first + 1) : 1;
        if (emit) {
            const int item = off.ditems + c.ditems, rows = off.prows + c.prows;
            for (int k = 0; k < np; ++k) {
                // piece k: the tiles of run first + k
                const long long lo = k == 0 ? u0 : (first + k) * d.run;
                const long long hi = k == np - 1 ? u0 + n : (first + k + 1) * d.run;
                p.ditems[item + k] = DecodeItem{r, g, (int)(lo - u0) * kDecodeChunk,
                                                min((int)(hi - u0) * kDecodeChunk, rq.s), k, np,
                                                np > 1 ? rows - g * nh * np : -1, q_off};
                if (d.cut && lo == (first + k) * d.run)
                    p.dec_first[first + k] = item + k;
            }
            if (!d.cut) {
                if (u0 == 0)
                    p.dec_first[0] = item;
                for (long long x = first + 1; x <= min((u0 + n) / d.run, (long long)p.dec_grid); ++x)
                    p.dec_first[x] = item + 1;
            }
            if (np > 1)
                p.citems[off.citems + c.citems] = CombineItem{q_off, 1, g * nh, nh, rows, np, off.cunits + c.cunits, 0};
        }
        c.ditems += np;
        if (np > 1) {
            c.prows += nh * np;
            c.citems += 1;
            c.cunits += nh;
        }
    }
    return c;
}

// dec_first of the runs behind the last tile.
__device__ void decode_stream_tail(const PlanParams &p, const DecodeStream &d, int n_items, int tid, int nthreads)
{
    const long long behind = d.cut || d.tiles == 0 ? (d.tiles + d.run - 1) / d.run : d.tiles / d.run + 1;
    for (long long x = behind + tid; x <= p.dec_grid; x += nthreads) p.dec_first[x] = n_items;
}

// What the block sums up (and takes the extremes of) before it walks the requests.
struct PlanTotals {
    long long tok, tiles, dprows, dtiles;
    int longest, shortest, dlongest;
};

template <bool STREAM>
__device__ __forceinline__ void warp_totals(PlanTotals &t)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        t.tok += __shfl_xor_sync(0xffffffffu, t.tok, o);
        t.tiles += __shfl_xor_sync(0xffffffffu, t.tiles, o);
        t.dprows += __shfl_xor_sync(0xffffffffu, t.dprows, o);
    }
    t.longest = __reduce_max_sync(0xffffffffu, t.longest);
    t.shortest = __reduce_min_sync(0xffffffffu, t.shortest);
    if (STREAM) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t.dtiles += __shfl_xor_sync(0xffffffffu, t.dtiles, o);
        t.dlongest = __reduce_max_sync(0xffffffffu, t.dlongest);
    }
}

// Over the block, for all its threads: the warps' totals meet in shared memory, and every warp adds them up.
__device__ void block_totals(PlanTotals &t)
{
    __shared__ PlanTotals red[kPlanThreads / 32];
    warp_totals<true>(t);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = t;
    __syncthreads();
    t = red[threadIdx.x & 31];
    warp_totals<true>(t);
}

// One request's part of the totals.
template <bool STREAM>
__device__ __forceinline__ void add_request(const PlanParams &p, const Req &rq, PlanTotals &t)
{
    t.tok += rq.q > 0 ? rq.q : 0;   // invalid requests still occupy their rows
    t.tiles += prefill_tiles<long long>(p, rq);
    t.longest = max(t.longest, longest_unit(p, rq));
    t.shortest = min(t.shortest, shortest_unit(p, rq));
    if (STREAM && p.dec_stream) {
        const int n = decode_tiles(p, rq);
        t.dtiles += (long long)n * (p.Hkv / p.dec_heads);
        t.dlongest = max(t.dlongest, n);
        t.dprows += decode_stream_rows(p, n);
    } else if (rq.valid && rq.q == 1) {
        const int ns = decode_splits(rq, p.max_splits, p.dec_keys);
        if (ns > 1) t.dprows += (long long)p.Hq * ns;
    }
}

// The flag of a batch of which nothing can be computed; 0: none.
__device__ __forceinline__ uint32_t plan_refused(const PlanParams &p, const PlanTotals &tot)
{
    return tot.tok != p.num_tokens ? CPSA_DEV_TOKENS_MISMATCH : tot.tiles > kMaxPlanTiles ? CPSA_DEV_PLAN_OVERFLOW : 0u;
}

__global__ void __launch_bounds__(kPlanThreads, 1) plan_kernel(PlanParams p)
{
    // dependents are released at the end (see plan_small_kernel)
    pdl_wait();
    // ---- pass 1: tokens, prefill tiles, decode tiles and partial rows
    PlanTotals tot{0, 0, 0, 0, 0, 0x7fffffff, 0};
    for (int base = 0; base < p.num_reqs; base += kPlanThreads) {
        const int r = base + threadIdx.x;
        if (r < p.num_reqs)
            add_request<true>(p, load_req(p, r), tot);
    }
    block_totals(tot);
    const long long tiles = tot.tiles;
    if (p.dec_stream)
        tot.dprows = decode_stream_bound(p, tot.dprows);
    if (const uint32_t bad = plan_refused(p, tot)) {
        if (threadIdx.x == 0) set_dev_error(p.dev_err, bad);
        if (threadIdx.x < kCntSlots) p.counts[threadIdx.x] = 0;
        for (int c = threadIdx.x; c <= p.chunk_grid; c += kPlanThreads) p.run_first[c] = 0;
        for (int c = threadIdx.x; p.dec_stream && c <= p.dec_grid; c += kPlanThreads) p.dec_first[c] = 0;
        return;
    }
    const int grid = max(1, p.chunk_grid);
    const SplitChoice sc = choose_split(p, tiles, tot.shortest, tot.longest, tot.dprows);
    DecodeStream ds{0, 1, false};
    if (p.dec_stream)
        ds = decode_stream(p, tot.dtiles, tot.dlongest, sc.max_splits);
    const int run = sc.run, max_splits = sc.max_splits;
    const bool split_prefill = sc.split_prefill;
    if (sc.clamped && threadIdx.x == 0)
        set_dev_error(p.dev_err, CPSA_DEV_SPLITS_CLAMPED);

    // ---- pass 2: offsets and lists, 1024 requests at a time
    __shared__ int s_qoff[kPlanThreads], s_toff[kPlanThreads], s_q[kPlanThreads], s_s[kPlanThreads];
    __shared__ int s_cnt[kPlanThreads][kScan], s_cuts[kPlanThreads];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int carry_a[2] = {0, 0};                        // tokens, tiles
    long long carry_d = 0;                          // streamed decode tiles
    int carry_b[kScan] = {0, 0, 0, 0, 0, 0};        // pieces, prows, cunits, citems, ditems, sunits
    for (int base = 0; base < p.num_reqs; base += kPlanThreads) {
        const int nloc = min(kPlanThreads, p.num_reqs - base);
        // (a) token and tile offsets: one thread per request
        Req mine{false, 0, 0, 0};
        {
            s_cuts[threadIdx.x] = 0;
            const int r = base + threadIdx.x;
            int va[2] = {0, 0};
            if (threadIdx.x < nloc) {
                mine = load_req(p, r);
                const Req &rq = mine;
                s_q[threadIdx.x] = rq.q;
                s_s[threadIdx.x] = rq.s;
                va[0] = rq.q > 0 ? rq.q : 0;
                va[1] = prefill_tiles(p, rq);
                if (!rq.valid)
                    set_dev_error(p.dev_err, (rq.q < 0 || rq.s < rq.q) ? CPSA_DEV_SEQ_LT_QUERY : CPSA_DEV_SEQ_GT_TABLE);
            }
            int ta[2];
            block_scan(va, ta);
            s_qoff[threadIdx.x] = carry_a[0] + va[0];
            s_toff[threadIdx.x] = carry_a[1] + va[1];
            if (threadIdx.x < nloc)
                p.cu_q[r] = carry_a[0] + va[0];
            carry_a[0] += ta[0];
            carry_a[1] += ta[1];
        }
        // streamed decode rows: one thread per request
        long long my_u0 = 0;
        Counts my_dec{0, 0, 0, 0, 0, 0};
        if (p.dec_stream) {
            long long vd[1] = {(long long)decode_tiles(p, mine) * (p.Hkv / p.dec_heads)}, td[1];
            block_scan(vd, td);
            my_u0 = carry_d + vd[0];
            carry_d += td[0];
            my_dec = decode_stream_work(p, ds, base + threadIdx.x, mine, my_u0, false, 0, Counts{0, 0, 0, 0, 0, 0});
        }
        __syncthreads();
        // (b) counts: run boundaries inside units, then one thread per request
        if (split_prefill)
            count_cuts(p, s_q, s_s, s_toff, nloc, carry_a[1], run, s_cuts);
        __syncthreads();
        // (c) list offsets: one thread per request
        {
            Counts c = threadIdx.x < nloc ? request_counts(p, mine, max_splits) : Counts{0, 0, 0, 0, 0, 0};
            add_cuts(p, s_cuts[threadIdx.x], c);
            int vb[kScan] = {c.pieces, c.prows + my_dec.prows, c.cunits + my_dec.cunits, c.citems + my_dec.citems,
                             c.ditems + my_dec.ditems, c.sunits};
            int tb[kScan];
            block_scan(vb, tb);
            for (int j = 0; j < kScan; ++j) s_cnt[threadIdx.x][j] = carry_b[j] + vb[j];
            for (int j = 0; j < kScan; ++j) carry_b[j] += tb[j];
        }
        __syncthreads();
        // (d) the lists: streamed decode rows, then one warp per request
        if (my_dec.ditems > 0) {
            const int *o = s_cnt[threadIdx.x];
            decode_stream_work(p, ds, base + threadIdx.x, mine, my_u0, true, s_qoff[threadIdx.x],
                               Counts{o[0], o[1], o[2], o[3], o[4], o[5]});
        }
        for (int l = warp; l < nloc; l += kPlanThreads / 32) {
            const Req rq = make_req(p, s_q[l], s_s[l]);
            const Counts off{s_cnt[l][0], s_cnt[l][1], s_cnt[l][2], s_cnt[l][3], s_cnt[l][4], s_cnt[l][5]};
            request_work(p, base + l, rq, s_toff[l], run, split_prefill, max_splits, s_qoff[l], off, lane);
        }
        __syncthreads();
    }
    __syncthreads();   // this block's piece writes are visible to the whole block
    const int n_pieces = (int)min((int64_t)carry_b[0], p.max_pitems);
    fill_run_first(p, n_pieces, grid, split_prefill, tiles, run, threadIdx.x, kPlanThreads);
    if (p.dec_stream)
        decode_stream_tail(p, ds, carry_b[4], threadIdx.x, kPlanThreads);
    if (threadIdx.x == 0) {
        p.cu_q[p.num_reqs] = carry_a[0];
        p.counts[kCntPrefill] = (int)min((int64_t)carry_b[0], p.max_pitems);
        p.counts[kCntCombine] = (int)min((int64_t)carry_b[3], p.max_citems);
        p.counts[kCntPartialRows] = carry_b[1];
        p.counts[kCntCombineUnits] = carry_b[2];
        p.counts[kCntDecode] = (int)min((int64_t)carry_b[4], p.max_ditems);
        p.counts[kCntRunTiles] = run;
        p.counts[kCntSplitUnits] = carry_b[5];
        for (int j = kCntSplitUnits + 1; j < kCntSlots; ++j) p.counts[j] = 0;
    }
    pdl_trigger();
}

// A batch of at most 32 requests as one warp, lane r holding request r, has it at first: totals, then
// offsets by warp scans, and the streamed decode rows' lists (STREAM: dec_stream).
struct SmallPlan {
    Req rq;                                   // of the lane's request
    int tok_off, tile_off, tok_total, tile_total;
    SplitChoice sc;
    DecodeStream ds;
    Counts off;                               // entries ahead of the other requests' lists
};

// False where the batch is refused (the lists are empty then).
template <bool STREAM>
__device__ __forceinline__ bool small_plan(const PlanParams &p, int lane, SmallPlan &w)
{
    const bool mine = lane < p.num_reqs;
    w.rq = Req{false, 0, 0, 0};
    if (mine)
        w.rq = load_req(p, lane);
    // totals in 64 bits first: the 32-bit scans below are only used once they fit
    PlanTotals tot{0, 0, 0, 0, 0, 0x7fffffff, 0};
    if (mine)
        add_request<STREAM>(p, w.rq, tot);
    warp_totals<STREAM>(tot);
    if (const uint32_t bad = plan_refused(p, tot)) {
        if (lane == 0) set_dev_error(p.dev_err, bad);
        if (lane < kCntSlots) p.counts[lane] = 0;
        for (int c = lane; c <= p.chunk_grid; c += 32) p.run_first[c] = 0;
        if (STREAM)
            for (int c = lane; c <= p.dec_grid; c += 32) p.dec_first[c] = 0;
        return false;
    }
    if (mine && !w.rq.valid)
        set_dev_error(p.dev_err, (w.rq.q < 0 || w.rq.s < w.rq.q) ? CPSA_DEV_SEQ_LT_QUERY : CPSA_DEV_SEQ_GT_TABLE);
    // (invalid requests still occupy their rows)
    w.tok_off = warp_excl_scan(mine && w.rq.q > 0 ? w.rq.q : 0, lane, w.tok_total);
    w.tile_off = warp_excl_scan(mine ? prefill_tiles(p, w.rq) : 0, lane, w.tile_total);
    if (mine)
        p.cu_q[lane] = w.tok_off;
    if (lane == 0)
        p.cu_q[p.num_reqs] = w.tok_total;
    w.sc = choose_split(p, tot.tiles, tot.shortest, tot.longest, STREAM ? decode_stream_bound(p, tot.dprows) : tot.dprows);
    if (w.sc.clamped && lane == 0)
        set_dev_error(p.dev_err, CPSA_DEV_SPLITS_CLAMPED);
    w.off = Counts{0, 0, 0, 0, 0, 0};
    w.ds = DecodeStream{0, 1, false};
    if (STREAM) {
        // streamed decode rows: a lane per request, ahead of the prefill requests' lists
        w.ds = decode_stream(p, tot.dtiles, tot.dlongest, w.sc.max_splits);
        long long u0 = (long long)decode_tiles(p, w.rq) * (p.Hkv / p.dec_heads);
        const long long own = u0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, u0, o);
            if (lane >= o) u0 += y;
        }
        u0 -= own;
        const Counts c = decode_stream_work(p, w.ds, lane, w.rq, u0, false, 0, w.off);
        Counts at;
        at.pieces = at.sunits = 0;
        at.prows = warp_excl_scan(c.prows, lane, w.off.prows);
        at.cunits = warp_excl_scan(c.cunits, lane, w.off.cunits);
        at.citems = warp_excl_scan(c.citems, lane, w.off.citems);
        at.ditems = warp_excl_scan(c.ditems, lane, w.off.ditems);
        decode_stream_work(p, w.ds, lane, w.rq, u0, true, w.tok_off, at);
    }
    return true;
}

// The lists' ends, with `end` entries in them: by all threads.
template <bool STREAM>
__device__ __forceinline__ void finish_plan(const PlanParams &p, const Counts &end, const SplitChoice &sc, const DecodeStream &ds,
                                            long long tiles, int nthreads)
{
    const int n_pieces = (int)min((int64_t)end.pieces, p.max_pitems);
    fill_run_first(p, n_pieces, max(1, p.chunk_grid), sc.split_prefill, tiles, sc.run, threadIdx.x, nthreads);
    if (STREAM)
        decode_stream_tail(p, ds, end.ditems, threadIdx.x, nthreads);
    if (threadIdx.x == 0) {
        p.counts[kCntPrefill] = n_pieces;
        p.counts[kCntCombine] = (int)min((int64_t)end.citems, p.max_citems);
        p.counts[kCntPartialRows] = end.prows;
        p.counts[kCntCombineUnits] = end.cunits;
        p.counts[kCntDecode] = (int)min((int64_t)end.ditems, p.max_ditems);
        p.counts[kCntRunTiles] = sc.run;
        p.counts[kCntSplitUnits] = end.sunits;
    } else if (threadIdx.x > kCntSplitUnits && threadIdx.x < kCntSlots) {
        p.counts[threadIdx.x] = 0;
    }
}

// The same lists by one warp, which walks the requests in order: every request's
// list offsets are the running totals of the ones before it.
template <bool STREAM>
__global__ void __launch_bounds__(32, 1) plan_small_kernel(PlanParams p)
{
    // The attention kernels that follow are released only at the end: CTAs
    // launched early wait beside this warp and halve its speed (measured), while
    // what they would overlap is short.
    pdl_wait();
    const int lane = threadIdx.x;
    SmallPlan w;
    if (!small_plan<STREAM>(p, lane, w))
        return;
    Counts off = w.off;
    for (int r = 0; r < p.num_reqs; ++r) {
        Req rr;
        rr.valid = __shfl_sync(0xffffffffu, w.rq.valid ? 1 : 0, r) != 0;
        rr.q = __shfl_sync(0xffffffffu, w.rq.q, r);
        rr.s = __shfl_sync(0xffffffffu, w.rq.s, r);
        rr.hist = __shfl_sync(0xffffffffu, w.rq.hist, r);
        const int qoff = __shfl_sync(0xffffffffu, w.tok_off, r);
        const int toff = __shfl_sync(0xffffffffu, w.tile_off, r);
        const Counts c = request_work(p, r, rr, toff, w.sc.run, w.sc.split_prefill, w.sc.max_splits, qoff, off, lane);
        off.pieces += c.pieces;
        off.prows += c.prows;
        off.cunits += c.cunits;
        off.citems += c.citems;
        off.ditems += c.ditems;
        off.sunits += c.sunits;
    }
    __syncwarp();   // the warp's piece writes are visible to all its lanes
    finish_plan<STREAM>(p, off, w.sc, w.ds, w.tile_total, 32);
    pdl_trigger();
}

// The same lists by a warp a request: the first warp begins as the one above; then all threads count
// the cuts, and every warp adds up the entries ahead of its request's and writes these.
template <bool STREAM>
__global__ void __launch_bounds__(kPlanThreads, 1) plan_warps_kernel(PlanParams p)
{
    __shared__ int s_q[32], s_s[32], s_qoff[32], s_toff[32], s_cuts[32], s_ok;
    __shared__ Counts s_cnt[32], s_end;   // a request's entries; all requests'
    __shared__ SmallPlan s_plan;          // of lane 0
    pdl_wait();                           // (dependents are released at the end, as above)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp == 0) {
        SmallPlan w;
        const bool ok = small_plan<STREAM>(p, lane, w);
        if (ok) {
            s_q[lane] = w.rq.q;
            s_s[lane] = w.rq.s;
            s_qoff[lane] = w.tok_off;
            s_toff[lane] = w.tile_off;
            s_cuts[lane] = 0;
            s_cnt[lane] = request_counts(p, w.rq, w.sc.max_splits);
            if (lane == 0)
                s_plan = w;
        }
        if (lane == 0)
            s_ok = ok;
    }
    __syncthreads();
    if (!s_ok)
        return;
    const SplitChoice sc = s_plan.sc;
    if (sc.split_prefill) {
        count_cuts(p, s_q, s_s, s_toff, p.num_reqs, s_plan.tile_total, sc.run, s_cuts);
        __syncthreads();
    }
    Counts b{0, 0, 0, 0, 0, 0}, off = s_plan.off;
    if (lane < warp) {                    // the requests ahead
        b = s_cnt[lane];
        add_cuts(p, s_cuts[lane], b);
    }
    off.pieces += __reduce_add_sync(0xffffffffu, b.pieces);
    off.prows += __reduce_add_sync(0xffffffffu, b.prows);
    off.cunits += __reduce_add_sync(0xffffffffu, b.cunits);
    off.citems += __reduce_add_sync(0xffffffffu, b.citems);
    off.ditems += __reduce_add_sync(0xffffffffu, b.ditems);
    off.sunits += __reduce_add_sync(0xffffffffu, b.sunits);
    const Counts c = request_work(p, warp, make_req(p, s_q[warp], s_s[warp]), s_toff[warp], sc.run, sc.split_prefill,
                                  sc.max_splits, s_qoff[warp], off, lane);
    if (warp == p.num_reqs - 1 && lane == 0)
        s_end = Counts{off.pieces + c.pieces, off.prows + c.prows, off.cunits + c.cunits,
                       off.citems + c.citems, off.ditems + c.ditems, off.sunits + c.sunits};
    __syncthreads();                      // the pieces are visible to all warps
    finish_plan<STREAM>(p, s_end, sc, s_plan.ds, s_plan.tile_total, blockDim.x);
    pdl_trigger();
}

}  // namespace

// Which kernel, by the number of requests alone: what else decides (whether one request holds most of
// the units) the host does not know. One warp walks every request's units itself, about 0.5 us
// per 32 units and 0.3 us a request; a warp a request walks them side by side, but for the price of
// barriers and of counting them first. Calls over a bf16 cache, 32/8 heads, D 128, replayed (other
// caches alike), by one warp and by a warp a request: a decode row and a chunk of 256 tokens at history
// 3000 56.8 and 58.6 us, three rows and that chunk 75.0 and 75.4, two prompts of 2500 124.3 and 121.3, four of
// 2000 163.2 and 152.1, four of 300 31.0 and 28.7, five rows 47.1 and 45.6. Past 32 requests, or by the block kernel:
// eight prompts of 1024 99.3 us, 95.3 by a warp a request; a chunk of 4096 beside eight rows 193.7 (its
// units walked twice then, once to count them) and 185.4.
constexpr int kPlanOneWarpReqs = 3;
constexpr int64_t kPlanOneWarpTokens = 8192;

cudaError_t launch_plan(const PlanParams &p, cudaStream_t s, bool early)
{
    if (p.num_reqs == 1 || (p.num_reqs <= kPlanOneWarpReqs && p.num_tokens <= kPlanOneWarpTokens))
        return launch_pdl(early, p.dec_stream ? plan_small_kernel<true> : plan_small_kernel<false>, dim3(1), dim3(32), 0, s, p);
    if (p.num_reqs <= 32)
        return launch_pdl(early, p.dec_stream ? plan_warps_kernel<true> : plan_warps_kernel<false>, dim3(1),
                          dim3(32 * p.num_reqs), 0, s, p);
    return launch_pdl(early, plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, p);
}

}  // namespace cpsa
