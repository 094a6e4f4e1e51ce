// Work list of the tcgen05 kernel in a language model's own attention, and the join of a prefix with what follows it.
//
// One block reads the offsets on the device (nothing returns to the host) and cuts units into items. A unit is a
// sequence with the keys that its mask lets through, or, with a prefix, one of:
//   - a sequence, whose items read the prefix first and then the sequence's own keys: one softmax over both;
//   - where sequences are short (`apart`): a group's queries of all its sequences over the prefix, so that tiles are
//     full and the prefix is read once per tile of the group instead of once per sequence, and a sequence over its own
//     keys. Both leave partial results, which window_join_kernel adds up row by row.
// Blocks of 256 rows, split items of 128 rows, cut key ranges and packed heads are those of cross attention (its list
// says more). Here a block's keys depend on its place: under a causal mask the last one of a sequence has the most. So
// units are ordered by their longest block, and a unit's blocks come last first, all heads of one after the other: long
// items start first, and what is left at the end is short.
#include <algorithm>

#include "block_sort.cuh"
#include "warp_mma.cuh"
#include "window.h"

namespace vit {
namespace {

constexpr int kThreads = kSortThreads;
// Three ways to make the list: up to 32 units by a warp, a unit per lane; up to kSmall (and where a prefix is apart) a unit
// per thread; more sorted by the block. Each is a kernel of its own, with and without prefixes: what it takes is latency,
// fetching its code included (all in one, a list of 1864 items took 2 us longer). With a prefix apart the second also
// chooses the length of runs, which the third leaves at the plan's shortest: sorted in place of a unit per thread, 254
// questions of 20 tokens behind two prefixes of 3000, 16 heads of 80 (256 units), take 236 us in a graph instead of 218;
// 100 of 30 behind one, 151 instead of 121.
enum { kByWarp, kByThread, kSorted };
constexpr int kSmall = 256;

// A unit's queries (rows [q0, q0 + qn), positions from p0 on) and its keys: the prefix rows [f0, f0 + fn), and the own
// keys from row k0 on (kn = 0: none).
struct Unit {
    int q0, qn, f0, fn, k0, kn, p0;
};
// what a unit's place in the slots is, for the join
struct UnitSlots {
    int q0, blocks, runs, slot;
};

struct Sched {
    CrossSegs s;
    int window, sinks;
    Groups groups;
    bool apart, own_few;
    int Hq, lg_pack, bn, run_tiles, num_sms;
    WsHeader *hdr;
    WinItem *items;
    CrossTile *tiles;
    CrossEmpty *empty;
    UnitSlots *units;
    float *part_s;
    int32_t *status;
};

// Unit u, and whether it can be used; `none` counts a sequence's queries that see nothing at all (its first rows).
template <bool PREFIX>
__device__ __forceinline__ bool load_unit(const Sched &p, int u, Unit &x, CrossEmpty &none, bool report)
{
    none = CrossEmpty{0, 0};
    x = Unit{0, 0, 0, 0, 0, 0, 0};
    if (PREFIX && p.apart && u < p.groups.G) {
        const int a = p.groups.bound(u), b = p.groups.bound(u + 1);
        const bool fine = p.groups.load(u, x.f0, x.fn);
        if (a < 0 || b < a || b > p.s.B) return false; // (reported with the groups)
        const int64_t q0 = p.s.cu_q[a], q1 = p.s.cu_q[b];
        if (!fine || q0 < 0 || q1 < q0 || q1 > p.s.Tq) return false;     // (the sequences report their offsets)
        x.q0 = (int)q0;
        x.qn = (int)(q1 - q0);
        return true;
    }
    const int b = PREFIX && p.apart ? u - p.groups.G : u;
    CrossSeg c;
    if (!load_seg(p.s, b, c, p.status, report)) return false;
    if (PREFIX && !p.apart) {
        if (!p.groups.load(p.groups.of(b), x.f0, x.fn)) return false;
    }
    const WinSeg w = win_seg(c);
    x.k0 = w.k0;
    x.kn = w.kn;
    x.q0 = w.q0;
    x.qn = w.qn;
    x.p0 = w.p0;
    if (PREFIX && x.fn > 0) {                          // all of them see the prefix
        x.q0 -= w.none;
        x.qn += w.none;
        x.p0 -= w.none;
    } else if (!PREFIX || !p.apart) {
        none = CrossEmpty{c.q0, w.none};
    }
    return true;
}

// What the queries [t, e) of a unit see between them, as an item says it.
struct Span {
    int f0, fn, lo, kn;
    __device__ int tiles(int bn) const { return (fn + bn - 1) / bn + (kn + bn - 1) / bn; }
};
template <bool PREFIX> __device__ __forceinline__ Span span_of(const Sched &p, const Unit &u, int t, int e)
{
    Span s{u.f0, u.fn, 0, 0};
    if (u.kn == 0) return s;
    const int first = u.p0 + t, last = u.p0 + e - 1;
    if (!PREFIX) {
        const WinRange r = win_range(first, p.window, p.sinks);
        s.f0 = u.k0;
        s.fn = r.first;
        s.lo = r.lo;
    }
    s.kn = max(0, last + 1 - s.lo);
    return s;
}

template <int MODE, bool PREFIX>
__global__ void __launch_bounds__(kThreads)
window_schedule_kernel(const Sched p)
{
    extern __shared__ unsigned long long s_key[];      // [NP]: longest block first, then index; later first item | index
    __shared__ int64_t s_warp[32];
    constexpr int KEPT = MODE == kByWarp ? 32 : MODE == kByThread ? kSmall : 1;
    __shared__ Unit s_unit[KEPT];                      // units in their order
    __shared__ int s_runs[KEPT];
    __shared__ int s_bad, s_used, s_total, s_tiles, s_all_split, s_more, s_empty, s_run;
    __shared__ unsigned long long s_best;
    grid_wait();
    grid_release();
    const int tid = threadIdx.x, n_units = !PREFIX ? p.s.B : p.own_few ? p.groups.G : p.apart ? p.groups.G + p.s.B : p.s.B;
    const bool apart = PREFIX && p.apart;
    int NP = 32;
    while (NP < n_units) NP <<= 1;
    int *s_tile = reinterpret_cast<int *>(s_key + NP); // [NP] first tile
    const int lg_tile = 7 - p.lg_pack;                 // tokens of a 128-row tile, log2
    const int packs = p.Hq >> p.lg_pack;
    auto longest = [&](const Unit &x) { return span_of<PREFIX>(p, x, max(0, x.qn - (1 << lg_tile)), x.qn).tiles(p.bn); };
    auto key_of = [&](bool use, const Unit &x, int i) {
        return ((unsigned long long)(use ? 0x7fffffffu - (uint32_t)longest(x) : 0xffffffffu) << 32) | (uint32_t)i;
    };
    auto blocks_of = [&](const Unit &x, int lg) { return packs * (int)(((unsigned)x.qn + (1u << lg) - 1u) >> lg); };
    auto runs_in = [&](int tiles, int run) { return run > 0 ? max(1, (tiles + run - 1) / run) : 1; };
    auto runs_of = [&](const Unit &x) { return runs_in(longest(x), p.run_tiles); };
    auto usable = [&](bool fine, const Unit &x) { return fine && x.qn > 0 && (x.fn > 0 || x.kn > 0); };
    // two-tile blocks of the batch: few of them means split items throughout
    auto split_all = [&](int64_t full) { return p.run_tiles > 0 || apart || 2 * full <= (int64_t)p.num_sms; };
    auto unfit = [&](int u, bool fine) {               // nothing is computed at all then
        const int b = apart ? u - p.groups.G : u;
        return (PREFIX && !fine) || (b >= 0 && p.s.cu_q[b + 1] < p.s.cu_q[b]);
    };
    bool wrong = false;                                // of a prefix call: then nothing is computed at all
    if constexpr (PREFIX) {
        for (int g = tid; g < p.groups.G; g += kThreads) {
            const int err = p.groups.error(g);
            if (err) report_error(p.status, err);
            wrong |= err != 0;
        }
        // (where sequences are no units: their rows have to lie inside their group's)
        if (p.own_few)
            for (int b = tid; b < p.s.B; b += kThreads) wrong |= p.s.cu_q[b + 1] < p.s.cu_q[b];
        wrong = __syncthreads_or(wrong);
    }
    if constexpr (MODE != kByWarp) {
        if (tid == 0) {
            s_bad = s_used = s_empty = 0;
            s_run = p.run_tiles;
            s_best = ~0ull;
        }
        __syncthreads();
    }
    if constexpr (MODE == kByWarp) {
        if (tid < 32) {
            Unit x;
            CrossEmpty none{0, 0};
            const bool fine = tid < n_units && load_unit<PREFIX>(p, tid, x, none, true);
            const bool bad = tid < n_units && unfit(tid, fine), use = usable(fine, x);
            int64_t full = use ? blocks_of(x, lg_tile + 1) : 0;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) full += __shfl_xor_sync(0xffffffffu, full, o);
            const bool all_split = split_all(full);
            const int n = use ? blocks_of(x, all_split ? lg_tile : lg_tile + 1) : 0, runs = use ? runs_of(x) : 1;
            int rank, at, tile_at;
            warp_place(key_of(use, x, tid), n * runs, runs > 1 ? n : 0, rank, at, tile_at);
            s_key[rank] = ((unsigned long long)at << 32) | (uint32_t)tid;
            s_tile[rank] = tile_at;
            s_unit[rank] = x;
            s_runs[rank] = runs;
            const unsigned used = __ballot_sync(0xffffffffu, use), any_bad = __ballot_sync(0xffffffffu, bad);
            const unsigned nones = __ballot_sync(0xffffffffu, fine && none.qn > 0);
            if (fine && none.qn > 0) p.empty[__popc(nones & ((1u << tid) - 1u))] = none;
            if (rank == 31) {                          // the last: its sums are all but its own
                s_total = at + n * runs;
                s_tiles = tile_at + (runs > 1 ? n : 0);
                s_used = __popc(used);
                s_empty = __popc(nones);
                s_all_split = all_split;
                s_bad = any_bad != 0;
                s_run = p.run_tiles;
            }
        }
        __syncthreads();
    } else if constexpr (MODE == kByThread) {
        // a unit's place is the number of units before it
        __shared__ int s_len[kSmall], s_blocks[kSmall];
        Unit x;
        CrossEmpty none{0, 0};
        const bool fine = tid < n_units && load_unit<PREFIX>(p, tid, x, none, true), use = usable(fine, x);
        const int len = use ? longest(x) : 0;
        const unsigned long long key = ((unsigned long long)(use ? 0x7fffffffu - (uint32_t)len : 0xffffffffu) << 32) | (uint32_t)tid;
        int64_t total_full, total, total_tiles;
        block_exclusive_scan(use ? blocks_of(x, lg_tile + 1) : 0, s_warp, &total_full);
        const bool all_split = split_all(total_full);
        const int blocks = use ? blocks_of(x, all_split ? lg_tile : lg_tile + 1) : 0;
        if (tid < n_units) {
            s_key[tid] = key;
            s_len[tid] = len;
            s_blocks[tid] = blocks;
            if (unfit(tid, fine)) s_bad = 1;
            if (use) atomicAdd(&s_used, 1);
            if (fine && none.qn > 0) p.empty[atomicAdd(&s_empty, 1)] = none;   // (in any order)
        }
        __syncthreads();
        if (apart) {
            // How long runs are best: an item takes a step for each two of its tiles, and about kItemSteps beside them. Of
            // units alike (the groups alone) as many rounds as it takes, else an even share and one item more. (32
            // questions of 8 to 131 tokens behind two prefixes, 16 heads of 80: 105 us in a graph at 0.5 and 1 step an
            // item, 91 to 92 at 1.5 to 8; 64 single tokens behind four prefixes 64 to 65 at all of them.)
            constexpr float kItemSteps = 2.5f;
            unsigned long long best = ~0ull;
            const int run = p.run_tiles + tid;
            if (tid < 128) {
                const float inv = 1.f / (float)run;
                float items = 0.f, steps = 0.f, most = 0.f;
                for (int u = 0; u < n_units; ++u) {
                    const float t = (float)s_len[u], n = fmaxf(1.f, floorf((t + run - 0.5f) * inv)), b = (float)s_blocks[u];
                    items += b * n;
                    steps += b * t * 0.5f;
                    if (b > 0.f) most = fmaxf(most, t / n);
                }
                const float share = p.own_few ? ceilf(items / p.num_sms) * (most * 0.5f + kItemSteps)
                                              : (steps + kItemSteps * items) / p.num_sms + most * 0.5f + kItemSteps;
                best = ((unsigned long long)__float_as_uint(share) << 32) | (uint32_t)tid;
            }
            if (tid < 128) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const unsigned long long y = __shfl_xor_sync(0xffffffffu, best, o);
                    best = y < best ? y : best;
                }
                if ((tid & 31) == 0) atomicMin(&s_best, best);
            }
            __syncthreads();
            if (tid == 0) s_run = p.run_tiles + (int)(uint32_t)s_best;
            __syncthreads();
        }
        const int runs = use ? runs_in(len, s_run) : 1;
        int rank = 0;
        if (tid < n_units)
            for (int u = 0; u < n_units; ++u) rank += s_key[u] < key;
        __syncthreads();
        if (tid < n_units) {
            s_unit[rank] = x;
            s_runs[rank] = runs;
            s_blocks[rank] = blocks;
            s_key[rank] = (uint32_t)tid;
        }
        __syncthreads();
        const int n = tid < n_units ? s_blocks[tid] : 0, r = tid < n_units ? s_runs[tid] : 1;
        const int64_t at = block_exclusive_scan((int64_t)n * r, s_warp, &total);
        const int64_t tile_at = block_exclusive_scan(r > 1 ? n : 0, s_warp, &total_tiles);
        if (tid < n_units) {
            s_key[tid] |= (unsigned long long)at << 32;
            s_tile[tid] = (int)tile_at;
        }
        if (tid == 0) {
            s_total = (int)total;
            s_tiles = (int)total_tiles;
            s_all_split = all_split;
        }
        __syncthreads();
    } else {
        for (int i = tid; i < NP; i += kThreads) {
            Unit x;
            CrossEmpty none{0, 0};
            const bool fine = i < n_units && load_unit<PREFIX>(p, i, x, none, true);
            if (i < n_units && unfit(i, fine)) s_bad = 1;
            const bool use = usable(fine, x);
            s_key[i] = key_of(use, x, i);
            if (use) atomicAdd(&s_used, 1);
            if (fine && none.qn > 0) p.empty[atomicAdd(&s_empty, 1)] = none;   // (in any order)
        }
        __syncthreads();
        block_sort(s_key, NP, tid);
        const int per = (n_units + kThreads - 1) / kThreads, lo = min(tid * per, s_used), hi = min(lo + per, s_used);
        auto unit_at = [&](int i) {
            Unit x;
            CrossEmpty none;
            load_unit<PREFIX>(p, (int)(s_key[i] & 0xffffffffu), x, none, false);
            return x;
        };
        int64_t mine = 0, total_full, n_items = 0, n_tiles = 0, total, total_tiles;
        for (int i = lo; i < hi; ++i) mine += blocks_of(unit_at(i), lg_tile + 1);
        block_exclusive_scan(mine, s_warp, &total_full);
        const bool all_split = split_all(total_full);
        const int lg_block = all_split ? lg_tile : lg_tile + 1;
        for (int i = lo; i < hi; ++i) {
            const Unit x = unit_at(i);
            const int n = blocks_of(x, lg_block), runs = runs_of(x);
            n_items += (int64_t)n * runs;
            if (runs > 1) n_tiles += n;
        }
        int64_t at = block_exclusive_scan(n_items, s_warp, &total);
        int64_t tile_at = block_exclusive_scan(n_tiles, s_warp, &total_tiles);
        for (int i = lo; i < hi; ++i) {
            const Unit x = unit_at(i);
            const int n = blocks_of(x, lg_block), runs = runs_of(x);
            s_key[i] = ((unsigned long long)at << 32) | (uint32_t)(s_key[i] & 0xffffffffu);
            s_tile[i] = (int)tile_at;
            at += (int64_t)n * runs;
            if (runs > 1) tile_at += n;
        }
        if (tid == 0) {
            s_total = (int)total;
            s_tiles = (int)total_tiles;
            s_all_split = all_split;
        }
        __syncthreads();
    }
    const bool bad = wrong || s_bad != 0, all_split = s_all_split != 0;
    const int total = bad ? 0 : s_total, lg_block = all_split ? lg_tile : lg_tile + 1;
    // where the items end in a wave that fills at most half the SMs, its items are cut into their tiles
    const int rest = total % p.num_sms, run_tiles = s_run;
    const int whole = run_tiles > 0 ? 0 : !all_split && 2 * rest <= p.num_sms ? total - rest : total;
    if (tid == 0) s_more = 0;
    __syncthreads();
    for (int i = tid; i < total; i += kThreads) {
        const int at_unit = place_of(s_key, s_used, i), n = i - (int)(s_key[at_unit] >> 32);
        const int unit = (int)(s_key[at_unit] & 0xffffffffu);
        Unit x;
        CrossEmpty none;
        if (MODE != kSorted) x = s_unit[at_unit];
        else load_unit<PREFIX>(p, unit, x, none, false);
        const int nq = (int)(((unsigned)x.qn + (1u << lg_block) - 1u) >> lg_block);
        const int runs = MODE != kSorted ? s_runs[at_unit] : runs_of(x);
        const int j = runs > 1 ? n / runs : n, run = n - j * runs, back = j / packs, qb = nq - 1 - back;
        const int h = j - back * packs;
        const int t = qb << lg_block, e = min(x.qn, t + (1 << lg_block));
        const Span s = span_of<PREFIX>(p, x, t, e);
        // the block's tiles, dealt evenly to as many runs as they fill
        const int tiles = runs > 1 ? s.tiles(p.bn) : 0, use = runs > 1 ? runs_in(tiles, run_tiles) : 1;
        if (apart && n == 0) p.units[unit] = UnitSlots{x.q0, nq, runs, i};
        if (run >= use) {
            if (apart)
                for (int r = 0; r < 128; ++r) p.part_s[(int64_t)i * 128 + r] = -INFINITY;
            continue;
        }
        WinItem it;
        it.q0 = x.q0 + t;
        it.q1 = x.q0 + x.qn;
        it.head = h << p.lg_pack;
        it.split = all_split || x.qn - t <= (1 << lg_tile);
        it.slot = runs > 1 || apart ? i : -1;
        it.p0 = x.p0 + t;
        it.pad = 0;
        int fa = 0, fb = s.fn, ka = 0, kb = s.kn;
        if (use > 1) {
            const int nf = (s.fn + p.bn - 1) / p.bn, a = (int)((int64_t)tiles * run / use);
            const int b = (int)((int64_t)tiles * (run + 1) / use);
            fa = min(s.fn, min(a, nf) * p.bn);
            fb = min(s.fn, min(b, nf) * p.bn);
            ka = min(s.kn, max(0, a - nf) * p.bn);
            kb = min(s.kn, max(0, b - nf) * p.bn);
        }
        it.f0 = s.f0 + fa;
        it.fn = fb - fa;
        it.kp = s.lo + ka;
        it.k0 = x.k0 + it.kp;
        it.kn = kb - ka;
        if (runs > 1 && run == 0 && !apart)
            p.tiles[s_tile[at_unit] + j] = CrossTile{it.q0, it.q1, it.head, i, use, {0, 0, 0}};
        if (i < whole) {
            p.items[i] = it;
        } else {                                       // (in any order: an item's result does not depend on its place)
            const int halves = it.split ? 1 : 2, at = whole + atomicAdd(&s_more, halves);
            it.split = 1;
            p.items[at] = it;
            if (halves == 2) {
                it.q0 += 1 << lg_tile;
                it.p0 += 1 << lg_tile;
                p.items[at + 1] = it;
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        WsHeader *hdr = p.hdr;
        hdr->n_long = whole + s_more;
        hdr->n_joins = bad || apart ? 0 : s_tiles;
        hdr->n_empty = bad ? 0 : s_empty;
        hdr->n_tiny = 0;
        hdr->bm_long = 1 << lg_block;
        hdr->tiny_max = 0;
        hdr->error = bad ? VIT_ERR_BAD_SEQLENS : 0;
        hdr->long_all_split = all_split ? 1 : 0;
        hdr->next_long = 0;
    }
}

// How the own keys' parts of the kernel for few query rows lie (cross_few.cu).
struct FewParts {
    const float *o, *s;           // [B][Hk][n_split][rows][D] and [..][rows]
    int Hk, group, n_split, rows, chunk;
};

// A row of sequence b: its parts over the prefix and over its own keys,
//   out = sum_s 2^(e_s - E) O_s / sum_s 2^(e_s - E), e_s the log2 of part s's sum,
// D / 8 lanes per row, 32 bytes of every part a lane. FEW: the own parts are those of the kernel for few query rows.
// Bound by latency: the offsets, then a row's weights, then its parts (1348 tokens of 16 heads of 80 in four parts, of
// 27 MB in L2: 32 us with a warp per row, 14 us so).
template <int D, bool FEW>
__global__ void __launch_bounds__(256, 3)
window_join_kernel(const Sched p, const float *part_o, const FewParts few, __nv_bfloat16 *out, int64_t out_stride,
                   float *lse)
{
    grid_wait();
    constexpr int CH = D / 8, R = 32 / CH;             // lanes of a row, rows of a warp
    const int lane = threadIdx.x & 31, b = blockIdx.y, sub = lane / CH, c8 = lane % CH * 8;
    const int error = p.hdr->error;
    int g, begin, f0, fn, err;
    const bool fine = p.groups.find(b, lane, false, g, begin, f0, fn, err);
    CrossSeg c;
    if (!load_seg(p.s, b, c, nullptr, false) || error != 0 || !fine) return;
    const int packs = p.Hq >> p.lg_pack, lg_tile = 7 - p.lg_pack, mask = (1 << lg_tile) - 1;
    const WinSeg w = win_seg(c);
    // a unit without keys has no slots
    UnitSlots own{0, 0, 0, 0}, pre{0, 0, 0, 0};
    if (FEW) own.runs = key_runs(w.kn, few.chunk);
    else if (w.kn > 0) own = p.units[p.groups.G + b];
    if (fn > 0) pre = p.units[g];
    const int before = c.q0 - p.s.cu_q[begin];         // rows of the group's sequences before this one
    const int64_t n_rows = (int64_t)c.qn * p.Hq;
    for (int64_t x0 = (int64_t)(blockIdx.x * 8 + (threadIdx.x >> 5)) * R; x0 < n_rows; x0 += (int64_t)8 * R * gridDim.x) {
        const int64_t x = x0 + sub;
        if (sub >= R || x >= n_rows) continue;
        const int tok = (int)(n_rows <= 0x7fffffff ? (uint32_t)x / (uint32_t)p.Hq : x / p.Hq);
        const int head = (int)(x - (int64_t)tok * p.Hq);
        const int pack = head >> p.lg_pack, in_pack = head & ((1 << p.lg_pack) - 1);
        // the first part's row of a unit's token t
        auto first = [&](const UnitSlots &u, int t) -> int64_t {
            const int64_t slot = u.slot + (int64_t)((u.blocks - 1 - (t >> lg_tile)) * packs + pack) * u.runs;
            return slot * 128 + ((t & mask) << p.lg_pack) + in_pack;
        };
        const int own_t = tok - w.none, own_runs = own_t < 0 ? 0 : own.runs;   // (the first may lie before the own keys)
        const float *ps = p.part_s + first(pre, before + tok), *po = part_o + first(pre, before + tok) * D + c8;
        const float *os, *oo;
        int step = 128;                                // rows between two runs' parts of a row
        if (FEW) {
            const int hk = head / few.group;
            const int64_t row = ((int64_t)b * few.Hk + hk) * few.n_split * few.rows + own_t * few.group + head - hk * few.group;
            os = few.s + row;
            oo = few.o + row * D + c8;
            step = few.rows;
        } else {
            os = p.part_s + first(own, own_t);
            oo = part_o + first(own, own_t) * D + c8;
        }
        float E = -INFINITY, sum = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int s = 0; s < pre.runs; ++s) E = fmaxf(E, ps[s * 128]);
#pragma unroll 2
        for (int s = 0; s < own_runs; ++s) E = fmaxf(E, os[s * step]);
        const float base = E == -INFINITY ? 0.f : E;
        auto add = [&](float e, const float *o) {
            const float y = wmma16::ex2(e - base);
            sum += y;
            if (y == 0.f) return;                      // (a part without weight was not written)
            const float4 u = *reinterpret_cast<const float4 *>(o), v = *reinterpret_cast<const float4 *>(o + 4);
            acc[0] = fmaf(y, u.x, acc[0]);
            acc[1] = fmaf(y, u.y, acc[1]);
            acc[2] = fmaf(y, u.z, acc[2]);
            acc[3] = fmaf(y, u.w, acc[3]);
            acc[4] = fmaf(y, v.x, acc[4]);
            acc[5] = fmaf(y, v.y, acc[5]);
            acc[6] = fmaf(y, v.z, acc[6]);
            acc[7] = fmaf(y, v.w, acc[7]);
        };
#pragma unroll 2
        for (int s = 0; s < pre.runs; ++s) add(ps[s * 128], po + (int64_t)s * 128 * D);
        for (int s = 0; s < own_runs; ++s) add(os[s * step], oo + (int64_t)s * step * D);
        const float inv = pre.runs + own_runs > 0 ? 1.f / sum : 0.f;   // keys, but no weight: 0 * inf; no keys: 0
        const int64_t t = (int64_t)c.q0 + tok;
        *reinterpret_cast<uint4 *>(out + t * out_stride + (int64_t)head * D + c8) =
            make_uint4(wmma16::pack_bf16(acc[0] * inv, acc[1] * inv), wmma16::pack_bf16(acc[2] * inv, acc[3] * inv),
                       wmma16::pack_bf16(acc[4] * inv, acc[5] * inv), wmma16::pack_bf16(acc[6] * inv, acc[7] * inv));
        if (lse && c8 == 0) lse[t * p.Hq + head] = (E + log2f(sum)) * 0.6931471805599453f;
    }
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

WinPlan win_plan(int64_t Tq, int B, int Hq, int Hk, int D, int max_q, int max_k, int window, int sinks, int G,
                 int64_t Tp, int max_p)
{
    WinPlan p;
    p.lg_pack = cross_pack(Hq / Hk);
    const int64_t tok = 128 >> p.lg_pack, packs = Hq >> p.lg_pack, bn = attn_long_bn(D);
    // tiles of the sequences, and of the groups
    const int64_t own = std::min(Tq / tok + B, (int64_t)B * cdiv(max_q, tok)), grouped = Tq / tok + G;
    const bool prefix = G > 0 && Tp > 0;
    // Apart where the sequences' tiles would be much emptier than the groups': otherwise a pass over both saves the
    // partial results and their join. In a graph, apart and together, 16 heads of 80, 16 sequences behind 4000 shared
    // keys: of 32 tokens (3.2 times the tiles) 37 and 58 us, of 43 (2.7) 48 and 58, of 55 (2.3) 58 and 58, of 64 (1.8) 60
    // and 58, of 85 (1.5) 72 and 59. Where the lines cross moves with the prefix's share of the work: 64 sequences behind
    // 1000 keys, 32 tokens (3.8) 62 and 70, 43 (2.9) 78 and 70, 55 (2.3) 89 and 71; 8 behind 9000, 55 (2.0) 58 and 60, 85
    // (1.3) 75 and 60.
    p.apart = prefix && own > 2 * grouped;
    p.own_few = p.apart && window_takes_few(B, Hq, Hk, D, max_q, max_k, 0, 0);
    p.units = p.own_few ? G : p.apart ? G + B : B;
    // key tiles of a block at most
    const int64_t own_keys = window > 0 ? std::min<int64_t>(max_k, (int64_t)window + 2 * tok - 1) : max_k;
    const int64_t first = prefix ? max_p : window > 0 ? std::min(sinks, max_k) : 0;
    const int64_t own_most = cdiv(own_keys, bn), first_most = cdiv(first, bn);
    const int64_t tiles = (p.apart ? own + grouped : own) * packs;
    p.run_tiles = 0;
    p.runs = 1;
    p.max_tiles = 0;
    // few tiles: cut their keys so that there is about one item per SM, of at least 512 keys each (a run writes and
    // re-reads 128 * D fp32 values)
    const int64_t least = 2 * cdiv(512, 2 * bn);
    if (p.apart) {
        const int64_t mine = p.own_few ? 0 : own;      // tiles of the list beside the groups'
        const int64_t work = (mine * own_most + grouped * first_most) * packs;
        const int64_t run = std::max(least, cdiv(work, 8 * kDesignSms));   // the shortest; the list may choose longer ones
        const int64_t r1 = cdiv(first_most, run), r2 = p.own_few ? 0 : cdiv(own_most, run);
        p.run_tiles = (int)run;
        p.runs = (int)std::max<int64_t>(1, std::max(r1, r2));
        p.max_items = (grouped * std::max<int64_t>(1, r1) + mine * std::max<int64_t>(1, r2)) * packs;
        p.slots = p.max_items;
    } else {
        const int64_t most = own_most + first_most;
        p.max_items = tiles;
        p.slots = 0;
        if (2 * tiles <= kDesignSms && tiles > 0) {
            const int64_t run = std::max(least, cdiv(most, kDesignSms / tiles)), runs = cdiv(most, run);
            if (runs > 1) {
                p.run_tiles = (int)run;
                p.runs = (int)runs;
                p.max_items = tiles * runs;
                p.max_tiles = tiles;
                p.slots = p.max_items;
            }
        }
    }
    p.off_items = sizeof(WsHeader);
    p.off_tiles = up(p.off_items + sizeof(WinItem) * (size_t)p.max_items);
    p.off_empty = up(p.off_tiles + sizeof(CrossTile) * (size_t)p.max_tiles);
    p.off_units = up(p.off_empty + sizeof(CrossEmpty) * (size_t)B);
    p.off_part_s = up(p.off_units + (p.apart ? sizeof(UnitSlots) * (size_t)p.units : 0));
    p.off_part_o = up(p.off_part_s + (size_t)p.slots * 128 * sizeof(float));
    p.off_few = up(p.off_part_o + (size_t)p.slots * 128 * (size_t)D * sizeof(float));
    p.few = FewPlan{};
    p.bytes = p.off_few;
    if (p.own_few) {
        p.few = window_few_plan(B, Hq, Hk, D, max_q, max_k, 0, 0);
        // One run each where that is enough blocks, and short ones. In a graph, one run and several, 8 key heads of 128: 64
        // sequences of 700 keys 68 and 74 us, of 2048 115 and 121, of 5000 221 and 226; of lengths from 20 up to 2048 82 and 82,
        // to 3000 103 and 101; 20 sequences up to 2000 53 and 53, up to 4000 76 and 68.
        if ((int64_t)B * Hk >= kDesignSms && max_k <= 2048) {
            p.few.chunk = std::max(64, (max_k + 63) / 64 * 64);
            p.few.n_split = p.few.room = 1;
        }
        p.bytes += sizeof(float) * (size_t)B * Hk * p.few.room * p.few.rows * (D + 1);
    }
    return p;
}

cudaError_t launch_window_tiles(const WinArgs &a, const WinPlan &pl, int num_sms, cudaStream_t stream)
{
    char *ws = static_cast<char *>(a.f.workspace);
    Sched p;
    p.s = a.f.segs;
    p.window = a.window;
    p.sinks = a.sinks;
    p.groups = a.groups;
    p.apart = pl.apart;
    p.own_few = pl.own_few;
    p.Hq = a.f.Hq;
    p.lg_pack = pl.lg_pack;
    p.bn = attn_long_bn(a.f.D);
    p.run_tiles = pl.run_tiles;
    p.num_sms = num_sms;
    p.hdr = reinterpret_cast<WsHeader *>(ws);
    p.items = reinterpret_cast<WinItem *>(ws + pl.off_items);
    p.tiles = reinterpret_cast<CrossTile *>(ws + pl.off_tiles);
    p.empty = reinterpret_cast<CrossEmpty *>(ws + pl.off_empty);
    p.units = reinterpret_cast<UnitSlots *>(ws + pl.off_units);
    p.part_s = reinterpret_cast<float *>(ws + pl.off_part_s);
    p.status = a.f.status;
    int np = 32;
    while (np < pl.units) np <<= 1;
    constexpr size_t each = sizeof(unsigned long long) + sizeof(int);
    auto kernel = [&](auto prefix) {
        constexpr bool P = decltype(prefix)::value;
        return pl.units <= 32 && !pl.apart ? window_schedule_kernel<kByWarp, P>
               : pl.units <= kSmall        ? window_schedule_kernel<kByThread, P>
                                           : window_schedule_kernel<kSorted, P>;
    };
    static DeviceOnce once;
    cudaError_t e = once.run([&] {
        constexpr int most = (int)each * 2 * VIT_MAX_SEGMENTS;
        const cudaError_t r = cudaFuncSetAttribute(window_schedule_kernel<kSorted, false>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        return r != cudaSuccess ? r : cudaFuncSetAttribute(window_schedule_kernel<kSorted, true>,
                                                           cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    });
    if (e != cudaSuccess) return e;
    {
        LaunchScope scope("window_schedule", stream);
        e = launch_chained(a.prefix ? kernel(std::true_type()) : kernel(std::false_type()), 1, kThreads, each * np, stream, p);
        if (e != cudaSuccess) return e;
    }
    WinLong cx{};
    cx.group = a.f.Hq / a.f.Hk;
    cx.lg_pack = pl.lg_pack;
    cx.empty = p.empty;
    cx.part_s = p.part_s;
    cx.part_o = reinterpret_cast<float *>(ws + pl.off_part_o);
    cx.window = a.window;
    cx.sinks = a.sinks;
    e = launch_window_long(a, cx, p.hdr, p.items, pl.max_items, num_sms, stream);
    if (e != cudaSuccess) return e;
    if (pl.apart) {
        FewParts few{};
        if (pl.own_few) {
            e = launch_window_few(a, pl.few, true, ws + pl.off_few, stream);
            if (e != cudaSuccess) return e;
            few.Hk = a.f.Hk;
            few.group = a.f.Hq / a.f.Hk;
            few.n_split = pl.few.n_split;
            few.rows = pl.few.rows;
            few.chunk = pl.few.chunk;
            few.o = reinterpret_cast<const float *>(ws + pl.off_few);
            few.s = few.o + (size_t)a.f.segs.B * a.f.Hk * pl.few.n_split * pl.few.rows * a.f.D;
        }
        LaunchScope scope("window_join", stream);
        // more blocks than fill the GPU once only cost their starts
        const int64_t most = cdiv((int64_t)a.f.segs.max_q * a.f.Hq, 8 * (32 / (a.f.D / 8)));
        const int64_t enough = cdiv(6 * kDesignSms, a.f.segs.B);
        const dim3 grid((unsigned)std::min(most, enough), (unsigned)a.f.segs.B);
        auto run = [&](auto kern) {
            return launch_chained(kern, grid, 256, 0, stream, p, cx.part_o, few, static_cast<__nv_bfloat16 *>(a.f.out),
                                  a.f.out_stride, a.f.lse);
        };
        auto pick = [&](auto d) {
            constexpr int D = decltype(d)::value;
            return pl.own_few ? run(window_join_kernel<D, true>) : run(window_join_kernel<D, false>);
        };
        switch (a.f.D) {
            case 32: return pick(std::integral_constant<int, 32>());
            case 64: return pick(std::integral_constant<int, 64>());
            case 80: return pick(std::integral_constant<int, 80>());
            case 96: return pick(std::integral_constant<int, 96>());
            default: return pick(std::integral_constant<int, 128>());
        }
    }
    if (pl.runs > 1) {
        LongPlan join{};
        join.max_tiles = pl.max_tiles;
        return launch_cross_tile_join(a.f, join, cx, p.hdr, p.tiles, stream);
    }
    return cudaSuccess;
}

}  // namespace vit
