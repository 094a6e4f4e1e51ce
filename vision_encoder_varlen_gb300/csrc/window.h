// Declarations shared by the translation units of a language model's own attention: a causal window over a
// sequence's keys with its first tokens kept visible, and a prefix that several sequences share.
#pragma once

#include "cross.h"

namespace vit {

// Work item of the tcgen05 kernel: its 128 (split) or 256 query rows see all of the keys [f0, f0 + fn) (a sequence's
// first tokens, or a prefix, which may be of another tensor), and of the keys [k0, k0 + kn), whose first one has
// position `kp` in its sequence, those that the mask lets through for a query of position p: j <= p and, with a
// window, p - j < window or j < sinks. Rows are packed as in CrossItem; token q0 has position p0.
struct alignas(16) WinItem {
    int f0, fn;
    int k0, kn;
    int q0, q1, head;
    int split;
    int slot;                     // place of the partial result, or -1: the result itself
    int kp, p0;
    int pad;
};
static_assert(sizeof(WinItem) == 48, "three 16-byte words");   // (as twelve 4-byte ones a list of 1168 took 9 us longer)
__device__ __forceinline__ int item_head(const WinItem &x) { return x.head; }
__device__ __forceinline__ bool item_split(const WinItem &x) { return x.split != 0; }

struct WinLong : CrossLong {
    int window, sinks;            // window 0: everything before a query
};

// Shared prefixes: the sequences [cu_g[g], cu_g[g+1]) (all of them without cu_g) see the rows [cu_p[g], cu_p[g+1]) of
// the prefix tensors.
struct Groups {
    const int32_t *cu_g, *cu_p;
    int64_t Tp;
    int G, max_p, B;

    __device__ int bound(int g) const { return cu_g ? cu_g[g] : g == 0 ? 0 : B; }
    // the prefix of group g: false where its rows are not in the tensor, or more than the bound
    __device__ bool load(int g, int &f0, int &fn) const
    {
        const int64_t a = cu_p[g], b = cu_p[g + 1];
        f0 = (int)a;
        fn = (int)(b - a);
        return a >= 0 && b >= a && b <= Tp && b - a <= max_p;
    }
    // Sequence b's group g and its prefix, for a converged warp, in one round of loads for up to 31 groups: false where
    // b's group is malformed, or any of up to 31. `err`: what is wrong, for one caller (`all`) also with other groups.
    __device__ bool find(int b, int lane, bool all, int &g, int &begin, int &f0, int &fn, int &err) const
    {
        int bad = 0;
        bool fine = true;
        if (G < 32) {
            const int at = lane <= G ? bound(lane) : 0, row = lane <= G ? cu_p[lane] : 0;
            const int at1 = __shfl_down_sync(0xffffffffu, at, 1), row1 = __shfl_down_sync(0xffffffffu, row, 1);
            if (lane < G) bad = check(lane, at, at1, row, row1);
            g = 31 - __clz(__ballot_sync(0xffffffffu, lane < G && at <= b) | 1u);
            begin = __shfl_sync(0xffffffffu, at, g);
            f0 = __shfl_sync(0xffffffffu, row, g);
            fn = __shfl_sync(0xffffffffu, row1, g) - f0;
        } else {
            g = of(b);
            begin = bound(g);
            load(g, f0, fn);
            bad = begin > b || bound(g + 1) <= b ? VIT_ERR_BAD_SEQLENS : error(g);
            fine = bad == 0;
            if (all)
                for (int i = lane; i < G; i += 32) bad = bad ? bad : error(i);
        }
        const unsigned any = __ballot_sync(0xffffffffu, bad != 0);
        err = any ? __shfl_sync(0xffffffffu, bad, __ffs(any) - 1) : 0;
        return fine && (any == 0 || G >= 32);
    }
    // group g's error: the groups follow one another and hold every sequence, their prefixes lie in the tensor
    __device__ int error(int g) const { return check(g, bound(g), bound(g + 1), cu_p[g], cu_p[g + 1]); }
    // [a, b) its sequences, [r0, r1) its prefix's rows
    __device__ int check(int g, int a, int b, int r0, int r1) const
    {
        if (a < 0 || b < a || b > B || (g == 0 && a != 0) || (g == G - 1 && b != B) || r0 < 0 || r1 < r0 || r1 > Tp)
            return VIT_ERR_BAD_SEQLENS;
        return r1 - r0 > max_p ? VIT_ERR_SEQLEN_EXCEEDS_MAX : 0;
    }
    // the group of sequence b: the last one that begins at or before it
    __device__ int of(int b) const
    {
        int lo = 0, hi = G;
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            if (bound(m) <= b) lo = m;
            else hi = m;
        }
        return lo;
    }
};

struct WinArgs {
    CrossArgs f;                  // the queries are the last ones of their sequence's keys
    int window, sinks;
    bool prefix;
    const void *kp, *vp;          // bf16 [Tp, Hk, D]
    int64_t kp_stride, vp_stride;
    Groups groups;
};

// The place of a sequence's queries among its keys. The first `none` queries lie before its first key (fewer keys than
// queries) and see none of them; the rest, from row q0 on, have positions p0, p0 + 1, ..
struct WinSeg {
    int q0, qn, k0, kn, p0, none;
};
__device__ __forceinline__ WinSeg win_seg(const CrossSeg &x)
{
    WinSeg w;
    w.none = x.qn > x.kn ? x.qn - x.kn : 0;
    w.q0 = x.q0 + w.none;
    w.qn = x.qn - w.none;
    w.k0 = x.k0;
    w.kn = x.kn;
    w.p0 = x.kn - w.qn;
    return w;
}

// The keys that queries of the positions [p, q] see between them: the `first` of the sequence and, behind a gap, those
// of the positions [lo, q] (first = 0 where there is no gap).
struct WinRange {
    int first, lo;
};
__host__ __device__ inline WinRange win_range(int p, int window, int sinks)
{
    const int lo = window > 0 && p >= window ? p - window + 1 : 0;
    return lo > sinks ? WinRange{sinks, lo} : WinRange{0, 0};
}

// How a call of the tcgen05 kernel is cut (a function of the sizes alone).
struct WinPlan {
    int lg_pack;
    int units;                    // sequences, or groups and sequences (apart)
    bool apart;                   // prefix and own keys are separate parts, joined by row
    bool own_few;                 // apart, and the own keys' parts are made by the kernel for few query rows
    FewPlan few;
    size_t off_few;
    int run_tiles;                // key tiles of an item at most (0: keys are not cut)
    int runs;                     // runs of a block at most
    int64_t max_items, max_tiles, slots;
    size_t off_items, off_tiles, off_empty, off_units, off_part_s, off_part_o, bytes;
};
WinPlan win_plan(int64_t Tq, int B, int Hq, int Hk, int D, int max_q, int max_k, int window, int sinks, int G,
                 int64_t Tp, int max_p);
cudaError_t launch_window_tiles(const WinArgs &a, const WinPlan &p, int num_sms, cudaStream_t stream);
cudaError_t launch_window_long(const WinArgs &a, const WinLong &cx, const WsHeader *hdr, const WinItem *items,
                               int64_t max_items, int num_sms, cudaStream_t stream);

// Work item of a gradient pass (as GradItem, with the part of the other side that the mask leaves). dk, dv: the 128
// keys from r0 on, the first at position rp, over the queries [l0, l0 + ln), the first at position lp. dq: the 128 / P
// tokens from r0 on, the first at position rp, over the keys [f0, f0 + fn), which all of them see, and [l0, l0 + ln),
// the first at position lp.
struct alignas(16) WinGradItem {
    int r0, r1, l0, ln;
    int head, tiles;
    int f0, fn;
    int rp, lp;
    int j0;                       // dk, dv: the item's first tile where a key tile's loop is cut into runs
    int slot;                     // place of such a run's sums, or -1: dk and dv themselves
};
static_assert(sizeof(WinGradItem) == 48, "three 16-byte words");
// A key tile whose loop is cut: the join adds the slots [slot, slot + runs).
struct WinGradTile {
    int r0, r1, head, slot, runs, pad[3];
};
struct WinGradPlan : GradPlan {
    int cut_over, run_tiles;      // a loop of more tiles than the first is cut into runs of the second at most (0: none)
    int max_cut, max_slots;       // key tiles cut, and their runs, at most
    size_t off_cut, off_sums;     // the sums: [slots][dk, dv][128][D] fp32
};
WinGradPlan window_grad_plan(int64_t Tq, int64_t Tk, int B, int Hq, int Hk, int D, int max_q, int max_k, int window,
                             int sinks);
cudaError_t launch_window_grad(const CrossGradArgs &a, const WinGradPlan &p, int window, int sinks, int num_sms,
                               cudaStream_t stream);

// few query rows (cross_few.cu)
bool window_takes_few(int B, int Hq, int Hk, int D, int max_q, int max_k, int window, int sinks);
FewPlan window_few_plan(int B, int Hq, int Hk, int D, int max_q, int max_k, int window, int sinks);
// `parts`: leave every run's partial result at `part` for another kernel to join
cudaError_t launch_window_few(const WinArgs &a, const FewPlan &p, bool parts, void *part, cudaStream_t stream);
// a prefix read by each of its sequences anew
bool prefix_takes_few(int B, int Hq, int Hk, int D, int max_q, int max_k, int max_p);
FewPlan prefix_few_plan(int B, int Hq, int Hk, int D, int max_q, int max_k, int max_p);

}  // namespace vit
