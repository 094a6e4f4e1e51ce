// Gradient of cross attention on the 5th-generation tensor cores (tcgen05 + TMEM + TMA).
//
//   p_ij  = exp(scale q_i k_j - lse_i)                 delta_i = sum_d do_i o_i
//   dv_j  = sum_i p_ij do_i                            ds_ij = p_ij (do_i v_j - delta_i)
//   dq_i  = scale sum_j ds_ij k_j                      dk_j = scale sum_i ds_ij q_i
// summed over the query heads that share a key head for dk and dv. P and dS are rounded to bf16 for
// their products (as P is in the forward pass), everything else is fp32.
//
// dq sums over keys and dk, dv sum over queries, so one pass over the tiles would have to add one of
// them up in memory with fp32 atomics, whose order changes the result. Instead there are two passes,
// each keeping its own sums in TMEM and recomputing S and dP (7 products instead of 5):
//   dk, dv   a tile of 128 keys stays, the queries of its heads stream by:
//            S^T = K Q^T, dP^T = V dO^T (SS MMAs), dV += P^T dO, dK += dS^T Q (TS MMAs: P and dS in TMEM)
//   dq       a tile of 128 query rows stays, the keys stream by:
//            S = Q K^T, dP = dO V^T, dQ += dS K
// which is the same kernel: two resident tiles X1, X2, two streamed ones Y1, Y2, S = X1 Y1^T,
// dP = X2 Y2^T, A1 += dS Y1 and (dk, dv only) A2 += P Y2. Statistics go by the streamed side in the
// first pass (read from shared memory) and by the row in the second. The passes do not depend on one
// another and are the two halves of one launch's blocks: those of dq come to SMs as those of dk, dv
// leave, and all of them wait for the launch that made the lists. (As two launches, the second released
// early, 532 instead of 541 us at 4 x 2048 x 4096, 16 heads of 80, and 792 instead of 795 at 128; but there only the
// first has waited for the lists, and what one launch has waited for is not visible to the next. Both
// kinds of items in one list, taken by the same blocks, was 10 % slower: the issuer's loop compiles worse.)
//
// Measured at 4 x 2048 queries over 4096 keys, 16 heads of 80: 541 us (1.11 PFLOP/s of the seven products; in
// launches of their own dk, dv 317 us, dq 211), the tensor pipe 43 to 50 % busy: bound by the exchange between the
// softmax groups and the issuer, whose products of one tile and sums of the one before take turns in one pipe, at
// 1.3 to 1.5 times the time that the MMAs need alone.
//
// delta comes from the stored bf16 out, as the interface has no other, except in sequences of 2 to 16 keys: where
// few keys carry a row, dP - delta cancels and leaves out's rounding. In the 2-norm dq is off by 0.35 % over 2
// keys, 0.28 over 4, 0.25 over 16 and 0.24 over 32 with delta from out, and by 0.24 % (its own rounding 0.17, that
// of dS the rest) over any number with delta from the scores. So few keys are one tile of the loop for dq, and one
// warp's lanes for dk, dv: S and dP are all there. (2000 sequences of 64 queries over 16 keys, 16 heads of 64: 1.31
// instead of 1.16 ms; over 32 keys, up to which it would go, 1.35 instead of 1.16.)
//
// Before them, one launch makes the two item lists (a block each) and the statistics -lse log2(e) and
// -delta of every (token, head) (the other blocks).
//
// Roles of a block (384 threads, one per SM, persistent over the item list):
//   warp 0       TMA producer: the X tiles and a ring of Y tiles of BN rows
//   warp 1       TMEM owner and MMA issuer: acc(j) as soon as P, dS of tile j are stored, then S, dP of
//                tile j + 2 into the TMEM stage that tile j leaves (MMAs of one thread run in order)
//   warps 2, 3   dk, dv: the statistics of each softmax group's next tile into shared memory; before that, where
//                asked for, zeros into the rows that belong to no sequence
//   warps 4-7, 8-11  the two softmax groups take alternate tiles: S, dP -> registers -> P, dS -> TMEM
//                over their own S and dP columns; at an item's end they write dk and dv (or half of dq each)
// TMEM (512 columns): A1 | A2 (dk, dv only) | two stages of S and dP (BN columns each).
// All tiles use slabs of W columns with a 2 W-byte swizzle, so that the same bytes serve as a K-major
// operand (of S and dP, reduced over D) and as an MN-major one (of the sums, reduced over rows).
// Streamed rows past the sequence's end enter the sums with P = dS = 0 and are zeroed in shared memory
// first (0 * NaN is NaN), the last 16-row step included.
//
// A causal window (WIN) leaves a tile only a part of the other side: a key tile the queries from its first key's position
// on, up to the window behind its last key's or, where it holds first tokens that stay visible, to the end; a query
// tile the first tokens and the run of keys that its rows see between them. Pairs that the mask excludes inside those
// tiles have P = dS = 0 exactly, whatever their scores are. delta is from the scores for every row that sees 2 to 16
// keys (the first rows of each sequence, all rows of a window of so many), made with the other statistics.
// A key tile that holds first tokens has all queries in its loop. Where that is more than an SM's even share of the work
// (long texts, a short window), the loop is cut into runs whose fp32 sums a last launch adds up in order: with 4 first
// tokens the call took 56 instead of 413 us for one text of 5200 tokens, 8 heads over one of 64, window 64, 400 instead
// of 1061 us for one of 16384, 32 over 8 of 128, window 128, and 421 instead of 1296 us for one of 32768, 16 over 4 of
// 64, window 512.
// Measured: four texts of 2500 to 5117 tokens, 16 heads of 80, window 1024: 381 us (0.28 of the floor with the other
// launches); three causal texts of 1500 to 2311, 32 heads over 8 of 128: 256 us. Bound by the hand-over between the issuer
// and the softmax groups, as without a mask: the tensor pipe is active 40 % of the time, DRAM at 1.3 TB/s.
#include <algorithm>
#include <type_traits>

#include "block_sort.cuh"
#include "cross.h"
#include "sm100.cuh"
#include "window.h"

namespace vit {
namespace {

using namespace sm100;

constexpr int kThreads = 384;
constexpr int kLaunchRegs = 168;
constexpr int kCtrlRegs = 88;
constexpr int kSoftmaxRegs = 208;
static_assert(128 * kCtrlRegs + 256 * kSoftmaxRegs <= kThreads * kLaunchRegs, "register split exceeds the launch pool");
constexpr int BM = 128;
constexpr long long kWaitBudget = 4000000000ll;
constexpr int kMaxY = 6;
constexpr int kItemRing = 4;           // windowed lists: items the producer may take ahead of the other roles
constexpr int kExactKeys = 16;         // sequences of 2 to so many keys have delta from the scores

template <int D, bool DKV> struct GradCfg {
    // Streamed rows per tile: what an MMA of 128 rows costs in shared memory (its A operand) and what a tile costs
    // in hand-overs go down with more of them, so as many as TMEM has room for beside the sums, (512 - sums) / 4,
    // and shared memory for four ring slots (64 at head_dim 128, with three). A pass alone, 16 heads, 4 x 2048 x 4096: dq at
    // head_dim 80 with 96 rows 211 us, 80 rows 240, 64 rows and three TMEM stages 275; at 64 with 112 rows 173,
    // 80 rows 209; at 96 with 80 rows and four slots 250, 96 rows and three 268; at 128 with 64 rows and three slots
    // 375, 80 rows and two 598. dk, dv at 80 with 80 rows 317, 48 rows and three stages 394.
    static constexpr int BN = DKV ? (D == 32 ? 112 : D == 64 ? 96 : D == 128 ? 64 : 80)
                                  : (D <= 64 ? 112 : D == 80 ? 96 : D == 96 ? 80 : 64);
    // columns of S and dP that a softmax thread has in registers at a time (tiles of more than 80 come in two parts)
    static constexpr int PART = BN <= 80 ? BN : (BN / 2 + 15) / 16 * 16;
    static constexpr int W = D % 64 == 0 ? 64 : D % 32 == 0 ? 32 : 16;   // columns of a slab
    static constexpr int SW = 2 * W;                       // its swizzle in bytes
    static constexpr int NS = D / W;                       // slabs
    static constexpr int X_SLAB = BM * SW, Y_SLAB = BN * SW;
    static constexpr int X_TILE = NS * X_SLAB, Y_TILE = NS * Y_SLAB;
    static constexpr int Y_PAIR = (2 * Y_TILE + 1023) / 1024 * 1024;
    static constexpr int BUDGET = 227 * 1024 - 1024 - 1280;   // without the alignment, the statistics and barriers
    // two X buffers, so that an item's tiles arrive while the one before it runs (with one, its Y loads wait as
    // well: 4 x 2048 x 4096 at head_dim 80 took 275 instead of 235 us for dq), and as many Y slots as fit, up to 6
    static constexpr int NY = (BUDGET - 4 * X_TILE) / Y_PAIR > 6 ? 6 : (BUDGET - 4 * X_TILE) / Y_PAIR;
    static constexpr int OFF_Y = 4 * X_TILE;
    static constexpr int DATA = OFF_Y + NY * Y_PAIR;
    static constexpr int SMEM = DATA + 1024 > 118 * 1024 ? DATA + 1024 : 118 * 1024;   // one block per SM
    static constexpr int LAYOUT = SW == 128 ? 2 : SW == 64 ? 4 : 6;
    static constexpr int TA1 = 0, TA2 = D, TSTAGE = DKV ? 2 * D : D; // TMEM columns; stage s: S at TSTAGE + 2 BN s, dP BN further
    static_assert(TSTAGE + 4 * BN <= 512, "TMEM budget");
    static_assert(X_TILE % 1024 == 0 && Y_SLAB % (8 * SW) == 0 && Y_TILE % (8 * SW) == 0, "slabs start on swizzle atoms");
    static_assert(NY <= kMaxY && BN % 16 == 0, "tile shapes");
};

struct Bars {
    uint64_t x_full[2], x_empty[2], y_full[kMaxY], y_empty[kMaxY];
    uint64_t s_full[2], p_full[2], stat[2], acc_done, acc_free, drain;
};

__device__ __forceinline__ uint32_t bar_addr(const uint64_t &b) { return smem_addr(&b); }

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.ftz.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// One pass over its list, by the blocks of a launch that take it.
struct Grad {
    const GradItem *items;
    const int32_t *n_items;
    CrossSegs segs;
    bool zero_rest;               // rows of no sequence get 0
    const float2 *stats;          // [Tq, Hq] {-lse log2(e), -delta}
    __nv_bfloat16 *out1, *out2;   // dk, dv; or dq
    int64_t out1_stride, out2_stride;
    int Hq, Hk, group, lg_pack;
    float scale, scale_log2;
    int first_block, n_blocks;
    int32_t *status;
};
struct GradMaps {
    CUtensorMap x1, x2, y1, y2;
};
struct WinGradMaps : GradMaps {
    CUtensorMap o1, o2;           // the outputs, in boxes of 32 rows
};
struct WinGrad : Grad {
    const WinGradItem *win_items;
    float *sums;                  // of the runs of cut loops
    int32_t *next;                // items handed out so far beyond each block's first
    int window, sinks;
};
__device__ __forceinline__ const GradItem *items_of(const Grad &p) { return p.items; }
__device__ __forceinline__ const WinGradItem *items_of(const WinGrad &p) { return p.win_items; }

template <int D> struct GradShared {
    Bars bars;
    uint32_t tmem;
    volatile int abort;
    alignas(16) float stat[2][2][GradCfg<D, true>::BN];    // dk, dv: [group][-lse2 | -delta][column]
};
template <int D> struct WinGradShared : GradShared<D> {
    uint64_t item_full[kItemRing], item_empty[kItemRing];
    int item[kItemRing];          // numbers of the items that the producer has taken (the list's length or more: the end)
};

template <int D, bool DKV, bool WIN>
__device__ __forceinline__ void grad_pass(const std::conditional_t<WIN, WinGradMaps, GradMaps> &tm,
                                          const std::conditional_t<WIN, WinGrad, Grad> &p,
                                          std::conditional_t<WIN, WinGradShared<D>, GradShared<D>> &sh)
{
    using C = GradCfg<D, DKV>;
    using GradItem = std::conditional_t<WIN, WinGradItem, vit::GradItem>;
    const GradItem *items = items_of(p);
    constexpr int BN = C::BN, NY = C::NY, W = C::W;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *base = reinterpret_cast<unsigned char *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    Bars &bars = sh.bars;
    uint32_t &s_tmem = sh.tmem;
    volatile int &s_abort = sh.abort;
    auto &s_stat = sh.stat;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar_addr(bars.x_full[i]), 1);
            mbar_init(bar_addr(bars.x_empty[i]), WIN ? 9 : 1);   // the issuer, and the softmax warps
            mbar_init(bar_addr(bars.s_full[i]), 1);
            mbar_init(bar_addr(bars.p_full[i]), 4);
            mbar_init(bar_addr(bars.stat[i]), 1);
        }
        for (int i = 0; i < NY; ++i) {
            mbar_init(bar_addr(bars.y_full[i]), 1);
            mbar_init(bar_addr(bars.y_empty[i]), 1);
        }
        mbar_init(bar_addr(bars.acc_done), 1);
        mbar_init(bar_addr(bars.acc_free), 8);
        mbar_init(bar_addr(bars.drain), 1);
        if constexpr (WIN) {
            for (int i = 0; i < kItemRing; ++i) {
                mbar_init(bar_addr(sh.item_full[i]), 1);
                mbar_init(bar_addr(sh.item_empty[i]), DKV ? 11 : 9);   // the issuer, the softmax warps, warps 2 and 3
            }
        }
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_addr(&s_tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    grid_wait();                           // the lists and statistics of the launch before
    grid_release();
    // Each role reads the block's place and the list's length for itself: kept from here on, either of them spills.
    auto block = [&] {
        uint32_t b;
        asm volatile("mov.u32 %0, %%ctaid.x;\n" : "=r"(b));
        return (int)b - p.first_block;
    };
    auto list_length = [&] { return *static_cast<const volatile int32_t *>(p.n_items); };
    // the first tile of an item's loop that is its own
    auto first_j = [&](const GradItem &it) -> int {
        if constexpr (WIN && DKV) return it.j0;
        else return 0;
    };
    // tiles of the keys that a windowed query tile reads first
    auto first_tiles = [&](const GradItem &it) -> int {
        if constexpr (WIN && !DKV) return (it.fn + BN - 1) / BN;
        else return 0;
    };

    auto wait = [&](const uint64_t &b, uint32_t parity) -> bool {
        if (mbar_wait(bar_addr(b), parity, (const volatile int *)&s_abort, kWaitBudget)) return true;
        if (!s_abort) {
            s_abort = 1;
            report_error(p.status, VIT_ERR_TIMEOUT);
        }
        return false;
    };
    auto wait_warp = [&](const uint64_t &b, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, wait(b, parity)) != 0;
    };
    // The items of a block: every n_blocks-th one, or, where their lengths differ (WIN), its first one and then the next
    // that no block has taken, which the producer takes from a counter and passes on through a ring. (Blocks of the
    // second pass start when those of the first leave, so that with a fixed share each the sum of both counts: three
    // texts of 1500 to 2311 tokens, 32 heads over 8 of 128, causal, 345 us.)
    uint32_t taken = 0;                    // by this role
    auto put = [&](int i) -> bool {        // the producer's
        if constexpr (WIN) {
            const uint32_t s = taken % kItemRing;
            if (taken >= kItemRing && !wait(sh.item_empty[s], (taken / kItemRing - 1) & 1)) return false;
            sh.item[s] = i;
            mbar_arrive(bar_addr(sh.item_full[s]));
            ++taken;
        }
        return true;
    };
    auto take = [&]() -> int {             // the other roles', by whole warps
        int i = 0x7fffffff;
        if constexpr (WIN) {
            const uint32_t s = taken % kItemRing;
            if (wait_warp(sh.item_full[s], (taken / kItemRing) & 1)) {
                i = *static_cast<volatile int *>(&sh.item[s]);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_addr(sh.item_empty[s]));
                ++taken;
            }
        }
        return i;
    };
    auto first_item = [&]() { return WIN ? take() : block(); };
    auto next_item = [&](int i) { return WIN ? take() : i + p.n_blocks; };
    // tokens of a streamed tile; tiles of an item; streamed rows of tile j inside the sequence
    const int y_tok = DKV ? BN >> p.lg_pack : BN;
    auto valid_rows = [&](const GradItem &it, int j) -> int {
        if constexpr (DKV) {
            const int nt = (it.ln + y_tok - 1) / y_tok;
            return min(y_tok, it.ln - j % nt * y_tok) << p.lg_pack;
        } else if constexpr (WIN) {
            const int nf = first_tiles(it);
            return min(BN, j < nf ? it.fn - j * BN : it.ln - (j - nf) * BN);
        } else {
            return min(BN, it.ln - j * BN);
        }
    };

    if (warp < 4) regs_dec<kCtrlRegs>();
    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            tma_prefetch_desc(&tm.x1);
            tma_prefetch_desc(&tm.x2);
            tma_prefetch_desc(&tm.y1);
            tma_prefetch_desc(&tm.y2);
            uint32_t xc = 0, yc = 0;
            bool ok = true;
            int after = 0;                                   // the item after this one
            auto on = [&](int i) {
                if constexpr (WIN) return after;
                else return i + p.n_blocks;
            };
            for (int i = block(), n_items = list_length(); ok && i < n_items; i = on(i)) {
                if (!(ok = put(i))) break;
                if constexpr (WIN) after = p.n_blocks + atomicAdd(p.next, 1);
                const GradItem it = items[i];
                if (it.tiles == 0) continue;
                const uint32_t xb = xc & 1;
                if (xc >= 2 && !(ok = wait(bars.x_empty[xb], (xc / 2 - 1) & 1))) break;
                mbar_arrive_expect_tx(bar_addr(bars.x_full[xb]), 2 * C::X_TILE);
#pragma unroll
                for (int s = 0; s < C::NS; ++s) {
                    unsigned char *x = base + xb * 2 * C::X_TILE + s * C::X_SLAB;
                    tma_load_3d(smem_addr(x), &tm.x1, W * s, it.head, it.r0, bar_addr(bars.x_full[xb]));
                    tma_load_3d(smem_addr(x + C::X_TILE), &tm.x2, W * s, it.head, it.r0, bar_addr(bars.x_full[xb]));
                }
                ++xc;
                const int nt = DKV ? (it.ln + y_tok - 1) / y_tok : 0;
                for (int j = 0; j < it.tiles; ++j, ++yc) {
                    const int s = yc % NY;
                    if (yc >= (uint32_t)NY && !(ok = wait(bars.y_empty[s], (yc / NY - 1) & 1))) break;
                    int head, row;
                    if constexpr (DKV) {
                        const int jj = j + first_j(it);
                        head = it.head * p.group + ((jj / nt) << p.lg_pack);
                        row = it.l0 + jj % nt * y_tok;
                    } else {
                        const int nf = first_tiles(it);
                        head = it.head / p.group;
                        row = it.l0 + (j - nf) * BN;
                        if constexpr (WIN) {
                            if (j < nf) row = it.f0 + j * BN;
                        }
                    }
                    mbar_arrive_expect_tx(bar_addr(bars.y_full[s]), 2 * C::Y_TILE);
#pragma unroll
                    for (int c = 0; c < C::NS; ++c) {
                        unsigned char *y = base + C::OFF_Y + s * C::Y_PAIR + c * C::Y_SLAB;
                        tma_load_3d(smem_addr(y), &tm.y1, W * c, head, row, bar_addr(bars.y_full[s]));
                        tma_load_3d(smem_addr(y + C::Y_TILE), &tm.y2, W * c, head, row, bar_addr(bars.y_full[s]));
                    }
                }
            }
            if (ok) ok = put(0x7fffffff);
            if (!ok) {
                // let every copy already issued land before this block's shared memory is released
                const int never = 0;
                for (uint32_t k = xc > 2 ? xc - 2 : 0; k < xc; ++k)
                    mbar_wait(bar_addr(bars.x_full[k & 1]), (k / 2) & 1, &never, 20000000ll);
                for (uint32_t k = yc > (uint32_t)NY ? yc - NY : 0; k < yc; ++k)
                    mbar_wait(bar_addr(bars.y_full[k % NY]), (k / NY) & 1, &never, 20000000ll);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (lane 0; all lanes zero tails)
        constexpr uint32_t ID_S = idesc_bf16(128, BN, 0, 0), ID_ACC = idesc_bf16(128, D, 0, 1);
        const uint32_t a_x = smem_addr(base), a_y = smem_addr(base + C::OFF_Y);
        const uint64_t dx0 = smem_desc(a_x, 16, 8 * C::SW, C::LAYOUT), dy0 = smem_desc(a_y, 16, 8 * C::SW, C::LAYOUT);
        const uint64_t dm0 = smem_desc(a_y, C::Y_SLAB, 8 * C::SW, C::LAYOUT);      // the same tile, MN-major
        uint32_t xc = 0;                                     // items before this item
        bool ok = true;
        const bool leader = elect_one();
        auto uni = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
        // the 16-row step in which a tile's `valid` rows end: its rows past them are zeroed
        auto zero_tail = [&](uint32_t slot, int valid) {
            if (!(valid & 15)) return;
            unsigned char *y = base + C::OFF_Y + slot * C::Y_PAIR;
            const int n = 16 - (valid & 15);
            for (int x = lane; x < n * C::NS * (W / 8) * (DKV ? 2 : 1); x += 32) {
                const int r = valid + x % n, c = x / n % (W / 8), sl = x / n / (W / 8);   // every 16 bytes of the row
                *reinterpret_cast<uint4 *>(y + (sl / C::NS) * C::Y_TILE + (sl % C::NS) * C::Y_SLAB + r * C::SW + 16 * c) =
                    make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
        };
        // leader: S and dP of a tile into its stage, in turn. The operands' places are worked out by the whole warp:
        // inside the elected thread's branch the compiler no longer knows them to be uniform, and every MMA waits
        // for its operands to be made so. Between the two groups of MMAs of a tile, and before the next tile's,
        // there is little arithmetic: the tensor pipe holds only about four MMAs while the issuer does other things.
        auto products = [&](uint32_t tS, uint64_t dx, uint64_t dy, uint32_t full) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    constexpr int PER = W / 16;
                    const uint32_t ox = w * C::X_TILE + (kk / PER) * C::X_SLAB + (kk % PER) * 32;
                    const uint32_t oy = w * C::Y_TILE + (kk / PER) * C::Y_SLAB + (kk % PER) * 32;
                    mma_ss(tS + w * BN, dx + (ox >> 4), dy + (oy >> 4), ID_S, kk > 0 ? 1u : 0u);
                }
            mma_commit(full);
        };
        // leader: the tile's part of the sums
        auto sums = [&](uint32_t tS, uint64_t dm, int steps, uint32_t acc, uint32_t empty) {
            auto step = [&](int kk) {
                if constexpr (DKV)
                    mma_ts(tmem + C::TA2, tS + kk * 8, dm + ((C::Y_TILE + kk * 16 * C::SW) >> 4), ID_ACC, kk > 0 ? 1u : acc);
                mma_ts(tmem + C::TA1, tS + BN + kk * 8, dm + ((kk * 16 * C::SW) >> 4), ID_ACC, kk > 0 ? 1u : acc);
            };
            if (steps == BN / 16) {
#pragma unroll
                for (int kk = 0; kk < BN / 16; ++kk) step(kk);
            } else {
                for (int kk = 0; kk < steps; ++kk) step(kk);
            }
            mma_commit(empty);
        };
        // the next tile to start: its ring slot and phase, and its operand; the next to add up; the stage of both
        constexpr uint32_t Y_STEP = C::Y_PAIR >> 4;
        uint32_t s_p = 0, ph_p = 0, s_a = 0, st = 0, ph_s = 0;
        uint64_t dy = dy0, dm = dm0;
        uint32_t tS = tmem + C::TSTAGE;
        constexpr uint32_t TS_SUM = 2 * C::TSTAGE + 2 * BN;   // of the two stages' columns
        const uint32_t a_sfull = bar_addr(bars.s_full[0]), a_yempty = bar_addr(bars.y_empty[0]);
        auto start = [&](uint64_t dx, uint32_t x_empty, int valid, bool last, uint32_t stage, uint32_t t) -> bool {
            if (!(ok = wait_warp(bars.y_full[s_p], ph_p))) return false;
            zero_tail(s_p, valid);
            tc_fence_after();
            if (leader) products(t, dx, dy, a_sfull + 8 * stage);
            if (last && leader) mma_commit(x_empty);
            __syncwarp();
            dy += Y_STEP;
            if (++s_p == (uint32_t)NY) {
                s_p = 0;
                dy = dy0;
                ph_p ^= 1u;
            }
            return true;
        };
        for (int i = first_item(), n_items = list_length(); ok && i < n_items; i = next_item(i)) {
            const GradItem it = items[i];
            const int n = uni(it.tiles);
            if (n == 0) continue;
            // tiles follow one another inside a head pack; the last one of a pack holds `tail` rows
            const int nt = DKV ? uni((it.ln + y_tok - 1) / y_tok) : WIN ? n : uni((it.ln + BN - 1) / BN);
            const int tail = uni(valid_rows(it, nt - 1)), tail_steps = (tail + 15) >> 4;
            // (a windowed query tile's first keys may end inside a tile of their own)
            const int nf = WIN && !DKV ? uni(first_tiles(it)) : 0;
            const int f_tail = WIN && !DKV ? uni(nf > 0 ? valid_rows(it, nf - 1) : BN) : BN, f_steps = (f_tail + 15) >> 4;
            int pj = WIN && DKV ? uni(first_j(it) % nt) : 0, aj = pj;   // place in its pack of the next tile to start, to add up
            auto next_valid = [&]() {
                const bool end = ++pj == nt;
                const int v = end ? tail : WIN && !DKV && pj == nf ? f_tail : BN;
                pj = end ? 0 : pj;
                return v;
            };
            const uint32_t xb = xc & 1, x_empty = bar_addr(bars.x_empty[0]) + 8 * xb;
            const uint64_t dx = dx0 + xb * (2 * C::X_TILE >> 4);
            if (!(ok = wait_warp(bars.x_full[xb], (xc / 2) & 1))) break;
            if (!start(dx, x_empty, next_valid(), n == 1, st, tS)) break;
            if (n > 1 && !start(dx, x_empty, next_valid(), n == 2, st ^ 1u, tmem + (TS_SUM - (tS - tmem)))) break;
            if (xc > 0 && !(ok = wait_warp(bars.acc_free, (xc - 1) & 1))) break;
            uint32_t acc = 0;
            for (int j = 0; j < n; ++j) {
                const bool end = ++aj == nt;
                const int steps = end ? tail_steps : WIN && !DKV && aj == nf ? f_steps : BN / 16;
                aj = end ? 0 : aj;
                if (!(ok = wait_warp(bars.p_full[st], ph_s))) break;
                tc_fence_after();
                if (leader) sums(tS, dm, steps, acc, a_yempty + 8 * s_a);
                if (j + 1 == n && leader) mma_commit(bar_addr(bars.acc_done));
                __syncwarp();
                acc = 1;
                dm += Y_STEP;
                if (++s_a == (uint32_t)NY) {
                    s_a = 0;
                    dm = dm0;
                }
                // the stage is free: its softmax group has read it, and the MMAs above run first
                if (j + 2 < n && !start(dx, x_empty, next_valid(), j + 3 == n, st, tS)) break;
                tS = tmem + (TS_SUM - (tS - tmem));
                ph_s ^= st;                                  // both stages share a phase: it turns after stage 1
                st ^= 1u;
            }
            ++xc;
        }
        if (leader) {
            // nothing this thread issued may still be running when TMEM is freed
            mma_commit(bar_addr(bars.drain));
            mbar_wait(bar_addr(bars.drain), 0, (const volatile int *)&s_abort, ok ? kWaitBudget : 200000000ll);
        }
        __syncwarp();
    } else if (warp < 4) {
        if (p.zero_rest && list_length() >= 0) {
            // the rows between and around the sequences, dealt to both warps of all blocks; gap b lies before sequence
            // b, and only k_len leaves gaps between sequences (none behind one that is malformed: all its rows stay)
            const CrossSegs &s = p.segs;
            const int64_t T = DKV ? s.Tk : s.Tq;
            const int32_t *cu = DKV ? s.cu_k : s.cu_q, *len = DKV ? s.k_len : nullptr;
            const int H = DKV ? p.Hk : p.Hq, gaps = len ? s.B + 1 : 2;
            for (int g0 = 0; g0 < gaps; g0 += 32) {
                const int b = len ? g0 + lane : lane * s.B;   // without k_len: gaps 0 and B
                int lo = 0, hi = 0;
                if (g0 + lane < gaps) {
                    hi = b < s.B ? cu[b] : (int)T;
                    if (b > 0) {
                        CrossSeg x;
                        lo = len && load_seg(s, b - 1, x, nullptr, false) ? x.k0 + x.kn : cu[b];
                    }
                    if (lo < 0 || hi > T) hi = lo;
                }
                for (unsigned todo = __ballot_sync(0xffffffffu, lo < hi); todo; todo &= todo - 1) {
                    const int src = __ffs(todo) - 1;
                    const int end = __shfl_sync(0xffffffffu, hi, src);
                    for (int64_t r = __shfl_sync(0xffffffffu, lo, src) + (int64_t)(2 * block() + warp - 2); r < end;
                         r += 2 * p.n_blocks)
                        for (int c = lane; c < H * (D / 8); c += 32) {
                            const uint4 z = make_uint4(0u, 0u, 0u, 0u);
                            *reinterpret_cast<uint4 *>(p.out1 + r * p.out1_stride + 8 * c) = z;
                            if constexpr (DKV) *reinterpret_cast<uint4 *>(p.out2 + r * p.out2_stride + 8 * c) = z;
                        }
                }
            }
            __syncwarp();
        }
        if constexpr (DKV) {
            // ------------------------------------------------------------ statistics of the streamed columns
            // Warp 2 + g stores those of group g's next tile as soon as every warp of the group has finished the one
            // before (the group's tiles share a TMEM stage, and p_full is their last arrival), read a tile ahead.
            const int grp = warp - 2;
            constexpr int PER = (BN + 31) / 32;
            uint32_t u0 = 0;
            bool ok = true;
            for (int i = first_item(), n_items = list_length(); ok && i < n_items; i = next_item(i)) {
                const GradItem it = items[i];
                const int n = it.tiles;
                if (n == 0) continue;
                const int nt = (it.ln + y_tok - 1) / y_tok;
                float2 v[PER];
                auto fetch = [&](int j) {
                    if (j >= n) return;
                    const int jj = j + first_j(it), valid = valid_rows(it, jj), tok0 = it.l0 + jj % nt * y_tok;
                    const int head0 = it.head * p.group + ((jj / nt) << p.lg_pack);
#pragma unroll
                    for (int e = 0; e < PER; ++e) {
                        const int c = lane + 32 * e;
                        v[e] = make_float2(0.f, 0.f);
                        if (c < valid)
                            v[e] = p.stats[(int64_t)(tok0 + (c >> p.lg_pack)) * p.Hq + head0 +
                                           (c & ((1 << p.lg_pack) - 1))];
                    }
                };
                int j = (int)((u0 ^ (uint32_t)grp) & 1);
                fetch(j);
                for (; j < n; j += 2) {
                    const uint32_t u = u0 + j;
                    if (u >= 2 && !(ok = wait_warp(bars.p_full[grp], (u / 2 - 1) & 1))) break;
#pragma unroll
                    for (int e = 0; e < PER; ++e) {
                        const int c = lane + 32 * e;
                        if (c < BN) {
                            s_stat[grp][0][c] = v[e].x;
                            s_stat[grp][1][c] = v[e].y;
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_addr(bars.stat[grp]));
                    fetch(j + 2);
                }
                u0 += n;
            }
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------ softmax groups
        regs_inc<kSoftmaxRegs>();
        const int grp = (warp - 4) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
        uint32_t u0 = 0, xc = 0;                              // tiles and items with tiles before this item
        // WIN: the X buffer that this warp's store still reads, or -1; it is given back behind the warp's next tile
        [[maybe_unused]] int pending = -1;
        [[maybe_unused]] auto release = [&] {
            if (pending >= 0 && lane == 0) {
                bulk_wait_read_all();
                mbar_arrive(bar_addr(bars.x_empty[pending]));
            }
            pending = -1;
        };
        bool ok = true;
        for (int i = first_item(), n_items = list_length(); ok && i < n_items; i = next_item(i)) {
            const GradItem it = items[i];
            const int n = it.tiles;
            // the row of the output that this lane holds
            int o_row, o_head;
            if constexpr (DKV) {
                o_row = it.r0 + row;
                o_head = it.head;
            } else {
                o_row = it.r0 + (row >> p.lg_pack);
                o_head = it.head + (row & ((1 << p.lg_pack) - 1));
            }
            const bool exists = o_row < it.r1;
            float2 st_row = make_float2(0.f, 0.f);
            if constexpr (!DKV) {
                if (exists && n > 0) st_row = p.stats[(int64_t)o_row * p.Hq + o_head];
            }
            const float *nl = s_stat[grp][0], *nd = s_stat[grp][1];
            // the item's tiles, as it has delta from the scores or not
            auto tiles = [&](auto exact) {
                for (int j = (int)((u0 ^ (uint32_t)grp) & 1); j < n; j += 2) {
                    const uint32_t u = u0 + j, st = u & 1;
                    const int valid = valid_rows(it, j + first_j(it));
                    if constexpr (DKV) {
                        if (!(ok = wait_warp(bars.stat[grp], (u / 2) & 1))) break;
                    }
                    if (!(ok = wait_warp(bars.s_full[st], (u / 2) & 1))) break;
                    tc_fence_after();
                    const uint32_t tS = t_lane + C::TSTAGE + st * 2 * BN, tD = tS + BN;
                    // WIN: what this lane sees of the tile: columns before `hi`, from `lo` on or before `sk`
                    [[maybe_unused]] int hi = valid, lo = 0, sk = 0;
                    if constexpr (WIN && DKV) {                // the columns of a token lie side by side
                        const int nt = (it.ln + y_tok - 1) / y_tok;
                        const int d = it.rp + row - (it.lp + (j + it.j0) % nt * y_tok);   // this key against the first token
                        lo = min(max(d, 0), BN) << p.lg_pack;
                        if (p.window > 0 && it.rp + row >= p.sinks)
                            hi = min(hi, min(max(d + p.window, 0), BN) << p.lg_pack);
                    } else if constexpr (WIN) {
                        const int nf = first_tiles(it);
                        if (j >= nf) {
                            const int kp = it.lp + (j - nf) * BN, d = it.rp + (row >> p.lg_pack) - kp;
                            hi = min(hi, d + 1);
                            if (p.window > 0) {
                                lo = d - p.window + 1;
                                sk = p.sinks - kp;
                            }
                        }
                    }
                    if constexpr (decltype(exact)::value) {
                        // few keys, all of them in this tile: delta = sum_j p_ij dP_ij, in dq over this lane's
                        // columns, in dk, dv for each column over the lanes of the one warp that has keys (what the
                        // others make of a delta that is half written goes to rows that do not exist)
                        auto products = [&](int c0, float row_nl, auto keep, float (&x)[16]) {
                            uint32_t s[16], d[16];
                            tmem_ld16(tS + c0, s);
                            tmem_ld16(tD + c0, d);
                            tmem_wait_ld();
                            reg_fence(s);
                            reg_fence(d);
#pragma unroll
                            for (int c = 0; c < 16; ++c) {
                                const float l = DKV ? nl[c0 + c] : row_nl;
                                const float pr = ex2(fmaf(__uint_as_float(s[c]), p.scale_log2, l));
                                const float y = pr * __uint_as_float(d[c]);
                                x[c] = keep(c0 + c) ? y : 0.f;
                            }
                        };
                        float x[16];
                        if constexpr (DKV) {
                            if (quarter == 0) {
#pragma unroll 1
                                for (int c0 = 0; c0 < valid; c0 += 16) {
                                    products(c0, 0.f, [&](int) { return exists; }, x);
                                    // sums over the lanes by halving: lane l ends with column l / 2
#pragma unroll
                                    for (int h = 0; h < 4; ++h)
#pragma unroll
                                        for (int i = 0; i < 8 >> h; ++i) {
                                            const bool up = (lane & (16 >> h)) != 0;
                                            const float a = x[i], b = x[i + (8 >> h)];
                                            x[i] = (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, 16 >> h);
                                        }
                                    x[0] += __shfl_xor_sync(0xffffffffu, x[0], 1);
                                    if ((lane & 1) == 0) s_stat[grp][1][c0 + (lane >> 1)] = -x[0];
                                }
                                __syncwarp();
                            }
                        } else {
                            float sum = 0.f;
#pragma unroll 1
                            for (int c0 = 0; c0 < valid; c0 += 16) {
                                products(c0, st_row.x, [&](int c) { return c < valid; }, x);
#pragma unroll
                                for (int c = 0; c < 16; ++c) sum += x[c];
                            }
                            st_row.y = -sum;
                        }
                    }
                    sk = min(sk, hi);
                    [[maybe_unused]] const bool edge = WIN && __any_sync(0xffffffffu, hi < BN || lo > 0);
                    const uint64_t sc2 = f2_splat(p.scale_log2);
                    const uint64_t nl_row = f2_splat(st_row.x), nd_row = f2_splat(st_row.y);
                    // columns [C0, C0 + CN): P and dS go where columns already read were
                    auto part = [&](auto c0, auto cn) {
                        constexpr int C0 = decltype(c0)::value, CN = decltype(cn)::value;
                        uint32_t sr[CN], dr[CN];
#pragma unroll
                        for (int c = 0; c < CN; c += 16)
                            tmem_ld16(tS + C0 + c, *reinterpret_cast<uint32_t(*)[16]>(sr + c));
#pragma unroll
                        for (int c = 0; c < CN; c += 16)
                            tmem_ld16(tD + C0 + c, *reinterpret_cast<uint32_t(*)[16]>(dr + c));
                        tmem_wait_ld();
                        reg_fence(sr);
                        reg_fence(dr);
                        [[maybe_unused]] ulonglong2 l4, d4;
#pragma unroll
                        for (int c = 0; c < CN; c += 2) {
                            uint64_t l2 = nl_row, d2 = nd_row;
                            if constexpr (DKV) {
                                if (c % 4 == 0) {
                                    l4 = *reinterpret_cast<const ulonglong2 *>(nl + C0 + c);
                                    d4 = *reinterpret_cast<const ulonglong2 *>(nd + C0 + c);
                                }
                                l2 = c % 4 == 0 ? l4.x : l4.y;
                                d2 = c % 4 == 0 ? d4.x : d4.y;
                            }
                            float x0, x1;
                            f2_split(f2_fma(f2_from_u32(sr[c], sr[c + 1]), sc2, l2), x0, x1);
                            float p0 = ex2(x0), p1 = ex2(x1);
                            uint64_t pp;
                            asm("mov.b64 %0, {%1, %2};\n" : "=l"(pp) : "f"(p0), "f"(p1));
                            float g0, g1;
                            f2_split(f2_mul(f2_add(f2_from_u32(dr[c], dr[c + 1]), d2), pp), g0, g1);
                            sr[c / 2] = pack_bf16x2(p0, p1);
                            dr[c / 2] = pack_bf16x2(g0, g1);
                        }
                        if constexpr (WIN) {                      // what is not seen: exactly 0, whatever was there
                            if (edge) {
#pragma unroll
                                for (int x = 0; x < CN; x += 32) {
                                    constexpr uint32_t LAST = CN % 32 ? (1u << CN % 32) - 1 : 0xffffffffu;
                                    const uint32_t seen = seen_bits(C0 + x, hi, lo, sk), all = x + 32 > CN ? LAST : 0xffffffffu;
                                    if (!__all_sync(0xffffffffu, (seen & all) == all)) {
#pragma unroll
                                        for (int c = 0; c < 32; ++c)
                                            if (x + c < CN && !(seen & (1u << c))) {
                                                const uint32_t other = c % 2 ? 0x0000ffffu : 0xffff0000u;
                                                sr[(x + c) / 2] &= other;
                                                dr[(x + c) / 2] &= other;
                                            }
                                    }
                                }
                            }
                        } else if (valid < C0 + CN) {             // columns past the end: exactly 0, whatever was there
#pragma unroll
                            for (int c = 0; c < CN; c += 2) {
                                const int x = C0 + c;
                                const uint32_t keep = x + 1 < valid ? 0xffffffffu : x < valid ? 0x0000ffffu : 0u;
                                sr[c / 2] &= keep;
                                dr[c / 2] &= keep;
                            }
                        }
                        if constexpr (DKV) {
#pragma unroll
                            for (int c = 0; c < CN / 2; c += 8)
                                tmem_st8(tS + C0 / 2 + c, *reinterpret_cast<const uint32_t(*)[8]>(sr + c));
                        }
#pragma unroll
                        for (int c = 0; c < CN / 2; c += 8)
                            tmem_st8(tD + C0 / 2 + c, *reinterpret_cast<const uint32_t(*)[8]>(dr + c));
                    };
                    using std::integral_constant;
                    auto parts = [&] {
                        part(integral_constant<int, 0>(), integral_constant<int, C::PART>());
                        if constexpr (C::PART < BN)
                            part(integral_constant<int, C::PART>(), integral_constant<int, BN - C::PART>());
                    };
                    if constexpr (WIN) {
                        if (!__any_sync(0xffffffffu, hi > 0 && (lo < hi || sk > 0))) {
                            // none of the warp's pairs is seen: P = dS = 0, without a look at S and dP
                            const uint32_t zero[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll
                            for (int c = 0; c < BN / 2; c += 8) {
                                if constexpr (DKV) tmem_st8(tS + c, zero);
                                tmem_st8(tD + c, zero);
                            }
                        } else {
                            parts();
                        }
                    } else {
                        parts();
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_addr(bars.p_full[st]));
                    if constexpr (WIN) release();
                }
            };
            using std::bool_constant;
            if constexpr (WIN) {
                tiles(bool_constant<false>());
            } else {
                if (it.exact) tiles(bool_constant<true>());
                else tiles(bool_constant<false>());
            }
            if (!ok) break;
            u0 += n;
            if constexpr (WIN) {
                // The item's sums: group 0 writes dk, group 1 dv; of dq each writes its slabs. They go through the X tiles,
                // which the item no longer needs (and which have the outputs' shape), and from there by TMA: a store of
                // 16 bytes per row by every lane took 12 % of the time at a window of 1024. Tiles that the sequence ends
                // in are written by row.
                constexpr int HALF = (C::NS + 1) / 2;
                auto write = [&](auto first, auto last) {
                    constexpr int S0 = decltype(first)::value, S1 = decltype(last)::value, COLS = (S1 - S0) * W;
                    const int which = DKV ? grp : 0;
                    uint32_t r[COLS > 0 ? COLS : 1];
#pragma unroll
                    for (int c = 0; c < COLS; ++c) r[c] = 0u;
                    const uint32_t xb = xc & 1;
                    if (n > 0) {
                        if (!(ok = wait_warp(bars.acc_done, xc & 1))) return;
                        ++xc;
                        tc_fence_after();
#pragma unroll
                        for (int c = 0; c < COLS; c += 8)
                            tmem_ld8(t_lane + (which ? C::TA2 : C::TA1) + S0 * W + c, *reinterpret_cast<uint32_t(*)[8]>(r + c));
                        tmem_wait_ld();
                        reg_fence(r);
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar_addr(bars.acc_free));
                    }
                    if constexpr (DKV) {
                        if (it.slot >= 0) {                  // a run's sums, as they are
                            float *to = p.sums + (((int64_t)it.slot * 2 + which) * BM + row) * D;
                            if (exists) {
#pragma unroll
                                for (int c = 0; c < COLS; c += 4)
                                    *reinterpret_cast<uint4 *>(to + c) = make_uint4(r[c], r[c + 1], r[c + 2], r[c + 3]);
                            }
                            if (lane == 0) mbar_arrive(bar_addr(bars.x_empty[xb]));
                            __syncwarp();
                            return;
                        }
                    }
                    // a query at position 0 sees one key, whose weight is 1 whatever its score: no dq, and no dk of a key that
                    // no other query sees
                    const bool alone = DKV ? it.ln == 1 && it.lp == 0 : it.rp + (row >> p.lg_pack) == 0;
                    const float f = which ? 1.f : alone ? 0.f : p.scale;
                    const bool whole = n > 0 && it.r0 + (DKV ? BM : BM >> p.lg_pack) <= it.r1;
                    unsigned char *x = base + (2 * xb + which) * C::X_TILE;
                    __nv_bfloat16 *dst = (which ? p.out2 + (int64_t)o_row * p.out2_stride
                                                : p.out1 + (int64_t)o_row * p.out1_stride) + (int64_t)o_head * D;
#pragma unroll
                    for (int c = 0; c < COLS; c += 8) {
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[e] = pack_bf16x2(__uint_as_float(r[c + 2 * e]) * f, __uint_as_float(r[c + 2 * e + 1]) * f);
                        const uint4 v = make_uint4(o[0], o[1], o[2], o[3]);
                        // 16-byte piece k of the row in slab s, where the swizzle puts it
                        const int s = S0 + c / W, k = c % W / 8;
                        const int at = C::SW == 128 ? k ^ (row & 7) : C::SW == 64 ? k ^ ((row >> 1) & 3) : k ^ ((row >> 2) & 1);
                        if (whole) *reinterpret_cast<uint4 *>(x + s * C::X_SLAB + row * C::SW + 16 * at) = v;
                        else if (exists) *reinterpret_cast<uint4 *>(dst + S0 * W + c) = v;
                    }
                    if (whole && COLS > 0) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
#pragma unroll
                            for (int s = S0; s < S1; ++s)
                                tma_store_3d(which ? &tm.o2 : &tm.o1, smem_addr(x + s * C::X_SLAB + 32 * quarter * C::SW),
                                             W * s, it.head, it.r0 + (DKV ? 32 * quarter : (32 * quarter) >> p.lg_pack));
                            bulk_commit();
                        }
                        pending = (int)xb;
                    } else if (n > 0 && lane == 0) {
                        mbar_arrive(bar_addr(bars.x_empty[xb]));
                    }
                    __syncwarp();
                };
                release();
                if (DKV) write(std::integral_constant<int, 0>(), std::integral_constant<int, C::NS>());
                else if (grp == 0) write(std::integral_constant<int, 0>(), std::integral_constant<int, HALF>());
                else write(std::integral_constant<int, HALF>(), std::integral_constant<int, C::NS>());
                if (!ok) break;
                continue;
            } else {
                // ---- the item's sums: group 0 writes dk, group 1 dv; of dq each writes half of the columns
                constexpr int COLS = DKV ? D : D / 2;
                const int col0 = DKV ? 0 : grp * COLS;
                const uint32_t tA = t_lane + (DKV && grp ? C::TA2 : C::TA1) + col0;
                __nv_bfloat16 *dst = DKV && grp ? p.out2 + (int64_t)o_row * p.out2_stride
                                                : p.out1 + (int64_t)o_row * p.out1_stride;
                dst += (int64_t)o_head * D + col0;
                const float f = DKV && grp ? 1.f : p.scale;
                if (n > 0) {
                    if (!(ok = wait_warp(bars.acc_done, xc & 1))) break;
                    ++xc;
                    tc_fence_after();
                }
#pragma unroll
                for (int c = 0; c < COLS; c += 8) {
                    uint32_t r[8];
                    if (n > 0) {
                        tmem_ld8(tA + c, r);
                        tmem_wait_ld();
                        reg_fence(r);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) r[e] = 0u;
                    }
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[e] = pack_bf16x2(__uint_as_float(r[2 * e]) * f, __uint_as_float(r[2 * e + 1]) * f);
                    if (exists) *reinterpret_cast<uint4 *>(dst + c) = make_uint4(o[0], o[1], o[2], o[3]);
                }
                if (n > 0) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_addr(bars.acc_free));
                }
            }
        }
        if constexpr (WIN) release();                         // (the shared memory goes with the block)
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Both passes: the first blocks take dk, dv, the rest dq. They do not depend on one another, and the blocks of the
// second come to SMs as those of the first leave.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
cross_grad_kernel(const __grid_constant__ GradMaps tm_dkv, const __grid_constant__ GradMaps tm_dq,
                  const __grid_constant__ Grad dkv, const __grid_constant__ Grad dq)
{
    __shared__ GradShared<D> sh;
    if ((int)blockIdx.x < dkv.n_blocks)
        grad_pass<D, true, false>(tm_dkv, dkv, sh);
    else
        grad_pass<D, false, false>(tm_dq, dq, sh);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
window_grad_kernel(const __grid_constant__ WinGradMaps tm_dkv, const __grid_constant__ WinGradMaps tm_dq,
                   const __grid_constant__ WinGrad dkv, const __grid_constant__ WinGrad dq)
{
    __shared__ WinGradShared<D> sh;
    if ((int)blockIdx.x < dkv.n_blocks)
        grad_pass<D, true, true>(tm_dkv, dkv, sh);
    else
        grad_pass<D, false, true>(tm_dq, dq, sh);
}

// ------------------------------------------------------------------ lists and statistics

// One list of work items by one block of 1024 threads: the dk, dv tiles (`keys`, ordered by query
// count) or the dq tiles (ordered by key count), longest loop first. Tiles without a loop are listed
// too: their gradients are 0.
template <bool W>
__device__ void make_list(bool keys, const CrossSegs &segs, int Hq, int Hk, int lg_pack, int bn, int32_t *counts,
                          std::conditional_t<W, WinGradItem, GradItem> *items, int32_t *status, int window, int sinks,
                          int cut_over, int run_tiles, int max_slots, WinGradTile *cut)
{
    constexpr int kThreads = kSortThreads;
    extern __shared__ unsigned long long s_key[];      // [NP] loop length descending, then index; later first item | index
    __shared__ int64_t s_warp[32];
    __shared__ int s_bad, s_used, s_total, s_more, s_cut, s_slots;
    const int tid = threadIdx.x, B = segs.B;
    const int lg_tile = keys ? 7 : 7 - lg_pack;        // rows (tokens) of a tile, log2
    const int heads = keys ? Hk : Hq >> lg_pack;       // tiles side by side
    auto rows_of = [&](const CrossSeg &x) { return keys ? x.kn : x.qn; };
    auto key_of = [&](bool use, const CrossSeg &x, int i) {
        return ((unsigned long long)(use ? 0x7fffffffu - (uint32_t)(keys ? x.qn : x.kn) : 0xffffffffu) << 32) | (uint32_t)i;
    };
    auto items_of = [&](const CrossSeg &x) { return heads * ((rows_of(x) + (1 << lg_tile) - 1) >> lg_tile); };
    auto decreases = [&](int i) { return segs.cu_q[i + 1] < segs.cu_q[i] || segs.cu_k[i + 1] < segs.cu_k[i]; };
    if (B <= 32) {
        // a warp: one sequence per lane
        if (tid < 32) {
            CrossSeg x;
            const bool fine = tid < B && load_seg(segs, tid, x, status, !keys);
            const bool bad = tid < B && decreases(tid), use = fine && rows_of(x) > 0;
            const int n = use ? items_of(x) : 0;
            int rank, at, none;
            warp_place(key_of(use, x, tid), n, 0, rank, at, none);
            s_key[rank] = ((unsigned long long)at << 32) | (uint32_t)tid;
            const unsigned used = __ballot_sync(0xffffffffu, use), any_bad = __ballot_sync(0xffffffffu, bad);
            if (rank == 31) {
                s_total = at + n;
                s_used = __popc(used);
                s_bad = any_bad != 0;
            }
        }
        __syncthreads();
    } else {
        int NP = 32;
        while (NP < B) NP <<= 1;
        if (tid == 0) s_bad = s_used = 0;
        __syncthreads();
        for (int i = tid; i < NP; i += kThreads) {
            CrossSeg x;
            const bool fine = i < B && load_seg(segs, i, x, status, !keys);
            if (i < B && decreases(i)) s_bad = 1;
            const bool use = fine && rows_of(x) > 0;
            s_key[i] = key_of(use, x, i);
            if (use) atomicAdd(&s_used, 1);
        }
        __syncthreads();
        block_sort(s_key, NP, tid);
        const int per = (B + kThreads - 1) / kThreads, lo = min(tid * per, s_used), hi = min(lo + per, s_used);
        auto seg_at = [&](int p) {
            CrossSeg x;
            load_seg(segs, (int)(s_key[p] & 0xffffffffu), x, nullptr, false);
            return x;
        };
        int64_t n = 0, total;
        for (int p = lo; p < hi; ++p) n += items_of(seg_at(p));
        int64_t at = block_exclusive_scan(n, s_warp, &total);
        for (int p = lo; p < hi; ++p) {
            const int k = items_of(seg_at(p));
            s_key[p] = ((unsigned long long)at << 32) | (uint32_t)(s_key[p] & 0xffffffffu);
            at += k;
        }
        if (tid == 0) s_total = (int)total;
        __syncthreads();
    }
    const int total = s_bad ? 0 : s_total;
    if (tid == 0) counts[keys] = s_bad ? -1 : total;   // -1: the call is left alone altogether
    if (W && tid == 0) {
        counts[2 + keys] = 0;
        s_more = s_cut = s_slots = 0;
    }
    if (W) __syncthreads();
    for (int i = tid; i < total; i += kThreads) {
        const int p = place_of(s_key, s_used, i), n = i - (int)(s_key[p] >> 32);
        CrossSeg x;
        load_seg(segs, (int)(s_key[p] & 0xffffffffu), x, nullptr, false);
        const int nr = (rows_of(x) + (1 << lg_tile) - 1) >> lg_tile;
        const int step = keys ? bn >> lg_pack : bn;
        if constexpr (W) {
            // all heads of a tile one after the other, the longest tiles first: a sequence's first keys, its last queries
            const int r = keys ? n / heads : nr - 1 - n / heads, h = n % heads;
            const int p0 = x.kn - x.qn, a = r << lg_tile, e = min(rows_of(x), a + (1 << lg_tile));
            WinGradItem it;
            it.r0 = (keys ? x.k0 : x.q0) + a;
            it.r1 = keys ? x.k0 + x.kn : x.q0 + x.qn;
            it.head = keys ? h : h << lg_pack;
            it.f0 = x.k0;
            it.fn = 0;
            if (keys) {                                // queries from the first key's position on
                const int lo = max(0, a - p0);
                const int64_t hi = window == 0 || a < sinks ? x.qn : (int64_t)e - 1 + window - p0;
                it.rp = a;
                it.lp = p0 + lo;
                it.l0 = x.q0 + lo;
                it.ln = (int)max((int64_t)0, min((int64_t)x.qn, hi) - lo);
                it.tiles = (it.ln + step - 1) / step * (Hq / Hk >> lg_pack);
            } else {                                   // (queries before the first key see nothing)
                const int last = p0 + e - 1;
                it.rp = p0 + a;
                it.lp = 0;
                it.ln = 0;
                if (last >= 0) {
                    const WinRange w = win_range(it.rp, window, sinks);
                    it.fn = w.first;
                    it.lp = w.lo;
                    it.ln = last + 1 - w.lo;
                }
                it.l0 = x.k0 + it.lp;
                it.tiles = (it.fn + step - 1) / step + (it.ln + step - 1) / step;
            }
            it.j0 = 0;
            it.slot = -1;
            if (keys && cut_over > 0 && it.tiles > cut_over) {
                // dealt evenly; its first run stands here, the others behind the list (in any order)
                const int all = it.tiles, runs = (all + run_tiles - 1) / run_tiles;
                const int slot = atomicAdd(&s_slots, runs);
                if (slot + runs <= max_slots) {        // (the plan has room for all of them)
                    const int more = total + atomicAdd(&s_more, runs - 1);
                    cut[atomicAdd(&s_cut, 1)] = WinGradTile{it.r0, min(it.r0 + 128, it.r1), it.head, slot, runs, {0, 0, 0}};
                    for (int k = 1; k < runs; ++k) {
                        it.j0 = (int)((int64_t)all * k / runs);
                        it.tiles = (int)((int64_t)all * (k + 1) / runs) - it.j0;
                        it.slot = slot + k;
                        items[more + k - 1] = it;
                    }
                    it.j0 = 0;
                    it.tiles = all / runs;
                    it.slot = slot;
                }
            }
            items[i] = it;
        } else {
            const int h = n / nr, r = n - h * nr;
            GradItem it;
            it.r0 = (keys ? x.k0 : x.q0) + (r << lg_tile);
            it.r1 = keys ? x.k0 + x.kn : x.q0 + x.qn;
            it.l0 = keys ? x.q0 : x.k0;
            it.ln = keys ? x.qn : x.kn;
            it.head = keys ? h : h << lg_pack;
            it.tiles = (it.ln + step - 1) / step * (keys ? Hq / Hk >> lg_pack : 1);
            it.exact = x.kn > 1 && x.kn <= kExactKeys;     // (one key: out is v, and nothing is lost)
            it.pad = 0;
            items[i] = it;
        }
    }
    if constexpr (W) {
        __syncthreads();
        if (keys && tid == 0) {
            if (!s_bad) counts[1] = total + s_more;
            counts[4] = s_cut;
        }
    }
}

struct Prepare {
    const __nv_bfloat16 *out, *dout;
    const float *lse;
    float2 *stats;                // {-lse log2(e), -delta} of every (token, head)
    int64_t rows, out_stride, dout_stride;
    CrossSegs segs;
    int Hq, Hk, lg_pack;
    int32_t *counts;
    void *dq, *dkv;               // the lists
    int32_t *status;
    // W: q, k and v for rows whose delta is from the scores
    const __nv_bfloat16 *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    int window, sinks;
    float scale_log2;
    int cut_over, run_tiles, max_slots;
    WinGradTile *cut;
};

// The keys that a token's rows see where those are 2 to kExactKeys: the first `first` of its sequence and `n` in all,
// the others from position lo on; else n = 0.
struct FewKeys {
    int64_t k0;
    int first, lo, n;
};
// cu_q: the list, or a copy of it in shared memory
__device__ __forceinline__ FewKeys few_keys(const Prepare &p, const int32_t *cu_q, int64_t t)
{
    const CrossSegs &s = p.segs;
    FewKeys none{0, 0, 0, 0};
    int b = 0, end = s.B;                              // the last sequence that begins at or before t (offsets that
    while (end - b > 1) {                              // decrease lead nowhere: the call computes nothing then)
        const int m = (b + end) >> 1;
        if (cu_q[m] <= t) b = m;
        else end = m;
    }
    CrossSeg x;
    if (!load_seg(s, b, x, nullptr, false) || t < x.q0 || t >= (int64_t)x.q0 + x.qn) return none;
    const int pos = x.kn - x.qn + (int)(t - x.q0);
    if (pos < 1) return none;
    const WinRange w = win_range(pos, p.window, p.sinks);
    const int64_t n = (int64_t)w.first + pos + 1 - w.lo;
    if (n < 2 || n > kExactKeys) return none;
    return FewKeys{x.k0, w.first, w.lo, (int)n};
}

// The statistics of a windowed call, by the blocks from `first_block` on. A warp takes up to kHeadSteps steps of
// 32 / (D / 16) heads of one token, 32 bytes of o and do a lane, so that what the token sees is looked up once for them; rows that see few keys are
// left to a second round, two lanes per key and a warp per row (one after the other in the first round, the 16 first
// tokens of a sequence alone took 40 us).
constexpr int kHeadSteps = 4;
template <int D>
__device__ void window_stats(const Prepare &p, int first_block)
{
    constexpr int CH = D / 16, R = 32 / CH, HEADS = R * kHeadSteps;
    extern __shared__ unsigned long long s_lists[];
    const int32_t *cu_q = p.segs.cu_q;
    if (p.segs.B <= 2 * kSortThreads) {                // (the searches' reads; the launch has room for the list)
        int32_t *copy = reinterpret_cast<int32_t *>(s_lists);
        for (int i = threadIdx.x; i < p.segs.B; i += kSortThreads) copy[i] = p.segs.cu_q[i];
        __syncthreads();
        cu_q = copy;
    }
    const int lane = threadIdx.x & 31;
    const int64_t n_tokens = p.rows / p.Hq;
    const int64_t warp = ((int64_t)(blockIdx.x - first_block) * blockDim.x + threadIdx.x) >> 5;
    const int64_t n_warps = ((int64_t)(gridDim.x - first_block) * blockDim.x) >> 5;
    auto load = [](const __nv_bfloat16 *x, bool live) {
        return live ? *reinterpret_cast<const uint4 *>(x) : make_uint4(0u, 0u, 0u, 0u);
    };
    auto dot = [](const uint4 &x, const uint4 &y, float s) {
        float a[8], b[8];
        rope::unpack8(x, a);
        rope::unpack8(y, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(a[e], b[e], s);
        return s;
    };
    {
        const int g = lane / CH, c = lane % CH, per_token = (p.Hq + HEADS - 1) / HEADS;
        for (int64_t w = warp; w < n_tokens * per_token; w += n_warps) {
            const int64_t t = per_token == 1 ? w : w >> 32 ? w / per_token : (int64_t)((uint32_t)w / (uint32_t)per_token);
            const int h0 = (int)(w - t * per_token) * HEADS;
            if (few_keys(p, cu_q, t).n > 0) continue;
            const __nv_bfloat16 *o = p.out + t * p.out_stride + 16 * c, *d = p.dout + t * p.dout_stride + 16 * c;
#pragma unroll
            for (int i = 0; i < kHeadSteps; ++i) {
                if (h0 + R * i >= p.Hq) break;
                const int h = h0 + R * i + g;
                const bool live = g < R && h < p.Hq;
                const __nv_bfloat16 *oh = o + (int64_t)h * D, *dh = d + (int64_t)h * D;
                const uint4 o0 = load(oh, live), o1 = load(oh + 8, live), d0 = load(dh, live), d1 = load(dh + 8, live);
                const float x = dot(o1, d1, dot(o0, d0, 0.f));
                float s = 0.f;                         // over the row's lanes
#pragma unroll
                for (int j = 0; j < CH; ++j) s += __shfl_sync(0xffffffffu, x, (g * CH + j) & 31);
                const int64_t r = t * p.Hq + h;
                if (live && c == 0) p.stats[r] = make_float2(-p.lse[r] * 1.4426950408889634f, -s);
            }
        }
    }
    // every row of a narrow window, else the first tokens of each sequence
    const bool narrow = p.window > 0 && (int64_t)p.window + p.sinks <= kExactKeys;
    const int64_t n_few = narrow ? p.rows : (int64_t)p.segs.B * kExactKeys * p.Hq;
    for (int64_t w = warp; w < n_few; w += n_warps) {
        int64_t t = w / p.Hq;
        const int h = (int)(w - t * p.Hq);
        if (!narrow) {
            CrossSeg x;
            const int b = (int)(t / kExactKeys), i = (int)(t % kExactKeys);
            if (!load_seg(p.segs, b, x, nullptr, false)) continue;
            const WinSeg s = win_seg(x);
            if (i >= s.qn) continue;
            t = (int64_t)s.q0 + i;
        }
        const FewKeys f = few_keys(p, cu_q, t);
        if (f.n == 0) continue;
        const int j = lane >> 1, part = (lane & 1) * (D / 2);
        const bool live = j < f.n;
        const int64_t row = f.k0 + (j < f.first ? j : f.lo + j - f.first), kv = (int64_t)(h / (p.Hq / p.Hk)) * D + part;
        const __nv_bfloat16 *q = p.q + t * p.q_stride + (int64_t)h * D + part, *k = p.k + row * p.k_stride + kv;
        const __nv_bfloat16 *d = p.dout + t * p.dout_stride + (int64_t)h * D + part, *v = p.v + row * p.v_stride + kv;
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int c = 0; c < D / 2; c += 8) {
            x = dot(load(q + c, live), load(k + c, live), x);
            y = dot(load(d + c, live), load(v + c, live), y);
        }
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        y += __shfl_xor_sync(0xffffffffu, y, 1);
        const int64_t r = t * p.Hq + h;
        const float nl = -p.lse[r] * 1.4426950408889634f;
        float s = live ? ex2(fmaf(x, p.scale_log2, nl)) * y : 0.f;     // delta = sum_j p_j (do v_j)
#pragma unroll
        for (int o = 2; o < 32; o *= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) p.stats[r] = make_float2(nl, -s);
    }
}

template <int D, bool W>
__global__ void __launch_bounds__(kSortThreads)
cross_grad_prepare_kernel(const Prepare p)
{
    using Item = std::conditional_t<W, WinGradItem, GradItem>;
    grid_wait();
    grid_release();
    if (blockIdx.x < 2) {
        const bool keys = blockIdx.x == 1;
        make_list<W>(keys, p.segs, p.Hq, p.Hk, p.lg_pack, keys ? GradCfg<D, true>::BN : GradCfg<D, false>::BN,
                     p.counts, static_cast<Item *>(keys ? p.dkv : p.dq), p.status, p.window, p.sinks, p.cut_over,
                     p.run_tiles, p.max_slots, p.cut);
        return;
    }
    if constexpr (W) {
        window_stats<D>(p, 2);
        return;
    }
    // D / 8 lanes per row, 16 bytes of o and do each
    constexpr int CH = D / 8, R = 32 / CH;
    const int lane = threadIdx.x & 31, g = lane / CH, c = lane % CH;
    const int64_t warp = ((int64_t)(blockIdx.x - 2) * blockDim.x + threadIdx.x) >> 5;
    const int64_t n_warps = ((int64_t)(gridDim.x - 2) * blockDim.x) >> 5;
    for (int64_t r0 = warp * R; r0 < p.rows; r0 += n_warps * R) {
        const int64_t r = r0 + g;
        const bool live = g < R && r < p.rows;
        float s = 0.f;
        if (live) {
            const int64_t t = r / p.Hq;
            const int h = (int)(r - t * p.Hq);
            float a[8], b[8];
            rope::unpack8(*reinterpret_cast<const uint4 *>(p.out + t * p.out_stride + (int64_t)h * D + 8 * c), a);
            rope::unpack8(*reinterpret_cast<const uint4 *>(p.dout + t * p.dout_stride + (int64_t)h * D + 8 * c), b);
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(a[e], b[e], s);
        }
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i) sum += __shfl_sync(0xffffffffu, s, (g * CH + i) & 31);
        if (live && c == 0) p.stats[r] = make_float2(-p.lse[r] * 1.4426950408889634f, -sum);
    }
}

// dk and dv of the key tiles whose loops were cut: their runs' sums in order. 32 blocks of 4 rows per
// tile: what it costs is the time of reading one run after the other.
template <int D>
__global__ void __launch_bounds__(256, 3)
window_grad_join_kernel(const int32_t *counts, const WinGradTile *cut, const float *sums, float scale, __nv_bfloat16 *dk,
                        __nv_bfloat16 *dv, int64_t dk_stride, int64_t dv_stride)
{
    grid_wait();
    grid_release();
    const int n = counts[1] < 0 ? 0 : counts[4];
    for (int b = blockIdx.x; b < 32 * n; b += gridDim.x) {
        const WinGradTile t = cut[b >> 5];
        for (int x = threadIdx.x; x < 2 * 4 * (D / 4); x += 256) {
            const int which = x / (4 * (D / 4)), r = (b & 31) * 4 + x / (D / 4) % 4, c = x % (D / 4) * 4;
            if (t.r0 + r >= t.r1) continue;
            const float *at = sums + (((int64_t)t.slot * 2 + which) * BM + r) * D + c;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
            for (int k = 0; k < t.runs; ++k) {
                const float4 v = *reinterpret_cast<const float4 *>(at + (int64_t)k * 2 * BM * D);
                sum.x += v.x;
                sum.y += v.y;
                sum.z += v.z;
                sum.w += v.w;
            }
            const float f = which ? 1.f : scale;
            __nv_bfloat16 *to = (which ? dv + (int64_t)(t.r0 + r) * dv_stride : dk + (int64_t)(t.r0 + r) * dk_stride);
            *reinterpret_cast<uint2 *>(to + (int64_t)t.head * D + c) =
                make_uint2(pack_bf16x2(sum.x * f, sum.y * f), pack_bf16x2(sum.z * f, sum.w * f));
        }
    }
}

// ------------------------------------------------------------------ host side

bool tile_map(CUtensorMap *m, const void *ptr, int64_t T, int H, int D, int64_t stride, int w, int pack, int rows)
{
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)H, (uint64_t)(T > 0 ? T : 1)};
    const uint64_t strides[2] = {(uint64_t)D * 2, (uint64_t)stride * 2};
    const uint32_t box[3] = {(uint32_t)w, (uint32_t)pack, (uint32_t)(rows / pack)};
    return encode_tiled_map(m, ptr, 3, dims, strides, box, 2 * w);
}

// A pass's tensor maps and parameters; its blocks are as many as its items at most.
template <int D, bool DKV>
bool make_pass(const CrossGradArgs &a, const GradPlan &pl, int num_sms, GradMaps &m, Grad &p)
{
    using C = GradCfg<D, DKV>;
    const CrossSegs &s = a.f.segs;
    const int pack = 1 << pl.lg_pack;
    // q and do, then k and v, as the resident or the streamed side
    const int qr = DKV ? C::BN : BM, kr = DKV ? BM : C::BN;
    CUtensorMap &q = DKV ? m.y1 : m.x1, &dout = DKV ? m.y2 : m.x2, &k = DKV ? m.x1 : m.y1, &v = DKV ? m.x2 : m.y2;
    if (!tile_map(&q, a.f.q, s.Tq, a.f.Hq, D, a.f.q_stride, C::W, pack, qr) ||
        !tile_map(&dout, a.dout, s.Tq, a.f.Hq, D, a.dout_stride, C::W, pack, qr) ||
        !tile_map(&k, a.f.k, s.Tk, a.f.Hk, D, a.f.k_stride, C::W, 1, kr) ||
        !tile_map(&v, a.f.v, s.Tk, a.f.Hk, D, a.f.v_stride, C::W, 1, kr))
        return false;
    char *ws = static_cast<char *>(a.f.workspace);
    p.items = reinterpret_cast<const GradItem *>(ws + (DKV ? pl.off_dkv : pl.off_dq));
    p.n_items = reinterpret_cast<const int32_t *>(ws) + (DKV ? 1 : 0);
    p.stats = reinterpret_cast<const float2 *>(ws + pl.off_stats);
    p.out1 = static_cast<__nv_bfloat16 *>(DKV ? a.dk : a.dq);
    p.out2 = static_cast<__nv_bfloat16 *>(a.dv);
    p.out1_stride = DKV ? a.dk_stride : a.dq_stride;
    p.out2_stride = a.dv_stride;
    p.Hq = a.f.Hq;
    p.group = a.f.Hq / a.f.Hk;
    p.lg_pack = pl.lg_pack;
    p.scale = a.f.scale_log2 * 0.6931471805599453f;
    p.scale_log2 = a.f.scale_log2;
    p.Hk = a.f.Hk;
    p.segs = s;
    p.zero_rest = a.zero_rest;
    p.status = a.f.status;
    const int64_t list = DKV ? pl.max_dkv : pl.max_dq, most = a.zero_rest ? num_sms : list;   // zeros: by every SM
    p.n_blocks = (int)(most < num_sms ? most : num_sms);
    return true;
}

template <int D, bool W>
cudaError_t launch_d(const CrossGradArgs &a, const std::conditional_t<W, WinGradPlan, GradPlan> &pl, int window,
                     int sinks, int num_sms, cudaStream_t stream)
{
    const CrossSegs &s = a.f.segs;
    char *ws = static_cast<char *>(a.f.workspace);

    Prepare r;
    r.out = static_cast<const __nv_bfloat16 *>(a.f.out);
    r.dout = static_cast<const __nv_bfloat16 *>(a.dout);
    r.lse = a.f.lse;
    r.stats = reinterpret_cast<float2 *>(ws + pl.off_stats);
    r.rows = s.Tq * a.f.Hq;
    r.out_stride = a.f.out_stride;
    r.dout_stride = a.dout_stride;
    r.segs = s;
    r.Hq = a.f.Hq;
    r.Hk = a.f.Hk;
    r.lg_pack = pl.lg_pack;
    r.counts = reinterpret_cast<int32_t *>(ws);
    r.dq = ws + pl.off_dq;
    r.dkv = ws + pl.off_dkv;
    r.status = a.f.status;
    r.q = static_cast<const __nv_bfloat16 *>(a.f.q);
    r.k = static_cast<const __nv_bfloat16 *>(a.f.k);
    r.v = static_cast<const __nv_bfloat16 *>(a.f.v);
    r.q_stride = a.f.q_stride;
    r.k_stride = a.f.k_stride;
    r.v_stride = a.f.v_stride;
    r.window = window;
    r.sinks = sinks;
    r.scale_log2 = a.f.scale_log2;
    r.cut_over = r.run_tiles = r.max_slots = 0;
    r.cut = nullptr;
    if constexpr (W) {
        r.cut_over = pl.cut_over;
        r.run_tiles = pl.run_tiles;
        r.max_slots = pl.max_slots;
        r.cut = reinterpret_cast<WinGradTile *>(ws + pl.off_cut);
    }
    int np = 32;
    while (np < s.B) np <<= 1;
    static DeviceOnce once_prepare;
    cudaError_t e = once_prepare.run([] {
        return cudaFuncSetAttribute(cross_grad_prepare_kernel<D, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)sizeof(unsigned long long) * VIT_MAX_SEGMENTS);
    });
    if (e != cudaSuccess) return e;
    {
        constexpr int per = 32 * (32 / (D / 8));             // rows of a block at a time
        constexpr int heads = kHeadSteps * (32 / (D / 16));
        const int64_t tasks = s.Tq * ((a.f.Hq + heads - 1) / heads);
        const int64_t want = W ? (tasks + 31) / 32 : (r.rows + per - 1) / per, cap = W ? num_sms - 2 : (int64_t)num_sms * 8;
        LaunchScope scope(W ? "window_grad_prepare" : "cross_grad_prepare", stream);
        e = launch_chained(cross_grad_prepare_kernel<D, W>, 2 + (unsigned)(want < cap ? want : cap), kSortThreads,
                           sizeof(unsigned long long) * (size_t)np, stream, r);
        if (e != cudaSuccess) return e;
    }

    std::conditional_t<W, WinGradMaps, GradMaps> m_dkv, m_dq;
    std::conditional_t<W, WinGrad, Grad> dkv, dq;
    if (!make_pass<D, true>(a, pl, num_sms, m_dkv, dkv) || !make_pass<D, false>(a, pl, num_sms, m_dq, dq))
        return cudaErrorInvalidValue;
    if constexpr (W) {
        constexpr int cols = GradCfg<D, true>::W;
        static_assert(cols == GradCfg<D, false>::W, "slabs of both passes");
        // (a side without rows has no items: nothing is stored there, but a map needs an address)
        const void *dq_at = s.Tq > 0 ? a.dq : a.dk, *dk_at = s.Tk > 0 ? a.dk : a.dq, *dv_at = s.Tk > 0 ? a.dv : a.dq;
        const int64_t nq = (int64_t)a.f.Hq * D, nk = (int64_t)a.f.Hk * D;
        if (!tile_map(&m_dkv.o1, dk_at, s.Tk, a.f.Hk, D, s.Tk > 0 ? a.dk_stride : nk, cols, 1, 32) ||
            !tile_map(&m_dkv.o2, dv_at, s.Tk, a.f.Hk, D, s.Tk > 0 ? a.dv_stride : nk, cols, 1, 32) ||
            !tile_map(&m_dq.o1, dq_at, s.Tq, a.f.Hq, D, s.Tq > 0 ? a.dq_stride : nq, cols, 1 << pl.lg_pack, 32))
            return cudaErrorInvalidValue;
        m_dq.o2 = m_dq.o1;
        dkv.win_items = static_cast<const WinGradItem *>(r.dkv);
        dq.win_items = static_cast<const WinGradItem *>(r.dq);
        dkv.sums = dq.sums = reinterpret_cast<float *>(ws + pl.off_sums);
        // (runs of cut loops are items as well)
        dkv.n_blocks = dkv.n_blocks + pl.max_slots < num_sms ? dkv.n_blocks + pl.max_slots : num_sms;
        dkv.next = r.counts + 3;
        dq.next = r.counts + 2;
        dkv.window = dq.window = window;
        dkv.sinks = dq.sinks = sinks;
        if (window == 1 && sinks == 0) dkv.scale = dq.scale = 0.f;     // every query sees one key
    }
    dkv.first_block = 0;
    dq.first_block = dkv.n_blocks;
    const int blocks = dkv.n_blocks + dq.n_blocks;
    if (blocks == 0) return cudaSuccess;
    constexpr int a1 = GradCfg<D, true>::SMEM, a2 = GradCfg<D, false>::SMEM, smem = a1 > a2 ? a1 : a2;
    static_assert(smem + sizeof(std::conditional_t<W, WinGradShared<D>, GradShared<D>>) <= 227 * 1024, "shared memory per block");
    auto kern = [] {
        if constexpr (W) return window_grad_kernel<D>;
        else return cross_grad_kernel<D>;
    }();
    static DeviceOnce once;
    e = once.run([&] {
        cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (r != cudaSuccess) return r;
        // the setmaxnreg split assumes exactly this launch budget
        cudaFuncAttributes fa;
        r = cudaFuncGetAttributes(&fa, kern);
        if (r != cudaSuccess) return r;
        return (fa.numRegs != kLaunchRegs || fa.maxThreadsPerBlock < kThreads) ? cudaErrorInvalidConfiguration
                                                                              : cudaSuccess;
    });
    if (e != cudaSuccess) return e;
    {
        LaunchScope scope(W ? "window_grad" : "cross_grad", stream);
        e = launch_chained(kern, (unsigned)blocks, kThreads, smem, stream, m_dkv, m_dq, dkv, dq);
    }
    if constexpr (W) {
        if (e == cudaSuccess && pl.cut_over > 0) {
            LaunchScope scope("window_grad_join", stream);
            const int want = 32 * pl.max_cut;
            e = launch_chained(window_grad_join_kernel<D>, (unsigned)(want < 4 * num_sms ? want : 4 * num_sms), 256, 0, stream,
                               r.counts, r.cut, dkv.sums, dkv.scale, static_cast<__nv_bfloat16 *>(a.dk),
                               static_cast<__nv_bfloat16 *>(a.dv), a.dk_stride, a.dv_stride);
        }
    }
    return e;
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

GradPlan grad_plan(int64_t Tq, int64_t Tk, int B, int Hq, int Hk, int D, int max_q, int max_k)
{
    GradPlan p;
    p.lg_pack = cross_pack(Hq / Hk);
    const int64_t tok = 128 >> p.lg_pack;
    auto tiles = [&](int64_t T, int64_t rows, int most) {
        const int64_t a = T / rows + B, b = (int64_t)B * ((most + rows - 1) / rows);
        return a < b ? a : b;
    };
    p.max_dq = tiles(Tq, tok, max_q) * (Hq >> p.lg_pack);
    p.max_dkv = tiles(Tk, 128, max_k) * Hk;
    p.off_dq = 256;
    p.off_dkv = up(p.off_dq + sizeof(GradItem) * (size_t)p.max_dq);
    p.off_stats = up(p.off_dkv + sizeof(GradItem) * (size_t)p.max_dkv);
    p.bytes = p.off_stats + sizeof(float2) * (size_t)Tq * Hq;
    return p;
}

// With a window: the same lists, of larger items, and runs of the dk, dv pass's long loops, which are those of the key
// tiles that hold first tokens. A loop is cut where it is longer than an SM's even share of both passes, that is two of
// this one's (cut from one on, two texts of 8192 tokens, 16 heads, window 256 lost 5 % to the join), than a loop without
// first tokens, and than 16 tiles; into runs of one such share (of two, one text of 32768 tokens, 4 heads, window 512
// took 537 instead of 421 us). That comes from what the call holds and not from max_q and max_k, so that results do not
// depend on these.
WinGradPlan window_grad_plan(int64_t Tq, int64_t Tk, int B, int Hq, int Hk, int D, int max_q, int max_k, int window,
                             int sinks)
{
    WinGradPlan p;
    static_cast<GradPlan &>(p) = grad_plan(Tq, Tk, B, Hq, Hk, D, max_q, max_k);
    p.cut_over = p.run_tiles = p.max_cut = p.max_slots = 0;
    if (window > 0 && sinks > 0) {
        const int bn = D == 32 ? GradCfg<32, true>::BN : D == 64 ? GradCfg<64, true>::BN
                       : D == 80 ? GradCfg<80, true>::BN : D == 96 ? GradCfg<96, true>::BN : GradCfg<128, true>::BN;
        const int64_t tok = bn >> p.lg_pack, packs = Hq / Hk >> p.lg_pack;
        auto loop = [&](int64_t queries) { return (queries + tok - 1) / tok * packs; };
        const int64_t some = loop(std::min<int64_t>(Tq, window + 127ll));
        const int64_t firsts = (std::min<int64_t>(sinks, Tk) + 127) / 128;
        const int64_t all = (Tk / 128 + B) * Hk * some + (Tq / tok + B) * packs * Hk * firsts;
        const int64_t share = (all + kDesignSms - 1) / kDesignSms;
        const int64_t over = std::max({2 * share, some, (int64_t)16}), run = std::max({share, some, (int64_t)8});
        if (loop(max_q) > over) {
            // All loops with first tokens are no more than kDesignSms runs: fewer tiles than that have more than a run,
            // and those have fewer than twice as many runs.
            const int64_t tiles = (int64_t)B * Hk * firsts, runs = tiles * ((loop(max_q) + run - 1) / run);
            p.cut_over = (int)over;
            p.run_tiles = (int)run;
            p.max_cut = (int)(tiles < kDesignSms ? tiles : kDesignSms);
            p.max_slots = (int)(runs < 2 * kDesignSms ? runs : 2 * kDesignSms);
        }
    }
    p.off_dkv = up(p.off_dq + sizeof(WinGradItem) * (size_t)p.max_dq);
    p.off_stats = up(p.off_dkv + sizeof(WinGradItem) * (size_t)(p.max_dkv + p.max_slots));
    p.off_cut = up(p.off_stats + sizeof(float2) * (size_t)Tq * Hq);
    p.off_sums = up(p.off_cut + sizeof(WinGradTile) * (size_t)p.max_cut);
    p.bytes = p.off_sums + sizeof(float) * 2 * BM * (size_t)D * (size_t)p.max_slots;
    return p;
}

cudaError_t launch_cross_grad(const CrossGradArgs &a, const GradPlan &p, int num_sms, cudaStream_t stream)
{
    switch (a.f.D) {
        case 32: return launch_d<32, false>(a, p, 0, 0, num_sms, stream);
        case 64: return launch_d<64, false>(a, p, 0, 0, num_sms, stream);
        case 80: return launch_d<80, false>(a, p, 0, 0, num_sms, stream);
        case 96: return launch_d<96, false>(a, p, 0, 0, num_sms, stream);
        case 128: return launch_d<128, false>(a, p, 0, 0, num_sms, stream);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_window_grad(const CrossGradArgs &a, const WinGradPlan &p, int window, int sinks, int num_sms,
                               cudaStream_t stream)
{
    switch (a.f.D) {
        case 32: return launch_d<32, true>(a, p, window, sinks, num_sms, stream);
        case 64: return launch_d<64, true>(a, p, window, sinks, num_sms, stream);
        case 80: return launch_d<80, true>(a, p, window, sinks, num_sms, stream);
        case 96: return launch_d<96, true>(a, p, window, sinks, num_sms, stream);
        case 128: return launch_d<128, true>(a, p, window, sinks, num_sms, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace vit
