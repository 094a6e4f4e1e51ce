// Work list of the tcgen05 kernel in cross attention, and the join of cut key ranges.
//
// One block reads the two offset lists on the device (nothing returns to the host, so a call can be
// captured in a graph): each sequence is checked by itself and left out when it is malformed (all of
// them when the query offsets decrease somewhere); the others are ordered by key count, longest first (an
// item's time goes by its keys, and the persistent kernel takes items in list order), and cut into items:
//   - 256 query rows (two tiles) per item, a last block of at most 128 rows, or every block of a
//     batch too small to occupy half the GPU otherwise, as a split item of one tile; where the list would end
//     in a wave for at most half the SMs, the items of that wave are cut into split items too (4 x 2048
//     queries over 4096 keys, 16 heads of 80: 169 -> 157 us; ragged batches of several waves gain 0 to 3 %);
//   - where the sizes bound the batch to at most half as many 128-row tiles as SMs, split items of
//     one tile and at most `chunk` keys each, whose partial results cross_tile_join adds up.
// A sequence with queries and no keys has no items; its rows go to a list of their own, from which the tcgen05
// kernel's idle warps write the zeros.
// Rows are packed: P query heads that share a key head lie side by side in a tile, so that short
// query sequences under grouped heads fill it and k and v are read once for all P.
//
// It is one block's latency, before the tcgen05 kernel can start: up to 32 sequences are ordered and counted by
// one warp in registers, more by the block; items are written by all threads, each finding its sequence.
#include "block_sort.cuh"
#include "cross.h"
#include "warp_mma.cuh"

namespace vit {
namespace {

constexpr int kThreads = kSortThreads;

__global__ void __launch_bounds__(kThreads)
cross_schedule_kernel(const CrossSegs segs, int Hq, int lg_pack, int chunk, int num_sms, WsHeader *hdr,
                      CrossItem *items, CrossTile *tiles, CrossEmpty *empty, int32_t *status)
{
    extern __shared__ unsigned long long s_key[];      // [NP]: key count descending, then index; later first item | index
    __shared__ int64_t s_warp[32];
    __shared__ int s_bad, s_used, s_total, s_tiles, s_all_split, s_more, s_empty;
    grid_wait();
    grid_release();
    const int tid = threadIdx.x, B = segs.B;
    int NP = 32;
    while (NP < B) NP <<= 1;
    int *s_tile = reinterpret_cast<int *>(s_key + NP); // [NP] first tile
    const int lg_tile = 7 - lg_pack;                   // tokens of a 128-row tile, log2
    const int packs = Hq >> lg_pack;
    // an unusable sequence sorts behind all others
    auto key_of = [&](bool use, const CrossSeg &x, int i) {
        return ((unsigned long long)(use ? 0x7fffffffu - (uint32_t)x.kn : 0xffffffffu) << 32) | (uint32_t)i;
    };
    auto blocks_of = [&](const CrossSeg &x, int lg) { return packs * ((x.qn + (1 << lg) - 1) >> lg); };
    auto runs_of = [&](const CrossSeg &x) { return chunk > 0 ? key_runs(x.kn, chunk) : 1; };
    // two-tile blocks of the batch: few of them means split items throughout
    auto split_all = [&](int64_t full) { return chunk > 0 || 2 * full <= (int64_t)num_sms; };
    if (B <= 32) {
        // a warp: one sequence per lane
        if (tid < 32) {
            CrossSeg x;
            const bool fine = tid < B && load_seg(segs, tid, x, status, true);
            // offsets that decrease somewhere could claim more rows than there are: no items at all then
            const bool bad = tid < B && segs.cu_q[tid + 1] < segs.cu_q[tid];
            const bool use = fine && x.qn > 0 && x.kn > 0, none = fine && x.qn > 0 && x.kn == 0;
            int64_t full = use ? blocks_of(x, lg_tile + 1) : 0;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) full += __shfl_xor_sync(0xffffffffu, full, o);
            const bool all_split = split_all(full);
            const int n = use ? blocks_of(x, all_split ? lg_tile : lg_tile + 1) : 0, runs = use ? runs_of(x) : 1;
            int rank, at, tile_at;
            warp_place(key_of(use, x, tid), n * runs, runs > 1 ? n : 0, rank, at, tile_at);
            s_key[rank] = ((unsigned long long)at << 32) | (uint32_t)tid;
            s_tile[rank] = tile_at;
            const unsigned used = __ballot_sync(0xffffffffu, use), any_bad = __ballot_sync(0xffffffffu, bad);
            const unsigned nones = __ballot_sync(0xffffffffu, none);
            if (none) empty[__popc(nones & ((1u << tid) - 1u))] = CrossEmpty{x.q0, x.qn};
            if (rank == 31) {                          // the last: its sums are all but its own
                s_total = at + n * runs;
                s_tiles = tile_at + (runs > 1 ? n : 0);
                s_used = __popc(used);
                s_empty = __popc(nones);
                s_all_split = all_split;
                s_bad = any_bad != 0;
            }
        }
        __syncthreads();
    } else {
        if (tid == 0) s_bad = s_used = s_empty = 0;
        __syncthreads();
        for (int i = tid; i < NP; i += kThreads) {
            CrossSeg x;
            const bool fine = i < B && load_seg(segs, i, x, status, true);
            if (i < B && segs.cu_q[i + 1] < segs.cu_q[i]) s_bad = 1;
            const bool use = fine && x.qn > 0 && x.kn > 0;
            s_key[i] = key_of(use, x, i);
            if (use) atomicAdd(&s_used, 1);
            if (fine && x.qn > 0 && x.kn == 0) empty[atomicAdd(&s_empty, 1)] = CrossEmpty{x.q0, x.qn};   // (in any order)
        }
        __syncthreads();
        block_sort(s_key, NP, tid);
        const int per = (B + kThreads - 1) / kThreads, lo = min(tid * per, s_used), hi = min(lo + per, s_used);
        auto seg_at = [&](int p) {
            CrossSeg x;
            load_seg(segs, (int)(s_key[p] & 0xffffffffu), x, nullptr, false);
            return x;
        };
        int64_t mine = 0, total_full, n_items = 0, n_tiles = 0, total, total_tiles;
        for (int p = lo; p < hi; ++p) mine += blocks_of(seg_at(p), lg_tile + 1);
        block_exclusive_scan(mine, s_warp, &total_full);
        const bool all_split = split_all(total_full);
        const int lg_block = all_split ? lg_tile : lg_tile + 1;
        for (int p = lo; p < hi; ++p) {
            const CrossSeg x = seg_at(p);
            const int n = blocks_of(x, lg_block), runs = runs_of(x);
            n_items += (int64_t)n * runs;
            if (runs > 1) n_tiles += n;
        }
        int64_t at = block_exclusive_scan(n_items, s_warp, &total);
        int64_t tile_at = block_exclusive_scan(n_tiles, s_warp, &total_tiles);
        for (int p = lo; p < hi; ++p) {
            const CrossSeg x = seg_at(p);
            const int n = blocks_of(x, lg_block), runs = runs_of(x);
            s_key[p] = ((unsigned long long)at << 32) | (uint32_t)(s_key[p] & 0xffffffffu);
            s_tile[p] = (int)tile_at;
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
    const bool bad = s_bad != 0, all_split = s_all_split != 0;
    const int total = bad ? 0 : s_total, lg_block = all_split ? lg_tile : lg_tile + 1;
    // where the items end in a wave that fills at most half the SMs, its items are cut into their tiles
    const int rest = total % num_sms, whole = !all_split && 2 * rest <= num_sms ? total - rest : total;
    if (tid == 0) s_more = 0;
    __syncthreads();
    for (int i = tid; i < total; i += kThreads) {
        const int p = place_of(s_key, s_used, i), n = i - (int)(s_key[p] >> 32);
        CrossSeg x;
        load_seg(segs, (int)(s_key[p] & 0xffffffffu), x, nullptr, false);
        const int nq = (x.qn + (1 << lg_block) - 1) >> lg_block, runs = runs_of(x);
        const int j = n / runs, run = n - j * runs, h = j / nq, qb = j - h * nq;
        CrossItem it;
        it.k0 = x.k0 + run * chunk;
        it.kn = runs > 1 ? min(chunk, x.kn - run * chunk) : x.kn;
        it.q0 = x.q0 + (qb << lg_block);
        it.q1 = x.q0 + x.qn;
        it.head = h << lg_pack;
        it.split = all_split || x.qn - (qb << lg_block) <= (1 << lg_tile);
        it.slot = runs > 1 ? i : -1;
        it.pad = 0;
        if (runs > 1 && run == 0) tiles[s_tile[p] + j] = CrossTile{it.q0, it.q1, it.head, i, runs, {0, 0, 0}};
        if (i < whole) {
            items[i] = it;
        } else {                                       // (in any order: an item's result does not depend on its place)
            const int halves = it.split ? 1 : 2, at = whole + atomicAdd(&s_more, halves);
            it.split = 1;
            items[at] = it;
            it.q0 += 1 << lg_tile;
            if (halves == 2) items[at + 1] = it;
        }
    }
    __syncthreads();
    if (tid == 0) {
        hdr->n_long = whole + s_more;
        hdr->n_joins = bad ? 0 : s_tiles;
        hdr->n_empty = bad ? 0 : s_empty;
        hdr->n_tiny = 0;
        hdr->bm_long = 1 << lg_block;
        hdr->tiny_max = 0;
        hdr->error = bad ? VIT_ERR_BAD_SEQLENS : 0;
        hdr->long_all_split = all_split ? 1 : 0;
        hdr->next_long = 0;
    }
}

// out = sum_s 2^(e_s - E) O_s / sum_s 2^(e_s - E) over a tile's key runs, one warp per row.
template <int D>
__global__ void __launch_bounds__(256)
cross_tile_join_kernel(const WsHeader *hdr, const CrossTile *tiles, const CrossLong cx, __nv_bfloat16 *out,
                       int64_t out_stride, float *lse, int Hq)
{
    grid_wait();
    const int n_tiles = hdr->n_joins, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n_rows = 16;                             // rows per block: a tile is dealt to 8 blocks
    for (int w = blockIdx.x; w < n_tiles * 8; w += gridDim.x) {
        const CrossTile t = tiles[w >> 3];
        for (int r = (w & 7) * n_rows + warp; r < ((w & 7) + 1) * n_rows; r += 8) {
            const int tok = t.q0 + (r >> cx.lg_pack), head = t.head + (r & ((1 << cx.lg_pack) - 1));
            if (tok >= t.q1) break;
            float E = -INFINITY;
            for (int s = lane; s < t.runs; s += 32) E = fmaxf(E, cx.part_s[(int64_t)(t.slot + s) * 128 + r]);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) E = fmaxf(E, __shfl_xor_sync(0xffffffffu, E, d));
            float sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
            const float base = E == -INFINITY ? 0.f : E;
#pragma unroll 4
            for (int s = 0; s < t.runs; ++s) {
                const int64_t row = (int64_t)(t.slot + s) * 128 + r;
                const float x = wmma16::ex2(cx.part_s[row] - base);
                sum += x;
                if (lane < D / 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(cx.part_o + row * D + 4 * lane);
                    acc[0] = fmaf(x, v.x, acc[0]);
                    acc[1] = fmaf(x, v.y, acc[1]);
                    acc[2] = fmaf(x, v.z, acc[2]);
                    acc[3] = fmaf(x, v.w, acc[3]);
                }
            }
            const float inv = 1.f / sum;               // (no weight in any run: 0 / 0)
            if (lane < D / 4)
                *reinterpret_cast<uint2 *>(out + (int64_t)tok * out_stride + (int64_t)head * D + 4 * lane) =
                    make_uint2(wmma16::pack_bf16(acc[0] * inv, acc[1] * inv),
                               wmma16::pack_bf16(acc[2] * inv, acc[3] * inv));
            if (lse && lane == 0) lse[(int64_t)tok * Hq + head] = (E + log2f(sum)) * 0.6931471805599453f;
        }
    }
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

// as many heads side by side as divide the group, up to 8 (a tile keeps 16 tokens at least)
int cross_pack(int group) { return group % 8 == 0 ? 3 : group % 4 == 0 ? 2 : group % 2 == 0 ? 1 : 0; }

LongPlan long_plan(int64_t Tq, int B, int Hq, int Hk, int D, int max_q, int max_k)
{
    LongPlan p;
    const int group = Hq / Hk;
    p.lg_pack = cross_pack(group);
    const int64_t tok = 128 >> p.lg_pack, packs = Hq >> p.lg_pack;
    int64_t tiles = Tq / tok + B;
    const int64_t by_seq = (int64_t)B * ((max_q + tok - 1) / tok);
    if (by_seq < tiles) tiles = by_seq;
    tiles *= packs;
    p.max_items = tiles;
    p.max_tiles = 0;
    p.chunk = 0;
    p.runs = 1;
    // few tiles: cut the keys so that they give about one item per SM, at least 512 keys each (a run
    // writes and re-reads 128 * D fp32 values)
    if (2 * tiles <= kDesignSms) {
        const int64_t want = kDesignSms / tiles;
        int64_t chunk = ((int64_t)max_k + want - 1) / want;
        if (chunk < 512) chunk = 512;
        const int64_t bn2 = 2 * attn_long_bn(D);
        chunk = (chunk + bn2 - 1) / bn2 * bn2;
        const int64_t runs = ((int64_t)max_k + chunk - 1) / chunk;
        if (runs > 1) {
            p.chunk = (int)chunk;
            p.runs = (int)runs;
            p.max_items = tiles * runs;
            p.max_tiles = tiles;
        }
    }
    p.off_items = sizeof(WsHeader);
    p.off_tiles = up(p.off_items + sizeof(CrossItem) * (size_t)p.max_items);
    p.off_empty = up(p.off_tiles + sizeof(CrossTile) * (size_t)p.max_tiles);
    p.off_part_s = up(p.off_empty + sizeof(CrossEmpty) * (size_t)B);
    const size_t slots = p.runs > 1 ? (size_t)p.max_items : 0;
    p.off_part_o = up(p.off_part_s + slots * 128 * sizeof(float));
    p.bytes = p.off_part_o + slots * 128 * (size_t)D * sizeof(float);
    return p;
}

cudaError_t launch_cross_schedule(const CrossArgs &a, const LongPlan &p, int num_sms, WsHeader *hdr, CrossItem *items,
                                  CrossTile *tiles, CrossEmpty *empty, cudaStream_t stream)
{
    int np = 32;
    while (np < a.segs.B) np <<= 1;
    constexpr size_t each = sizeof(unsigned long long) + sizeof(int);
    static DeviceOnce once;
    cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(cross_schedule_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)each * VIT_MAX_SEGMENTS);
    });
    if (e != cudaSuccess) return e;
    LaunchScope scope("cross_schedule", stream);
    return launch_chained(cross_schedule_kernel, 1, kThreads, each * np, stream, a.segs, a.Hq, p.lg_pack, p.chunk,
                          num_sms, hdr, items, tiles, empty, a.status);
}

cudaError_t launch_cross_tile_join(const CrossArgs &a, const LongPlan &p, const CrossLong &cx, const WsHeader *hdr,
                                   const CrossTile *tiles, cudaStream_t stream)
{
    const unsigned blocks = (unsigned)(p.max_tiles * 8);
    LaunchScope scope("cross_tile_join", stream);
    auto run = [&](auto kern) {
        return launch_chained(kern, blocks, 256, 0, stream, hdr, tiles, cx, static_cast<__nv_bfloat16 *>(a.out),
                              a.out_stride, a.lse, a.Hq);
    };
    switch (a.D) {
        case 32: return run(cross_tile_join_kernel<32>);
        case 64: return run(cross_tile_join_kernel<64>);
        case 80: return run(cross_tile_join_kernel<80>);
        case 96: return run(cross_tile_join_kernel<96>);
        case 128: return run(cross_tile_join_kernel<128>);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace vit
