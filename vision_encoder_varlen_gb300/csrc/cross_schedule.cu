// Work list of the tcgen05 kernel in cross attention, and the join of cut key ranges.
//
// One block reads the two offset lists on the device (nothing returns to the host, so a call can be
// captured in a graph): each sequence is checked by itself and left out when it is malformed (all of
// them when the query offsets decrease somewhere); the others are ordered by key count, longest first (an item's time goes by its keys, and the
// persistent kernel takes items in list order), and cut into items:
//   - 256 query rows (two tiles) per item, a last block of at most 128 rows, or every block of a
//     batch too small to occupy half the GPU otherwise, as a split item of one tile;
//   - where the sizes bound the batch to at most half as many 128-row tiles as SMs, split items of
//     one tile and at most `chunk` keys each, whose partial results cross_tile_join adds up.
// Rows are packed: P query heads that share a key head lie side by side in a tile, so that short
// query sequences under grouped heads fill it and k and v are read once for all P.
#include "block_sort.cuh"
#include "cross.h"
#include "warp_mma.cuh"

namespace vit {
namespace {

constexpr int kThreads = kSortThreads;

__global__ void __launch_bounds__(kThreads)
cross_schedule_kernel(const CrossSegs segs, int Hq, int lg_pack, int chunk, int num_sms, WsHeader *hdr,
                      CrossItem *items, CrossTile *tiles, int32_t *status)
{
    extern __shared__ unsigned long long s_key[];      // [NP]: key count descending, then index
    __shared__ int64_t s_warp[32];
    __shared__ int s_bad;
    grid_release();
    const int tid = threadIdx.x, B = segs.B;
    int NP = 1;
    while (NP < B) NP <<= 1;
    if (tid == 0) s_bad = 0;
    __syncthreads();
    for (int i = tid; i < NP; i += kThreads) {
        CrossSeg x;
        const bool fine = i < B && load_seg(segs, i, x, status, true);
        // offsets that decrease somewhere could claim more rows than there are: no items at all then
        if (i < B && segs.cu_q[i + 1] < segs.cu_q[i]) s_bad = 1;
        const bool use = fine && x.qn > 0 && x.kn > 0;
        s_key[i] = use ? ((unsigned long long)(0x7fffffffu - (uint32_t)x.kn) << 32) | (uint32_t)i : ~0ull;
    }
    __syncthreads();
    if (s_bad) {
        if (tid == 0) {
            hdr->n_long = hdr->reserved = hdr->n_tiny = hdr->next_long = 0;
            hdr->error = VIT_ERR_BAD_SEQLENS;
        }
        return;
    }
    block_sort(s_key, NP, tid);

    const int lg_tile = 7 - lg_pack;                   // tokens of a 128-row tile, log2
    const int packs = Hq >> lg_pack;
    const int per = (B + kThreads - 1) / kThreads, lo = min(tid * per, B), hi = min(lo + per, B);
    auto seg_at = [&](int p, CrossSeg &x) -> bool {
        if (s_key[p] == ~0ull) return false;
        load_seg(segs, (int)(s_key[p] & 0xffffffffu), x, nullptr, false);
        return true;
    };
    // two-tile blocks of the batch: few of them means split items throughout
    int64_t mine = 0, total_full;
    for (int p = lo; p < hi; ++p) {
        CrossSeg x;
        if (seg_at(p, x)) mine += (int64_t)packs * ((x.qn + (2 << lg_tile) - 1) >> (lg_tile + 1));
    }
    block_exclusive_scan(mine, s_warp, &total_full);
    const bool all_split = chunk > 0 || 2 * total_full <= (int64_t)num_sms;
    const int lg_block = all_split ? lg_tile : lg_tile + 1;
    int64_t n_items = 0, n_tiles = 0, total, total_tiles;
    for (int p = lo; p < hi; ++p) {
        CrossSeg x;
        if (!seg_at(p, x)) continue;
        const int64_t n = (int64_t)packs * ((x.qn + (1 << lg_block) - 1) >> lg_block);
        const int runs = chunk > 0 ? key_runs(x.kn, chunk) : 1;
        n_items += n * runs;
        if (runs > 1) n_tiles += n;
    }
    int64_t at = block_exclusive_scan(n_items, s_warp, &total);
    int64_t tile_at = block_exclusive_scan(n_tiles, s_warp, &total_tiles);
    // a sequence's items by the thread that holds it when they are few, else by all threads in turn
    for (int p = lo; p < hi; ++p) {
        CrossSeg x;
        if (!seg_at(p, x)) continue;
        const int nq = (x.qn + (1 << lg_block) - 1) >> lg_block;
        const int runs = chunk > 0 ? key_runs(x.kn, chunk) : 1;
        s_key[p] = ((unsigned long long)at << 32) | (uint32_t)(s_key[p] & 0xffffffffu);   // first item | sequence
        if (runs > 1) {
            for (int i = 0; i < packs * nq; ++i) {
                const int h = i / nq, qb = i - h * nq;
                tiles[tile_at + i] = CrossTile{x.q0 + (qb << lg_block), x.q0 + x.qn, h << lg_pack,
                                               (int)(at + (int64_t)i * runs), runs, {0, 0, 0}};
            }
            tile_at += (int64_t)packs * nq;
        }
        at += (int64_t)packs * nq * runs;
    }
    __syncthreads();
    const int lane = tid & 31, warp = tid >> 5;
    for (int p = warp; p < B; p += kThreads / 32) {
        if (s_key[p] == ~0ull) break;                  // the unused sequences are last
        CrossSeg x;
        load_seg(segs, (int)(s_key[p] & 0xffffffffu), x, nullptr, false);
        const int first = (int)(s_key[p] >> 32);
        const int nq = (x.qn + (1 << lg_block) - 1) >> lg_block;
        const int runs = chunk > 0 ? key_runs(x.kn, chunk) : 1;
        const int n = packs * nq * runs;
        for (int i = lane; i < n; i += 32) {
            const int run = i % runs, j = i / runs, h = j / nq, qb = j - h * nq;
            const int q0 = x.q0 + (qb << lg_block), left = x.qn - (qb << lg_block);
            CrossItem it;
            it.k0 = x.k0 + run * chunk;
            it.kn = runs > 1 ? min(chunk, x.kn - run * chunk) : x.kn;
            it.q0 = q0;
            it.q1 = x.q0 + x.qn;
            it.head = h << lg_pack;
            it.split = all_split || left <= (1 << lg_tile);
            it.slot = runs > 1 ? first + i : -1;
            it.pad = 0;
            items[first + i] = it;
        }
    }
    if (tid == 0) {
        hdr->n_long = (int32_t)total;
        hdr->reserved = (int32_t)total_tiles;
        hdr->n_tiny = 0;
        hdr->bm_long = 1 << lg_block;
        hdr->tiny_max = 0;
        hdr->error = 0;
        hdr->long_all_split = all_split ? 1 : 0;
        hdr->next_long = 0;
    }
}

// out = sum_s 2^(e_s - E) O_s / sum_s 2^(e_s - E) over a tile's key runs, one warp per row.
template <int D>
__global__ void __launch_bounds__(256)
cross_tile_join_kernel(const WsHeader *__restrict__ hdr, const CrossTile *__restrict__ tiles, const CrossLong cx,
                       __nv_bfloat16 *__restrict__ out, int64_t out_stride, float *__restrict__ lse, int Hq)
{
    grid_wait();
    const int n_tiles = hdr->reserved, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
#pragma unroll 4
            for (int s = 0; s < t.runs; ++s) {
                const int64_t row = (int64_t)(t.slot + s) * 128 + r;
                const float x = wmma16::ex2(cx.part_s[row] - E);
                sum += x;
                if (lane < D / 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(cx.part_o + row * D + 4 * lane);
                    acc[0] = fmaf(x, v.x, acc[0]);
                    acc[1] = fmaf(x, v.y, acc[1]);
                    acc[2] = fmaf(x, v.z, acc[2]);
                    acc[3] = fmaf(x, v.w, acc[3]);
                }
            }
            const float inv = 1.f / sum;
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
    p.off_part_s = up(p.off_tiles + sizeof(CrossTile) * (size_t)p.max_tiles);
    const size_t slots = p.runs > 1 ? (size_t)p.max_items : 0;
    p.off_part_o = up(p.off_part_s + slots * 128 * sizeof(float));
    p.bytes = p.off_part_o + slots * 128 * (size_t)D * sizeof(float);
    return p;
}

cudaError_t launch_cross_schedule(const CrossArgs &a, const LongPlan &p, int num_sms, WsHeader *hdr, CrossItem *items,
                                  CrossTile *tiles, cudaStream_t stream)
{
    int np = 1;
    while (np < a.segs.B) np <<= 1;
    static DeviceOnce once;
    cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(cross_schedule_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)sizeof(unsigned long long) * VIT_MAX_SEGMENTS);
    });
    if (e != cudaSuccess) return e;
    LaunchScope scope("cross_schedule", stream);
    cross_schedule_kernel<<<1, kThreads, sizeof(unsigned long long) * (size_t)np, stream>>>(
        a.segs, a.Hq, p.lg_pack, p.chunk, num_sms, hdr, items, tiles, a.status);
    return cudaGetLastError();
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
