// Cross attention with few query rows: single new tokens, short continuations, small sets of latent
// queries (at most 32 rows of max_q * (Hq / Hk) that share one key head).
//
//   o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  s_j = scale q k_j,  m = max_j s_j,
// over one sequence's keys. With so few rows the cost is reading k and v once (4 D bytes per key and
// key head against 4 D rows flops), so the work is laid out for loads: a block takes one (sequence,
// key head, run of `chunk` keys), all query rows of the group at once so that k and v are read only
// once, and a producer warp keeps whole 64-key tiles in flight (TMA into a ring of three slots; two or
// more blocks share an SM). The keys of a sequence are split over blocks so that a few long sequences
// still fill the GPU; each block leaves (m, l, O) of its run and a second
// kernel joins a row's runs in order (results do not depend on timing). With one run per sequence the
// block writes the result itself.
//
// HBM bound. Measured: 48 single tokens of 32 heads over 8 of 128, up to 8191 states each (326 MB), 62 us
// with the join (5.3 TB/s; the kernel alone 58 us, 5.7 TB/s, the rate of a copy of that size); three single
// tokens over 1601 states 17.5 us in a graph, of which the two launches are most.
//
// Inside a block a warp takes one 16-row tile and a group of 16 keys of every 64-key tile: S = Q K^T and
// O += P V by m16n8k16 MMAs (the rows are far too few for 128-row tcgen05 tiles to pay: the tensor pipe is
// idle either way), softmax statistics in fp32 registers, P rounded to bf16 as in
// the other attention kernels, O rescaled only when a row's maximum grows by more than 2^8. The key
// groups are joined through shared memory at the end.
//
// Keys past the run's end score -inf, and their V rows are zeroed in shared memory before use: what
// lies there (the next sequence, padding, Inf or NaN) enters nothing.
#include "cross.h"
#include "sm100.cuh"
#include "warp_mma.cuh"

namespace vit {
namespace {

constexpr int kTile = 64;                     // keys per ring slot
constexpr int kStages = 3;                    // 96 KB at head_dim 128: two blocks of an SM keep 192 KB in flight
constexpr long long kWaitBudget = 4000000000ll;

// A tile of `kTile` rows of D columns as TMA leaves it: 64-column slabs with 128-byte swizzle, then one
// slab of the remaining 16 or 32 columns with 32- or 64-byte swizzle.
template <int D> struct Tile {
    static constexpr int N128 = D / 64, REM = D % 64;
    static constexpr int BYTES = kTile * D * 2;
    // byte offset of the 16-byte chunk c of row r
    __device__ static __forceinline__ uint32_t at(int r, int c) {
        if (REM == 0 || c < 8 * N128) return (c >> 3) * (kTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
        const int rc = c - 8 * N128;
        if constexpr (REM == 32) return N128 * kTile * 128 + r * 64 + ((rc ^ ((r >> 1) & 3)) << 4);
        return N128 * kTile * 128 + r * 32 + ((rc ^ ((r >> 2) & 1)) << 4);
    }
};

struct Few {
    __nv_bfloat16 *out;
    const __nv_bfloat16 *q;
    float *lse;
    int Hq, Hk, group;
    int64_t q_stride, out_stride;
    float scale_log2;
    CrossSegs segs;
    int32_t *status;
    int chunk, n_split, rows;                 // rows: max_q * group, the partial rows of a split
    float *part_o, *part_s;                   // [B][Hk][n_split][rows][D] and [..][rows] (log2 of the run's sum)
};

// Warps of a block: MT row tiles x 4 key groups.
constexpr int kGroups = 4;
template <int MT> constexpr int kMmaWarps = MT * kGroups;

template <int D, int MT>
__global__ void __launch_bounds__(32 * kMmaWarps<MT> + 32)
cross_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_kr,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_vr, const Few p)
{
    using T = Tile<D>;
    constexpr int NK = D / 16, KQ = kGroups, NW = kMmaWarps<MT>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *ring = reinterpret_cast<unsigned char *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t s_full[kStages], s_empty[kStages];
    __shared__ volatile int s_abort;
    __shared__ float s_m[NW][16], s_l[NW][16];

    grid_wait();
    grid_release();                                           // the join may take its place already
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = blockIdx.z, hk = blockIdx.x, b = blockIdx.y;   // later runs last: ragged lengths leave them empty
    CrossSeg seg;
    // a sequence without keys is left to the join, or to split 0 where there is none
    if (!load_seg(p.segs, b, seg, p.status, threadIdx.x == 0 && split == 0 && hk == 0)) return;
    if (seg.qn == 0) return;
    const int first = split * p.chunk;
    const bool only = p.n_split == 1;
    if (first >= seg.kn && !(only && seg.kn == 0)) return;
    const int n_keys = min(p.chunk, seg.kn - first);          // of this run
    const int n_tiles = (n_keys + kTile - 1) / kTile;
    const int n_rows = seg.qn * p.group;

    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int i = 0; i < kStages; ++i) {
            sm100::mbar_init(sm100::smem_addr(&s_full[i]), 1);
            sm100::mbar_init(sm100::smem_addr(&s_empty[i]), NW);
        }
        sm100::fence_mbar_init();
    }
    __syncthreads();
    auto wait = [&](uint64_t &bar, uint32_t parity) {
        if (sm100::mbar_wait(sm100::smem_addr(&bar), parity, (const volatile int *)&s_abort, kWaitBudget)) return true;
        if (!s_abort) {
            s_abort = 1;
            report_error(p.status, VIT_ERR_TIMEOUT);
        }
        return false;
    };

    float o[NK * 2][4];                                       // 16 rows x D, as D / 8 accumulator tiles
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};   // rows lane / 4 and lane / 4 + 8
    bool ok = true;
    const int row_tile = warp / KQ, quarter = warp % KQ;
    if (warp == NW) {
        // ---- producer
        if (lane == 0) {
            int i = 0;
            for (; i < n_tiles; ++i) {
                const int s = i % kStages;
                if (i >= kStages && !wait(s_empty[s], (i / kStages - 1) & 1)) break;
                const uint32_t bar = sm100::smem_addr(&s_full[s]), dst = sm100::smem_addr(ring) + s * 2 * T::BYTES;
                const int row = seg.k0 + first + i * kTile;
                sm100::mbar_arrive_expect_tx(bar, 2 * T::BYTES);
#pragma unroll
                for (int x = 0; x < T::N128; ++x) {
                    sm100::tma_load_2d(dst + x * kTile * 128, &tm_k, hk * D + 64 * x, row, bar);
                    sm100::tma_load_2d(dst + T::BYTES + x * kTile * 128, &tm_v, hk * D + 64 * x, row, bar);
                }
                if constexpr (T::REM > 0) {
                    sm100::tma_load_2d(dst + T::N128 * kTile * 128, &tm_kr, hk * D + 64 * T::N128, row, bar);
                    sm100::tma_load_2d(dst + T::BYTES + T::N128 * kTile * 128, &tm_vr, hk * D + 64 * T::N128, row, bar);
                }
            }
            // after a wait that gave up: let what was issued land before the shared memory goes
            if (i < n_tiles) {
                const int never = 0;
                for (int k = i > kStages ? i - kStages : 0; k < i; ++k)
                    sm100::mbar_wait(sm100::smem_addr(&s_full[k % kStages]), (k / kStages) & 1, &never, 20000000ll);
            }
        }
    } else {
        // ---- 16 query rows against 16 keys of every tile
        const int g = lane >> 2, c = lane & 3;
        uint32_t qa[NK][4];
        const int r0 = row_tile * 16 + g, r1 = r0 + 8;       // row r: token r / group, head hk * group + r % group
        auto q_row = [&](int r) {
            return p.q + (int64_t)(seg.q0 + r / p.group) * p.q_stride + (int64_t)(hk * p.group + r % p.group) * D + 2 * c;
        };
        const __nv_bfloat16 *qa_p = r0 < n_rows ? q_row(r0) : nullptr, *qb_p = r1 < n_rows ? q_row(r1) : nullptr;
#pragma unroll
        for (int kk = 0; kk < NK; ++kk) {
            qa[kk][0] = qa_p ? *reinterpret_cast<const uint32_t *>(qa_p + 16 * kk) : 0u;
            qa[kk][1] = qb_p ? *reinterpret_cast<const uint32_t *>(qb_p + 16 * kk) : 0u;
            qa[kk][2] = qa_p ? *reinterpret_cast<const uint32_t *>(qa_p + 16 * kk + 8) : 0u;
            qa[kk][3] = qb_p ? *reinterpret_cast<const uint32_t *>(qb_p + 16 * kk + 8) : 0u;
        }
#pragma unroll
        for (int j = 0; j < 2 * NK; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.f;

        for (int i = 0; i < n_tiles; ++i) {
            const int s = i % kStages;
            ok = __all_sync(0xffffffffu, wait(s_full[s], (i / kStages) & 1));
            if (!ok) break;
            unsigned char *kt = ring + s * 2 * T::BYTES, *vt = kt + T::BYTES;
            const int key0 = 16 * quarter;
            const int live = n_keys - i * kTile - key0;       // of this warp's 16 keys
            if (live > 0) {
                const uint32_t ka = sm100::smem_addr(kt), va = sm100::smem_addr(vt);
                float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                // ldmatrix: lane l gives the row address of matrix l / 8: keys (l & 7) + 8 (l / 16), chunk (l / 8) & 1
                const int kr = key0 + (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;
#pragma unroll
                for (int kk = 0; kk < NK; ++kk) {
                    uint32_t b0, b1, b2, b3;
                    wmma16::ldsm_x4(ka + T::at(kr, 2 * kk + kc), b0, b1, b2, b3);
                    wmma16::mma16816(sc[0], qa[kk], b0, b1);
                    wmma16::mma16816(sc[1], qa[kk], b2, b3);
                }
                if (live < 16) {
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (8 * n + 2 * c + (e & 1) >= live) sc[n][e] = -INFINITY;
                    // V rows past the end: zero them (this warp alone reads its 16 keys)
                    for (int x = lane; x < (16 - live) * (D / 8); x += 32)
                        *reinterpret_cast<uint4 *>(vt + T::at(key0 + live + x / (D / 8), x % (D / 8))) =
                            make_uint4(0u, 0u, 0u, 0u);
                    __syncwarp();
                }
                float pr[2][4];
                bool grew = false;
                float alpha[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {                 // rows g and g + 8
                    float mx = fmaxf(fmaxf(sc[0][2 * h], sc[0][2 * h + 1]), fmaxf(sc[1][2 * h], sc[1][2 * h + 1]));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    mx *= p.scale_log2;
                    alpha[h] = 1.f;
                    if (mx > m_run[h] + 8.f) {
                        alpha[h] = wmma16::ex2(m_run[h] - mx);
                        m_run[h] = mx;
                        grew = true;
                    }
                    float sum = 0.f;
                    const float base = m_run[h] == -INFINITY ? 0.f : m_run[h];   // scores of -inf: weight 0
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float v = wmma16::ex2(fmaf(sc[n][2 * h + e], p.scale_log2, -base));
                            pr[n][2 * h + e] = v;
                            sum += v;
                        }
                    l_run[h] = l_run[h] * alpha[h] + sum;     // per lane: joined over the quad at the end
                }
                if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                    for (int j = 0; j < 2 * NK; ++j) {
                        o[j][0] *= alpha[0];
                        o[j][1] *= alpha[0];
                        o[j][2] *= alpha[1];
                        o[j][3] *= alpha[1];
                    }
                }
                const uint32_t pa[4] = {wmma16::pack_bf16(pr[0][0], pr[0][1]), wmma16::pack_bf16(pr[0][2], pr[0][3]),
                                        wmma16::pack_bf16(pr[1][0], pr[1][1]), wmma16::pack_bf16(pr[1][2], pr[1][3])};
                // transposed: matrices (keys 0-7, chunk 2j), (keys 8-15, 2j), (keys 0-7, 2j + 1), (keys 8-15, 2j + 1)
                const int vr = key0 + (lane & 15), vc = lane >> 4;
#pragma unroll
                for (int j = 0; j < NK; ++j) {
                    uint32_t b0, b1, b2, b3;
                    wmma16::ldsm_x4_t(va + T::at(vr, 2 * j + vc), b0, b1, b2, b3);
                    wmma16::mma16816(o[2 * j], pa, b0, b1);
                    wmma16::mma16816(o[2 * j + 1], pa, b2, b3);
                }
            }
            __syncwarp();
            if (lane == 0) sm100::mbar_arrive(sm100::smem_addr(&s_empty[s]));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l_run[h] += __shfl_xor_sync(0xffffffffu, l_run[h], 1);
            l_run[h] += __shfl_xor_sync(0xffffffffu, l_run[h], 2);
            if (c == 0) {
                s_m[warp][g + 8 * h] = m_run[h];
                s_l[warp][g + 8 * h] = l_run[h];
            }
        }
    }
    if (!__syncthreads_and(ok && !s_abort)) return;           // the ring is free from here on
    // ---- join the key groups of each row tile: weights first, then O by halving
    float *acc = reinterpret_cast<float *>(ring);             // [row tile][2][16][D]
    float M[2], L[2];
    const int g = lane >> 2, c = lane & 3;
    if (warp < NW) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int w0 = KQ * row_tile, r = g + 8 * h;
            M[h] = s_m[w0][r];
#pragma unroll
            for (int x = 1; x < KQ; ++x) M[h] = fmaxf(M[h], s_m[w0 + x][r]);
            L[h] = 0.f;
            // a group without keys, or whose scores are all -inf, has m = -inf and l = 0: weight 0
            const float base = M[h] == -INFINITY ? 0.f : M[h];
#pragma unroll
            for (int x = 0; x < KQ; ++x) L[h] += s_l[w0 + x][r] * wmma16::ex2(s_m[w0 + x][r] - base);
            const float f = wmma16::ex2(m_run[h] - base);
#pragma unroll
            for (int j = 0; j < 2 * NK; ++j) {
                o[j][2 * h] *= f;
                o[j][2 * h + 1] *= f;
            }
        }
    }
    auto place = [&](int j, int h, int half) {
        return acc + ((row_tile * 2 + half) * 16 + g + 8 * h) * D + 8 * j + 2 * c;
    };
#pragma unroll
    for (int n = KQ / 2; n > 0; n /= 2) {                     // groups 2, 3 into 0, 1; then 1 into 0
        const int give = n;
        if (warp < NW && quarter >= give && quarter < give + n)
#pragma unroll
            for (int j = 0; j < 2 * NK; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<float2 *>(place(j, h, quarter - give)) = make_float2(o[j][2 * h], o[j][2 * h + 1]);
        __syncthreads();
        if (warp < NW && quarter < n)
#pragma unroll
            for (int j = 0; j < 2 * NK; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float2 v = *reinterpret_cast<const float2 *>(place(j, h, quarter));
                    o[j][2 * h] += v.x;
                    o[j][2 * h + 1] += v.y;
                }
        __syncthreads();
    }
    if (warp >= NW || quarter != 0) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = row_tile * 16 + g + 8 * h;
        if (r >= n_rows) continue;
        if (only) {
            const int64_t tok = seg.q0 + r / p.group;
            const int head = hk * p.group + r % p.group;
            const float inv = seg.kn > 0 ? 1.f / L[h] : 0.f;  // no key at all: 0, and lse = -inf
            __nv_bfloat16 *dst = p.out + tok * p.out_stride + (int64_t)head * D + 2 * c;
#pragma unroll
            for (int j = 0; j < 2 * NK; ++j)
                *reinterpret_cast<uint32_t *>(dst + 8 * j) = wmma16::pack_bf16(o[j][2 * h] * inv, o[j][2 * h + 1] * inv);
            if (p.lse && c == 0) p.lse[tok * p.Hq + head] = (M[h] + log2f(L[h])) * 0.6931471805599453f;
        } else {
            const int64_t row = (((int64_t)b * p.Hk + hk) * p.n_split + split) * p.rows + r;
            float *dst = p.part_o + row * D + 2 * c;
            const float inv = L[h] == 0.f ? 0.f : 1.f / L[h];   // every score -inf: a run of weight 0
#pragma unroll
            for (int j = 0; j < 2 * NK; ++j)
                *reinterpret_cast<float2 *>(dst + 8 * j) = make_float2(o[j][2 * h] * inv, o[j][2 * h + 1] * inv);
            if (c == 0) p.part_s[row] = M[h] + log2f(L[h]);
        }
    }
}

// out = sum_s 2^(e_s - E) O_s / sum_s 2^(e_s - E), e_s the log2 of run s's sum: a row by one warp, or
// (WIDE, many runs) by the eight warps of a block, each every eighth run, added up in warp order.
template <int D, bool WIDE>
__global__ void __launch_bounds__(256)
cross_join_kernel(const Few p)
{
    __shared__ float s_acc[WIDE ? 8 : 1][WIDE ? D : 1], s_sum[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.y;
    CrossSeg seg;
    grid_wait();                                              // the runs' results
    if (!load_seg(p.segs, b, seg, nullptr, false)) return;
    const int n_rows = seg.qn * p.Hq;                         // (token, head) rows of the sequence
    const int runs = key_runs(seg.kn, p.chunk);
    const int x = WIDE ? (int)blockIdx.x : (int)blockIdx.x * 8 + warp;
    if (x >= n_rows) return;
    const int tok = x / p.Hq, head = x - tok * p.Hq, hk = head / p.group;
    const int r = tok * p.group + head - hk * p.group;
    const int64_t row0 = ((int64_t)b * p.Hk + hk) * p.n_split * p.rows + r;
    float E = -INFINITY;
    for (int s = lane; s < runs; s += 32) E = fmaxf(E, p.part_s[row0 + (int64_t)s * p.rows]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) E = fmaxf(E, __shfl_xor_sync(0xffffffffu, E, d));
    const float base = E == -INFINITY ? 0.f : E;
    const float first = E == -INFINITY && runs > 0 ? NAN : 0.f;   // keys, but no weight: 0 / 0; no keys: 0
    float sum = 0.f, acc[4] = {first, first, first, first};
    const bool col = lane < D / 4;
#pragma unroll 4
    for (int s = WIDE ? warp : 0; s < runs; s += WIDE ? 8 : 1) {
        const int64_t row = row0 + (int64_t)s * p.rows;
        const float w = wmma16::ex2(p.part_s[row] - base);
        sum += w;
        if (col) {
            const float4 v = *reinterpret_cast<const float4 *>(p.part_o + row * D + 4 * lane);
            acc[0] = fmaf(w, v.x, acc[0]);
            acc[1] = fmaf(w, v.y, acc[1]);
            acc[2] = fmaf(w, v.z, acc[2]);
            acc[3] = fmaf(w, v.w, acc[3]);
        }
    }
    if constexpr (WIDE) {
        if (col) *reinterpret_cast<float4 *>(&s_acc[warp][4 * lane]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        if (lane == 0) s_sum[warp] = sum;
        __syncthreads();
        if (warp > 0) return;
        for (int w = 1; w < 8; ++w) {
            sum += s_sum[w];
            if (col)
                for (int e = 0; e < 4; ++e) acc[e] += s_acc[w][4 * lane + e];
        }
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    const int64_t t = seg.q0 + tok;
    if (col)
        *reinterpret_cast<uint2 *>(p.out + t * p.out_stride + (int64_t)head * D + 4 * lane) =
            make_uint2(wmma16::pack_bf16(acc[0] * inv, acc[1] * inv), wmma16::pack_bf16(acc[2] * inv, acc[3] * inv));
    if (p.lse && lane == 0) p.lse[t * p.Hq + head] = (E + log2f(sum)) * 0.6931471805599453f;
}

bool kv_map(CUtensorMap *m, const void *ptr, int64_t T, int H, int D, int64_t stride, int cols)
{
    const uint64_t dims[2] = {(uint64_t)H * D, (uint64_t)(T > 0 ? T : 1)};
    const uint64_t strides[1] = {(uint64_t)stride * 2};
    const uint32_t box[2] = {(uint32_t)cols, (uint32_t)kTile};
    return encode_tiled_map(m, ptr, 2, dims, strides, box, cols * 2);
}

template <int D, int MT>
cudaError_t launch_mt(const CrossArgs &a, const FewPlan &pl, const Few &p, cudaStream_t stream)
{
    constexpr int rem = Tile<D>::REM > 0 ? Tile<D>::REM : 64, wide = D >= 64 ? 64 : rem;
    CUtensorMap mk, mkr, mv, mvr;
    const CrossSegs &s = a.segs;
    if (!kv_map(&mk, a.k, s.Tk, a.Hk, D, a.k_stride, wide) || !kv_map(&mv, a.v, s.Tk, a.Hk, D, a.v_stride, wide))
        return cudaErrorInvalidValue;
    mkr = mk;
    mvr = mv;
    if (rem != wide &&
        (!kv_map(&mkr, a.k, s.Tk, a.Hk, D, a.k_stride, rem) || !kv_map(&mvr, a.v, s.Tk, a.Hk, D, a.v_stride, rem)))
        return cudaErrorInvalidValue;
    constexpr int smem = kStages * 2 * Tile<D>::BYTES + 1024;
    static_assert(kStages * 2 * Tile<D>::BYTES >= 2 * MT * 16 * D * 4, "the joins reuse the ring");
    auto kern = cross_few_kernel<D, MT>;
    static DeviceOnce once;
    cudaError_t e = once.run([&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
    if (e != cudaSuccess) return e;
    {
        LaunchScope scope("cross_few", stream);
        e = launch_chained(kern, dim3(a.Hk, s.B, pl.n_split), 32 * kMmaWarps<MT> + 32, smem, stream, mk, mkr, mv, mvr, p);
    }
    if (e != cudaSuccess || pl.n_split == 1) return e;
    LaunchScope scope("cross_join", stream);
    const int rows = s.max_q * a.Hq;
    // with more than 16 runs a warp per row is too few loads in flight (147 runs: 37 us)
    return pl.n_split > 16 ? launch_chained(cross_join_kernel<D, true>, dim3(rows, s.B), 256, 0, stream, p)
                           : launch_chained(cross_join_kernel<D, false>, dim3((rows + 7) / 8, s.B), 256, 0, stream, p);
}

template <int D> cudaError_t launch_d(const CrossArgs &a, const FewPlan &pl, cudaStream_t stream)
{
    Few p;
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.q = static_cast<const __nv_bfloat16 *>(a.q);
    p.lse = a.lse;
    p.Hq = a.Hq;
    p.Hk = a.Hk;
    p.group = a.Hq / a.Hk;
    p.q_stride = a.q_stride;
    p.out_stride = a.out_stride;
    p.scale_log2 = a.scale_log2;
    p.segs = a.segs;
    p.status = a.status;
    p.chunk = pl.chunk;
    p.n_split = pl.n_split;
    p.rows = pl.rows;
    const size_t n = (size_t)a.segs.B * a.Hk * pl.n_split * pl.rows;
    p.part_o = static_cast<float *>(a.workspace);
    p.part_s = p.part_o + n * D;
    switch (pl.row_tiles) {
        case 1: return launch_mt<D, 1>(a, pl, p, stream);
        default: return launch_mt<D, 2>(a, pl, p, stream);
    }
}

}  // namespace

// Keys per split: enough blocks to fill the GPU about eight times over where the sequences are long
// enough (ragged lengths then even out; 4, 16 and 32 times were slower on 48 single tokens over up to
// 8191 keys: 72, 64, 68 against 62 us), but at least 128 keys (two tiles) and, since a split leaves
// rows * D fp32 values that are written and read again, at least 16 keys per row (at most 1/8 of the
// traffic). Runs of equal length, in whole tiles.
FewPlan few_plan(int B, int Hq, int Hk, int D, int max_q, int max_k)
{
    FewPlan p;
    p.rows = max_q * (Hq / Hk);
    p.row_tiles = p.rows <= 16 ? 1 : 2;
    const int64_t pairs = (int64_t)B * Hk, want = kDesignSms * 8;
    const int64_t least = 16 * p.rows > 128 ? 16 * p.rows : 128;
    int64_t n = (want + pairs / 2) / pairs;
    const int64_t most = ((int64_t)max_k + least - 1) / least;
    if (n > most) n = most;
    if (n < 1) n = 1;
    int64_t chunk = ((int64_t)max_k + n - 1) / n;
    chunk = (chunk + kTile - 1) / kTile * kTile;
    if (chunk < kTile) chunk = kTile;
    n = max_k > 0 ? ((int64_t)max_k + chunk - 1) / chunk : 1;
    p.chunk = (int)chunk;
    p.n_split = (int)n;
    p.partial_bytes = n > 1 ? sizeof(float) * (size_t)pairs * n * p.rows * (D + 1) : 0;
    return p;
}

// Few rows take this kernel. Up to 16 rows always; up to 32 where all the keys are at most 32 MiB, and
// launches dominate (8 rows x 4 heads over 4096 keys of 8 heads of 128: 22 us here, 28 us by the tcgen05
// kernel; over 8 such sequences 61 and 53 us, over 32 of 16 heads of 80 118 and 92 us; with four row
// tiles, 64 rows over 16 sequences of 256 to 4097 keys, 87 and 58 us).
bool takes_few(int B, int Hq, int Hk, int D, int max_q, int max_k)
{
    const int64_t rows = (int64_t)max_q * (Hq / Hk);
    return rows <= 16 || (rows <= 32 && (int64_t)B * max_k * Hk * D * 4 <= ((int64_t)32 << 20));
}

cudaError_t launch_cross_few(const CrossArgs &a, const FewPlan &p, cudaStream_t stream)
{
    switch (a.D) {
        case 32: return launch_d<32>(a, p, stream);
        case 64: return launch_d<64>(a, p, stream);
        case 80: return launch_d<80>(a, p, stream);
        case 96: return launch_d<96>(a, p, stream);
        case 128: return launch_d<128>(a, p, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace vit
