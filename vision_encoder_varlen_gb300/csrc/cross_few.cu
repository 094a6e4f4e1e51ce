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
//
// A causal window (W): the keys that a sequence's queries see between them are its first `sn` tokens, in tiles of
// their own, and the run of positions from `lo` on; a run of `chunk` keys counts along both. Keys outside are not
// loaded, and where there is more than one query each masks for itself what another one sees. HBM bound like the rest: 48
// single tokens over padded caches of up to 16383 keys, window 4096, 32 heads over 8 of 128: 61 us with the join, 5.4 TB/s
// of the visible keys (0.80 of a copy). A prefix takes the place of the first tokens where reading it for each sequence
// is cheap: three single tokens behind 1601 shared keys 12 us in a graph, 27 with one pass for all of them, of which the
// launches are most.
#include <type_traits>

#include "cross.h"
#include "sm100.cuh"
#include "warp_mma.cuh"
#include "window.h"

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
    bool parts;                               // W: leave the runs' partial results even where there is only one run
    int window, sinks;                        // W: as in WinLong
    bool prefix;
    Groups groups;
};

// The keys of a sequence as the runs count them: [0, head) are the rows from f0 on, padded to whole tiles (its first sn
// tokens, or the prefix), and head + i is position lo + i of its own; n in all. A query before the first own key sees the
// prefix alone, or nothing (`none` of them).
struct Keys {
    int f0, sn, head, lo, n, none;
};
__device__ __forceinline__ Keys window_keys(const Few &p, int b, const CrossSeg &x, int f0, int fn)
{
    const WinSeg w = win_seg(x);
    Keys k{x.k0, 0, 0, 0, 0, w.none};
    if (p.prefix) {
        k.f0 = f0;
        k.sn = fn;
        if (fn > 0) k.none = 0;
    } else {
        const WinRange r = win_range(w.p0, p.window, p.sinks);
        k.sn = r.first;
        k.lo = r.lo;
    }
    k.head = (k.sn + kTile - 1) / kTile * kTile;
    k.n = x.qn > k.none ? k.head + w.kn - k.lo : 0;
    return k;
}

// Warps of a block: MT row tiles x 4 key groups.
constexpr int kGroups = 4;
template <int MT> constexpr int kMmaWarps = MT * kGroups;

// W: the tensors of the keys that are read first
struct FewMaps {
    CUtensorMap k, kr, v, vr;
};
struct NoMaps {};

template <int D, int MT, bool W>
__global__ void __launch_bounds__(32 * kMmaWarps<MT> + 32)
cross_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_kr,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_vr,
                 const __grid_constant__ std::conditional_t<W, FewMaps, NoMaps> tm_f, const Few p)
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
    [[maybe_unused]] int f0 = 0, fn = 0;                      // W: the prefix
    if constexpr (W) {
        if (p.prefix) {
            int g, begin, err;
            const bool fine = p.groups.find(b, lane, (split | hk | b) == 0, g, begin, f0, fn, err);
            if (err && threadIdx.x == 0 && split == 0 && hk == 0) report_error(p.status, err);
            if (!fine) return;
        }
    }
    // a sequence without keys is left to the join, or to split 0 where there is none
    if (!load_seg(p.segs, b, seg, p.status, threadIdx.x == 0 && split == 0 && hk == 0)) return;
    if (seg.qn == 0) return;
    const int first = split * p.chunk;
    const bool only = p.n_split == 1 && !(W && p.parts);
    Keys keys{0, 0, 0, 0, 0, 0};
    int p0 = 0;                                               // position of the first query
    if constexpr (W) {
        keys = window_keys(p, b, seg, f0, fn);
        // queries that see nothing: zeros, by the first run's block
        if (split == 0 && !p.parts)
            for (int x = threadIdx.x; x < keys.none * p.group * (D / 8); x += 32 * NW + 32) {
                const int r = x / (D / 8), c = x % (D / 8), head = hk * p.group + r % p.group;
                const int64_t t = seg.q0 + r / p.group;
                *reinterpret_cast<uint4 *>(p.out + t * p.out_stride + (int64_t)head * D + 8 * c) = make_uint4(0u, 0u, 0u, 0u);
                if (p.lse && c == 0) p.lse[t * p.Hq + head] = -INFINITY;
            }
        if (first >= keys.n) return;
        p0 = seg.kn - seg.qn + keys.none;
        seg.q0 += keys.none;
        seg.qn -= keys.none;
    } else {
        if (first >= seg.kn && !(only && seg.kn == 0)) return;
    }
    const int n_keys = min(p.chunk, (W ? keys.n : seg.kn) - first);   // of this run
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
                int row = seg.k0 + first + i * kTile;
                const CUtensorMap *mk = &tm_k, *mkr = &tm_kr, *mv = &tm_v, *mvr = &tm_vr;
                if constexpr (W) {
                    if (first + i * kTile >= keys.head) {
                        row += keys.lo - keys.head;
                    } else {
                        row += keys.f0 - seg.k0;
                        mk = &tm_f.k;
                        mkr = &tm_f.kr;
                        mv = &tm_f.v;
                        mvr = &tm_f.vr;
                    }
                }
                sm100::mbar_arrive_expect_tx(bar, 2 * T::BYTES);
#pragma unroll
                for (int x = 0; x < T::N128; ++x) {
                    sm100::tma_load_2d(dst + x * kTile * 128, mk, hk * D + 64 * x, row, bar);
                    sm100::tma_load_2d(dst + T::BYTES + x * kTile * 128, mv, hk * D + 64 * x, row, bar);
                }
                if constexpr (T::REM > 0) {
                    sm100::tma_load_2d(dst + T::N128 * kTile * 128, mkr, hk * D + 64 * T::N128, row, bar);
                    sm100::tma_load_2d(dst + T::BYTES + T::N128 * kTile * 128, mvr, hk * D + 64 * T::N128, row, bar);
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
            int live = n_keys - i * kTile - key0;             // of this warp's 16 keys
            int kp = first + i * kTile + key0;                // W: position of the first of them
            if constexpr (W) {
                if (kp < keys.head) live = keys.sn - kp;
                else kp += keys.lo - keys.head;
            }
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
                if constexpr (W) {
                    if (seg.qn > 1 && first + i * kTile >= keys.head) {
                        // rows g and g + 8: keys up to `hi`, from `lo` on or before `sk`
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int hi = p0 + (row_tile * 16 + g + 8 * h) / p.group - kp;
                            const int lo = p.window > 0 ? hi - p.window + 1 : 0, sk = p.sinks - kp;
#pragma unroll
                            for (int n = 0; n < 2; ++n)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const int x = 8 * n + 2 * c + e;
                                    if (x > hi || (x < lo && x >= sk)) sc[n][2 * h + e] = -INFINITY;
                                }
                        }
                    }
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
            const float inv = W || seg.kn > 0 ? 1.f / L[h] : 0.f;   // no key at all: 0, and lse = -inf
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
template <int D, bool WIDE, bool W>
__global__ void __launch_bounds__(256, W ? 4 : 0)
cross_join_kernel(const Few p)
{
    __shared__ float s_acc[WIDE ? 8 : 1][WIDE ? D : 1], s_sum[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.y;
    CrossSeg seg;
    grid_wait();                                              // the runs' results
    [[maybe_unused]] int f0 = 0, fn = 0;
    if constexpr (W) {
        int g, begin, err;
        if (p.prefix && !p.groups.find(b, lane, false, g, begin, f0, fn, err)) return;
    }
    if (!load_seg(p.segs, b, seg, nullptr, false)) return;
    int n_keys = seg.kn;
    if constexpr (W) {                                        // (queries that see nothing are written already)
        const Keys keys = window_keys(p, b, seg, f0, fn);
        n_keys = keys.n;
        seg.q0 += keys.none;
        seg.qn -= keys.none;
    }
    const int n_rows = seg.qn * p.Hq;                         // (token, head) rows of the sequence
    const int runs = key_runs(n_keys, p.chunk);
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

// a tensor's maps: the wide one and that of the remaining columns
template <int D> bool kv_maps(CUtensorMap *m, CUtensorMap *mr, const void *ptr, int64_t T, int H, int64_t stride)
{
    constexpr int rem = Tile<D>::REM > 0 ? Tile<D>::REM : 64, wide = D >= 64 ? 64 : rem;
    if (!kv_map(m, ptr, T, H, D, stride, wide)) return false;
    *mr = *m;
    return rem == wide || kv_map(mr, ptr, T, H, D, stride, rem);
}

template <int D, int MT, bool W>
cudaError_t launch_mt(const CrossArgs &a, const WinArgs *wa, const FewPlan &pl, const Few &p, cudaStream_t stream)
{
    CUtensorMap mk, mkr, mv, mvr;
    const CrossSegs &s = a.segs;
    if (!kv_maps<D>(&mk, &mkr, a.k, s.Tk, a.Hk, a.k_stride) || !kv_maps<D>(&mv, &mvr, a.v, s.Tk, a.Hk, a.v_stride))
        return cudaErrorInvalidValue;
    std::conditional_t<W, FewMaps, NoMaps> first;
    if constexpr (W) {
        first = FewMaps{mk, mkr, mv, mvr};
        if (p.prefix && (!kv_maps<D>(&first.k, &first.kr, wa->kp, p.groups.Tp, a.Hk, wa->kp_stride) ||
                         !kv_maps<D>(&first.v, &first.vr, wa->vp, p.groups.Tp, a.Hk, wa->vp_stride)))
            return cudaErrorInvalidValue;
    }
    constexpr int smem = kStages * 2 * Tile<D>::BYTES + 1024;
    static_assert(kStages * 2 * Tile<D>::BYTES >= 2 * MT * 16 * D * 4, "the joins reuse the ring");
    auto kern = cross_few_kernel<D, MT, W>;
    static DeviceOnce once;
    cudaError_t e = once.run([&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
    if (e != cudaSuccess) return e;
    {
        LaunchScope scope(W ? "window_few" : "cross_few", stream);
        e = launch_chained(kern, dim3(a.Hk, s.B, pl.n_split), 32 * kMmaWarps<MT> + 32, smem, stream, mk, mkr, mv, mvr,
                           first, p);
    }
    if (e != cudaSuccess || pl.n_split == 1 || p.parts) return e;
    LaunchScope scope("cross_join", stream);
    const int rows = s.max_q * a.Hq;
    // with more than 16 runs a warp per row is too few loads in flight (147 runs: 37 us)
    return pl.n_split > 16 ? launch_chained(cross_join_kernel<D, true, W>, dim3(rows, s.B), 256, 0, stream, p)
                           : launch_chained(cross_join_kernel<D, false, W>, dim3((rows + 7) / 8, s.B), 256, 0, stream, p);
}

template <int D, bool W>
cudaError_t launch_d(const CrossArgs &a, const WinArgs *wa, const FewPlan &pl, bool parts, void *part, cudaStream_t stream)
{
    Few p{};
    if constexpr (W) {
        p.window = wa->window;
        p.sinks = wa->sinks;
        p.prefix = wa->prefix && !parts;       // (else the prefix is another kernel's)
        p.groups = wa->groups;
    }
    p.parts = parts;
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
    p.part_o = static_cast<float *>(part);
    p.part_s = p.part_o + n * D;
    switch (pl.row_tiles) {
        case 1: return launch_mt<D, 1, W>(a, wa, pl, p, stream);
        default: return launch_mt<D, 2, W>(a, wa, pl, p, stream);
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
    p.n_split = p.room = (int)n;
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

// Keys that the runs of a windowed call count at most: everything in one piece where no window leaves a gap behind the
// first tokens, else those in whole tiles and what the queries of a sequence see between them.
static int window_most(int max_q, int max_k, int window, int sinks)
{
    if (window == 0 || (int64_t)window + sinks >= max_k) return max_k;
    const int64_t own = (int64_t)window + max_q - 1, head = ((int64_t)sinks + kTile - 1) / kTile * kTile;
    const int64_t most = head + own, all = (int64_t)max_k + kTile;
    return (int)(most < all ? most : all);
}
bool window_takes_few(int B, int Hq, int Hk, int D, int max_q, int max_k, int window, int sinks)
{
    return takes_few(B, Hq, Hk, D, max_q, window_most(max_q, max_k, window, sinks));
}
// A second round of blocks for less than half the places of the first is not begun: the places that shared memory leaves,
// and those that registers leave to two row tiles (nine warps) from head_dim 64 on. Three single tokens behind 1601 shared
// keys: 14 runs of 24 pairs, where 304 blocks of one row tile fit at head_dim 128. Two row tiles, 32 rows, 8 key heads: 7
// sequences of 1100 keys at head_dim 128, 112 blocks 19.5 us in a graph, 168 27.1; 5 of 1600, 120 19.2, 160 23.0; 13 of
// 1200 at 64, 208 19.0, 312 22.4. At head_dim 32 registers leave 4 and 3 places of 8, but counting those was slower: 20
// of 1600, 320 blocks 25.7, 640 24.6; one row, 40 of 1000, 1280 blocks 16.4, 960 14.6.
static FewPlan one_round(int B, int Hq, int Hk, int D, int max_q, int most)
{
    FewPlan p = few_plan(B, Hq, Hk, D, max_q, most);
    const int64_t pairs = (int64_t)B * Hk;
    auto round = [&](int blocks) {
        const int64_t fit = (int64_t)kDesignSms * blocks;
        if (pairs * p.n_split > fit && 2 * pairs * p.n_split < 3 * fit && pairs <= fit) {
            const int64_t n = fit / pairs;
            p.chunk = (int)((((int64_t)most + n - 1) / n + kTile - 1) / kTile * kTile);
            p.n_split = (int)(((int64_t)most + p.chunk - 1) / p.chunk);
        }
    };
    round(227 * 1024 / (kStages * 4 * kTile * D + 2048));
    p.room = p.n_split;
    if (p.row_tiles == 2 && D >= 64) round(D <= 80 ? 2 : 1);
    p.partial_bytes = p.room > 1 ? sizeof(float) * (size_t)pairs * p.room * p.rows * (D + 1) : 0;
    return p;
}
FewPlan window_few_plan(int B, int Hq, int Hk, int D, int max_q, int max_k, int window, int sinks)
{
    return one_round(B, Hq, Hk, D, max_q, window_most(max_q, max_k, window, sinks));
}

static int prefix_most(int max_k, int max_p)
{
    const int64_t most = ((int64_t)max_p + kTile - 1) / kTile * kTile + max_k;
    return most < 0x7fff0000 ? (int)most : 0x7fff0000;
}
// Behind prefixes: few rows where reading the prefix for each sequence anew costs less than the launches that share it, up to
// 96 MB. In a graph, anew and shared, single tokens of 32 heads over 8 of 128: 8 sequences behind 1000 keys (34 MB) 17 and
// 28 us, behind 2000 (66) 27 and 27, 2900 (94) 29 and 29, 4000 (128) 32 and 29, 8000 (253) 41 and 32; 16 behind 1450 (94) 29
// and 27, 2500 (159) 34 and 29; 3 behind 8000 (95) 29 and 31, 16 000 (189) 39 and 36.
bool prefix_takes_few(int B, int Hq, int Hk, int D, int max_q, int max_k, int max_p)
{
    const int64_t keys = prefix_most(max_k, max_p);
    return keys < 0x7fff0000 && takes_few(B, Hq, Hk, D, max_q, (int)keys) &&
           B * keys * Hk * D * 4 <= ((int64_t)96 << 20);
}
FewPlan prefix_few_plan(int B, int Hq, int Hk, int D, int max_q, int max_k, int max_p)
{
    return one_round(B, Hq, Hk, D, max_q, prefix_most(max_k, max_p));
}

cudaError_t launch_cross_few(const CrossArgs &a, const FewPlan &p, cudaStream_t stream)
{
    switch (a.D) {
        case 32: return launch_d<32, false>(a, nullptr, p, false, a.workspace, stream);
        case 64: return launch_d<64, false>(a, nullptr, p, false, a.workspace, stream);
        case 80: return launch_d<80, false>(a, nullptr, p, false, a.workspace, stream);
        case 96: return launch_d<96, false>(a, nullptr, p, false, a.workspace, stream);
        case 128: return launch_d<128, false>(a, nullptr, p, false, a.workspace, stream);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_window_few(const WinArgs &a, const FewPlan &p, bool parts, void *part, cudaStream_t stream)
{
    switch (a.f.D) {
        case 32: return launch_d<32, true>(a.f, &a, p, parts, part, stream);
        case 64: return launch_d<64, true>(a.f, &a, p, parts, part, stream);
        case 80: return launch_d<80, true>(a.f, &a, p, parts, part, stream);
        case 96: return launch_d<96, true>(a.f, &a, p, parts, part, stream);
        case 128: return launch_d<128, true>(a.f, &a, p, parts, part, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace vit
