// Rotary positions with three axes (time, height, width) for images and video, fused with the
// per-head RMS norm of q and k, and their gradient; plus the positions themselves.
//
// Pair m < D/2 of a head turns by a_m = pos[axis(m)] * inv_freq[m], where axis(m) comes from the
// three section lengths s_t + s_h + s_w = D/2:
//   blocked   the first s_t pairs follow time, the next s_h height, the last s_w width;
//   cycled    pair m follows height if m = 1 (mod 3) and m < 3 s_h, width if m = 2 (mod 3) and
//             m < 3 s_w, else time.
//   xn = x * rsqrt(mean(x^2) + eps) * w            (or xn = x)
//   (y1, y2) = (x1 cos a - x2 sin a, x2 cos a + x1 sin a)     over pairs (m, m + D/2) or (2m, 2m + 1)
// all in fp32, rounded to bf16 once at the end. The gradient turns back and differentiates the norm:
//   dz = R(-a) dy,  dn = dz w,  dx = r (dn - xh mean(dn xh)),  dw = sum over rows of dz xh,
//   r = rsqrt(mean(x^2) + eps), xh = x r.
//
// The angle: the product of an int32 position and an fp32 frequency needs 55 bits before it is
// reduced (position 10^6 at frequency 1 leaves an fp32 product with 0.06 rad of error), so it is
// formed and reduced by 2 pi exactly enough: as a product and its rounding error in fp32 where the
// position fits 22 bits, in fp64 beyond (GB300's fp64 rate is low). The remainder in about [-pi, pi]
// then goes through __sincosf, whose absolute error there is 2^-21. All heads of a token share it.
//
// HBM bound: 4 T (Hq + Hk) D bytes forward, 6 T (Hq + Hk) D backward. Measured: 36771 tokens of 16 + 16
// heads of 80, 75 us forward with their positions (5.0 TB/s; a plain copy of as many bytes 63 us); 40013 tokens
// of 16 + 4 heads of 128, 126 us backward (4.9 TB/s). Issue slots are 66 and 60 % busy, but fewer instructions
// (the weights unpacked once in shared memory; a variant for whole tokens) changed nothing forward, and cost 7 %
// backward (bank conflicts); blocks of one token per warp instead of resident ones 82 us forward.
// Rows of one warp's loads straight into registers took 108 and 176 us. One warp owns a token (or,
// when there are fewer tokens than warps to fill the GPU, a slice of a token's heads): it builds the
// token's cos/sin row in its own part of shared memory and then walks the heads, so no barrier
// wider than a warp is needed. A head row belongs to D/16 lanes, lane c holding the 16-byte chunks
// c and c + D/16, so every rotated pair lies in one thread; a warp handles 32 / (D/16) rows per
// step. Rows arrive through asynchronous copies a fixed number of steps ahead (across tokens), each
// lane copying into shared memory exactly the bytes that it will read itself, so the loads in flight
// need neither registers nor a barrier. The gradient's weight sums stay in registers (a
// lane's columns never change), are joined per block in shared memory in a fixed order, and a
// second kernel adds the blocks' partial sums.
#include <limits.h>

#include "internal.h"
#include "rope_math.cuh"

namespace vit {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

struct Mrope {
    const __nv_bfloat16 *q_in, *k_in;          // forward input, or (gradient) the normed call's input
    __nv_bfloat16 *q_out, *k_out;              // forward output, or dx
    const __nv_bfloat16 *dq, *dk;              // gradient: dy
    int64_t q_in_stride, k_in_stride, q_out_stride, k_out_stride, dq_stride, dk_stride;
    int64_t T;
    int Hq, Hk;
    const int32_t *pos;
    const float *inv_freq;
    int s_t, s_h, s_w;
    bool cycled;
    const __nv_bfloat16 *norm_w;
    float eps;
    int slices;                                // a token's heads are dealt to this many warps
    float *part;                               // gradient: [blocks][2][D] sums of dz * xh
};

__device__ __forceinline__ int axis_of(const Mrope &p, int m) {
    if (p.cycled) {
        const int a = m % 3;
        return a == 1 ? (m < 3 * p.s_h ? 1 : 0) : a == 2 ? (m < 3 * p.s_w ? 2 : 0) : 0;
    }
    return m < p.s_t ? 0 : m < p.s_t + p.s_h ? 1 : 2;
}

// pos * f reduced to about [-pi, pi], as an fp32 value
__device__ __forceinline__ float reduced_angle(int pos, float f) {
    if ((unsigned)pos + (1u << 22) < (1u << 23) && fabsf(f) <= 1.f) {      // (abs(-2^31) is negative)
        // pos is exact in fp32 and p + e is the exact product; the multiple n of 2 pi (|n| < 2^20) is
        // taken off in two parts, 2 pi = C1 + C2 to 2^-50 (Cody and Waite): the error stays below 2^-21
        const float x = (float)pos, p = x * f, e = fmaf(x, f, -p);
        const float n = rintf(p * 0.159154943f);
        constexpr float C1 = 6.28318548f, C2 = -1.74845553e-7f;
        return fmaf(-n, C2, fmaf(-n, C1, p)) + e;
    }
    const double a = (double)pos * (double)f;
    const double n = rint(a * 0.15915494309189535);                 // 1 / (2 pi)
    return (float)fma(n, -6.283185307179586, a);
}

// The pairs whose cos/sin a lane makes for every token: 2 lane and 2 lane + 1 (D/4 lanes have some).
struct LanePairs {
    float f0, f1;
    int a0, a1;
};
template <int D> __device__ __forceinline__ LanePairs lane_pairs(const Mrope &p, int lane) {
    LanePairs x{0.f, 0.f, 0, 0};
    if (lane < D / 4) {
        x.f0 = p.inv_freq[2 * lane];
        x.f1 = p.inv_freq[2 * lane + 1];
        x.a0 = axis_of(p, 2 * lane);
        x.a1 = axis_of(p, 2 * lane + 1);
    }
    return x;
}
// cos/sin of a token's pairs as {cos m, cos m+1, sin m, sin m+1}, m even
template <int D> __device__ __forceinline__ void fill_turns(const LanePairs &x, const int *pos, int lane, float4 *cs) {
    if (lane < D / 4) {
        float c0, s0, c1, s1;
        __sincosf(reduced_angle(pos[x.a0], x.f0), &s0, &c0);
        __sincosf(reduced_angle(pos[x.a1], x.f1), &s1, &c1);
        cs[lane] = make_float4(c0, c1, s0, s1);
    }
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// A lane's way over its warp's rows, `ROWS` head rows per step: unit after unit (a token, or a slice
// of its heads), and in each the q rows and then the k rows. `at` is the
// lane's own place in the current row of one tensor; only a change of part computes an address anew.
template <int D> struct Walk {
    int64_t u, t;                              // unit and its token
    char *at;                                  // this lane's chunk c of row (first row of the step + g)
    int left;                                  // rows of the part from the step's first on
    int part;                                  // 0: q, 1: k
};
struct Side {                                  // one tensor pair (q, k) that a walk goes over
    char *q, *k;
    int64_t q_stride, k_stride;                // token strides, bytes
};
template <int D> struct Way {
    int64_t units, stride;
    int slices, per, Hq, rows;
    int off;                                   // the lane's bytes from a row's start: row g, chunk c

    // the first rows at or after (unit w.u, part w.part)
    __device__ __forceinline__ void enter(Walk<D> &w, const Side &s) const {
        for (; w.u < units; w.u += stride, w.part = 0) {
            w.t = slices == 1 ? w.u : w.u / slices;
            const int lo = slices == 1 ? 0 : (int)(w.u - w.t * slices) * per, hi = min(rows, lo + per);
            for (; w.part < 2; ++w.part) {
                const int first = w.part ? max(lo, Hq) - Hq : lo, last = w.part ? hi - Hq : min(hi, Hq);
                w.left = last - first;
                if (w.left > 0) {
                    w.at = (w.part ? s.k + w.t * s.k_stride : s.q + w.t * s.q_stride) + (int64_t)first * (2 * D) + off;
                    return;
                }
            }
        }
    }
    __device__ __forceinline__ bool done(const Walk<D> &w) const { return w.u >= units; }
    __device__ __forceinline__ void step(Walk<D> &w, const Side &s, int n) const {
        w.left -= n;
        w.at += n * (2 * D);
        if (w.left <= 0) {
            ++w.part;
            enter(w, s);
        }
    }
};

// A lane's 16 elements as eight pairs, for the packed fp32 instructions: pairs 0..3 are the chunk of
// the first half, 4..7 that of the second.
__device__ __forceinline__ void unpack16(const uint4 &a, const uint4 &b, uint64_t *x) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = rope::f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack_pair(uint64_t x) {
    float lo, hi;
    rope::f2_split(x, lo, hi);
    return rope::pack2(lo, hi);
}
__device__ __forceinline__ void pack16(const uint64_t *x, uint4 &a, uint4 &b) {
    a = make_uint4(pack_pair(x[0]), pack_pair(x[1]), pack_pair(x[2]), pack_pair(x[3]));
    b = make_uint4(pack_pair(x[4]), pack_pair(x[5]), pack_pair(x[6]), pack_pair(x[7]));
}
__device__ __forceinline__ float pair_sum(uint64_t x) {
    float lo, hi;
    rope::f2_split(x, lo, hi);
    return lo + hi;
}

// y = R(a) x on the 16 elements of a lane; cs: the lane's turns of its two chunks' pairs
// (rotate-half: the four entries of chunk c in cs[0..3]; interleaved: two of each chunk)
template <bool IL>
__device__ __forceinline__ void turn(uint64_t *x, const float4 *cs) {
    using rope::f2;
    using rope::f2_fma;
    using rope::f2_mul;
    if constexpr (!IL) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {                          // elements 2i, 2i + 1 of both chunks
            const float4 t = cs[i];
            const uint64_t c = f2(t.x, t.y), s = f2(t.z, t.w);
            const uint64_t n = f2(-t.z, -t.w);
            const uint64_t a = x[i], b = x[4 + i];
            x[i] = f2_fma(b, n, f2_mul(a, c));
            x[4 + i] = f2_fma(a, s, f2_mul(b, c));
        }
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) {                          // one rotated pair each
            const float4 t = cs[q >> 1];
            const float c = (q & 1) ? t.y : t.x, s = (q & 1) ? t.w : t.z;
            float a, b;
            rope::f2_split(x[q], a, b);
            x[q] = f2_fma(f2(b, a), f2(-s, s), f2_mul(x[q], f2(c, c)));
        }
    }
}

template <int D> struct Shape {
    static constexpr int CH = D / 16;          // lanes per row
    static constexpr int ROWS = 32 / CH;       // rows a warp handles at a time
};

// sum over the CH lanes of a row's group, added in lane order
template <int D> __device__ __forceinline__ float group_sum(float v, int first) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < Shape<D>::CH; ++i) s += __shfl_sync(0xffffffffu, v, (first + i) & 31);
    return s;
}

// steps in flight: 40 and 64 KB of a block (forward: 4 steps 78 us, 5 75, 6 77, 8, of which fewer blocks fit, 97)
constexpr int kAheadFwd = 5, kAheadBwd = 4;

template <int D, bool IL>
__global__ void __launch_bounds__(kThreads, 3)
mrope_kernel(const Mrope p)
{
    constexpr int CH = Shape<D>::CH, ROWS = Shape<D>::ROWS, AHEAD = kAheadFwd;
    extern __shared__ uint4 s_rows[];                      // [warp][step][chunk a, b][lane]
    __shared__ int s_pos[kWarps][AHEAD][4];               // the steps' positions, copied with their rows
    __shared__ float4 s_cs[kWarps][D / 4];
    __shared__ uint4 s_w[2][D / 8];
    grid_wait();
    grid_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane / CH, c = lane % CH;               // row of the step, chunk of the row
    const int my_row = g < ROWS ? g : INT_MAX;             // lanes past the last group have none
    const int first = g * CH;
    if (p.norm_w) {
        for (int i = threadIdx.x; i < D / 4; i += kThreads)
            s_w[i / (D / 8)][i % (D / 8)] = reinterpret_cast<const uint4 *>(p.norm_w)[i];
        __syncthreads();
    }
    const float4 *cs_a = s_cs[warp] + (IL ? 2 * c : 4 * c), *cs_b = cs_a + D / 8;
    uint4 *mine = s_rows + warp * (AHEAD * 64) + lane;
    const uint32_t mine_a = (uint32_t)__cvta_generic_to_shared(mine);
    const uint32_t pos_a = (uint32_t)__cvta_generic_to_shared(&s_pos[warp][0][lane & 3]);
    const int rows = p.Hq + p.Hk;
    const Way<D> way{p.T * p.slices, (int64_t)gridDim.x * kWarps, p.slices, (rows + p.slices - 1) / p.slices, p.Hq, rows,
                     2 * (g * D + 8 * c)};
    const Side in{(char *)p.q_in, (char *)p.k_in, 2 * p.q_in_stride, 2 * p.k_in_stride};
    const Side out{(char *)p.q_out, (char *)p.k_out, 2 * p.q_out_stride, 2 * p.k_out_stride};
    const LanePairs pairs = lane_pairs<D>(p, lane);

    Walk<D> fetch;
    fetch.u = (int64_t)blockIdx.x * kWarps + warp;
    fetch.part = 0;
    Walk<D> at = fetch;
    way.enter(fetch, in);
    way.enter(at, out);
    auto request = [&](int slot) {                         // this lane's chunks of the fetch step's rows
        if (!way.done(fetch)) {
            if (lane < 3) copy4(pos_a + slot * 16, p.pos + 3 * fetch.t + lane);
            if (my_row < fetch.left) {
                copy16(mine_a + slot * 1024, fetch.at);
                copy16(mine_a + slot * 1024 + 512, fetch.at + D);
            }
            way.step(fetch, in, ROWS);
        }
        copies_commit();
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) request(i);
    int64_t turned = -1;                                   // the unit whose turns are in cs
    float4 cs[4];
    int slot = 0;
    while (!way.done(at)) {
        copies_wait<AHEAD - 1>();
        if (at.u != turned) {
            __syncwarp();                                  // the copied position is there, the last turns were read
            fill_turns<D>(pairs, s_pos[warp][slot], lane, s_cs[warp]);
            turned = at.u;
            __syncwarp();
            cs[0] = cs_a[0];                               // the lane's turns, for all rows of the token
            cs[1] = cs_a[1];
            cs[2] = IL ? cs_b[0] : cs_a[2];
            cs[3] = IL ? cs_b[1] : cs_a[3];
        }
        const bool row = my_row < at.left;
        uint4 va = make_uint4(0u, 0u, 0u, 0u), vb = va;
        if (row) {
            va = mine[slot * 64];
            vb = mine[slot * 64 + 32];
        }
        uint64_t x[8];
        unpack16(va, vb, x);
        if (p.norm_w) {
            uint64_t sq = rope::f2_mul(x[0], x[0]);
#pragma unroll
            for (int e = 1; e < 8; ++e) sq = rope::f2_fma(x[e], x[e], sq);
            const float inv = rsqrtf(group_sum<D>(pair_sum(sq), first) * (1.f / D) + p.eps);
            uint64_t w[8];
            unpack16(s_w[at.part][c], s_w[at.part][CH + c], w);
            const uint64_t inv2 = rope::f2(inv, inv);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = rope::f2_mul(x[e], rope::f2_mul(inv2, w[e]));
        }
        turn<IL>(x, cs);
        if (row) {
            uint4 ya, yb;
            pack16(x, ya, yb);
            *reinterpret_cast<uint4 *>(at.at) = ya;
            *reinterpret_cast<uint4 *>(at.at + D) = yb;
        }
        request(slot);                                     // read above: the slot is free
        if (++slot == AHEAD) slot = 0;
        way.step(at, out, ROWS);
    }
}

// The gradient's way over its units, `rows` head rows at a time, among the rows [h0, h1) of a token's
// Hq + Hk. (It goes over three tensors: row numbers and unpacked arithmetic, 128 us for 40013 tokens of
// 16 + 4 heads of 128, were faster here than the forward kernel's places and pairs, 137 us.)
struct RowWalk {
    int64_t u, t;
    int r, hi;
    __device__ __forceinline__ bool done(int64_t units) const { return u >= units; }
    __device__ __forceinline__ void enter(const Mrope &p, int64_t units, int64_t stride, int per, int h0, int h1) {
        for (; u < units; u += stride) {
            t = p.slices == 1 ? u : u / p.slices;
            const int lo = p.slices == 1 ? 0 : (int)(u - t * p.slices) * per;
            r = max(lo, h0);
            hi = min(lo + per, h1);
            if (r < hi) return;
        }
    }
    __device__ __forceinline__ void step(const Mrope &p, int64_t units, int64_t stride, int per, int h0, int h1,
                                         int rows) {
        r += rows;
        if (r >= hi) {
            u += stride;
            enter(p, units, stride, per, h0, h1);
        }
    }
};

// dz = R(-a) dy on the 16 elements of a lane; cs: the lane's turns of its two chunks' pairs
template <bool IL>
__device__ __forceinline__ void turn_back(float *xa, float *xb, const float4 *cs_a, const float4 *cs_b) {
    if constexpr (!IL) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float4 t = cs_a[i / 2];
            const float s0 = -t.z, s1 = -t.w;
            const float a0 = xa[i], a1 = xa[i + 1], b0 = xb[i], b1 = xb[i + 1];
            xa[i] = fmaf(a0, t.x, -b0 * s0);
            xb[i] = fmaf(b0, t.x, a0 * s0);
            xa[i + 1] = fmaf(a1, t.y, -b1 * s1);
            xb[i + 1] = fmaf(b1, t.y, a1 * s1);
        }
    } else {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float *x = half ? xb : xa;
            const float4 *cs = half ? cs_b : cs_a;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 t = cs[q >> 1];
                const float c = (q & 1) ? t.y : t.x, s = -((q & 1) ? t.w : t.z);
                const float a = x[2 * q], b = x[2 * q + 1];
                x[2 * q] = fmaf(a, c, -b * s);
                x[2 * q + 1] = fmaf(b, c, a * s);
            }
        }
    }
}

__device__ __forceinline__ uint4 pack8(const float *x) {
    return make_uint4(rope::pack2(x[0], x[1]), rope::pack2(x[2], x[3]), rope::pack2(x[4], x[5]),
                      rope::pack2(x[6], x[7]));
}

template <int D, bool IL>
__global__ void __launch_bounds__(kThreads)
mrope_bwd_kernel(const Mrope p)
{
    constexpr int CH = Shape<D>::CH, ROWS = Shape<D>::ROWS, AHEAD = kAheadBwd;
    extern __shared__ uint4 s_rows[];                      // [warp][step][dy a, dy b, x a, x b][lane]
    __shared__ int s_pos[kWarps][AHEAD][4];               // the steps' positions, copied with their rows
    __shared__ float4 s_cs[kWarps][D / 4];
    __shared__ uint4 s_w[2][D / 8];
    __shared__ float s_sum[kWarps][2][D];
    grid_wait();
    grid_release();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane / CH, c = lane % CH;
    const bool live = g < ROWS;
    const int first = g * CH;
    const bool norm = p.norm_w != nullptr;
    if (norm) {
        for (int i = threadIdx.x; i < D / 4; i += kThreads)
            s_w[i / (D / 8)][i % (D / 8)] = reinterpret_cast<const uint4 *>(p.norm_w)[i];
        __syncthreads();
    }
    const float4 *cs_a = s_cs[warp] + (IL ? 2 * c : 4 * c), *cs_b = cs_a + D / 8;
    uint4 *mine = s_rows + warp * (AHEAD * 128) + lane;
    const uint32_t mine_a = (uint32_t)__cvta_generic_to_shared(mine);
    const int rows = p.Hq + p.Hk, per = (rows + p.slices - 1) / p.slices;
    const int64_t units = p.T * p.slices, stride = (int64_t)gridDim.x * kWarps;
    const LanePairs pairs = lane_pairs<D>(p, lane);
    // all q rows, then all k rows: one set of sums in registers at a time (both at once spilled)
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const int h0 = which ? p.Hq : 0, h1 = which ? rows : p.Hq;
        const __nv_bfloat16 *dy0 = which ? p.dk : p.dq, *x0 = which ? p.k_in : p.q_in;
        __nv_bfloat16 *dx0 = which ? p.k_out : p.q_out;
        const int64_t dy_s = which ? p.dk_stride : p.dq_stride, x_s = which ? p.k_in_stride : p.q_in_stride;
        const int64_t dx_s = which ? p.k_out_stride : p.q_out_stride;
        float acc[16];                                    // this lane's columns of the weight sums
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] = 0.f;
        RowWalk fetch;
        fetch.u = (int64_t)blockIdx.x * kWarps + warp;
        fetch.enter(p, units, stride, per, h0, h1);
        auto request = [&](int slot) {
            if (!fetch.done(units)) {
                const int r = fetch.r + g;
                if (lane < 3) copy4((uint32_t)__cvta_generic_to_shared(&s_pos[warp][slot][lane]), p.pos + 3 * fetch.t + lane);
                if (live && r < fetch.hi) {
                    const int64_t off = (int64_t)(r - h0) * D + 8 * c;
                    const __nv_bfloat16 *dy = dy0 + fetch.t * dy_s + off;
                    copy16(mine_a + slot * 2048, dy);
                    copy16(mine_a + slot * 2048 + 512, dy + D / 2);
                    if (norm) {
                        const __nv_bfloat16 *x = x0 + fetch.t * x_s + off;
                        copy16(mine_a + slot * 2048 + 1024, x);
                        copy16(mine_a + slot * 2048 + 1536, x + D / 2);
                    }
                }
                fetch.step(p, units, stride, per, h0, h1, ROWS);
            }
            copies_commit();
        };
        RowWalk at = fetch;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) request(i);
        int64_t turned = -1;
        int slot = 0;
        while (!at.done(units)) {
            copies_wait<AHEAD - 1>();
            if (at.u != turned) {
                __syncwarp();
                fill_turns<D>(pairs, s_pos[warp][slot], lane, s_cs[warp]);
                turned = at.u;
                __syncwarp();
            }
            const int r = at.r + g;
            const bool row = live && r < at.hi;
            uint4 va = make_uint4(0u, 0u, 0u, 0u), vb = va, ua = va, ub = va;
            if (row) {
                va = mine[slot * 128];
                vb = mine[slot * 128 + 32];
                if (norm) {
                    ua = mine[slot * 128 + 64];
                    ub = mine[slot * 128 + 96];
                }
            }
            float da[8], db[8];
            rope::unpack8(va, da);
            rope::unpack8(vb, db);
            turn_back<IL>(da, db, cs_a, cs_b);           // dz
            if (norm) {
                float xa[8], xb[8], dna[8], dnb[8];       // x, dn = dz w
                rope::unpack8(ua, xa);
                rope::unpack8(ub, xb);
                rope::unpack8(s_w[which][c], dna);
                rope::unpack8(s_w[which][CH + c], dnb);
                float ss = 0.f, dot = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dna[e] *= da[e];
                    dnb[e] *= db[e];
                    ss = fmaf(xa[e], xa[e], fmaf(xb[e], xb[e], ss));
                    dot = fmaf(dna[e], xa[e], fmaf(dnb[e], xb[e], dot));
                }
                // lanes without a row add nothing to the sums, whatever eps is
                const float r_rms = rsqrtf(group_sum<D>(ss, first) * (1.f / D) + p.eps);
                const float inv = row ? r_rms : 0.f;
                const float k = inv * inv * (group_sum<D>(dot, first) * (1.f / D));
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    acc[e] = fmaf(da[e], xa[e] * inv, acc[e]);
                    acc[8 + e] = fmaf(db[e], xb[e] * inv, acc[8 + e]);
                    da[e] = inv * fmaf(-xa[e], k, dna[e]);
                    db[e] = inv * fmaf(-xb[e], k, dnb[e]);
                }
            }
            if (row) {
                __nv_bfloat16 *dx = dx0 + at.t * dx_s + (int64_t)(r - h0) * D + 8 * c;
                *reinterpret_cast<uint4 *>(dx) = pack8(da);
                *reinterpret_cast<uint4 *>(dx + D / 2) = pack8(db);
            }
            request(slot);
            if (++slot == AHEAD) slot = 0;
            at.step(p, units, stride, per, h0, h1, ROWS);
        }
        copies_wait<0>();
        if (!p.part) continue;
        // a warp's groups hold the same columns: join them in group order
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            float s = 0.f;
#pragma unroll 1
            for (int i = 0; i < ROWS; ++i) s += __shfl_sync(0xffffffffu, acc[e], (i * CH + c) & 31);
            if (g == 0) s_sum[warp][which][e < 8 ? 8 * c + e : D / 2 + 8 * c + e - 8] = s;
        }
    }
    if (!p.part) return;
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += s_sum[w][i / D][i % D];
        p.part[(int64_t)blockIdx.x * 2 * D + i] = s;
    }
}

// Blocks and slices: one warp per token where tokens alone fill the GPU; otherwise a token's heads
// are cut into slices of at least one step's rows, up to about 16 warps per SM in all.
template <int D> void shape(Mrope &p, int num_sms, int64_t max_blocks, unsigned *blocks) {
    const int rows = p.Hq + p.Hk;
    const int most = (rows + Shape<D>::ROWS - 1) / Shape<D>::ROWS;
    int64_t s = (int64_t)num_sms * 16 / (p.T > 0 ? p.T : 1);
    if (s < 1) s = 1;
    if (s > most) s = most;
    p.slices = (int)s;
    const int64_t want = (p.T * p.slices + kWarps - 1) / kWarps;
    *blocks = (unsigned)(want < max_blocks ? want : max_blocks);
}

template <int D> cudaError_t launch_fwd(Mrope p, bool il, int num_sms, cudaStream_t stream) {
    unsigned blocks;
    shape<D>(p, num_sms, (int64_t)num_sms * 3, &blocks);   // resident blocks: 80 registers, 53 KB each
    constexpr int smem = kWarps * kAheadFwd * 1024;
    auto kern = il ? mrope_kernel<D, true> : mrope_kernel<D, false>;
    static DeviceOnce once[2];
    cudaError_t e = once[il].run([&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
    if (e != cudaSuccess) return e;
    LaunchScope scope("qk_norm_mrope", stream);
    return launch_chained(kern, blocks, kThreads, smem, stream, p);
}

template <int D> cudaError_t launch_bwd(Mrope p, bool il, float *dnorm_w, int num_sms, cudaStream_t stream) {
    unsigned blocks;
    int64_t most = (int64_t)num_sms * 2;                 // resident blocks: 128 registers, 77 KB each
    if (most > kMropeParts) most = kMropeParts;
    shape<D>(p, num_sms, most, &blocks);
    if (!dnorm_w) p.part = nullptr;
    if (blocks > 0) {
        constexpr int smem = kWarps * kAheadBwd * 2048;
        auto kern = il ? mrope_bwd_kernel<D, true> : mrope_bwd_kernel<D, false>;
        static DeviceOnce once[2];
        cudaError_t e = once[il].run([&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
        if (e != cudaSuccess) return e;
        LaunchScope scope("qk_norm_mrope_bwd", stream);
        e = launch_chained(kern, blocks, kThreads, smem, stream, p);
        if (e != cudaSuccess) return e;
    }
    if (!dnorm_w) return cudaSuccess;
    return launch_column_sum(p.part, (int)blocks, 1, 2 * D, dnorm_w, nullptr, nullptr, stream);
}

Mrope params(const MropeArgs &a) {
    Mrope p{};
    p.q_in = static_cast<const __nv_bfloat16 *>(a.q_in);
    p.k_in = static_cast<const __nv_bfloat16 *>(a.k_in);
    p.q_out = static_cast<__nv_bfloat16 *>(a.q_out);
    p.k_out = static_cast<__nv_bfloat16 *>(a.k_out);
    p.dq = static_cast<const __nv_bfloat16 *>(a.dq);
    p.dk = static_cast<const __nv_bfloat16 *>(a.dk);
    p.q_in_stride = a.q_in_stride;
    p.k_in_stride = a.k_in_stride;
    p.q_out_stride = a.q_out_stride;
    p.k_out_stride = a.k_out_stride;
    p.dq_stride = a.dq_stride;
    p.dk_stride = a.dk_stride;
    p.T = a.T;
    p.Hq = a.Hq;
    p.Hk = a.Hk;
    p.pos = a.pos;
    p.inv_freq = a.inv_freq;
    p.s_t = a.sections[0];
    p.s_h = a.sections[1];
    p.s_w = a.sections[2];
    p.cycled = a.cycled;
    p.norm_w = static_cast<const __nv_bfloat16 *>(a.norm_w);
    p.eps = a.eps;
    p.part = a.part;
    return p;
}

constexpr int kPosThreads = 256;

// (time, row, column) of every token of clips packed one after the other, frames row-major one
// after the other inside a clip, and the clips' offsets: every block scans the grid list in shared
// memory, so no pass over blocks is needed. Latency bound at a batch's sizes: a thread's tokens are few, and
// the scan takes two barriers.
__global__ void __launch_bounds__(kPosThreads)
grid_positions_kernel(const int32_t *grid_thw, int n, int64_t T, int32_t *pos, int32_t *cu_out, int32_t *status)
{
    extern __shared__ int64_t s_cu[];          // [n + 1]
    __shared__ int64_t s_part[kPosThreads / 32];
    grid_wait();
    grid_release();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // tokens of clip i; a product past any T this call takes is an error, not an overflow
    auto size = [&](int i) -> int64_t {
        const int64_t t = grid_thw[3 * i], h = grid_thw[3 * i + 1], w = grid_thw[3 * i + 2];
        if (t < 0 || h < 0 || w < 0) return -1;
        const int64_t hw = h * w;
        if (t == 0 || hw == 0) return 0;
        return (hw > T || t > T || t * hw > T) ? -1 : t * hw;
    };
    const int per = (n + kPosThreads - 1) / kPosThreads;
    const int lo = min(tid * per, n), hi = min(lo + per, n);
    int64_t local = 0;
    int bad = 0;
    for (int i = lo; i < hi; ++i) {
        const int64_t s = size(i);
        bad |= s < 0;
        local += s < 0 ? 0 : s;
    }
    int64_t run = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
    }
    if (lane == 31) s_part[warp] = run;
    bad = __syncthreads_or(bad);
    run -= local;
    for (int w = 0; w < warp; ++w) run += s_part[w];
    if (tid == 0) s_cu[0] = 0;
    for (int i = lo; i < hi; ++i) {
        const int64_t s = size(i);
        run += s < 0 ? 0 : s;
        s_cu[i + 1] = run;
    }
    __syncthreads();
    if (bad || s_cu[n] != T) {
        if (blockIdx.x == 0 && tid == 0) report_error(status, VIT_ERR_GRID_MISMATCH);
        return;
    }
    if (blockIdx.x == 0 && cu_out)
        for (int i = tid; i <= n; i += kPosThreads) cu_out[i] = (int32_t)s_cu[i];
    if (!pos) return;
    for (int64_t t = (int64_t)blockIdx.x * kPosThreads + tid; t < T; t += (int64_t)gridDim.x * kPosThreads) {
        int a = 0, b = n;                      // s_cu[a] <= t < s_cu[b]; ends on the last such a (empty clips skipped)
        while (b - a > 1) {
            const int m = (a + b) >> 1;
            if (s_cu[m] <= t) a = m; else b = m;
        }
        const unsigned h = (unsigned)grid_thw[3 * a + 1], w = (unsigned)grid_thw[3 * a + 2];
        const unsigned off = (unsigned)(t - s_cu[a]), row = off / w;
        pos[3 * t] = (int32_t)(row / h);
        pos[3 * t + 1] = (int32_t)(row % h);
        pos[3 * t + 2] = (int32_t)(off % w);
    }
}

}  // namespace

cudaError_t launch_grid_positions(const int32_t *grid_thw, int n, int64_t T, int32_t *pos, int32_t *cu_seqlens,
                                  int32_t *status, int num_sms, cudaStream_t stream)
{
    const size_t smem = sizeof(int64_t) * (size_t)(n + 1);
    static DeviceOnce once;
    cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(grid_positions_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)(sizeof(int64_t) * (VIT_MAX_SEGMENTS + 1)));
    });
    if (e != cudaSuccess) return e;
    // a token per thread up to four blocks an SM; a long list, which every block scans, is worth fewer blocks
    const int64_t want = pos ? (T + kPosThreads - 1) / kPosThreads : 1, most = (int64_t)num_sms * (n <= 1024 ? 4 : 1);
    const unsigned blocks = (unsigned)(want < 1 ? 1 : want < most ? want : most);
    LaunchScope scope("grid_positions", stream);
    return launch_chained(grid_positions_kernel, blocks, kPosThreads, smem, stream, grid_thw, n, T, pos, cu_seqlens,
                          status);
}

cudaError_t launch_mrope(const MropeArgs &a, int num_sms, cudaStream_t stream)
{
    const Mrope p = params(a);
    switch (a.D) {
        case 32: return launch_fwd<32>(p, a.interleaved, num_sms, stream);
        case 64: return launch_fwd<64>(p, a.interleaved, num_sms, stream);
        case 80: return launch_fwd<80>(p, a.interleaved, num_sms, stream);
        case 96: return launch_fwd<96>(p, a.interleaved, num_sms, stream);
        case 128: return launch_fwd<128>(p, a.interleaved, num_sms, stream);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_mrope_bwd(const MropeArgs &a, float *dnorm_w, int num_sms, cudaStream_t stream)
{
    const Mrope p = params(a);
    switch (a.D) {
        case 32: return launch_bwd<32>(p, a.interleaved, dnorm_w, num_sms, stream);
        case 64: return launch_bwd<64>(p, a.interleaved, dnorm_w, num_sms, stream);
        case 80: return launch_bwd<80>(p, a.interleaved, dnorm_w, num_sms, stream);
        case 96: return launch_bwd<96>(p, a.interleaved, dnorm_w, num_sms, stream);
        case 128: return launch_bwd<128>(p, a.interleaved, dnorm_w, num_sms, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace vit
